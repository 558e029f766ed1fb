"""Cases of a trained scorer's operators: embedding rows with their gradient by sorted tokens, gated products
(dense, and one pair of matrices per expert) with their gradients, and log probabilities of given tokens with
entropy, best alternatives and gradient.

Every case runs in its plain form (``own`` false: elementary torch operations in float32, rounded once at the
end) or through the library's entry points (``own`` true).  The same inputs feed both.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # the rows of the 2048 candidates that a search returned for one query, 128 wide as the index's
        {"name": "embed_query", "op": "embed", "tokens": 2048, "rows": 1000000, "width": 128, "type": "f16"},
        # a training batch of popular and rare tokens
        {"name": "embed_batch", "op": "embed", "tokens": 65536, "rows": 131072, "width": 1024, "type": "bf16"},
        # gradient of a small table, sizes that fill no tile
        {"name": "embed_grad_odd", "op": "embed_grad", "tokens": 3001, "rows": 5003, "width": 250, "type": "f32"},
        # gradient of the training batch above
        {"name": "embed_grad_batch", "op": "embed_grad", "tokens": 65536, "rows": 131072, "width": 1024,
         "type": "bf16"},
        # one token: the weights' bytes are the cost
        {"name": "gated_one", "op": "gated", "tokens": 1, "ins": 4096, "outs": 8192, "experts": 0, "act": "silu",
         "keep": False, "type": "bf16"},
        # a serving step: 32 tokens with 2 of 32 experts each; some experts see no row
        {"name": "gated_experts_step", "op": "gated", "tokens": 64, "ins": 1024, "outs": 1024, "experts": 32,
         "act": "gelu", "keep": False, "type": "f16"},
        # a forward pass of a training step that keeps what its gradient needs
        {"name": "gated_batch", "op": "gated", "tokens": 8192, "ins": 2048, "outs": 8192, "experts": 0, "act": "silu",
         "keep": True, "type": "bf16"},
        # gradients at sizes that fill no tile, float32 as the rerank's weights
        {"name": "gated_grad_odd", "op": "gated_grad", "tokens": 1001, "ins": 250, "outs": 999, "experts": 0,
         "act": "gelu", "type": "f32"},
        # gradients of a training step: 8192 tokens with 2 of 8 experts each
        {"name": "gated_grad_experts", "op": "gated_grad", "tokens": 16384, "ins": 1024, "outs": 2048, "experts": 8,
         "act": "silu", "type": "bf16"},
        # one generated token with its best alternatives
        {"name": "logprobs_one", "op": "logprobs", "tokens": 1, "vocab": 131072, "top": 8, "scale": 1.25,
         "masked": 0.0, "grad": False, "type": "bf16"},
        # 256 queries, each over the 2048 candidates of its search: the chosen one, the 16 best, the gradient
        {"name": "logprobs_candidates", "op": "logprobs", "tokens": 256, "vocab": 2048, "top": 16, "scale": 1.0,
         "masked": 0.1, "grad": True, "type": "f32"},
        # a training step's loss with an entropy term, rows that end inside every tile
        {"name": "logprobs_train", "op": "logprobs", "tokens": 4096, "vocab": 50021, "top": 0, "scale": 1.0,
         "masked": 0.0, "grad": True, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "gated", "gated_grad", "logprobs", "logprobs"])
    case = {"op": op, "type": rng.choice(["f32", "f16", "bf16"])}
    if op in ("embed", "embed_grad"):
        width = _log(rng, 16, 4096)
        case.update(tokens=_log(rng, 1, min(262144, 67108864 // width)),
                    rows=_log(rng, 16, min(1000000, 134217728 // width)), width=width)
    elif op == "logprobs":
        vocab = _log(rng, 2, 200000)
        case.update(vocab=vocab, tokens=_log(rng, 1, min(16384, 67108864 // vocab)),
                    top=rng.choice([0, 1, rng.randint(2, 16)]), scale=rng.choice([1.0, 1.0, 0.5, 1.6]),
                    masked=rng.choice([0.0, 0.1, 0.6]), grad=rng.random() < 0.5)
        case["top"] = min(case["top"], vocab)
    else:
        experts = rng.choice([0, 0, rng.randint(2, 48)])
        ins, outs = _log(rng, 16, 4096), _log(rng, 16, 4096)
        if experts:   # so that all matrices together hold at most 64 M values
            ins, outs = min(ins, 1024), min(outs, 2048)
            outs = min(outs, 33554432 // (experts * ins))
        case.update(tokens=_log(rng, 1, 4096 if op == "gated" else 2048), ins=ins, outs=outs, experts=experts,
                    act=rng.choice(["silu", "gelu", "relu"]))
        if op == "gated":
            case["keep"] = rng.random() < 0.5
    return case


def _popular(g, n, rows):
    """n tokens, the r-th most popular with a probability near 1 / r; the popular ones lie anywhere."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.clamp(torch.exp(u * math.log(rows + 1)).long() - 1, 0, rows - 1)
    return (rank * 2654435761 + 12345) % rows


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    T = case["tokens"]
    if op in ("embed", "embed_grad"):
        V, D = case["rows"], case["width"]
        ids = _popular(g, T, V)
        gone = torch.rand(T, generator=g, device="cuda") < 0.01
        st = {"ids": torch.where(gone, torch.full_like(ids, -1), ids), "scale": math.sqrt(D)}
        st.update({"table": (normal(V, D) / math.sqrt(D)).to(dt)} if op == "embed" else {"d_out": normal(T, D).to(dt)})
        return st
    if op == "logprobs":
        V = case["vocab"]
        x = 2.0 * normal(T, V)
        tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
        if case["masked"]:
            shut = torch.rand((T, V), generator=g, device="cuda") < case["masked"]
            shut.scatter_(1, tokens[:, None], False)   # a token that was given is open
            x = torch.where(shut, torch.full_like(x, -math.inf), x)
        padding = torch.rand(T, generator=g, device="cuda") < 0.02
        return {"logits": x.to(dt), "tokens": torch.where(padding, torch.full_like(tokens, -1), tokens),
                "d_logprobs": normal(T), "d_entropy": 0.1 * normal(T)}
    K, N, E = case["ins"], case["outs"], case["experts"]
    many = (E,) if E else ()
    st = {"x": normal(T, K).to(dt), "offsets": None}
    for name in ("w_gate", "w_up"):
        st[name] = (normal(*many, N, K) / math.sqrt(K)).to(dt)
    if E:   # rows sorted by expert, some experts liked more than others
        liked = torch.randn(E, generator=g, device="cuda")
        ids = (normal(T, E) + liked).argmax(1)
        st["offsets"] = (ids[None, :] < torch.arange(E + 1, device="cuda")[:, None]).sum(1).to(torch.int32)
    if op == "gated_grad":
        st["dh"] = normal(T, N).to(dt)
        gate, up = _projections(st, case)   # what the forward pass kept
        st["gate"], st["up"] = gate.to(dt), up.to(dt)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    return st


# ---- plain forms -------------------------------------------------------------------------------------

def _plain_embed(st):
    ids, table = st["ids"], st["table"]
    there = (ids >= 0) & (ids < table.shape[0])
    rows = table[torch.where(there, ids, torch.zeros_like(ids))].float() * st["scale"]
    return torch.where(there[:, None], rows, torch.zeros_like(rows)).to(table.dtype)


def _plain_embed_grad(st, case):
    ids, d = st["ids"], st["d_out"]
    there = (ids >= 0) & (ids < case["rows"])
    at = torch.where(there, ids, torch.full_like(ids, case["rows"]))   # a last row takes what is dropped
    out = torch.zeros((case["rows"] + 1, case["width"]), device="cuda")
    out.index_add_(0, at, d.float() * st["scale"])
    return out[:-1].to(d.dtype)


def _parts(st, case):
    """(first row, end, its gate and up matrices) of every expert that has rows."""
    if not case["experts"]:
        return [(0, case["tokens"], 0, st["w_gate"][None], st["w_up"][None])]
    ends = st["offsets"].tolist()
    return [(a, b, e, st["w_gate"], st["w_up"]) for e, (a, b) in enumerate(zip(ends, ends[1:])) if a < b]


def _projections(st, case):
    x = st["x"].float()
    gate, up = (torch.empty((case["tokens"], case["outs"]), device="cuda") for _ in range(2))
    for a, b, e, w_gate, w_up in _parts(st, case):
        gate[a:b] = x[a:b] @ w_gate[e].float().t()
        up[a:b] = x[a:b] @ w_up[e].float().t()
    return gate, up


def _activation(v, act):
    """Its value and slope."""
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v)), (v > 0).float()
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-v))
        return v * s, s * (1.0 + v * (1.0 - s))
    cdf = 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v * cdf, cdf + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)


def _plain_gated(st, case):
    gate, up = _projections(st, case)
    dt = st["x"].dtype
    h = (_activation(gate, case["act"])[0] * up).to(dt)
    return [h, gate.to(dt), up.to(dt)] if case["keep"] else [h]


def _plain_gated_grad(st, case):
    dt, x, dh = st["x"].dtype, st["x"].float(), st["dh"].float()
    value, slope = _activation(st["gate"].float(), case["act"])
    d_gate, d_up = dh * st["up"].float() * slope, dh * value
    dx = torch.zeros_like(x)
    dw_gate, dw_up = torch.zeros_like(st["w_gate"]), torch.zeros_like(st["w_up"])
    for a, b, e, w_gate, w_up in _parts(st, case):
        dx[a:b] = d_gate[a:b] @ w_gate[e].float() + d_up[a:b] @ w_up[e].float()
        (dw_gate[e] if case["experts"] else dw_gate).copy_(d_gate[a:b].t() @ x[a:b])
        (dw_up[e] if case["experts"] else dw_up).copy_(d_up[a:b].t() @ x[a:b])
    return [dx.to(dt), dw_gate, dw_up]


def _plain_logprobs(st, case):
    x, tokens = st["logits"].float() * case["scale"], st["tokens"]
    there = (tokens >= 0) & (tokens < case["vocab"])
    at = torch.where(there, tokens, torch.zeros_like(tokens))[:, None]
    z = x - x.amax(1, keepdim=True)
    log_sum = torch.log(torch.exp(z).sum(1, keepdim=True))
    logp = z - log_sum
    p = torch.exp(logp)
    part = torch.where(p > 0, logp, torch.zeros_like(logp)) * p
    entropy = -part.sum(1)
    zero = torch.zeros_like(entropy)
    out = [torch.where(there, logp.gather(1, at)[:, 0], zero), entropy]
    if case["top"]:
        # by the logits themselves: scaled ones may tie where these do not
        best = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True)[1][:, :case["top"]]
        value = logp.gather(1, best)
        out += [torch.where(value == -math.inf, torch.full_like(best, -1), best), value]
    if case["grad"]:
        d = torch.where(there, st["d_logprobs"], zero)[:, None]
        grad = -p * d - (part + p * entropy[:, None]) * st["d_entropy"][:, None]
        grad.scatter_add_(1, at, d)
        out.append((grad * case["scale"]).to(st["logits"].dtype))
    return out


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "embed":
            return _plain_embed(state)
        if op == "embed_grad":
            return _plain_embed_grad(state, case)
        if op == "gated":
            return _plain_gated(state, case)
        if op == "gated_grad":
            return _plain_gated_grad(state, case)
        return _plain_logprobs(state, case)
    from int8_ivf_ann_amd import svt
    if op == "embed":
        return svt.svt_embedding(state["table"], state["ids"], scale=state["scale"])
    if op == "embed_grad":
        return svt.svt_embedding_backward(state["d_out"], state["ids"], case["rows"], scale=state["scale"])
    if op == "gated":
        out = svt.svt_gated_linear(state["x"], state["w_gate"], state["w_up"], offsets=state["offsets"],
                                   activation=case["act"], keep=case["keep"])
        return list(out) if case["keep"] else [out]
    if op == "gated_grad":
        return list(svt.svt_gated_linear_backward(state["dh"], state["x"], state["w_gate"], state["w_up"],
                                                  state["gate"], state["up"], offsets=state["offsets"],
                                                  activation=case["act"]))
    logprobs, entropy, norms, *best = svt.svt_token_logprobs(state["logits"], state["tokens"], top=case["top"],
                                                             scale=case["scale"])
    out = [logprobs, entropy, *best]
    if case["grad"]:
        out.append(svt.svt_token_logprobs_backward(state["logits"], state["tokens"], norms, entropy,
                                                   state["d_logprobs"], state["d_entropy"], scale=case["scale"]))
    return out


# ---- the definition in 64 bits -----------------------------------------------------------------------

def _exact_act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    return v * (torch.sigmoid(v) if act == "silu" else 0.5 * torch.special.erfc(-v / math.sqrt(2)))


def _exact_slope(v, act):
    if act == "relu":
        return torch.heaviside(v, torch.zeros_like(v))
    if act == "silu":
        s = torch.sigmoid(v)
        return s + v * s * torch.sigmoid(-v)
    return 0.5 * torch.special.erfc(-v / math.sqrt(2)) + v * torch.exp(-v.square() / 2) / math.sqrt(2 * math.pi)


def _exact_logprobs(st, case):
    T, V, K, scale = case["tokens"], case["vocab"], case["top"], case["scale"]
    logprobs, entropy, ids, values, grads = [], [], [], [], []
    step = max(1, 33554432 // V)
    for a in range(0, T, step):
        raw = st["logits"][a:a + step].double()
        token = st["tokens"][a:a + step]
        given = token >= 0
        onehot = torch.zeros_like(raw)
        onehot[given.nonzero()[:, 0], token[given]] = 1.0
        logp = raw * scale - torch.logsumexp(raw * scale, 1, keepdim=True)
        p = logp.exp()
        h = torch.special.entr(p).sum(1)
        finite = torch.nan_to_num(logp, neginf=0.0)
        logprobs.append((finite * onehot).sum(1))
        entropy.append(h)
        left = raw.clone()
        for _ in range(K):
            v = left.max(1, keepdim=True)[0]
            first = (left == v).to(torch.int8).argmax(1, keepdim=True)
            ids.append(torch.where(v > -math.inf, first, -1)[:, 0])
            values.append(torch.where(v > -math.inf, logp.gather(1, first), -math.inf)[:, 0])
            left.scatter_(1, first, -math.inf)
        if K:
            ids[-K:] = [torch.stack(ids[-K:], 1)]
            values[-K:] = [torch.stack(values[-K:], 1)]
        if case["grad"]:
            d = st["d_logprobs"][a:a + step].double()[:, None] * given[:, None]
            dh = st["d_entropy"][a:a + step].double()[:, None]
            grads.append(scale * (d * (onehot - p) - dh * p * (finite + h[:, None])))
    out = [torch.cat(logprobs), torch.cat(entropy)]
    if K:
        out += [torch.cat(ids), torch.cat(values)]
    return out + ([torch.cat(grads)] if case["grad"] else [])


def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if op == "embed":
        wide = torch.cat((st["table"].new_zeros((1, case["width"])), st["table"]))   # row 0: no token
        return torch.cat([wide[i + 1].double() * st["scale"] for i in st["ids"].split(8192)])
    if op == "embed_grad":
        ids, order = torch.sort(st["ids"], stable=True)
        first = int((ids < 0).sum())
        ids, order = ids[first:], order[first:]
        out = torch.zeros((case["rows"], case["width"]), dtype=torch.float64, device="cuda")
        named, counts = torch.unique_consecutive(ids, return_counts=True)
        step = max(1, 67108864 // max(1, len(ids)))
        for c in range(0, case["width"], step):   # sums of runs, as differences of running sums
            d = torch.nn.functional.pad(st["d_out"][order, c:c + step].double().cumsum(0), (0, 0, 1, 0))
            ends = counts.cumsum(0)
            out[named, c:c + step] = (d[ends] - d[ends - counts]) * st["scale"]
        return out
    if op == "logprobs":
        return _exact_logprobs(st, case)
    T, K, N, E = case["tokens"], case["ins"], case["outs"], case["experts"]
    w_gate, w_up = (st[k].reshape(-1, N, K) for k in ("w_gate", "w_up"))
    ends = st["offsets"].tolist() if E else [0, T]
    if op == "gated":
        gate = torch.cat([st["x"][ends[e]:ends[e + 1]].double() @ w_gate[e].double().T for e in range(len(w_gate))])
        up = torch.cat([st["x"][ends[e]:ends[e + 1]].double() @ w_up[e].double().T for e in range(len(w_up))])
        h = _exact_act(gate, case["act"]) * up
        return [h, gate, up] if case["keep"] else [h]
    dx, dwg, dwu = [], [], []
    for e in range(len(w_gate)):
        rows = slice(ends[e], ends[e + 1])
        gate, up, dh, x = (st[k][rows].double() for k in ("gate", "up", "dh", "x"))
        d_gate, d_up = dh * up * _exact_slope(gate, case["act"]), dh * _exact_act(gate, case["act"])
        both = torch.cat((d_gate, d_up), 1)
        dx.append(both @ torch.cat((w_gate[e], w_up[e])).double())
        dw = both.T @ x
        dwg.append(dw[:N])
        dwu.append(dw[N:])
    shape = st["w_gate"].shape
    return [torch.cat(dx), torch.stack(dwg).view(shape), torch.stack(dwu).view(shape)]


def _distinct(tokens, rows):
    """How many distinct rows the tokens name, about."""
    u = np.random.default_rng(0).random(tokens)
    return len(np.unique(np.clip(np.exp(u * math.log(rows + 1)).astype(np.int64) - 1, 0, rows - 1)))


def _seen(experts, rows):
    """How many of the experts get at least one of the rows, on average: only their matrices are read."""
    if not experts:
        return 1.0
    rng = np.random.default_rng(0)
    ids = (rng.standard_normal((8, rows, experts)) + rng.standard_normal((8, 1, experts))).argmax(2)
    return float(np.mean([len(np.unique(v)) for v in ids]))


def work(case):
    op, b, T = case["op"], SIZE[case["type"]], case["tokens"]
    if op == "embed":
        D = case["width"]
        return {"bytes": 8 * T + (T + _distinct(T, case["rows"])) * D * b, "flops": T * D}
    if op == "embed_grad":
        D = case["width"]
        return {"bytes": 8 * T + (T + case["rows"]) * D * b, "flops": 2 * T * D}
    if op == "logprobs":
        n, K = T * case["vocab"], case["top"]
        # the softmax of a row is known only once it has been read, but a row fits on the chip: read and written once
        return {"bytes": n * b * (2 if case["grad"] else 1) + T * (16 + 12 * K) + (8 * T if case["grad"] else 0),
                "flops": n * (12 if case["grad"] else 6)}
    K, N = case["ins"], case["outs"]
    matrices = int(2 * N * K * b * _seen(case["experts"], T))
    if op == "gated":
        return {"bytes": matrices + T * (K + (3 if case["keep"] else 1) * N) * b, "flops": 4 * T * N * K}
    return {"bytes": matrices + 2 * max(1, case["experts"]) * N * K * b + T * (2 * K + 3 * N) * b,
            "flops": 8 * T * N * K}
