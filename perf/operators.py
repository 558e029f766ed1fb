"""Cases of the routed-expert operators: the router's choice, tokens sorted by expert, the exchange of rows
with its gradient, and products with 4-bit weights (dense, and one matrix per expert).

Every case runs in its plain form (``own`` false: elementary torch operations in float32, rounded once at
the end) or through the library's entry points (``own`` true).  The same inputs feed both.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the 2048 candidates that a search returned for one query, each sent to 2 of 8 scorers
        {"name": "route_one_query", "op": "route", "tokens": 2048, "experts": 8, "top": 2, "type": "f32",
         "renormalise": True, "masked": 0.0, "grad": False},
        # a training step of the router over 32 queries' candidates: choice, weights, gradient of the logits
        {"name": "route_train", "op": "route", "tokens": 65536, "experts": 64, "top": 8, "type": "bf16",
         "renormalise": False, "masked": 0.05, "grad": True},
        # one serving step of 64 requests
        {"name": "sort_step", "op": "sort", "tokens": 64, "experts": 32, "top": 4, "dropped": 0.1},
        # 256 queries' 2048 candidates each
        {"name": "sort_batch", "op": "sort", "tokens": 524288, "experts": 64, "top": 2, "dropped": 0.0},
        # one query's candidates to the experts and back, rows as wide as the index's embeddings
        {"name": "exchange_one_query", "op": "exchange", "tokens": 2048, "width": 128, "experts": 8, "top": 2,
         "type": "f16"},
        # 32 queries' candidates with hidden rows
        {"name": "exchange_batch", "op": "exchange", "tokens": 65536, "width": 1024, "experts": 64, "top": 2,
         "type": "bf16"},
        # gradients at sizes that fill no tile, float32 as the rerank's weights
        {"name": "exchange_grad_odd", "op": "exchange_grad", "tokens": 2047, "width": 250, "experts": 12, "top": 3,
         "type": "f32"},
        # gradients of a training step
        {"name": "exchange_grad_batch", "op": "exchange_grad", "tokens": 32768, "width": 1024, "experts": 64,
         "top": 4, "type": "bf16"},
        # one token through a large layer: the weights' bytes are the cost
        {"name": "linear_one", "op": "linear", "rows": 1, "outs": 16384, "ins": 4096, "group": 128, "type": "bf16",
         "scales": "bf16", "zeros": False, "relu": False},
        # a few tokens, sizes that end inside tiles and groups, with the fused epilogue
        {"name": "linear_ragged", "op": "linear", "rows": 13, "outs": 1000, "ins": 1000, "group": 64, "type": "f16",
         "scales": "f16", "zeros": True, "relu": True},
        # a serving step: 32 tokens, 2 of 64 experts each, most experts see one row, some none
        {"name": "experts_step", "op": "experts", "rows": 64, "experts": 64, "outs": 2048, "ins": 1024, "group": 64,
         "type": "bf16", "scales": "bf16", "zeros": True, "relu": True},
        # one query's 2048 candidates to 2 of 8 experts each
        {"name": "experts_query", "op": "experts", "rows": 4096, "experts": 8, "outs": 1024, "ins": 256, "group": 32,
         "type": "f16", "scales": "f32", "zeros": False, "relu": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "sort", "exchange", "exchange_grad", "linear", "experts"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op in ("route", "sort"):
        experts = _log(rng, 2, 256)
        top = rng.randint(1, min(8, experts))
        if op == "sort":
            return {"op": op, "tokens": _log(rng, 1, 1048576 // top), "experts": experts, "top": top,
                    "dropped": rng.choice([0.0, 0.0, 0.3])}
        return {"op": op, "tokens": _log(rng, 1, 65536 * 64 // max(64, experts)), "experts": experts, "top": top,
                "type": kind, "renormalise": rng.random() < 0.5, "masked": rng.choice([0.0, 0.05, 0.5]),
                "grad": rng.random() < 0.5}
    if op in ("exchange", "exchange_grad"):
        width = _log(rng, 16, 4096)
        experts = _log(rng, 2, 128)
        top = rng.randint(1, min(6, experts))
        most = 96 * 1024 * 1024 // (width * (1 + 2 * top))
        return {"op": op, "tokens": _log(rng, 1, min(65536, most)), "width": width, "experts": experts, "top": top,
                "type": kind}
    group = rng.choice([32, 64, 128])
    case = {"op": op, "group": group, "type": kind, "scales": rng.choice(["f32", "f16", "bf16"]),
            "zeros": rng.random() < 0.5, "relu": rng.random() < 0.5}
    if op == "linear":
        case.update(rows=_log(rng, 1, 64), outs=_log(rng, 16, 16384), ins=_log(rng, 16, 4096))
    else:
        case.update(rows=_log(rng, 1, 1024), experts=rng.randint(2, 64), outs=_log(rng, 64, 2048),
                    ins=_log(rng, 64, 1024))
    return case


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _choice(g, tokens, experts, top, dropped=0.0):
    """Distinct experts per token, some experts liked more than others; dropped entries are -1."""
    liked = torch.randn(experts, generator=g, device="cuda")
    score = torch.randn((tokens, experts), generator=g, device="cuda") + liked
    ids = torch.sort(score, dim=1, descending=True)[1][:, :top].to(torch.int32)
    if dropped:
        gone = torch.rand((tokens, top), generator=g, device="cuda") < dropped
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.contiguous()


def _inputs(case, seed):
    g = _gen(seed)
    op, dt = case["op"], TYPES.get(case.get("type"))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if op == "route":
        T, E = case["tokens"], case["experts"]
        logits = 1.5 * normal(T, E) + 0.5 * normal(E)
        if case["masked"]:
            shut = torch.rand((T, E), generator=g, device="cuda") < case["masked"]
            logits = torch.where(shut, torch.full_like(logits, -math.inf), logits)
        return {"logits": logits.to(dt), "d_weights": normal(T, case["top"])}
    if op == "sort":
        return {"experts": _choice(g, case["tokens"], case["experts"], case["top"], case["dropped"])}
    if op in ("exchange", "exchange_grad"):
        T, D, K = case["tokens"], case["width"], case["top"]
        st = {"experts": _choice(g, T, case["experts"], K)}
        w = torch.rand((T, K), generator=g, device="cuda") + 0.05
        st["weights"] = w / w.sum(1, keepdim=True)
        st["x" if op == "exchange" else "dy"] = normal(T, D).to(dt)
        st["rows"] = normal(T * K, D).to(dt)
        if op == "exchange_grad":
            st["d_rows"] = normal(T * K, D).to(dt)
            order, position, offsets = _sorted(st["experts"], case["experts"])
            st["position"] = position
        return st
    E, R, N, K, G = case.get("experts", 1), case["rows"], case["outs"], case["ins"], case["group"]
    groups = -(-K // G)
    q = torch.empty((E, N, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, N, groups), dtype=TYPES[case["scales"]], device="cuda")
    z = torch.empty((E, N, groups), dtype=torch.uint8, device="cuda") if case["zeros"] else None
    for e in range(E):   # weights of a layer, quantised group by group
        w = torch.zeros((N, groups * G), device="cuda")
        w[:, :K] = normal(N, K) / math.sqrt(K)
        w = w.view(N, groups, G)
        if case["zeros"]:
            lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
            se = ((hi - lo) / 15).to(s.dtype).float()
            ze = torch.round(-lo / se).clamp(0, 15)
            z[e] = ze.to(torch.uint8)
        else:
            se = (w.abs().amax(2) / 7).to(s.dtype).float()
            ze = torch.full_like(se, 8.0)
        s[e] = se.to(s.dtype)
        qe = (torch.round(w / se[..., None]) + ze[..., None]).clamp(0, 15)
        q[e] = qe.view(N, groups * G)[:, :K].to(torch.uint8)
    if K % 2:
        q = torch.nn.functional.pad(q, (0, 1))
    st = {"nibbles": q[..., 0::2] | (q[..., 1::2] << 4), "scales": s, "zeros": z,
          "x": normal(R, K).to(dt), "bias": 0.1 * normal(E, N) if case["relu"] else None, "offsets": None}
    if op == "experts":
        ids = _choice(g, R, E, 1)
        st["offsets"] = _sorted(ids, E)[2]
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if case["op"] in ("linear", "experts") and own:
        from int8_ivf_ann_amd import svt
        st["packed"] = svt.svt_quant_pack(st["nibbles"], st["scales"], st["zeros"], case["ins"], case["group"])
    st["case"] = case
    return st


# ---- plain forms -------------------------------------------------------------------------------------

def _sorted(ids, experts):
    """order [T*K]: the sorted entries' flat indexes (-1 behind the last); position [T, K]: where each entry
    went (-1: dropped); offsets [E + 1]."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= experts), torch.full_like(flat, experts), flat)
    by, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(by, torch.arange(experts + 1, device=ids.device))
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    position = torch.where(key < experts, place, torch.full_like(place, -1)).view(ids.shape)
    order = torch.where(by < experts, order, torch.full_like(order, -1))
    return order.to(torch.int32), position.to(torch.int32), offsets.to(torch.int32)


def _plain_route(st, case):
    x = st["logits"].float()
    K = case["top"]
    value, ids = torch.sort(x, dim=1, descending=True, stable=True)
    value, ids = value[:, :K], ids[:, :K]
    shut = value == -math.inf
    top = torch.where(shut[:, :1], torch.zeros_like(value[:, :1]), value[:, :1])
    e = torch.exp(value - top)
    everything = torch.exp(x - top)
    total = (e if case["renormalise"] else everything).sum(1, keepdim=True)
    total = torch.where(total == 0, torch.ones_like(total), total)
    weights = e / total
    out = [torch.where(shut, torch.full_like(ids, -1), ids).to(torch.int32), weights]
    if case["grad"]:
        dw = torch.where(shut, torch.zeros_like(weights), st["d_weights"])
        dot = (dw * weights).sum(1, keepdim=True)
        if case["renormalise"]:
            d = torch.zeros_like(x)
        else:
            d = -everything / total * dot
        d.scatter_add_(1, ids, weights * (dw - dot if case["renormalise"] else dw))
        out.append(d.to(st["logits"].dtype))
    return out


def _plain_exchange(st, case):
    order, position, offsets = _sorted(st["experts"], case["experts"])
    T, K = position.shape
    sent = st["x"][(order // K).long()]
    y = torch.zeros(st["x"].shape, device="cuda")
    for j in range(K):
        y += st["weights"][:, j:j + 1] * st["rows"][position[:, j].long()].float()
    return sent, y.to(st["x"].dtype)


def _plain_exchange_grad(st, case):
    position, dy = st["position"].long(), st["dy"].float()
    T, K = position.shape
    d_rows = torch.empty(st["rows"].shape, device="cuda", dtype=st["rows"].dtype)
    d_weights = torch.empty((T, K), device="cuda")
    dx = torch.zeros_like(dy)
    for j in range(K):
        at = position[:, j]
        d_rows[at] = (st["weights"][:, j:j + 1] * dy).to(d_rows.dtype)
        d_weights[:, j] = (dy * st["rows"][at].float()).sum(1)
        dx += st["d_rows"][at].float()
    return d_rows, d_weights, dx.to(st["dy"].dtype)


def _plain_weights(st, case, e):
    K, G = case["ins"], case["group"]
    b = st["nibbles"][e]
    q = torch.stack((b & 15, b >> 4), 2).reshape(b.shape[0], -1)[:, :K].float()
    s = st["scales"][e].float().repeat_interleave(G, 1)[:, :K]
    z = 8.0 if st["zeros"] is None else st["zeros"][e].float().repeat_interleave(G, 1)[:, :K]
    return (q - z) * s


def _plain_linear(st, case):
    E = st["nibbles"].shape[0]
    x = st["x"].float()
    y = torch.zeros((x.shape[0], case["outs"]), device="cuda")
    ends = [0, x.shape[0]] if st["offsets"] is None else st["offsets"].tolist()
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a < b:
            y[a:b] = x[a:b] @ _plain_weights(st, case, e).t()
            if case["relu"]:
                y[a:b] += st["bias"][e]
    if case["relu"]:
        y = torch.where(y < 0, torch.zeros_like(y), y)
    return y.to(st["x"].dtype)


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "route":
            return _plain_route(state, case)
        if op == "sort":
            order, position, offsets = _sorted(state["experts"], case["experts"])
            return offsets, order, position
        if op == "exchange":
            return _plain_exchange(state, case)
        if op == "exchange_grad":
            return _plain_exchange_grad(state, case)
        return _plain_linear(state, case)
    from int8_ivf_ann_amd import svt
    if op == "route":
        ids, weights = svt.svt_route(state["logits"], case["top"], renormalise=case["renormalise"])
        if not case["grad"]:
            return [ids, weights]
        d = svt.svt_route_backward(state["logits"], ids, weights, state["d_weights"],
                                   renormalise=case["renormalise"])
        return [ids, weights, d]
    if op == "sort":
        return svt.svt_expert_sort(state["experts"], case["experts"])
    if op == "exchange":
        offsets, order, position = svt.svt_expert_sort(state["experts"], case["experts"])
        sent = svt.svt_expert_dispatch(state["x"], position)
        return sent, svt.svt_expert_combine(state["rows"], position, state["weights"])
    if op == "exchange_grad":
        d_rows, d_weights = svt.svt_expert_combine_backward(state["dy"], state["rows"], state["position"],
                                                            state["weights"])
        return d_rows, d_weights, svt.svt_expert_dispatch_backward(state["d_rows"], state["position"])
    return svt.svt_quant_linear(state["x"], state["packed"], offsets=state["offsets"], bias=state["bias"],
                                activation="relu" if case["relu"] else "none")


# ---- the definition in 64 bits -----------------------------------------------------------------------

def exact(case, seed):
    st = {k: (v.cpu() if isinstance(v, torch.Tensor) else v) for k, v in _inputs(case, seed).items()} \
        if case["op"] in ("route", "sort") else _inputs(case, seed)
    op = case["op"]
    if op == "route":
        x = st["logits"].double().numpy()
        T, E = x.shape
        K = case["top"]
        best = np.argsort(-x, axis=1, kind="stable")[:, :K]
        picked = np.take_along_axis(x, best, 1)
        open_ = picked > -np.inf
        with np.errstate(divide="ignore", invalid="ignore"):
            base = picked if case["renormalise"] else x
            m = x.max(1, keepdims=True)
            m[~np.isfinite(m)] = 0.0
            log_z = m + np.log(np.exp(base - m).sum(1, keepdims=True))
            w = np.where(open_, np.exp(picked - log_z), 0.0)
            out = [torch.from_numpy(np.where(open_, best, -1).astype(np.int32)), torch.from_numpy(w)]
            if case["grad"]:
                g = np.where(open_, st["d_weights"].double().numpy(), 0.0)
                mean = (g * w).sum(1, keepdims=True)
                chosen = np.zeros((T, E))
                np.put_along_axis(chosen, best, np.where(open_, g, 0.0), 1)
                if case["renormalise"]:
                    p = np.zeros((T, E))
                    np.put_along_axis(p, best, w, 1)
                else:
                    p = np.where(x > -np.inf, np.exp(x - log_z), 0.0)
                out.append(torch.from_numpy(p * (chosen - mean)))
        return out
    if op == "sort":
        ids = st["experts"].numpy().reshape(-1)
        lists = [np.nonzero(ids == e)[0] for e in range(case["experts"])]
        offsets = np.cumsum([0] + [len(v) for v in lists]).astype(np.int32)
        order = np.full(ids.shape, -1, np.int32)
        order[:offsets[-1]] = np.concatenate(lists)
        position = np.full(ids.shape, -1, np.int32)
        position[order[:offsets[-1]]] = np.arange(offsets[-1])
        return tuple(torch.from_numpy(v) for v in (offsets, order, position.reshape(st["experts"].shape)))
    if op in ("exchange", "exchange_grad"):
        ids = st["experts"].cpu().numpy()
        T, K = ids.shape
        order = np.concatenate([np.nonzero(ids.reshape(-1) == e)[0] for e in range(case["experts"])])
        at = np.empty(T * K, np.int64)
        at[order] = np.arange(T * K)
        at = torch.from_numpy(at.reshape(T, K)).cuda()
        if op == "exchange":
            sent = torch.empty((T * K, case["width"]), dtype=st["x"].dtype, device="cuda")
            sent[at.reshape(-1)] = st["x"].repeat_interleave(K, 0)
            y = torch.empty((T, case["width"]), dtype=torch.float64, device="cuda")
            for a in range(0, T, 4096):
                y[a:a + 4096] = (st["rows"][at[a:a + 4096]].double() * st["weights"][a:a + 4096, :, None].double()).sum(1)
            return sent, y
        d_rows = torch.empty((T * K, case["width"]), dtype=torch.float64, device="cuda")
        d_w = torch.empty((T, K), dtype=torch.float64, device="cuda")
        dx = torch.empty((T, case["width"]), dtype=torch.float64, device="cuda")
        for a in range(0, T, 4096):
            dy, to = st["dy"][a:a + 4096].double(), at[a:a + 4096]
            d_rows[to] = st["weights"][a:a + 4096, :, None].double() * dy[:, None, :]
            d_w[a:a + 4096] = (st["rows"][to].double() * dy[:, None, :]).sum(2)
            dx[a:a + 4096] = st["d_rows"][to].double().sum(1)
        return d_rows, d_w, dx
    K, G, E = case["ins"], case["group"], st["nibbles"].shape[0]
    out = []
    ends = [0, case["rows"]] if st["offsets"] is None else st["offsets"].tolist()
    for e in range(E):
        x = st["x"][ends[e]:ends[e + 1]].double()
        if not len(x):
            continue
        y = torch.zeros((len(x), case["outs"]), dtype=torch.float64, device="cuda")
        for g in range(-(-K // G)):
            k = range(g * G, min(K, g * G + G))
            both = st["nibbles"][e][:, g * G // 2:(k[-1] // 2) + 1].double()
            high = torch.floor(both / 16)
            low = both - 16 * high
            zero = 8.0 if st["zeros"] is None else st["zeros"][e][:, g].double()[:, None]
            scale = st["scales"][e][:, g].double()[:, None]
            xg = x[:, k[0]:k[-1] + 1]
            y += (xg[:, 0::2] @ ((low - zero) * scale).t())
            if len(k) > 1:
                y += (xg[:, 1::2] @ ((high - zero) * scale)[:, :len(k) // 2].t())
        if case["relu"]:
            y = torch.clamp(y + st["bias"][e].double(), min=0)
        out.append(y)
    return torch.cat(out)


def _seen(experts, rows):
    """How many of the experts get at least one of the rows, on average: only their matrices are read."""
    if experts == 1:
        return 1.0
    rng = np.random.default_rng(0)
    liked = rng.standard_normal((16, 1, experts))
    ids = (rng.standard_normal((16, rows, experts)) + liked).argmax(2)
    return float(np.mean([len(np.unique(v)) for v in ids]))


def work(case):
    op = case["op"]
    b = {"f32": 4, "f16": 2, "bf16": 2}.get(case.get("type"))
    if op == "route":
        T, E, K = case["tokens"], case["experts"], case["top"]
        grad = T * E * b + T * K * 4 if case["grad"] else 0
        return {"bytes": T * E * b + T * K * 8 + grad, "flops": T * E * (8 if case["grad"] else 4)}
    if op == "sort":
        n = case["tokens"] * case["top"]
        return {"bytes": 12 * n + 4 * (case["experts"] + 1), "flops": 2 * n}
    if op == "exchange":
        T, D, K = case["tokens"], case["width"], case["top"]
        return {"bytes": T * D * b * (2 + 2 * K) + T * K * 8, "flops": 2 * T * K * D}
    if op == "exchange_grad":
        T, D, K = case["tokens"], case["width"], case["top"]
        return {"bytes": T * D * b * (2 + 3 * K) + T * K * 12, "flops": 4 * T * K * D}
    E, R, N, K, G = case.get("experts", 1), case["rows"], case["outs"], case["ins"], case["group"]
    sb = {"f32": 4, "f16": 2, "bf16": 2}[case["scales"]] + (1 if case["zeros"] else 0)
    matrix = N * ((K + 1) // 2) + N * (-(-K // G)) * sb + (4 * N if case["relu"] else 0)
    return {"bytes": int(_seen(E, R) * matrix) + R * (K + N) * b, "flops": 2 * R * N * K}
