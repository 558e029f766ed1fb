"""CPU oracle of the routed-expert operators: the router's choice, tokens sorted by expert, the exchange of
rows with its gradients, and products with 4-bit weights.

TEST INFRASTRUCTURE ONLY.  It shares no code with the GPU library.  Plain numpy in float64, following the
definitions step by step:

  p = softmax(l) over the experts with l > -inf (NaN: shut; +inf: the largest finite float32)
  s_j = the top best by (l desc, id asc);  w_j = p_{s_j}, or exp(l_{s_j}) / sum_m exp(l_{s_m})
  position = offsets[e] + (earlier valid entries of e);  rows[position[t][j]] = x[t]
  y[t] = sum_j w[t][j] rows[position[t][j]]
  W[n][k] = s[n][k // group] (q[n][k] - z[n][k // group]);  y = act(W x + b)
"""
from __future__ import annotations

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def _clean(logits):
    l = np.array(logits, np.float64)
    l[np.isnan(l)] = -np.inf
    return np.minimum(l, FLT_MAX)


def route(logits, top, renormalise):
    """(experts int32 [T, top], weights float64 [T, top], per-weight sensitivity [T, top]): the last is
    |l_s - max| + sum_i p_i |l_i - max|, the relative error of a weight per relative error of a difference."""
    l = _clean(logits)
    T, E = l.shape
    ids = np.full((T, top), -1, np.int32)
    w = np.zeros((T, top))
    sens = np.zeros((T, top))
    for t in range(T):
        best = [e for e in sorted(range(E), key=lambda e: (-l[t, e], e)) if l[t, e] > -np.inf][:top]
        if not best:
            continue
        pool = np.array(best) if renormalise else np.nonzero(l[t] > -np.inf)[0]
        m = l[t, best[0]]
        e = np.exp(l[t, pool] - m)
        spread = float(np.sum(e * (m - l[t, pool])) / e.sum())
        ids[t, :len(best)] = best
        w[t, :len(best)] = np.exp(l[t, best] - m) / e.sum()
        sens[t, :len(best)] = (m - l[t, best]) + spread
    return ids, w, sens


def route_backward(logits, ids, w, dw, renormalise):
    """(d_logits float64 [T, E], magnitude [T, E], sensitivity [T, E]) given the weights w as they were returned."""
    l = _clean(logits)
    T, E = l.shape
    d, mag, sens = np.zeros((T, E)), np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        ok = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        dot = sum(w[t, j] * dw[t, j] for j in ok)
        adot = sum(abs(w[t, j] * dw[t, j]) for j in ok)
        if renormalise:
            for j in ok:
                d[t, ids[t, j]] += w[t, j] * (dw[t, j] - dot)
                mag[t, ids[t, j]] += w[t, j] * (abs(dw[t, j]) + adot)
            continue
        open_ = l[t] > -np.inf
        if not open_.any():
            continue
        m = l[t].max()
        e = np.where(open_, np.exp(l[t] - m), 0.0)
        p = e / e.sum()
        g, ag = np.zeros(E), np.zeros(E)
        for j in ok:
            g[ids[t, j]] += dw[t, j]
            ag[ids[t, j]] += abs(dw[t, j])
        d[t] = p * (g - dot)
        mag[t] = p * (ag + adot)
        away = np.where(open_, m - np.where(open_, l[t], m), 0.0)
        sens[t] = away + float(np.sum(p * away))
    return d, mag, sens


def sort(experts, n_experts):
    """(offsets int32 [E + 1], order int32 [T * top], position int32 [T, top])."""
    flat = np.asarray(experts).reshape(-1)
    lists = [[] for _ in range(n_experts)]
    for i, e in enumerate(flat.tolist()):
        if 0 <= e < n_experts:
            lists[e].append(i)
    offsets, order, position = [0], np.full(flat.shape, -1, np.int32), np.full(flat.shape, -1, np.int32)
    for v in lists:
        for r, i in enumerate(v, start=offsets[-1]):
            order[r], position[i] = i, r
        offsets.append(offsets[-1] + len(v))
    return np.array(offsets, np.int32), order, position.reshape(np.asarray(experts).shape)


def dispatch(x, position, rows):
    """rows, changed in place where an entry names them."""
    for t in range(position.shape[0]):
        for p in position[t]:
            if 0 <= p < rows.shape[0]:
                rows[p] = x[t]
    return rows


def combine(rows, position, weights):
    """(y float64, sum of magnitudes float64)."""
    T, K = position.shape
    y, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(K):
            if 0 <= position[t, j] < rows.shape[0]:
                v = (1.0 if weights is None else float(weights[t, j])) * rows[position[t, j]].astype(np.float64)
                y[t] += v
                mag[t] += np.abs(v)
    return y, mag


def combine_backward(dy, rows, position, weights, d_rows):
    """(d_rows float64, changed where an entry names them; d_weights; magnitude of d_weights)."""
    T, K = position.shape
    dw, mag = np.zeros((T, K)), np.zeros((T, K))
    for t in range(T):
        g = dy[t].astype(np.float64)
        for j in range(K):
            p = position[t, j]
            if 0 <= p < rows.shape[0]:
                r = rows[p].astype(np.float64)
                d_rows[p] = float(weights[t, j]) * g
                dw[t, j] = float(g @ r)
                mag[t, j] = float(np.abs(g) @ np.abs(r))
    return d_rows, dw, mag


def unpack(nibbles, n_in):
    """q [.., n_in] from bytes holding two (even input in the low half)."""
    b = np.asarray(nibbles)
    q = np.empty(b.shape[:-1] + (2 * b.shape[-1],), np.uint8)
    q[..., 0::2], q[..., 1::2] = b & 15, b >> 4
    return q[..., :n_in]


def linear(x, q, scales, zeros, group, offsets, bias, relu, y):
    """(y float64, changed where a matrix names a row; magnitude sum_g |s| sum_k |x| (q + z) + |b|).  q [M, N, K]."""
    M, N, K = q.shape
    mag = np.zeros(y.shape)
    ends = [0, x.shape[0]] if offsets is None else np.clip(offsets, 0, x.shape[0]).tolist()
    for e in range(M):
        a, b = ends[e], ends[e + 1]
        if a >= b:
            continue
        z = np.full(scales[e].shape, 8.0) if zeros is None else zeros[e].astype(np.float64)
        s = np.repeat(scales[e].astype(np.float64), group, 1)[:, :K]
        z = np.repeat(z, group, 1)[:, :K]
        qe = q[e].astype(np.float64)
        xe = x[a:b].astype(np.float64)
        v = xe @ ((qe - z) * s).T
        mag[a:b] = np.abs(xe) @ ((qe + z) * np.abs(s)).T
        if bias is not None:
            v = v + bias[e].astype(np.float64)
            mag[a:b] += np.abs(bias[e].astype(np.float64))
        y[a:b] = np.where(v < 0, 0.0, v) if relu else v
    return y, mag
