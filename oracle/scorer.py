"""CPU oracle of the trained scorer's operators: embedding rows and their gradient, gated products and their
gradients, log probabilities of given tokens with entropy, best alternatives and gradient.

TEST INFRASTRUCTURE ONLY.  It shares no code with the GPU library.  Plain numpy in float64, following the
definitions step by step:

  out[i] = s table[ids[i]] (zeros outside);  d_table[v] = s sum_{i: ids[i] = v} d_out[i]
  z = s l over the tokens with l > -inf (NaN: shut; +inf: the largest finite float32);  p = softmax(z)
  logp = log p of the token;  H = -sum p log p;  dl_i = s (d ([i = t] - p_i) - dH p_i (log p_i + H))
  g = x Wg^T, u = x Wu^T, h = act(g) u;  dg = dh u act'(g), du = dh act(g),
  dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, row by row with the expert's matrices
"""
from __future__ import annotations

import math

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def embedding(table, ids, scale):
    out = np.zeros((len(ids), table.shape[1]))
    for i, v in enumerate(ids):
        if 0 <= v < len(table):
            out[i] = scale * table[v]
    return out


def embedding_backward(d_out, ids, n_rows, scale):
    """(d_table float64 [n_rows, D], sum of the parts' sizes, number of parts [n_rows])."""
    d, size, n = np.zeros((n_rows, d_out.shape[1])), np.zeros((n_rows, d_out.shape[1])), np.zeros(n_rows, np.int64)
    for i, v in enumerate(ids):
        if 0 <= v < n_rows:
            d[v] += scale * d_out[i]
            size[v] += abs(scale) * np.abs(d_out[i])
            n[v] += 1
    return d, size, n


class Row:
    """One row of logits: p, logp, entropy and what error bounds need."""

    def __init__(self, logits, scale):
        l = np.array(logits, np.float64)
        l[np.isnan(l)] = -np.inf
        self.l = l = np.minimum(l, FLT_MAX)
        self.open = l > -np.inf
        self.scale = scale
        n = len(l)
        self.p, self.logp = np.zeros(n), np.full(n, -np.inf)
        self.peak = self.log_z = self.entropy = 0.0
        self.away = np.zeros(n)      # (peak - l) scale of open tokens
        if self.open.any():
            self.peak = float(l[self.open].max())
            self.away[self.open] = (self.peak - l[self.open]) * scale
            e = np.where(self.open, np.exp(-self.away), 0.0)
            self.log_z = math.log(e.sum())
            self.logp[self.open] = -self.away[self.open] - self.log_z
            self.p = np.where(self.open, np.exp(self.logp), 0.0)
            self.entropy = float(-np.sum(self.p[self.p > 0] * self.logp[self.p > 0]))
        self.spread = float(np.sum(np.where(self.p > 0, self.p * self.away, 0.0)))

    def top(self, k):
        """(tokens int64 [k], logp [k])."""
        best = [i for i in np.lexsort((np.arange(len(self.l)), -self.l)) if self.open[i]][:k]
        ids, lp = np.full(k, -1, np.int64), np.full(k, -np.inf)
        ids[:len(best)] = best
        lp[:len(best)] = self.logp[best]
        return ids, lp

    def backward(self, token, d, dh):
        given = 0 <= token < len(self.l)
        d = d if given else 0.0
        lp = np.where(self.p > 0, self.logp, 0.0)
        g = -self.p * (d + dh * (lp + self.entropy))
        if given and self.open[token]:
            g[token] += d
        return self.scale * g


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activation(v, act):
    """Its value and slope."""
    if act == "none":
        return v, np.ones_like(v)
    if act == "relu":
        return np.maximum(v, 0.0), (v > 0).astype(np.float64)
    if act == "silu":
        s = np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))
        return v * s, s * (1.0 + v * (1.0 - s))
    cdf = 0.5 * _erfc(-v / math.sqrt(2.0))   # 1 + erf would lose the far end
    return v * cdf, cdf + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)


def _rows_of(n_rows, offsets, n_matrices):
    if offsets is None:
        return [(0, 0, n_rows)]
    ends = [min(max(int(o), 0), n_rows) for o in offsets]
    return [(e, ends[e], ends[e + 1]) for e in range(n_matrices) if ends[e] < ends[e + 1]]


def gated(x, w_gate, w_up, act, offsets=None):
    """(h, gate, up, sum |x||Wg|, sum |x||Wu|); w [M, N, K].  Rows that no matrix names: NaN."""
    out = [np.full((len(x), w_gate.shape[1]), np.nan) for _ in range(5)]
    for e, a, b in _rows_of(len(x), offsets, len(w_gate)):
        out[1][a:b], out[2][a:b] = x[a:b] @ w_gate[e].T, x[a:b] @ w_up[e].T
        out[3][a:b], out[4][a:b] = np.abs(x[a:b]) @ np.abs(w_gate[e]).T, np.abs(x[a:b]) @ np.abs(w_up[e]).T
        out[0][a:b] = activation(out[1][a:b], act)[0] * out[2][a:b]
    return out


def gated_backward(dh, x, w_gate, w_up, gate, up, act, offsets=None):
    """(dx, dWg, dWu) and of each the sum of its parts' sizes."""
    M = len(w_gate)
    dx, sx = np.full(x.shape, np.nan), np.full(x.shape, np.nan)
    dw = [np.zeros(w_gate.shape) for _ in range(4)]
    for e, a, b in _rows_of(len(x), offsets, M):
        value, slope = activation(gate[a:b], act)
        dg, du = dh[a:b] * up[a:b] * slope, dh[a:b] * value
        dx[a:b] = dg @ w_gate[e] + du @ w_up[e]
        sx[a:b] = np.abs(dg) @ np.abs(w_gate[e]) + np.abs(du) @ np.abs(w_up[e])
        dw[0][e], dw[1][e] = dg.T @ x[a:b], du.T @ x[a:b]
        dw[2][e], dw[3][e] = np.abs(dg).T @ np.abs(x[a:b]), np.abs(du).T @ np.abs(x[a:b])
    return dx, dw[0], dw[1], sx, dw[2], dw[3]
