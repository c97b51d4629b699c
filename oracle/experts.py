"""FP64 definitions of the expert operators: routing by scores and groups, the
expert-sorted row layout, the experts' products and the projection with
low-rank adapters.

TEST INFRASTRUCTURE ONLY, like the rest of this package: it shares no code
with the CUDA library.  Every floating-point step is IEEE double; results are
returned unrounded, with the sums of absolute terms that forward-error bounds
need.  The functions are written as loops over tokens, experts and adapters
and are pinned by ``tests/test_oracle_experts.py``.
"""

from __future__ import annotations

import numpy as np

from .oracle import bf16_bits_to_f64

__all__ = ["group_topk_route", "expert_map", "silu", "expert_linear", "adapter_linear"]


def group_topk_route(logits, k, scale, bias=None, n_group=1, topk_group=1, group_top=2, scores="sigmoid",
                     renormalize=True):
    """ids [T, k] int32 and weights [T, k] float64 of the score routing: one
    token after the other, one choice after the other."""
    lg = np.asarray(logits, np.float32).astype(np.float64)
    T, E = lg.shape
    size = E // n_group
    ids = np.zeros((T, k), np.int32)
    w = np.zeros((T, k))
    b = None if bias is None else np.asarray(bias, np.float32).astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        for t in range(T):
            z = np.where(np.isnan(lg[t]), -np.inf, lg[t])
            if scores == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-z))
            else:
                m = z.max()
                e = np.where(z == m, 1.0, np.exp(z - m)) if m > -np.inf else np.zeros(E)
                s = e / e.sum() if e.sum() > 0 else e
            if b is None:
                key, val = z, (z if group_top == 1 else s)
            else:
                key = s + b
                key = np.where(np.isnan(key), -np.inf, key)
                val = key
            groups = []
            for g in range(n_group):
                v = -np.sort(-val[g * size:(g + 1) * size])
                gs = v[0] + v[1] if group_top == 2 and size > 1 else v[0]
                groups.append(-np.inf if np.isnan(gs) else gs)
            left = list(range(n_group))
            inside = np.zeros(E, bool)
            for _ in range(topk_group):
                g = max(left, key=lambda i: (groups[i], -i))
                left.remove(g)
                inside[g * size:(g + 1) * size] = True
            free = [i for i in range(E) if inside[i]]
            for j in range(k):
                i = max(free, key=lambda i: (key[i], -i))
                free.remove(i)
                ids[t, j], w[t, j] = i, s[i]
            if renormalize:
                total = w[t].sum()
                w[t] = w[t] / total if total > 0 else 0.0
    return ids, scale * w


def expert_map(topk_ids, E, block=1, n_rows=None):
    """(row_map, row_token, offsets, counts) of the expert-sorted layout."""
    ids = np.asarray(topk_ids)
    T, k = ids.shape
    need = T * k + min(E, T * k) * (block - 1)
    n_rows = need if n_rows is None else n_rows
    row_map = np.full((T, k), -1, np.int32)
    row_token = np.full(n_rows, -1, np.int32)
    offsets, counts = np.zeros(E + 1, np.int32), np.zeros(E, np.int32)
    at = 0
    for e in range(E):
        offsets[e] = at
        for t, j in zip(*np.nonzero(ids == e)):  # row-major: ascending (token, slot)
            row_map[t, j] = at + counts[e]
            row_token[at + counts[e]] = t
            counts[e] += 1
        at += -(-counts[e] // block) * block
    offsets[E] = at
    return row_map, row_token, offsets, counts


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def _activate(y, S, dy, act):
    """act(y) and the first-order image of the error dy of y."""
    if act is None:
        return y, dy
    h = y.shape[-1] // 2
    g, u, dg, du = y[..., :h], y[..., h:], dy[..., :h], dy[..., h:]
    sg = silu(g)
    # |silu'| <= 1.1; second-order term kept
    return sg * u, 1.1 * dg * np.abs(u) + np.abs(sg) * du + 1.1 * dg * du


def expert_linear(x_bits, w_bits, offsets, counts, row_token=None, act=None, rel=0.0):
    """Dict of unrounded rows: {row: (values, error bound)} over the segments;
    the bound is the image of an error of rel * sum|terms| in every sum."""
    x = bf16_bits_to_f64(x_bits)
    out = {}
    for e in range(len(counts)):
        if counts[e] == 0:
            continue
        w = bf16_bits_to_f64(w_bits[e])
        rows = np.arange(offsets[e], offsets[e] + counts[e])
        src = rows if row_token is None else row_token[rows]
        xr = x[src]
        y, S = xr @ w.T, np.abs(xr) @ np.abs(w).T
        val, err = _activate(y, S, rel * S, act)
        for i, r in enumerate(rows):
            out[int(r)] = (val[i], err[i])
    return out


def adapter_linear(x_bits, w_bits, a_bits, b_bits, ids, scale, act=None, rel=0.0, rel_low=0.0):
    """(values, error bound) [T, N or N/2]; rel as in expert_linear, rel_low
    the relative rounding of the low-rank product."""
    x, w = bf16_bits_to_f64(x_bits), bf16_bits_to_f64(w_bits)
    y, S = x @ w.T, np.abs(x) @ np.abs(w).T
    dy = rel * S
    for t, a in enumerate(ids):
        if a < 0 or a >= len(scale):
            continue
        A, B = bf16_bits_to_f64(a_bits[a]), bf16_bits_to_f64(b_bits[a])
        sc = float(np.float32(scale[a]))
        v, Sv = sc * (A @ x[t]), abs(sc) * (np.abs(A) @ np.abs(x[t]))
        dv = rel * Sv + rel_low * np.abs(v)
        y[t] += B @ v
        dy[t] += np.abs(B) @ dv + rel * (np.abs(B) @ np.abs(v))
    return _activate(y, None, dy, act)
