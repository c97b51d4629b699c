"""FP64 definitions of microscaled 4-bit floating point: what codes and scales
stand for, the quantisation of a row, products.

TEST INFRASTRUCTURE ONLY, like the rest of this package: it shares no code
with the CUDA library.  Roundings are searches in the tables of all values;
pinned by ``tests/test_oracle_fp4.py``.
"""

from __future__ import annotations

import numpy as np

__all__ = ["FP4_BLOCK", "fp4_e2m1", "fp4_scale_values", "fp4_values", "fp4_quantize", "fp4_tiled_scales", "fp4_linear"]

FP4_BLOCK = {"nvfp4": 16, "mxfp4": 32}

# the values of the sixteen codes
fp4_e2m1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def fp4_scale_values(fmt):
    """float64 [256]: what each scale byte stands for (E4M3 without sign: the
    top bit is not part of the number)."""
    b = np.arange(256)
    if fmt == "mxfp4":
        v = np.exp2(b - 127.0)
        v[255] = np.nan
        return v
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 512.0, np.exp2(e - 7.0) * (1 + m / 8.0))
    v[(b & 127) == 127] = np.nan
    return v


def fp4_values(codes, scales, fmt, g=1.0):
    """float64 [.., K]: codes [.., K / 2] bytes times scales times g."""
    two = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    return fp4_e2m1[two] * np.repeat(fp4_scale_values(fmt)[scales], FP4_BLOCK[fmt], axis=-1) * g


def _nearest(v, table):
    """Index of the entry of an ascending table nearest to each v, between two the even one."""
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    below, above = v - table[lo], table[hi] - v
    return np.where(above < below, hi, np.where(below < above, lo, np.where(lo % 2 == 0, lo, hi)))


def fp4_quantize(x, fmt, g=1.0):
    """x [T, K] of BF16 numbers -> (codes [T, K / 2], scales [T, K / block])
    uint8, choices made on quotients in double precision: a quotient of these
    short numbers is a midpoint exactly or lies 2^-36 of itself beside it."""
    x = np.asarray(x, np.float64)
    b = x.reshape(len(x), -1, FP4_BLOCK[fmt])
    bad = ~np.isfinite(b).all(axis=2) | (not 2.0 ** -100 <= g <= 2.0 ** 100)
    b = np.where(bad[:, :, None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    table = fp4_scale_values(fmt)
    if fmt == "nvfp4":
        scales = _nearest(amax / (6.0 * g), table[:127])
    else:
        scales = np.clip(np.frexp(np.where(amax > 0, amax, 2.0 ** -140))[1] - 1 - 2 + 127, 0, 254)
    s = table[scales] * g
    v = np.abs(b) / np.where(s > 0, s, 1.0)[:, :, None]
    v = np.where((s > 0)[:, :, None], v, 0.0)
    # a block whose scale is zero has no codes; neither has one that is not finite
    keep = (s > 0) & ~bad
    code = np.where(keep[:, :, None], _nearest(v, fp4_e2m1[:8]) + 8 * np.signbit(b), 0).reshape(x.shape).astype(np.uint8)
    scales = np.where(bad, 0x7F if fmt == "nvfp4" else 0xFF, scales).astype(np.uint8)
    return code[:, 0::2] | code[:, 1::2] << 4, scales


def fp4_tiled_scales(scales, fmt, act):
    """scales [E, N, K / block] in the order of the products: [expert][tile of
    128 rows][256 elements of K][word of four scales][row % 32][row / 32][4],
    with SwiGLU 16 gate rows and their 16 up rows in turn; zeros elsewhere."""
    E, N, cols = scales.shape
    per = 256 // FP4_BLOCK[fmt]
    stages = -(-cols // per)
    n_out = N // 2 if act else N
    tiles = -(-n_out // (64 if act else 128))
    out = np.zeros((E, tiles, stages, per // 4, 32, 4, 4), np.uint8)
    for m in range(tiles):
        for r in range(128):
            if act:
                o = m * 64 + r // 32 * 16 + r % 16
                row = o + (n_out if r % 32 >= 16 else 0)
            else:
                o = row = m * 128 + r
            if o >= n_out:
                continue
            padded = np.zeros((E, stages * per), np.uint8)
            padded[:, :cols] = scales[:, row]
            out[:, m, :, :, r % 32, r // 32] = padded.reshape(E, stages, per // 4, 4)
    return out.reshape(-1)


def fp4_linear(x, w, factor, act, rel):
    """(out, err) float64 [n, N or N / 2] of rows x [n, K] and weights w [N, K],
    given as values: act(factor * (w @ x)), and the error of sums that are off by
    `rel` of their absolute terms, of the FP32 steps behind them (factor 2^-24,
    activation 2^-20) and of the rounding to BF16 (2^-8)."""
    f = abs(float(factor))
    y, dy = factor * (x @ w.T), (np.abs(x) @ np.abs(w).T) * f * rel
    dy = dy + 2.0 ** -24 * np.abs(y)
    if act:
        h = y.shape[1] // 2
        with np.errstate(over="ignore"):
            gate, up, dg, du = y[:, :h], y[:, h:], dy[:, :h], dy[:, h:]
            s = gate / (1 + np.exp(-gate))
        y, dy = s * up, 1.1 * dg * (np.abs(up) + du) + np.abs(s) * du
        dy = dy + 2.0 ** -20 * np.abs(y)
    return y, dy + 2.0 ** -8 * (np.abs(y) + dy) + 2.0 ** -133
