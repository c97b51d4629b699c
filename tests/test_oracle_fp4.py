"""Pins of the 4-bit definitions (no GPU): library conversions, closed forms,
exact rational arithmetic."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle as O
from moe_decode_layer_logits_gb300.inputs import draw_bf16

G = [1.0, 0.0017, 0.75, 3.0e-5, 12.5]


def f64(bits):
    return O.bf16_bits_to_f64(bits)


def test_scale_bytes_are_the_library_types():
    b = torch.arange(256, dtype=torch.uint8)
    e4m3 = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.fp4_scale_values("nvfp4")[:128], e4m3[:128], equal_nan=True)
    assert np.array_equal(O.fp4_scale_values("nvfp4")[128:], e4m3[:128], equal_nan=True)   # the top bit is no sign
    e8m0 = O.fp4_scale_values("mxfp4")
    assert e8m0[0] == 2.0 ** -127 and e8m0[127] == 1.0 and e8m0[254] == 2.0 ** 127 and np.isnan(e8m0[255])


def test_codes_by_hand():
    codes = np.array([[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]], np.uint8)
    v = O.fp4_values(codes, np.array([[0x40]], np.uint8), "nvfp4", 0.5)      # E4M3 2.0, times 0.5
    assert v.tolist() == [[0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantize_ties_by_hand(fmt):
    # amax 6: the scale is 1; every midpoint goes to the code whose last bit is 0
    x = np.zeros((1, O.FP4_BLOCK[fmt]))
    x[0, :16] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, .26]
    codes, scales = O.fp4_quantize(x, fmt)
    assert O.fp4_scale_values(fmt)[scales[0, 0]] == 1
    v = O.fp4_values(codes, scales, fmt)[0, :16]
    assert v.tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, .5]
    assert (codes[0, 4] & 15) == 8                                          # a negative zero keeps its sign


def test_powers_of_two_by_hand():
    # floor(log2 amax) - 2: 7.9 has the scale of 4, and is cut to 6
    x = np.zeros((4, 32))
    x[:, 0] = [4, 7.9375, 8, 2.0 ** -130]
    codes, scales = O.fp4_quantize(x, "mxfp4")
    assert scales[:, 0].tolist() == [127, 127, 128, 0]
    assert O.fp4_values(codes, scales, "mxfp4")[:, 0].tolist() == [4, 6, 8, 0]   # 2^-130 is a quarter step: to zero


def test_not_finite_blocks_and_zero_blocks():
    for bad in (np.inf, -np.inf, np.nan):
        x = np.ones((1, 64))
        x[0, 20] = bad
        for fmt, at, nan in (("nvfp4", 1, 0x7F), ("mxfp4", 0, 0xFF)):
            codes, scales = O.fp4_quantize(x, fmt)
            assert scales[0, at] == nan and (np.delete(scales[0], at) != nan).all()
    codes, scales = O.fp4_quantize(-np.zeros((1, 32)), "nvfp4")
    assert not codes.any() and not scales.any()
    assert (O.fp4_quantize(np.ones((1, 32)), "nvfp4", 2.0 ** -101)[1] == 0x7F).all()


@pytest.mark.parametrize("g", G)
def test_quantize_against_exact_fractions(g):
    rng = np.random.default_rng([1, int(g * 1e6)])
    g = float(np.float32(g))
    bits = draw_bf16(rng, (24, 16), 1.0)
    x = f64(bits)
    x[12:] = np.round(x[12:] * 4) / 4                                       # full of ties when g is 1
    codes, scales = O.fp4_quantize(x, "nvfp4", g)
    e4m3 = [Fraction(v) for v in O.fp4_scale_values("nvfp4")[:127]]
    e2m1 = [Fraction(v) for v in O.fp4_e2m1[:8]]

    def nearest(v, table):
        return min(range(len(table)), key=lambda i: (abs(table[i] - v), i % 2))

    G_ = Fraction(g)
    for r in range(len(x)):
        top = max(abs(Fraction(v)) for v in x[r])
        s = nearest(top / (6 * G_), e4m3)
        assert s == scales[r, 0]
        for i, v in enumerate(x[r]):
            c = nearest(abs(Fraction(v)) / (e4m3[s] * G_), e2m1) if s else 0
            assert c == (codes[r, i // 2] >> 4 * (i % 2)) & 7


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("act,N,K", [(None, 8, 128), (None, 264, 640), ("swiglu", 16, 128), ("swiglu", 272, 384)])
def test_tiled_scales_hold_every_scale_once(fmt, act, N, K):
    cols = K // O.FP4_BLOCK[fmt]
    s = np.random.default_rng(2).integers(1, 255, (3, N, cols)).astype(np.uint8)
    t = O.fp4_tiled_scales(s, fmt, act)
    assert np.array_equal(np.bincount(t, minlength=256)[1:], np.bincount(s.reshape(-1), minlength=256)[1:])
    # one of them by hand: expert 2, the last row, the last scale
    row, per = N - 1, 256 // O.FP4_BLOCK[fmt]
    n_out = N // 2 if act else N
    o = row - (n_out if act else 0)
    tile, r = (o // 64, o % 64 // 16 * 32 + 16 + o % 16) if act else (o // 128, o % 128)
    tiles, stages = -(-n_out // (64 if act else 128)), -(-cols // per)
    at = (((2 * tiles + tile) * stages + (cols - 1) // per) * (per // 4) + (cols - 1) % per // 4) * 512 + r % 32 * 16 + r // 32 * 4 + 3
    assert t[at] == s[2, row, cols - 1]


def test_linear_is_the_matrix_product():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((5, 64)), rng.standard_normal((12, 64))
    y, err = O.fp4_linear(x, w, 0.5, None, 0.0)
    assert np.allclose(y, 0.5 * np.einsum("rk,nk->rn", x, w), rtol=1e-13) and (err >= 2.0 ** -8 * np.abs(y)).all()
    z, _ = O.fp4_linear(x, w, 0.5, "swiglu", 0.0)
    t = torch.from_numpy(y)
    assert np.allclose(z, (torch.nn.functional.silu(t[:, :6]) * t[:, 6:]).numpy(), rtol=1e-13)
