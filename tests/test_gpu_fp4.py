"""GPU tests of the 4-bit operators against their FP64 definitions.

Tolerances, derived from the arithmetic:

* Codes, scales and the order of the weights' scales are exact.
* A dequantised value is code * scale * global scale rounded to BF16 once: within
  half a step, 2^-8 of itself (exact without a global scale).
* Products: an element is a code times a scale, at most 6 bits, so every product
  is exact in FP32.  A tensor-core step adds 64 products to the accumulator,
  scale block by scale block: K / 16 sums, each within 2^-23 of the sum of
  absolute terms S, the 64 products of one step within another 64 * 2^-23:
  |y - y64| <= (K/16 + 64) * 2^-23 * S; the split sums of a small batch add up to
  152 pieces, each addition within 2^-24 of S.  The factor, the activation and
  the rounding as in oracle.fp4_linear.
"""

import numpy as np
import pytest
import torch

import moe_decode_layer_logits_gb300 as M_
import oracle as O
from _guard import Guarded, check_all
from moe_decode_layer_logits_gb300 import _lib as L
from moe_decode_layer_logits_gb300.inputs import draw_bf16
from test_gpu_experts import M, dev, devn, host16, values  # noqa: F401

pytestmark = pytest.mark.gpu


def rel_sum(K):
    return (K / 16 + 64) * 2.0 ** -23 + 152 * 2.0 ** -24


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------

def run_quantize(M, bits, fmt, g=None):
    T, K = bits.shape
    codes, scales = Guarded((T, K // 2), torch.uint8, fill=7), Guarded((T, K // O.FP4_BLOCK[fmt]), torch.uint8, fill=7)
    gs = None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")
    M.moe_fp4_quantize(dev(bits), format=fmt, global_scale=gs, codes=codes.t, scales=scales.t)
    check_all(codes=codes, scales=scales)
    return codes.t, scales.t, gs


def check_quantize(M, bits, fmt, g=None):
    g = None if g is None else float(np.float32(g))
    codes, scales, gs = run_quantize(M, bits, fmt, g)
    want_c, want_s = O.fp4_quantize(O.bf16_bits_to_f64(bits), fmt, 1.0 if g is None else g)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    out = Guarded(bits.shape, torch.bfloat16, fill=3.0)
    M.moe_fp4_dequantize(codes, scales, format=fmt, global_scale=gs, out=out.t)
    check_all(out=out)
    want = O.fp4_values(want_c, want_s, fmt, 1.0 if g is None else g)
    got = values(out.t)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), ~fine)
    assert np.array_equal(host16(out.t)[fine], O.f64_to_bf16_bits(want[fine]))


@pytest.mark.parametrize("fmt,T,K", [("nvfp4", 1, 64), ("nvfp4", 1, 6144), ("nvfp4", 37, 1088), ("nvfp4", 300, 2048),
                                     ("mxfp4", 1, 128), ("mxfp4", 3, 6144), ("mxfp4", 65, 1152), ("mxfp4", 257, 384)])
def test_quantize(M, fmt, T, K):
    rng = np.random.default_rng([300, T, K])
    bits = draw_bf16(rng, (T, K), 1.0)
    wide = O.f64_to_bf16_bits(O.bf16_bits_to_f64(bits) * np.exp(2 * rng.standard_normal(K)))
    for g in (None, 0.0018, 1.0, 0.125, 3.7) if fmt == "nvfp4" else (None,):
        check_quantize(M, bits, fmt, g)
        check_quantize(M, wide, fmt, g)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantize_ties_zeros_and_the_ends_of_the_range(M, fmt):
    rng = np.random.default_rng(301)
    K = 256
    rows = [np.round(rng.standard_normal(K) * 8) / 4,                 # quarters: ties at scales of 1, 2, ..
            np.round(rng.standard_normal(K) * 3), np.zeros(K), -np.zeros(K),
            rng.standard_normal(K) * 2.0 ** -128, rng.standard_normal(K) * 2.0 ** -132, rng.standard_normal(K) * 2.0 ** 125,
            np.where(rng.random(K) < 0.02, 448.0 * 6, 0.01), np.full(K, 2.0 ** -9), np.full(K, 3.3e38), np.full(K, 2.0 ** -133)]
    bits = O.f64_to_bf16_bits(np.stack(rows))
    check_quantize(M, bits, fmt)
    if fmt == "nvfp4":
        for g in (2.0 ** -100, 2.0 ** -133 * 2 ** 40, 1.1e-20, 6.0, 2.0 ** 100):
            check_quantize(M, bits, fmt, g)


def test_quantize_global_scales_that_bring_midpoints_next_to_bf16_numbers(M):
    # g such that midpoint * scale * g is a BF16 number, or a few, 30 and 40 units of FP32's last place beside one
    rng = np.random.default_rng(305)
    bits = draw_bf16(rng, (64, 256), 1.0)
    for ms in (1.0, 1.25 * 1.375, 1.75 * 1.875, 1.5 * 1.125):
        for off in (0, 1, -1, 3, -30, 30, 40, -40):
            near = np.float32(1.0078125 / 256) / np.float32(ms)
            g = (near.view(np.int32) + np.int32(off)).view(np.float32)
            x = bits.copy()
            # elements that sit at such midpoints: x = m s g for many m and s, rounded to BF16
            at = np.outer(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]), 2.0 ** np.arange(-6, 8) * ms).reshape(-1)[:64] * float(g)
            x[:, 3::16] = O.f64_to_bf16_bits(np.resize(at, (64, 16)))
            check_quantize(M, x, "nvfp4", float(g))
            check_quantize(M, O.f64_to_bf16_bits(O.bf16_bits_to_f64(x) * 2.0 ** -9), "nvfp4", float(g))


def test_quantize_ties_of_global_scales_of_few_bits(M):
    # all with 8 bits, and some of 9: elements on midpoints of blocks' scales, beside them, and far above the largest
    rng = np.random.default_rng(307)
    m = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    for mantissa in [*range(128, 256), *(k + 0.5 for k in range(128, 256, 9))]:
        g = float(np.float32(mantissa * 2.0 ** (-8 - mantissa % 5)))
        x = rng.standard_normal((18, 256)) * 2.0 ** rng.integers(-6, 4, (18, 16)).repeat(16, axis=1) * g * 6
        x[16] *= 2.0 ** 20  # scales that stop at 448
        x[17, ::16] = 3e38
        _, s = O.fp4_quantize(O.bf16_bits_to_f64(O.f64_to_bf16_bits(x)), "nvfp4", g)
        s = O.fp4_scale_values("nvfp4")[s] * g
        for i in range(7):
            x[:, i + 2::16] = m[i] * s * (1 + rng.integers(-1, 2, s.shape) * 2.0 ** -8)
        x[:, 10::16], x[:, 11::16] = 0.0, -0.0
        bits = O.f64_to_bf16_bits(x * rng.choice([-1, 1], x.shape))
        check_quantize(M, bits, "nvfp4", g)
        check_quantize(M, O.f64_to_bf16_bits(O.bf16_bits_to_f64(bits) * 2.0 ** -100), "nvfp4", g * 2.0 ** -94)


def test_quantize_global_scales_from_the_largest_element(M):
    # g = amax / (448 * 6), as calibration sets it: 0.75 * 448 * g and 0.875 * 384 * g are then next to BF16 numbers
    rng = np.random.default_rng(306)
    for mantissa in range(128):
        top = float(np.float32(2.0 ** (mantissa % 9 - 3) * (1 + mantissa / 128)))
        x = O.bf16_bits_to_f64(draw_bf16(rng, (16, 512), 1.0)) * rng.choice([0.05, 0.3, 1.0], (16, 32)).repeat(16, axis=1) * top
        # elements on and beside midpoints of the blocks' scales
        g = np.float32(top) / np.float32(448 * 6)
        _, s = O.fp4_quantize(np.clip(x, -top, top), "nvfp4", float(g))
        s = O.fp4_scale_values("nvfp4")[s] * float(g)
        m = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
        for i in range(7):
            x[:, i + 2::16] = m[i] * s * (1 + rng.integers(-1, 2, s.shape) * 2.0 ** -8)
        bits = O.f64_to_bf16_bits(np.clip(x, -top, top) * rng.choice([-1, 1], x.shape))
        check_quantize(M, bits, "nvfp4", g)


def test_quantize_every_bf16_as_the_largest_of_its_block(M):
    # 2^15 blocks: the largest takes every value, the others lie below it
    rng = np.random.default_rng(302)
    top = np.arange(0x7F80, dtype=np.uint16)
    x = O.bf16_bits_to_f64(top)[:, None] * rng.uniform(-1, 1, (len(top), 64))
    bits = O.f64_to_bf16_bits(x)
    bits[:, 5::16] = top[:, None]
    for g in (None, 0.0018, 1.3):
        check_quantize(M, bits, "nvfp4", g)
    check_quantize(M, np.concatenate([bits, bits], axis=1), "mxfp4")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantize_what_is_not_finite(M, fmt):
    bits = draw_bf16(np.random.default_rng(303), (6, 256), 1.0)
    for r, b in enumerate((0x7F80, 0xFF80, 0x7FC0, 0xFFFF, 0x7F81)):
        bits[r, 33 + 17 * r] = b
    check_quantize(M, bits, fmt)
    if fmt == "nvfp4":
        for g in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -101, 2.0 ** 101):
            codes, scales, _ = run_quantize(M, bits, fmt, g)
            assert (scales == 0x7F).all() and not codes.any()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,K", [(1, 64), (37, 1088), (300, 2048)])
def test_tensors_that_begin_between_sectors(M, fmt, T, K):
    # 16 bytes behind a multiple of 32: the same values, and nothing written beside them
    K = K if fmt == "nvfp4" else K * 2
    x = dev(draw_bf16(np.random.default_rng([308, T, K]), (T, K), 1.0))
    codes, scales = M.moe_fp4_quantize(x, format=fmt)
    at = torch.empty(T * K + 16, dtype=torch.bfloat16, device="cuda")
    at = at[8 if at.data_ptr() % 32 == 0 else 0:][:T * K].view(T, K)
    assert at.data_ptr() % 32 == 16
    at.copy_(x)
    for got, want in zip(M.moe_fp4_quantize(at, format=fmt), (codes, scales)):
        assert torch.equal(got, want)
    whole = torch.full((T * K + 32,), 7.0, dtype=torch.bfloat16, device="cuda")
    first = 8 if whole.data_ptr() % 32 == 0 else 16
    out = whole[first:first + T * K].view(T, K)
    assert out.data_ptr() % 32 == 16
    M.moe_fp4_dequantize(codes, scales, format=fmt, out=out)
    assert torch.equal(out, M.moe_fp4_dequantize(codes, scales, format=fmt))
    assert bool((whole[:first] == 7).all()) and bool((whole[first + T * K:] == 7).all())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_dequantize_every_code_with_every_scale(M, fmt):
    B = O.FP4_BLOCK[fmt]
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(-1, B // 2), (1, 1)).reshape(1, -1)   # 512 elements
    codes = np.repeat(codes, 256, axis=0)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 512 // B, axis=1)
    for g in (None, 0.37):
        if g is not None and fmt == "mxfp4":
            continue
        gs = None if g is None else torch.tensor([g], device="cuda")
        out = M.moe_fp4_dequantize(devn(codes), devn(scales), format=fmt, global_scale=gs)
        with np.errstate(over="ignore"):
            want = O.fp4_values(codes, scales, fmt, 1.0 if g is None else float(np.float32(g)))
        fine = ~np.isnan(want)
        assert np.array_equal(np.isnan(values(out)), ~fine)
        assert np.array_equal(host16(out)[fine], O.f64_to_bf16_bits(want[fine]))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("E,N,K", [(1, 16, 128), (3, 272, 384), (2, 2064, 1152), (5, 128, 256)])
def test_weight_scales(M, fmt, act, E, N, K):
    s = np.random.default_rng(304).integers(0, 256, (E, N, K // O.FP4_BLOCK[fmt])).astype(np.uint8)
    want = O.fp4_tiled_scales(s, fmt, act)
    out = Guarded(want.shape, torch.uint8)
    M.moe_fp4_weight_scales(devn(s), format=fmt, act=act, out=out.t)
    check_all(out=out)
    assert np.array_equal(out.t.cpu().numpy(), want)


def test_rows_beyond_31_bits(M):
    # elements, then codes, whose numbers pass 2^31 and 2^32
    T, K = 70000, 65536
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 32767, 32768, 65535, 65536, T - 1], device="cuda")
    x[at, 100:164] = torch.arange(64, device="cuda", dtype=torch.bfloat16)
    codes, scales = M.moe_fp4_quantize(x)
    few, few_s = M.moe_fp4_quantize(x[at])
    assert torch.equal(codes[at], few) and torch.equal(scales[at], few_s)
    back = M.moe_fp4_dequantize(codes, scales)
    assert torch.equal(back[at], M.moe_fp4_dequantize(few, few_s))
    assert int((back != 0).sum()) == int((back[at] != 0).sum())


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def draw_four(rng, shape, std, fmt, g=1.0):
    """(codes, scales, values): rows of a normal distribution in 4 bits."""
    flat = O.bf16_bits_to_f64(draw_bf16(rng, (int(np.prod(shape[:-1])), shape[-1]), std))
    codes, scales = O.fp4_quantize(flat, fmt, g)
    v = O.fp4_values(codes, scales, fmt)
    return tuple(a.reshape(*shape[:-1], -1) for a in (codes, scales, v))


def check_rows(got, want, err, what):
    d = np.abs(got - want)
    bad = ~(d <= err)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, the worst {float((d / err)[bad].max()):.2f} times "
                           f"the bound, first at {np.argwhere(bad)[0]}")


def draw_linear(T, N, K, fmt, seed=0):
    rng = np.random.default_rng([310, seed, T, N, K])
    x, xs, xv = draw_four(rng, (T, K), 1.0, fmt)
    w, ws, wv = draw_four(rng, (N, K), 0.05, fmt, 0.001 if fmt == "nvfp4" else 1.0)
    return dict(x=x, xs=xs, xv=xv, w=w, ws=ws, wv=wv)


def run_linear(M, c, fmt, act, factor=None, **kw):
    T, N = len(c["x"]), len(c["w"])
    out, flag = Guarded((T, N // 2 if act else N), torch.bfloat16, fill=3.0), Guarded((1,), torch.int32, fill=0)
    M.moe_fp4_linear(devn(c["x"]), devn(c["xs"]), devn(c["w"]), M.moe_fp4_weight_scales(devn(c["ws"]), format=fmt, act=act),
                     format=fmt, factor=None if factor is None else torch.tensor([factor], device="cuda"), act=act,
                     out=out.t, err_flag=flag.t, **kw)
    check_all(out=out, flag=flag)
    return out.t, int(flag.t.item())


LINEAR = [  # T, N, K
    (1, 4096, 6144), (1, 16, 128), (1, 8, 128), (2, 528, 1152), (7, 272, 256), (16, 256, 384), (17, 2056, 640), (33, 144, 2048),
    (64, 1024, 2048), (65, 272, 512), (128, 256, 896), (129, 144, 1408), (200, 264, 128), (255, 512, 256), (300, 528, 1152),
    (513, 16, 256), (700, 384, 384), (1000, 256, 640), (1100, 2048, 256), (2100, 128, 128),
    (1, 4096, 256), (31, 9728, 512), (64, 8192, 768), (95, 4608, 384), (90, 16384, 256), (5, 20480, 128),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("T,N,K", LINEAR)
def test_linear(M, T, N, K, act, fmt):
    if act and N % 16:
        N += 8
    factor = None if N == 16 else 0.0031
    c = draw_linear(T, N, K, fmt)
    out, flag = run_linear(M, c, fmt, act, factor)
    assert flag == 0
    want, err = O.fp4_linear(c["xv"], c["wv"], 1.0 if factor is None else float(np.float32(factor)), act, rel_sum(K))
    check_rows(values(out), want, err, f"T={T} N={N} K={K}")


def test_linear_of_words_of_scales_that_end_inside_a_stage(M):
    for K in (64, 192, 320, 448, 1088):
        c = draw_linear(40, 136, K, "nvfp4")
        out, _ = run_linear(M, c, "nvfp4", None)
        want, err = O.fp4_linear(c["xv"], c["wv"], 1.0, None, rel_sum(K))
        check_rows(values(out), want, err, f"K={K}")


def test_linear_scales_that_start_on_any_word(M):
    for fmt, T, K in (("nvfp4", 40, 512), ("mxfp4", 40, 512), ("nvfp4", 300, 256), ("mxfp4", 300, 512)):
        c = draw_linear(T, 144, K, fmt)
        want, _ = run_linear(M, c, fmt, None)
        room = torch.zeros(c["xs"].size + 16, dtype=torch.uint8, device="cuda")
        for at in (4, 8, 12):
            xs = room[at:at + c["xs"].size].view(c["xs"].shape)
            xs.copy_(devn(c["xs"]))
            got = M.moe_fp4_linear(devn(c["x"]), xs, devn(c["w"]), M.moe_fp4_weight_scales(devn(c["ws"]), format=fmt), format=fmt)
            assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [5, 300])
def test_linear_scales_of_any_size(M, T, fmt):
    # whole numbers as codes, scales far apart: a misplaced scale changes sums by orders of magnitude
    rng = np.random.default_rng([311, T])
    N, K, B = 144, 512, O.FP4_BLOCK[fmt]
    x, w = (rng.integers(0, 256, (n, K // 2)).astype(np.uint8) for n in (T, N))
    lo, hi = (8, 120) if fmt == "nvfp4" else (110, 145)
    xs, ws = (rng.integers(lo, hi, (n, K // B)).astype(np.uint8) for n in (T, N))
    c = dict(x=x, xs=xs, w=w, ws=ws)
    out, _ = run_linear(M, c, fmt, None)
    want, err = O.fp4_linear(O.fp4_values(x, xs, fmt), O.fp4_values(w, ws, fmt), 1.0, None, rel_sum(K))
    check_rows(values(out), want, err, "any size")


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("T,N,K", [(3, 4096, 2048), (100, 4096, 2048), (3, 8192, 1024), (20, 65536, 512), (300, 8192, 2048), (1200, 8192, 4096)])
def test_linear_leaves_nan_where_a_wait_ran_out(M, T, N, K, act):  # single CTAs, pairs
    c = draw_linear(T, N, K, "nvfp4")
    want, flag = run_linear(M, c, "nvfp4", act)
    assert flag == 0
    for stage in (0, 1):
        M.moe_debug_withhold_expert_stage(stage)
        out, flag = run_linear(M, c, "nvfp4", act)
        assert flag & L.MOE_FLAG_TIMEOUT
        lost = torch.isnan(out)
        assert torch.equal(out[~lost], want[~lost]) and 0 < int(lost.sum()) < out.numel()
    again, flag = run_linear(M, c, "nvfp4", act)
    assert flag == 0 and torch.equal(again, want)


def test_linear_same_bits_again(M):
    for T, N, K in ((2, 4096, 2048), (50, 6144, 1024), (90, 16384, 512), (700, 1024, 512)):
        c = draw_linear(T, N, K, "nvfp4")
        a, _ = run_linear(M, c, "nvfp4", "swiglu")
        for _ in range(3):
            assert torch.equal(run_linear(M, c, "nvfp4", "swiglu")[0], a)


def test_linear_swiglu_over_the_range_of_its_gate(M):
    # y = the weight itself (one element of x is 1): gates from -150 to 150 and beyond, ups of 1
    rng = np.random.default_rng(312)
    n_out, K = 2048, 64
    w, ws = np.zeros((2 * n_out, K // 2), np.uint8), np.full((2 * n_out, K // 16), 0x38, np.uint8)
    w[:n_out, 0], ws[:n_out, 0] = rng.integers(1, 16, n_out), rng.integers(0x18, 0x60, n_out)
    w[n_out:, 0] = 2                                       # 1.0
    x, xs = np.zeros((1, K // 2), np.uint8), np.full((1, K // 16), 0x38, np.uint8)
    x[0, 0] = 2
    gate = O.fp4_values(w, ws, "nvfp4")[:n_out, 0]
    assert gate.min() < -90 and gate.max() > 90 and (np.abs(gate) < 0.1).any()
    with np.errstate(over="ignore"):
        want = gate / (1 + np.exp(-gate))
    for T in (1, 1200):                                    # (1200: pairs)
        rep = {"x": np.repeat(x, T, 0), "xs": np.repeat(xs, T, 0), "w": w, "ws": ws}
        got = values(run_linear(M, rep, "nvfp4", "swiglu")[0])
        # FP32's exponential ends at e^88.7: below, the result is 0 instead of some 1e-37
        err = (2.0 ** -8 + 2.0 ** -20) * np.abs(want) + np.where(gate < -88, 1e-36, 2.0 ** -133)
        check_rows(got, np.repeat(want[None], T, 0), np.repeat(err[None], T, 0), "range of the gate")
    big = run_linear(M, {"x": x, "xs": xs, "w": w, "ws": ws}, "nvfp4", "swiglu", 3e38)[0]
    got = values(big)[0]
    assert np.all(np.isposinf(got[gate * 3e38 > 3.4e38])) and not np.isnan(got[gate > 0]).any()


def test_linear_empty_batch(M):
    c = draw_linear(1, 64, 128, "nvfp4")
    assert run_linear(M, {**c, "x": c["x"][:0], "xs": c["xs"][:0]}, "nvfp4", None)[0].shape == (0, 64)


def draw_layer(seed, T, E, k, K, N, fmt, block=1, gather=True, hot=None):
    rng = np.random.default_rng([320, seed, T, E, k, K, N])
    ids = rng.random((T, E)).argsort(1)[:, :k].astype(np.int32)
    if hot is not None:
        ids[:, 0] = hot                                   # (a second slot may hold it too)
    row_map, row_token, offsets, counts = O.expert_map(ids, E, block)
    x, xs, xv = draw_four(rng, (T if gather else len(row_token), K), 1.0, fmt)
    w, ws, wv = draw_four(rng, (E, N, K), 0.05, fmt, 0.001 if fmt == "nvfp4" else 1.0)
    return dict(ids=ids, row_map=row_map, row_token=row_token, offsets=offsets, counts=counts, x=x, xs=xs, xv=xv, w=w, ws=ws,
                wv=wv, factor=rng.uniform(0.5, 2, E).astype(np.float32) * 0.001)


def run_expert(M, c, fmt, act, gather, factor=True, **kw):
    n, N = len(c["row_token"]), c["w"].shape[1]
    out, flag = Guarded((n, N // 2 if act else N), torch.bfloat16, fill=3.0), Guarded((1,), torch.int32, fill=0)
    M.moe_fp4_expert_linear(devn(c["x"]), devn(c["xs"]), devn(c["w"]),
                            M.moe_fp4_weight_scales(devn(c["ws"]), format=fmt, act=act), devn(c["offsets"]),
                            devn(c["counts"]), format=fmt, factor=devn(c["factor"]) if factor else None,
                            row_token=devn(c["row_token"]) if gather else None, act=act, out=out.t, err_flag=flag.t, **kw)
    check_all(out=out, flag=flag)
    return out.t, int(flag.t.item())


def check_expert(M, c, fmt, act, gather, what, factor=True):
    out, flag = run_expert(M, c, fmt, act, gather, factor)
    assert flag == 0
    got, seen = values(out), np.zeros(len(out), bool)
    for e, (off, cnt) in enumerate(zip(c["offsets"], c["counts"])):
        if cnt == 0:
            continue
        rows = np.arange(off, off + cnt)
        x = c["xv"][c["row_token"][rows] if gather else rows]
        want, err = O.fp4_linear(x, c["wv"][e], float(c["factor"][e]) if factor else 1.0, act, rel_sum(x.shape[1]))
        check_rows(got[rows], want, err, f"{what} expert {e}")
        seen[rows] = True
    assert np.all(got[~seen] == 3.0), f"{what}: rows of no segment were written"


EXPERT = [  # T, E, k, K, N, block, gather, hot
    (1, 8, 8, 6144, 256, 1, True, None), (1, 4, 1, 128, 16, 1, True, None), (1, 64, 8, 256, 4096, 1, True, None),
    (3, 16, 4, 1152, 2064, 1, True, None), (64, 40, 8, 512, 256, 1, True, None), (5, 8, 2, 128, 16, 1, True, None),
    (64, 40, 8, 128, 272, 16, True, None), (37, 24, 6, 1152, 528, 1, False, None), (130, 8, 3, 256, 144, 128, False, 2),
    (700, 6, 2, 128, 256, 1, True, 3), (513, 3, 3, 384, 272, 8, False, None), (300, 1, 1, 128, 384, 1, True, None),
    (40, 1024, 8, 128, 32, 1, True, None), (2000, 16, 4, 256, 512, 1, True, None), (2500, 2, 1, 1024, 128, 1, True, 1),
    (257, 1, 1, 4096, 1024, 1, False, None), (600, 5, 2, 128, 336, 1, True, 4), (600, 5, 2, 128, 336, 8, False, 4),
    (820, 3, 1, 128, 528, 1, True, 1), (820, 3, 1, 256, 272, 1, False, 1), (1400, 8, 2, 640, 272, 1, True, 5),
    (1024, 2, 1, 128, 512, 1, True, 0), (1500, 4, 2, 1152, 528, 1, True, None), (1500, 4, 2, 1152, 512, 1, False, 0),
    (9, 200, 4, 2048, 64, 1, False, None),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("T,E,k,K,N,block,gather,hot", EXPERT)
def test_expert_linear(M, T, E, k, K, N, block, gather, hot, act, fmt):
    c = draw_layer(1, T, E, k, K, N, fmt, block, gather, hot)
    check_expert(M, c, fmt, act, gather, f"T={T} E={E} k={k} K={K} N={N}", factor=T % 2 == 0)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 207, 208, 209, 255, 256,
                                  257, 415, 416, 417, 513])
def test_expert_linear_segment_lengths(M, rows):
    # one expert of each length beside an empty one and one of a single row
    rng = np.random.default_rng([321, rows])
    K, N = 128, 272
    counts = np.array([0, rows, 0, 1, 0], np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    for fmt, act in (("nvfp4", None), ("nvfp4", "swiglu"), ("mxfp4", None)):
        x, xs, xv = draw_four(rng, (9, K), 1.0, fmt)
        w, ws, wv = draw_four(rng, (5, N, K), 0.1, fmt)
        c = dict(x=x, xs=xs, xv=xv, w=w, ws=ws, wv=wv, offsets=offsets, counts=counts, factor=np.ones(5, np.float32),
                 row_token=rng.integers(0, 9, rows + 1).astype(np.int32))
        check_expert(M, c, fmt, act, True, f"rows={rows}")


def test_expert_linear_of_no_rows_writes_nothing(M):
    c = draw_layer(2, 20, 8, 2, 128, 32, "nvfp4")
    c["counts"] = np.zeros_like(c["counts"])
    check_expert(M, c, "nvfp4", None, True, "no rows")


def test_expert_linear_bad_tokens_and_segments(M):
    c = draw_layer(3, 50, 8, 3, 256, 48, "nvfp4")
    bad = c["row_token"].copy()
    at = [0, 17, 149]
    bad[at] = [-1, 50, 2 ** 31 - 1]
    out, flag = run_expert(M, {**c, "row_token": bad}, "nvfp4", None, True)
    assert flag == L.MOE_FLAG_BAD_INDEX
    assert np.all(values(out)[at] == 0)
    clean, _ = run_expert(M, c, "nvfp4", None, True)
    keep = np.setdiff1d(np.arange(150), at)
    assert np.array_equal(host16(out)[keep], host16(clean)[keep])
    # an expert whose segment leaves the rows is skipped
    for off, cnt in [(-1, 4), (149, 2), (0, -3), (2 ** 31 - 1, 2 ** 31 - 1), (151, 1)]:
        d = {**c, "offsets": c["offsets"].copy(), "counts": c["counts"].copy()}
        lo, n = int(c["offsets"][2]), int(c["counts"][2])
        d["offsets"][2], d["counts"][2] = off, cnt
        out, flag = run_expert(M, d, "nvfp4", None, True)
        assert flag == L.MOE_FLAG_BAD_INDEX
        got, ref = host16(out), host16(clean)
        mine = np.zeros(150, bool)
        mine[lo:lo + n] = True
        assert np.array_equal(got[~mine], ref[~mine]) and np.all(values(out)[mine] == 3.0)


@pytest.mark.parametrize("T", [40, 400])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_expert_linear_nan_scales_stay_in_their_rows(M, fmt, T):
    c = draw_layer(4, T, 6, 2, 512, 64, fmt, block=16, gather=False)
    nan = 0x7F if fmt == "nvfp4" else 0xFF
    free = np.nonzero(c["row_token"] < 0)[0]
    xs = c["xs"].copy()
    xs[free] = nan                                         # in the padding rows
    clean, _ = run_expert(M, c, fmt, "swiglu", False)
    out, _ = run_expert(M, {**c, "xs": xs}, fmt, "swiglu", False)
    assert np.array_equal(host16(out), host16(clean))
    row = int(c["row_map"][7, 1])
    xs[row, 3] = nan                                       # one block of a live row
    out, _ = run_expert(M, {**c, "xs": xs}, fmt, None, False)
    plain, _ = run_expert(M, c, fmt, None, False)
    keep = np.arange(len(xs)) != row
    assert np.array_equal(host16(out)[keep], host16(plain)[keep])
    assert np.isnan(values(out)[row]).all()


@pytest.mark.parametrize("T,E,k", [(2, 12, 3), (90, 12, 3), (900, 4, 2)])
def test_expert_linear_same_bits_again(M, T, E, k):
    c = draw_layer(5, T, E, k, 1152, 272, "nvfp4")
    a, _ = run_expert(M, c, "nvfp4", "swiglu", True)
    for _ in range(3):
        b, _ = run_expert(M, c, "nvfp4", "swiglu", True)
        assert torch.equal(a, b)


def test_expert_linear_overlapping_segments_take_nothing(M):
    for n in (60, 600):
        c = draw_layer(8, n, 4, 2, 128, 32, "nvfp4")
        c["counts"] = np.full(4, n, np.int32)
        c["offsets"] = np.array([0, 5, 10, 15], np.int32)
        out, flag = run_expert(M, c, "nvfp4", None, True)
        assert flag == L.MOE_FLAG_BAD_INDEX and np.all(values(out) == 3.0)


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("T,gather", [(2, True), (2, False), (300, True), (300, False)])
def test_expert_linear_leaves_nan_where_a_wait_ran_out(M, T, gather, act):
    c = draw_layer(6, T, 4, 2, 2048, 4096, "nvfp4", gather=gather)
    want, flag = run_expert(M, c, "nvfp4", act, gather)
    assert flag == 0
    for stage in (0, 2):
        M.moe_debug_withhold_expert_stage(stage)
        out, flag = run_expert(M, c, "nvfp4", act, gather)
        assert flag & L.MOE_FLAG_TIMEOUT
        lost = torch.isnan(out)
        assert torch.equal(out[~lost], want[~lost]) and 0 < int(lost.sum()) < out.numel()
    again, flag = run_expert(M, c, "nvfp4", act, gather)
    assert flag == 0 and torch.equal(again, want)


def test_expert_linear_without_any_token(M):
    # no rows of x at all: every named token is outside, its row is zeros
    c = draw_layer(7, 1, 2, 1, 128, 32, "nvfp4")
    d = {**c, "x": c["x"][:0], "xs": c["xs"][:0], "row_token": np.array([0, -1, 5], np.int32),
         "offsets": np.array([0, 2, 3], np.int32), "counts": np.array([2, 1], np.int32)}
    out, flag = run_expert(M, d, "nvfp4", None, True)
    assert not out.any() and flag == L.MOE_FLAG_BAD_INDEX


def halves(seed, *shape):
    """Codes and, as FP32, their values, for scales of 1: products are multiples
    of a quarter, and sums of some hundred of them are exact in FP32."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device="cuda", dtype=torch.uint8)
    table = torch.tensor(O.fp4_e2m1, dtype=torch.float32, device="cuda")
    return codes, lambda c: table[torch.stack([c & 15, c >> 4], dim=-1).long()].flatten(-2)


def ones(*shape):
    return torch.full(shape, 0x38, dtype=torch.uint8, device="cuda")      # E4M3 1.0


@pytest.mark.parametrize("E,rows", [(80, 1), (80, 96)])
def test_expert_linear_more_pieces_than_a_walker_keeps(M, E, rows):
    # 512 (pairs: 256) weight tiles an expert: over 256 tiles a CTA or pair
    N, K = 65536, 64
    x, val = halves(1, E * rows, K)
    w, _ = halves(2, E, N, K)
    off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * rows
    out = M.moe_fp4_expert_linear(x, ones(E * rows, 4), w, M.moe_fp4_weight_scales(ones(E, N, 4)), off,
                                  torch.full((E,), rows, device="cuda", dtype=torch.int32))
    for e in range(E):
        want = (val(x[e * rows:(e + 1) * rows]) @ val(w[e]).T).to(torch.bfloat16)
        assert torch.equal(out[e * rows:(e + 1) * rows], want), e


def test_products_with_offsets_beyond_31_bits(M):
    # outputs, then rows of x, whose offsets in elements pass 2^31 and 2^32
    n, N, K = 70000, 65536, 64
    x, val = halves(3, n, K)
    w, _ = halves(4, N, K)
    t = M.moe_fp4_weight_scales(ones(N, 4))
    out = M.moe_fp4_linear(x, ones(n, 4), w, t)
    at = torch.tensor([0, 1, 32767, 32768, 65535, 65536, n - 1], device="cuda")
    assert torch.equal(out[at], (val(x[at]) @ val(w).T).to(torch.bfloat16))
    del out
    n, K, N = 140000, 65536, 16
    x = torch.zeros(n, K // 2, dtype=torch.uint8, device="cuda")
    some, _ = halves(5, n, 64)
    x[:, 20000:20032] = some
    xs = ones(n, K // 16)
    w, _ = halves(6, 1, N, K)
    t = M.moe_fp4_weight_scales(ones(1, N, K // 16))
    want = (val(some) @ val(w[0, :, 20000:20032]).T).to(torch.bfloat16)
    seg = torch.tensor([0, n], device="cuda", dtype=torch.int32)
    back = torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.int32)
    for tok, ref in ((None, want), (back, want.flip(0))):
        assert torch.equal(M.moe_fp4_expert_linear(x, xs, w, t, seg, seg[1:], row_token=tok), ref)
    few = torch.tensor([n - 1, 0, 65536, 131072], device="cuda", dtype=torch.int32)
    four = torch.tensor([0, 4], device="cuda", dtype=torch.int32)
    assert torch.equal(M.moe_fp4_expert_linear(x, xs, w, t, four, four[1:], row_token=few), want[few.long()])


@pytest.mark.parametrize("T,N,K", [(3, 512, 256), (1200, 8192, 4096)])
def test_linear_behind_a_kernel_that_runs_long(M, T, N, K):
    # An expert map of 2^30 slots lets its dependents start at once and runs for
    # longer than the probes of one bounded wait last: the call behind it must not
    # give up, nor read its inputs, which the kernel between them writes, too early.
    c = draw_linear(T, N, K, "nvfp4")
    want, _ = run_linear(M, c, "nvfp4", "swiglu")
    ids = torch.randint(0, 1024, (1 << 25, 32), dtype=torch.int32, device="cuda")
    x, xs = devn(c["x"]), devn(c["xs"])
    late, late_s = torch.zeros_like(x), torch.zeros_like(xs)
    w, t = devn(c["w"]), M.moe_fp4_weight_scales(devn(c["ws"]), act="swiglu")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    M.moe_expert_map(ids, 1024)
    late.copy_(x)
    late_s.copy_(xs)
    out = M.moe_fp4_linear(late, late_s, w, t, act="swiglu", err_flag=flag)
    torch.cuda.synchronize()
    assert int(flag.item()) == 0 and torch.equal(out, want)
    M.moe_expert_map(ids, 1024)
    out = M.moe_fp4_linear(x, xs, w, t, act="swiglu", err_flag=flag)
    assert int(flag.item()) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("T", [2, 1200])
def test_quantised_rows_are_read_behind_the_kernel_that_writes_them(M, T):
    # quantisation and product back to back, over and over, on new rows each time
    N, K = 8192, 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    rows = torch.randn(6, T, K, generator=g, device="cuda", dtype=torch.bfloat16)
    w, ws = M.moe_fp4_quantize(torch.randn(N, K, generator=g, device="cuda", dtype=torch.bfloat16))
    t = M.moe_fp4_weight_scales(ws)
    codes, scales = torch.empty(T, K // 2, dtype=torch.uint8, device="cuda"), torch.empty(T, K // 16, dtype=torch.uint8, device="cuda")
    want = []
    for r in rows:
        q = M.moe_fp4_quantize(r)
        torch.cuda.synchronize()
        want.append(M.moe_fp4_linear(*q, w, t))
        torch.cuda.synchronize()
    got = [M.moe_fp4_linear(*M.moe_fp4_quantize(r, codes=codes, scales=scales), w, t) for r in rows]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# products large enough for pairs of CTAs (against 64-bit products on the GPU)
# ---------------------------------------------------------------------------

def in_pairs(n_rows, E, N, K):
    """Whether a call of these sizes runs in pairs: it has a workspace then."""
    return L.lib().moe_fp4_linear_workspace(n_rows, E, N, K) > 0


def bytes_of(seed, lo, hi, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.uint8)


def decoded(codes, scales, fmt):
    e2m1 = torch.tensor(O.fp4_e2m1, device="cuda")
    scale = torch.tensor(O.fp4_scale_values(fmt), device="cuda")
    two = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    return e2m1[two.long()] * scale[scales.long()].repeat_interleave(O.FP4_BLOCK[fmt], dim=-1)


def reference(x, w, factor, act):
    """O.fp4_linear on the GPU."""
    rel = rel_sum(x.shape[1])
    y, dy = factor * (x @ w.T), (x.abs() @ w.abs().T) * abs(factor) * rel
    dy += 2.0 ** -24 * y.abs()
    if act:
        h = y.shape[1] // 2
        gate, up, dg, du = y[:, :h], y[:, h:], dy[:, :h], dy[:, h:]
        s = gate / (1 + torch.exp(-gate))
        y, dy = s * up, 1.1 * dg * (up.abs() + du) + s.abs() * du
        dy = dy + 2.0 ** -20 * y.abs()
    return y, dy + 2.0 ** -8 * (y.abs() + dy) + 2.0 ** -133


LENGTHS = [1, 15, 0, 16, 17, 128, 129, 192, 207, 208, 209, 224, 225, 240, 241, 255, 256, 257, 0, 272, 415, 416, 417, 511, 512, 513, 700]


def large_case(fmt, act, N, K, gather, lengths=LENGTHS, seed=0):
    counts = torch.tensor(lengths, dtype=torch.int32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int32), torch.cumsum(counts, 0, dtype=torch.int32)])
    E, n = len(lengths), int(offsets[-1])
    n_x = 500 if gather else n
    B = O.FP4_BLOCK[fmt]
    lo, hi = (40, 70) if fmt == "nvfp4" else (120, 130)
    assert in_pairs(n, E, N, K)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(x=bytes_of(seed + 1, 0, 256, n_x, K // 2), xs=bytes_of(seed + 2, lo, hi, n_x, K // B),
             w=bytes_of(seed + 3, 0, 256, E, N, K // 2), ws=bytes_of(seed + 4, lo, hi, E, N, K // B), offsets=offsets.cuda(),
             counts=counts.cuda(), factor=torch.rand(E, generator=g, device="cuda") * 0.01,
             token=torch.randint(0, n_x, (n,), generator=g, device="cuda", dtype=torch.int32) if gather else None)
    c["t"] = M_.moe_fp4_weight_scales(c["ws"], format=fmt, act=act)
    return c, n


def run_large(c, n, fmt, act):
    N = c["w"].shape[1]
    out, flag = Guarded((n, N // 2 if act else N), torch.bfloat16, fill=3.0), Guarded((1,), torch.int32, fill=0)
    M_.moe_fp4_expert_linear(c["x"], c["xs"], c["w"], c["t"], c["offsets"], c["counts"], format=fmt, factor=c["factor"],
                             row_token=c["token"], act=act, out=out.t, err_flag=flag.t)
    check_all(out=out, flag=flag)
    return out.t, int(flag.t.item())


def check_large(c, n, fmt, act, out, skip=None):
    x = decoded(c["x"], c["xs"], fmt)
    for e, (off, cnt) in enumerate(zip(c["offsets"].tolist(), c["counts"].tolist())):
        rows = torch.arange(off, off + cnt, device="cuda")
        if skip is not None:
            rows = rows[~skip[rows]]
        want, err = reference(x[c["token"][rows].long()] if c["token"] is not None else x[rows], decoded(c["w"][e], c["ws"][e], fmt),
                              float(c["factor"][e]), act)
        d = (out[rows].double() - want).abs()
        assert bool((d <= err).all()), (e, cnt, float((d / err).max()))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("N,K,gather", [(4112, 1408, True), (4112, 1536, False), (8208, 640, False), (8240, 768, True), (2064, 2816, True)])
def test_pairs_segment_lengths(M, N, K, gather, act, fmt):
    c, n = large_case(fmt, act, N, K, gather)
    out, flag = run_large(c, n, fmt, act)
    assert flag == 0
    check_large(c, n, fmt, act, out)


@pytest.mark.parametrize("act", [None, "swiglu"])
def test_pairs_word_long_scales(M, act):
    # rows' scales that start and end on any word
    c, n = large_case("nvfp4", act, 4112, 1344, True)
    check_large(c, n, "nvfp4", act, run_large(c, n, "nvfp4", act)[0])
    c, n = large_case("nvfp4", act, 4112, 1536, True)
    want, _ = run_large(c, n, "nvfp4", act)
    room = torch.zeros(c["xs"].numel() + 16, dtype=torch.uint8, device="cuda")
    c["xs"] = room[4:4 + c["xs"].numel()].view(c["xs"].shape).copy_(c["xs"])
    assert torch.equal(run_large(c, n, "nvfp4", act)[0], want)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("T,N,K", [(1024, 8192, 4096), (1111, 8208, 4224), (1800, 16400, 1152), (2305, 4112, 3712), (9000, 2064, 2048)])
def test_pairs_of_one_segment(M, T, N, K, act, fmt):
    assert in_pairs(T, 1, N, K)
    B = O.FP4_BLOCK[fmt]
    lo, hi = (40, 70) if fmt == "nvfp4" else (120, 130)
    x, xs, w, ws = bytes_of(1, 0, 256, T, K // 2), bytes_of(2, lo, hi, T, K // B), bytes_of(3, 0, 256, N, K // 2), bytes_of(4, lo, hi, N, K // B)
    f = torch.tensor([0.003], device="cuda")
    out, flag = Guarded((T, N // 2 if act else N), torch.bfloat16, fill=3.0), Guarded((1,), torch.int32, fill=0)
    M.moe_fp4_linear(x, xs, w, M.moe_fp4_weight_scales(ws, format=fmt, act=act), format=fmt, factor=f, act=act, out=out.t, err_flag=flag.t)
    check_all(out=out, flag=flag)
    assert int(flag.t.item()) == 0
    wv = decoded(w, ws, fmt)
    for a in range(0, T, 2048):
        want, err = reference(decoded(x[a:a + 2048], xs[a:a + 2048], fmt), wv, float(f), act)
        d = (out.t[a:a + 2048].double() - want).abs()
        assert bool((d <= err).all()), float((d / err).max())


def test_pairs_bad_tokens_and_nan_scales_stay_in_their_rows(M):
    c, n = large_case("nvfp4", "swiglu", 4112, 1536, True)
    clean, _ = run_large(c, n, "nvfp4", "swiglu")
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[torch.tensor([0, 31, 400, 4000, n - 1], device="cuda")] = True
    token = c["token"].clone()
    token[bad] = torch.tensor([-1, 500, 2 ** 31 - 1, -7, 501], dtype=torch.int32, device="cuda")
    out, flag = run_large({**c, "token": token}, n, "nvfp4", "swiglu")
    assert flag == L.MOE_FLAG_BAD_INDEX and not out[bad].any() and torch.equal(out[~bad], clean[~bad])
    xs = c["xs"].clone()
    xs[77, 90] = 0x7F
    out, flag = run_large({**c, "xs": xs}, n, "nvfp4", "swiglu")
    hit = c["token"] == 77
    assert flag == 0 and hit.any() and torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])
    again, _ = run_large(c, n, "nvfp4", "swiglu")
    assert torch.equal(again, clean)


@pytest.mark.parametrize("gather", [True, False])
def test_pairs_leave_nan_where_a_wait_ran_out(M, gather):
    c, n = large_case("nvfp4", "swiglu", 4112, 1536, gather)
    want, _ = run_large(c, n, "nvfp4", "swiglu")
    for stage in (0, 2, 40):
        M.moe_debug_withhold_expert_stage(stage)
        out, flag = run_large(c, n, "nvfp4", "swiglu")
        assert flag & L.MOE_FLAG_TIMEOUT
        lost = torch.isnan(out)
        assert torch.equal(out[~lost], want[~lost]) and 0 < int(lost.sum()) < out.numel()
    again, flag = run_large(c, n, "nvfp4", "swiglu")
    assert flag == 0 and torch.equal(again, want)


def test_pairs_captured_on_two_streams(M):
    """Two graphs of large products, whose workspaces are their own, replayed at once."""
    cases = [large_case("nvfp4", "swiglu", 4112, 1536, True, seed=s) for s in (0, 50)]
    want = [run_large(c, n, "nvfp4", "swiglu")[0].clone() for c, n in cases]
    graphs, outs = [], []
    call = lambda c: M.moe_fp4_expert_linear(c["x"], c["xs"], c["w"], c["t"], c["offsets"], c["counts"], factor=c["factor"],
                                             row_token=c["token"], act="swiglu")
    for c, _ in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(c))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for out, ref in zip(outs, want):
        assert torch.equal(out, ref)


# ---------------------------------------------------------------------------
# together: a layer whose experts work in 4 bits
# ---------------------------------------------------------------------------

def prepare_layer(M, T, H, I, E, fmt, seed=0):
    rng = np.random.default_rng([330, seed, T, H])
    f = lambda *s, std=0.05: dev(draw_bf16(rng, s, std))
    g = dict(x=f(T, H, std=1.0), w_gate=f(E, H), residual=f(T, H, std=1.0),
             gamma=devn((1 + 0.1 * rng.standard_normal(H)).astype(np.float32)))
    one = torch.tensor([0.002], device="cuda") if fmt == "nvfp4" else None
    for name, e, n, k, act in (("w13", E, 2 * I, H, "swiglu"), ("w2", E, H, I, None), ("s13", 1, 2 * I, H, "swiglu"),
                               ("s2", 1, H, I, None)):
        codes, scales = M.moe_fp4_quantize(f(e * n, k), format=fmt, global_scale=one)
        shape = (e, n) if e > 1 else (n,)
        g[name] = codes.reshape(*shape, k // 2)
        g[name + "s"] = scales.reshape(*shape, -1)
        g[name + "t"] = M.moe_fp4_weight_scales(g[name + "s"], format=fmt, act=act)
    g["g"] = one
    g["factor"] = None if one is None else one.square().expand(E).contiguous()
    return g


def layer(M, g, E, k, fmt):
    """Router, routing, map, experts and shared expert in 4 bits, tail."""
    logits = M.moe_router_logits_fp32(g["x"], g["w_gate"])
    ids, w = M.moe_topk_route(logits, k, 2.5)
    row_map, row_token, offsets, counts = M.moe_expert_map(ids, E)
    one = None if g["factor"] is None else g["factor"][:1]
    x = M.moe_fp4_quantize(g["x"], format=fmt, global_scale=g["g"])
    h = M.moe_fp4_expert_linear(*x, g["w13"], g["w13t"], offsets, counts, format=fmt, factor=g["factor"], row_token=row_token,
                                act="swiglu")
    hq = M.moe_fp4_quantize(h, format=fmt, global_scale=g["g"])
    rows = M.moe_fp4_expert_linear(*hq, g["w2"], g["w2t"], offsets, counts, format=fmt, factor=g["factor"])
    sh = M.moe_fp4_linear(*x, g["s13"], g["s13t"], format=fmt, factor=one, act="swiglu")
    sq = M.moe_fp4_quantize(sh, format=fmt, global_scale=g["g"])
    shared = M.moe_fp4_linear(*sq, g["s2"], g["s2t"], format=fmt, factor=one)
    ro, no = M.moe_finalize_add_rmsnorm(rows, row_map, w, shared, g["residual"], g["gamma"], 1e-6)
    return dict(ids=ids, w=w, row_map=row_map, row_token=row_token, offsets=offsets, counts=counts, x=x[0], xs=x[1], h=h,
                hq=hq[0], hs=hq[1], rows=rows, sh=sh, sq=sq[0], ss=sq[1], shared=shared, ro=ro, no=no)


@pytest.mark.parametrize("T,H,I,E,k,fmt", [(1, 512, 128, 16, 4, "nvfp4"), (28, 640, 192, 24, 3, "nvfp4"),
                                           (300, 256, 128, 16, 4, "mxfp4"), (1100, 128, 64, 16, 4, "nvfp4")])
def test_layer_step_by_step(M, T, H, I, E, k, fmt):
    """Each step against its definition on the GPU's own inputs of that step."""
    g = prepare_layer(M, T, H, I, E, fmt)
    o = layer(M, g, E, k, fmt)
    n = {name: v.cpu().numpy() for name, v in {**g, **o}.items() if v is not None and v.dtype in (torch.uint8, torch.int32)}
    gs = float(g["g"].item()) if g["g"] is not None else 1.0
    f = float(g["factor"][0].item()) if g["factor"] is not None else 1.0
    for src, codes, scales in ((g["x"], "x", "xs"), (o["h"], "hq", "hs"), (o["sh"], "sq", "ss")):
        c, s = O.fp4_quantize(values(src), fmt, gs)
        assert np.array_equal(o[codes].cpu().numpy(), c) and np.array_equal(n[scales], s)
    xq, hq, sq = (O.fp4_values(o[a].cpu().numpy(), n[b], fmt) for a, b in (("x", "xs"), ("hq", "hs"), ("sq", "ss")))
    for got, x, w, tok, act in ((o["h"], xq, "w13", True, "swiglu"), (o["rows"], hq, "w2", False, None)):
        got, wv = values(got), O.fp4_values(n[w], n[w + "s"], fmt)
        for e in range(E):
            rows = np.arange(n["offsets"][e], n["offsets"][e] + n["counts"][e])
            want, err = O.fp4_linear(x[n["row_token"][rows] if tok else rows], wv[e], f, act, rel_sum(x.shape[1]))
            check_rows(got[rows], want, err, f"{w} expert {e}")
    for got, x, w, act in ((o["sh"], xq, "s13", "swiglu"), (o["shared"], sq, "s2", None)):
        want, err = O.fp4_linear(x, O.fp4_values(n[w], n[w + "s"], fmt), f, act, rel_sum(x.shape[1]))
        check_rows(values(got), want, err, w)
    ref = O.finalize_add_rmsnorm(host16(o["rows"]), n["row_map"], o["w"].cpu().numpy(), host16(o["shared"]), None,
                                 host16(g["residual"]), g["gamma"].cpu().numpy(), 1e-6)
    from _tol import check_bf16, tail_deltas
    dr, dn = tail_deltas(ref, k + 2, g["gamma"].cpu().numpy(), 1e-6)
    check_bf16(f"fp4 layer T={T} residual_out", host16(o["ro"]), ref["residual_out"], ref["r"], dr)
    check_bf16(f"fp4 layer T={T} normed", host16(o["no"]), ref["normed"], ref["normed64"], dn)


@pytest.mark.parametrize("T", [1, 40, 1100])
def test_layer_captured_and_replayed(M, T):
    H, I, E, k, fmt = 256, 128, 16, 4, "nvfp4"
    g = prepare_layer(M, T, H, I, E, fmt)
    eager = layer(M, g, E, k, fmt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(M, g, E, k, fmt)
    for _ in range(3):
        for v in out.values():
            v.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for name in eager:
        assert torch.equal(eager[name], out[name]), name
    g2 = prepare_layer(M, T, H, I, E, fmt, seed=1)         # new inputs in the same buffers
    for name, v in g.items():
        v.copy_(g2[name])
    graph.replay()
    fresh = layer(M, g2, E, k, fmt)
    for name in fresh:
        assert torch.equal(fresh[name], out[name]), name


@pytest.mark.parametrize("T", [2, 60, 1100])
def test_layers_on_two_streams_at_once(M, T):
    H, I, E, k, fmt = 512, 256, 16, 4, "nvfp4"
    g = prepare_layer(M, T, H, I, E, fmt)
    want = layer(M, g, E, k, fmt)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append(layer(M, g, E, k, fmt))
    for st in (streams[0], streams[1].cuda_stream):        # an explicit stream, and its handle
        got.append({"x": M.moe_fp4_quantize(g["x"], global_scale=g["g"], stream=st)[0],
                    "h": M.moe_fp4_expert_linear(want["x"], want["xs"], g["w13"], g["w13t"], want["offsets"], want["counts"],
                                                 factor=g["factor"], row_token=want["row_token"], act="swiglu", stream=st),
                    "shared": M.moe_fp4_linear(want["sq"], want["ss"], g["s2"], g["s2t"], factor=g["factor"][:1], stream=st)})
    torch.cuda.synchronize()
    for o in got:
        for name in o:
            assert torch.equal(o[name], want[name]), name


def test_workspaces_of_two_graphs_are_apart(M):
    """Two captured layers replayed at the same time on two streams."""
    inputs = [prepare_layer(M, 50, 512, 256, 16, "nvfp4", seed=s) for s in (0, 1)]
    layer(M, inputs[0], 16, 4, "nvfp4")
    torch.cuda.synchronize()
    graphs, outs = [], []
    for g in inputs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(layer(M, g, 16, 4, "nvfp4"))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for g, out in zip(inputs, outs):
        fresh = layer(M, g, 16, 4, "nvfp4")
        for name in fresh:
            assert torch.equal(fresh[name], out[name]), name


@pytest.mark.parametrize("call", ["quantize", "dequantize", "scales", "linear", "expert"])
@pytest.mark.parametrize("T", [2, 1100])
def test_refused_launch_is_reported_and_the_next_call_is_clean(M, call, T):
    g = prepare_layer(M, T, 256, 128, 16, "nvfp4")
    o = layer(M, g, 16, 4, "nvfp4")
    run = {"quantize": lambda: M.moe_fp4_quantize(g["x"], global_scale=g["g"])[0],
           "dequantize": lambda: M.moe_fp4_dequantize(o["x"], o["xs"], global_scale=g["g"]),
           "scales": lambda: M.moe_fp4_weight_scales(g["w13s"], act="swiglu"),
           "linear": lambda: M.moe_fp4_linear(o["sq"], o["ss"], g["s2"], g["s2t"], factor=g["factor"][:1]),
           "expert": lambda: M.moe_fp4_expert_linear(o["hq"], o["hs"], g["w2"], g["w2t"], o["offsets"], o["counts"],
                                                     factor=g["factor"])}[call]
    want = run()
    M.moe_debug_fail_next_launch(True)
    try:
        with pytest.raises(M.MoeTailError) as ei:
            run()
    finally:
        M.moe_debug_fail_next_launch(False)
    assert ei.value.status == L.MOE_ERR_CUDA
    assert torch.equal(run(), want)
