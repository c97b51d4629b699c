"""Host side of the 4-bit operators, no GPU: argument checks of the C ABI
(every refused case fails a host check, nothing is launched) and of the
binding."""

import pytest

from moe_decode_layer_logits_gb300 import _lib as L
from test_abi_experts import INVALID, MISALIGNED, NULL, OK, P, UNSUPPORTED, lib  # noqa: F401

NV, MX = L.MOE_FP4_NV, L.MOE_FP4_MX
ROWS = dict(x=P, g=NULL, codes=P, scales=P, T=4, K=256, fmt=NV)


@pytest.mark.parametrize("name", ["moe_fp4_quantize", "moe_fp4_dequantize"])
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(K=-64), INVALID), (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID),
    (dict(K=96), UNSUPPORTED), (dict(K=64, fmt=MX), UNSUPPORTED), (dict(K=65600), UNSUPPORTED),
    (dict(T=1 << 62), UNSUPPORTED), (dict(fmt=MX, g=P), INVALID),
    (dict(x=NULL), INVALID), (dict(codes=NULL), INVALID), (dict(scales=NULL), INVALID),
    (dict(x=P + 8), MISALIGNED), (dict(codes=P + 8), MISALIGNED), (dict(scales=P + 2), MISALIGNED), (dict(g=P + 2), MISALIGNED),
    (dict(T=0, x=NULL, codes=NULL, scales=NULL), OK),
])
def test_row_argument_checks(lib, name, kw, want):
    a = {**ROWS, **kw}
    if name == "moe_fp4_quantize":
        got = lib.moe_fp4_quantize(a["x"], a["g"], a["codes"], a["scales"], a["T"], a["K"], a["fmt"], None)
    else:
        got = lib.moe_fp4_dequantize(a["codes"], a["scales"], a["g"], a["x"], a["T"], a["K"], a["fmt"], None)
    assert got == want


SC = dict(scales=P, tiled=P, E=4, N=64, K=256, fmt=NV, act=0)


@pytest.mark.parametrize("kw,want", [
    (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(fmt=2), INVALID), (dict(act=2), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(N=60), UNSUPPORTED), (dict(N=72, act=1), UNSUPPORTED), (dict(K=32), UNSUPPORTED),
    (dict(K=64, fmt=MX), UNSUPPORTED), (dict(N=65544), UNSUPPORTED),
    (dict(scales=NULL), INVALID), (dict(tiled=NULL), INVALID), (dict(scales=P + 2), MISALIGNED), (dict(tiled=P + 8), MISALIGNED),
])
def test_weight_scales_argument_checks(lib, kw, want):
    a = {**SC, **kw}
    assert lib.moe_fp4_weight_scales(a["scales"], a["tiled"], a["E"], a["N"], a["K"], a["fmt"], a["act"], None) == want


@pytest.mark.parametrize("E,N,K,fmt,act,want", [
    (1, 128, 256, NV, 0, 2048), (1, 8, 64, NV, 0, 2048), (3, 264, 640, MX, 0, 3 * 3 * 3 * 1024),
    (2, 272, 256, NV, 1, 2 * 3 * 2048), (1, 60, 256, NV, 0, -1), (0, 64, 256, NV, 0, -1), (1, 64, 100, NV, 0, -1),
    (1, 64, 256, 5, 0, -1), (1025, 64, 256, NV, 0, -1),
])
def test_weight_scales_bytes(lib, E, N, K, fmt, act, want):
    assert lib.moe_fp4_weight_scales_bytes(E, N, K, fmt, act) == want


LIN = dict(x=P, xs=P, n_x=4, tok=P, w=P, ws=P, f=P, offsets=P, counts=P, out=P, n_rows=32, E=16, N=64, K=256, fmt=NV, act=0,
           work=P, nb=1 << 40, err=NULL)

COMMON = [
    (dict(n_rows=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(act=2), INVALID), (dict(fmt=2), INVALID),
    (dict(nb=-1), INVALID), (dict(N=60), UNSUPPORTED), (dict(N=72, act=1), UNSUPPORTED), (dict(K=96), UNSUPPORTED),
    (dict(K=64, fmt=MX), UNSUPPORTED), (dict(N=65544), UNSUPPORTED), (dict(K=65600), UNSUPPORTED),
    (dict(n_rows=1 << 31), UNSUPPORTED), (dict(n_rows=(1 << 31) - 1, N=65536), UNSUPPORTED),
    (dict(x=NULL), INVALID), (dict(xs=NULL), INVALID), (dict(w=NULL), INVALID), (dict(ws=NULL), INVALID),
    (dict(out=NULL), INVALID), (dict(x=P + 8), MISALIGNED), (dict(xs=P + 2), MISALIGNED), (dict(w=P + 8), MISALIGNED),
    (dict(ws=P + 8), MISALIGNED), (dict(f=P + 2), MISALIGNED), (dict(out=P + 8), MISALIGNED), (dict(work=P + 8), MISALIGNED),
    (dict(err=P + 2), MISALIGNED),
]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(n_rows=0, x=NULL, xs=NULL, w=NULL, out=NULL), OK),
])
def test_linear_argument_checks(lib, kw, want):
    a = {**LIN, **kw}
    assert lib.moe_fp4_linear(a["x"], a["xs"], a["w"], a["ws"], a["f"], a["out"], a["n_rows"], a["N"], a["K"], a["fmt"],
                              a["act"], a["work"], a["nb"], a["err"], None) == want


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(n_x=-1), INVALID), (dict(E=0), INVALID), (dict(E=1025), UNSUPPORTED), (dict(n_x=1 << 31), UNSUPPORTED),
    (dict(tok=NULL, n_x=31), INVALID), (dict(offsets=NULL), INVALID), (dict(counts=NULL), INVALID),
    (dict(tok=P + 2), MISALIGNED), (dict(offsets=P + 2), MISALIGNED), (dict(counts=P + 2), MISALIGNED),
    (dict(n_rows=0, x=NULL, xs=NULL, tok=NULL, w=NULL, out=NULL, offsets=NULL, counts=NULL), OK),
])
def test_expert_linear_argument_checks(lib, kw, want):
    a = {**LIN, **kw}
    assert lib.moe_fp4_expert_linear(a["x"], a["xs"], a["n_x"], a["tok"], a["w"], a["ws"], a["f"], a["offsets"], a["counts"],
                                     a["out"], a["n_rows"], a["E"], a["N"], a["K"], a["fmt"], a["act"], a["work"], a["nb"],
                                     a["err"], None) == want


def test_workspace_that_is_too_small_is_refused(lib):
    for n_rows in (1, 64, 4096):
        need = lib.moe_fp4_linear_workspace(n_rows, 1, 4096, 6144)
        assert need >= 0
        if need > 0:
            a = (P, P, P, P, NULL, P, n_rows, 4096, 6144, NV, 0)
            assert lib.moe_fp4_linear(*a, P, need - 1, NULL, None) == INVALID
            assert lib.moe_fp4_linear(*a, NULL, 0, NULL, None) == INVALID
    assert lib.moe_fp4_linear_workspace(-1, 1, 64, 64) == -1
    assert lib.moe_fp4_linear_workspace(8, 0, 64, 64) == -1


def test_binding_refuses_before_anything_is_launched(lib):
    import torch
    import moe_decode_layer_logits_gb300 as M
    z, u8 = torch.zeros, torch.uint8
    with pytest.raises(TypeError, match="CUDA"):
        M.moe_fp4_quantize(z(4, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="x must be"):
        M.moe_fp4_quantize(z(4, 64))
    with pytest.raises(ValueError, match="format"):
        M.moe_fp4_quantize(z(4, 64, dtype=torch.bfloat16), format="fp4")
    with pytest.raises(ValueError, match="multiple of 128"):
        M.moe_fp4_quantize(z(4, 64, dtype=torch.bfloat16), format="mxfp4")
    with pytest.raises(ValueError, match="one element"):
        M.moe_fp4_quantize(z(4, 64, dtype=torch.bfloat16), global_scale=z(2))
    with pytest.raises(ValueError, match="scales must have the shape"):
        M.moe_fp4_dequantize(z(4, 32, dtype=u8), z(4, 2, dtype=u8))
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_fp4_dequantize(z(32, 64, dtype=u8).t(), z(64, 4, dtype=u8))
    with pytest.raises(ValueError, match="scales must be"):
        M.moe_fp4_weight_scales(z(8, dtype=u8))
    with pytest.raises(ValueError, match="range"):
        M.moe_fp4_weight_scales(z(60, 4, dtype=u8))
    x, xs, w = z(4, 32, dtype=u8), z(4, 4, dtype=u8), z(8, 32, dtype=u8)
    ws = z(2048, dtype=u8)
    with pytest.raises(ValueError, match="x must be"):
        M.moe_fp4_linear(x, xs, w[:, :16], ws)
    with pytest.raises(ValueError, match="w_scales"):
        M.moe_fp4_linear(x, xs, w, ws[:1024])
    with pytest.raises(ValueError, match="factor"):
        M.moe_fp4_linear(x, xs, w, ws, factor=z(2))
    with pytest.raises(ValueError, match="offsets"):
        M.moe_fp4_expert_linear(x, xs, w[None], ws, z(5), z(1))
    with pytest.raises(TypeError, match="counts"):
        M.moe_fp4_expert_linear(x, xs, w[None], ws, z(1, dtype=torch.int32), z(1))
    with pytest.raises(ValueError, match="act"):
        M.moe_fp4_linear(x, xs, w, ws, act="relu")
