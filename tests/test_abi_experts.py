"""Host side of the expert operators, no GPU: argument checks of the C ABI
(every refused case fails a host check, nothing is launched) and of the
binding."""

import os

import pytest

from moe_decode_layer_logits_gb300 import _lib as L
from moe_decode_layer_logits_gb300.build import LIB as LIB_PATH, build_library

P = 0x10000     # fake, 16-byte aligned, never dereferenced
NULL = None
INVALID, UNSUPPORTED, MISALIGNED, OK = (L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_MISALIGNED, L.MOE_OK)


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake-pointer argument checks run only without a visible GPU")
    if not os.path.exists(LIB_PATH):
        build_library()
    return L.lib()


ROUTE = dict(logits=P, bias=P, ids=P, w=P, T=4, E=64, k=8, n_group=8, topk_group=4, group_top=2,
             score=L.MOE_SCORE_SIGMOID, renorm=1, scale=2.5)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=33), INVALID),
    (dict(k=9, topk_group=1), INVALID),                  # 8 experts in one group
    (dict(n_group=0), INVALID), (dict(n_group=7), INVALID), (dict(topk_group=0), INVALID),
    (dict(topk_group=9), INVALID), (dict(group_top=0), INVALID), (dict(group_top=3), INVALID),
    (dict(score=2), INVALID), (dict(renorm=2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("-inf")), INVALID), (dict(E=2048), UNSUPPORTED), (dict(n_group=64, topk_group=32), UNSUPPORTED),
    (dict(T=1 << 31), UNSUPPORTED),
    (dict(logits=NULL), INVALID), (dict(ids=NULL), INVALID), (dict(w=NULL), INVALID),
    (dict(logits=P + 2), MISALIGNED), (dict(bias=P + 1), MISALIGNED), (dict(ids=P + 2), MISALIGNED),
    (dict(w=P + 2), MISALIGNED),
    (dict(T=0, logits=NULL, ids=NULL, w=NULL, bias=NULL), OK),
])
def test_group_route_argument_checks(lib, kw, want):
    a = {**ROUTE, **kw}
    assert lib.moe_group_topk_route(a["logits"], a["bias"], a["ids"], a["w"], a["T"], a["E"], a["k"], a["n_group"],
                                    a["topk_group"], a["group_top"], a["score"], a["renorm"], a["scale"], None) == want


@pytest.mark.parametrize("T,E,k,block,want", [
    (0, 8, 2, 16, 0), (1, 8, 2, 1, 2), (1, 8, 2, 16, 2 + 2 * 15), (100, 8, 2, 16, 200 + 8 * 15),
    (-1, 8, 2, 1, -1), (1, 0, 2, 1, -1), (1, 8, 0, 1, -1), (1, 8, 2, 0, -1), (1 << 40, 8, 2, 1, -1),
])
def test_expert_rows(lib, T, E, k, block, want):
    assert lib.moe_expert_rows(T, E, k, block) == want


MAP = dict(ids=P, row_map=P, row_token=P, offsets=P, counts=P, n_rows=64, T=4, E=16, k=8, block=1)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=33), INVALID), (dict(block=0), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(block=4097), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
    (dict(n_rows=1 << 31), UNSUPPORTED), (dict(n_rows=31), INVALID), (dict(n_rows=32 + 16 * 3 - 1, block=4), INVALID),
    (dict(ids=NULL), INVALID), (dict(row_map=NULL), INVALID), (dict(row_token=NULL), INVALID),
    (dict(offsets=NULL), INVALID), (dict(counts=NULL), INVALID),
    (dict(ids=P + 2), MISALIGNED), (dict(row_map=P + 1), MISALIGNED), (dict(row_token=P + 2), MISALIGNED),
    (dict(offsets=P + 2), MISALIGNED), (dict(counts=P + 2), MISALIGNED),
])
def test_expert_map_argument_checks(lib, kw, want):
    a = {**MAP, **kw}
    assert lib.moe_expert_map(a["ids"], a["row_map"], a["row_token"], a["offsets"], a["counts"], a["n_rows"], a["T"],
                              a["E"], a["k"], a["block"], None) == want


LIN = dict(x=P, n_x=4, tok=P, w=P, offsets=P, counts=P, out=P, n_rows=32, E=16, N=64, K=64, act=0, ws=P, nb=1 << 40,
           err=NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(n_x=-1), INVALID), (dict(n_rows=-1), INVALID), (dict(E=0), INVALID), (dict(N=0), INVALID),
    (dict(K=0), INVALID), (dict(act=2), INVALID), (dict(nb=-1), INVALID),
    (dict(N=60), UNSUPPORTED), (dict(N=72, act=1), UNSUPPORTED), (dict(K=68), UNSUPPORTED), (dict(E=1025), UNSUPPORTED),
    (dict(N=65544), UNSUPPORTED), (dict(K=65544), UNSUPPORTED), (dict(n_rows=1 << 31), UNSUPPORTED),
    (dict(n_x=1 << 31), UNSUPPORTED), (dict(n_rows=(1 << 31) - 1, N=65536), UNSUPPORTED),
    (dict(tok=NULL, n_x=31), INVALID),                    # fewer rows than the segments may name
    (dict(x=NULL), INVALID), (dict(w=NULL), INVALID), (dict(offsets=NULL), INVALID), (dict(counts=NULL), INVALID),
    (dict(out=NULL), INVALID),
    (dict(x=P + 8), MISALIGNED), (dict(w=P + 8), MISALIGNED), (dict(out=P + 8), MISALIGNED), (dict(tok=P + 2), MISALIGNED),
    (dict(offsets=P + 2), MISALIGNED), (dict(counts=P + 2), MISALIGNED), (dict(ws=P + 8), MISALIGNED),
    (dict(err=P + 2), MISALIGNED),
    (dict(n_rows=0, x=NULL, tok=NULL, w=NULL, out=NULL), OK),
])
def test_expert_linear_argument_checks(lib, kw, want):
    a = {**LIN, **kw}
    assert lib.moe_expert_linear(a["x"], a["n_x"], a["tok"], a["w"], a["offsets"], a["counts"], a["out"], a["n_rows"],
                                 a["E"], a["N"], a["K"], a["act"], a["ws"], a["nb"], a["err"], None) == want


def test_workspace_that_is_too_small_is_refused(lib):
    for n_rows, E, N, K in [(8, 16, 4096, 6144), (512, 256, 4096, 6144), (65536, 256, 4096, 6144)]:
        need = lib.moe_expert_linear_workspace(n_rows, E, N, K)
        assert need >= 0
        if need > 0:
            a = (P, n_rows, P, P, P, P, P, n_rows, E, N, K, 0)
            assert lib.moe_expert_linear(*a, P, need - 1, NULL, None) == INVALID
            assert lib.moe_expert_linear(*a, NULL, 0, NULL, None) == INVALID
    for T in (1, 64, 4096):
        need = lib.moe_adapter_linear_workspace(T, 4096, 6144, 16, 8)
        assert need >= 0
        if need > 0:
            a = (P, P, P, P, P, P, P, T, 4096, 6144, 16, 8, 0)
            assert lib.moe_adapter_linear(*a, P, need - 1, NULL, None) == INVALID
    assert lib.moe_expert_linear_workspace(-1, 16, 64, 64) == -1
    assert lib.moe_expert_linear_workspace(8, 0, 64, 64) == -1
    assert lib.moe_adapter_linear_workspace(8, 64, 64, 0, 4) == -1


ADA = dict(x=P, w=P, a=P, b=P, ids=P, scale=P, out=P, T=4, N=64, K=64, R=16, L=3, act=0, ws=P, nb=1 << 40, err=NULL)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(R=0), INVALID), (dict(L=0), INVALID),
    (dict(act=-1), INVALID), (dict(nb=-1), INVALID),
    (dict(N=60), UNSUPPORTED), (dict(K=60), UNSUPPORTED), (dict(N=72, act=1), UNSUPPORTED), (dict(R=12), UNSUPPORTED),
    (dict(R=264), UNSUPPORTED), (dict(L=1025), UNSUPPORTED), (dict(T=1 << 28), UNSUPPORTED),
    (dict(x=NULL), INVALID), (dict(w=NULL), INVALID), (dict(a=NULL), INVALID), (dict(b=NULL), INVALID),
    (dict(ids=NULL), INVALID), (dict(scale=NULL), INVALID), (dict(out=NULL), INVALID),
    (dict(x=P + 8), MISALIGNED), (dict(w=P + 8), MISALIGNED), (dict(a=P + 8), MISALIGNED), (dict(b=P + 8), MISALIGNED),
    (dict(out=P + 8), MISALIGNED), (dict(ids=P + 2), MISALIGNED), (dict(scale=P + 2), MISALIGNED),
    (dict(ws=P + 8), MISALIGNED), (dict(err=P + 2), MISALIGNED),
    (dict(T=0, x=NULL, ids=NULL, out=NULL), OK),
])
def test_adapter_linear_argument_checks(lib, kw, want):
    a = {**ADA, **kw}
    assert lib.moe_adapter_linear(a["x"], a["w"], a["a"], a["b"], a["ids"], a["scale"], a["out"], a["T"], a["N"], a["K"],
                                  a["R"], a["L"], a["act"], a["ws"], a["nb"], a["err"], None) == want


def test_binding_refuses_before_anything_is_launched(lib):
    import torch
    import moe_decode_layer_logits_gb300 as M
    z = torch.zeros
    with pytest.raises(TypeError, match="CUDA"):
        M.moe_group_topk_route(z(4, 16), 2, 1.0)
    with pytest.raises(TypeError, match="CUDA"):
        M.moe_expert_map(z(4, 2, dtype=torch.int32), 16)
    with pytest.raises(ValueError, match="shape"):
        M.moe_group_topk_route(z(4, 16), 2, 1.0, bias=z(15))
    with pytest.raises(ValueError, match="x must be"):
        M.moe_expert_linear(z(4, 16), z(2, 8, 24), z(2), z(2))
    with pytest.raises(ValueError, match="act"):
        M.moe_expert_linear(z(4, 16), z(2, 8, 16), z(2), z(2), act="relu")
    with pytest.raises(ValueError, match="offsets"):
        M.moe_expert_linear(z(4, 16), z(2, 8, 16), z(5), z(2))
    b = torch.bfloat16
    with pytest.raises(ValueError, match="adapter_b"):
        M.moe_adapter_linear(z(4, 16, dtype=b), z(8, 16, dtype=b), z(2, 8, 16, dtype=b), z(2, 9, 8, dtype=b), z(4), z(2))
    with pytest.raises(TypeError, match="w must be"):
        M.moe_adapter_linear(z(4, 16, dtype=b), z(8, 16), z(2, 8, 16, dtype=b), z(2, 8, 8, dtype=b), z(4), z(2))
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_group_topk_route(z(16, 4).t(), 2, 1.0)
    with pytest.raises(ValueError, match="range"):
        M.moe_expert_rows(1, 8, 0)
