"""GPU tests of the expert operators against their FP64 definitions.

Tolerances, derived from the arithmetic:

* ids, maps, offsets and counts are exact.
* Routing weights: a sigmoid or a softmax term is an expf (2 ulp = 4u with
  u = 2^-24), a sum, a quotient (u each); the softmax adds u * |l - l_max| from
  the subtraction and a sum of E terms (E/32 in a lane, 5 across lanes); the
  renormalising sum has k terms; two more roundings follow.  So
  |w - w64| <= w64 * u * (2 * (D + E/32 + 12) + k + 4), D the largest
  |l - l_max| of the row (softmax only).
* Products: exact BF16 products, FP32 sums.  A tensor-core sum adds 16 products
  to the accumulator per step, each step within 2^-23 of the sum of absolute
  terms S, the 16 products of one step within another 16 * 2^-23:
  |y - y64| <= (K/16 + 16) * 2^-23 * S.
  SwiGLU carries that through silu(g) * u (|silu'| <= 1.1) and adds 2^-20
  relative (expf, quotient, product).  The low-rank product of an adapter is
  carried with 16 significant bits, so it is within 2^-16 of itself.
* The one rounding to BF16 is within half a step, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import oracle as O
from _guard import Guarded, check_all
from moe_decode_layer_logits_gb300 import _lib as L
from moe_decode_layer_logits_gb300.inputs import draw_bf16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import os
    from moe_decode_layer_logits_gb300 import build
    if not os.path.exists(build.LIB):
        build.build_library()
    import moe_decode_layer_logits_gb300 as m
    m.lib()
    return m


def dev(b):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(torch.bfloat16).cuda()


def devn(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host16(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def values(t):
    return O.bf16_bits_to_f64(host16(t))


def rel_sum(K):
    return (K / 16 + 16) * 2.0 ** -23


def check_rows(got, want, err, what):
    tol = np.abs(want) * (2.0 ** -8 + 2.0 ** -20) + err * 1.01 + 1e-38
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3], tol[bad][:3])


# ---------------------------------------------------------------------------
# routing by scores and groups
# ---------------------------------------------------------------------------

ROUTE = [  # T, E, k, n_group, topk_group, group_top, scores, bias, renormalize
    (1, 256, 8, 8, 4, 2, "sigmoid", True, True),
    (64, 256, 8, 8, 4, 2, "sigmoid", True, True),
    (300, 256, 8, 1, 1, 2, "sigmoid", True, True),
    (65, 168, 6, 1, 1, 2, "softmax", False, False),
    (33, 160, 6, 8, 3, 1, "softmax", False, True),
    (40, 160, 6, 8, 3, 2, "softmax", False, True),
    (40, 160, 6, 8, 3, 1, "softmax", True, False),
    (40, 160, 6, 8, 3, 1, "sigmoid", False, True),
    (17, 256, 8, 16, 3, 2, "sigmoid", False, True),
    (29, 1024, 32, 32, 7, 2, "sigmoid", True, True),
    (29, 1024, 32, 1, 1, 2, "softmax", True, True),
    (9, 512, 17, 4, 2, 2, "softmax", True, True),
    (9, 400, 9, 4, 4, 1, "sigmoid", True, False),
    (12, 32, 7, 32, 9, 2, "sigmoid", True, True),     # groups of one expert
    (12, 62, 4, 31, 2, 2, "sigmoid", True, True),     # groups of two, k takes all of them
    (5, 1, 1, 1, 1, 1, "softmax", True, True),
    (7, 3, 3, 1, 1, 2, "sigmoid", True, False),
    (3, 40, 20, 2, 1, 2, "sigmoid", True, True),      # k takes the whole group
    (1000, 64, 4, 8, 4, 2, "sigmoid", True, True),
]


def check_route(M, lg, k, kw, scale=2.5):
    T, E = lg.shape
    ids, w = Guarded((T, k), torch.int32), Guarded((T, k), torch.float32)
    dkw = {**kw, "bias": None if kw.get("bias") is None else devn(kw["bias"])}
    M.moe_group_topk_route(devn(lg), k, scale, topk_ids=ids.t, topk_w=w.t, **dkw)
    check_all(ids=ids, w=w)
    rids, rw = O.group_topk_route(lg, k, scale, **kw)
    assert np.array_equal(ids.t.cpu().numpy(), rids)
    D = 0.0
    if kw.get("scores") == "softmax":
        f = np.where(np.isfinite(lg), lg, 0.0).astype(np.float64)
        D = (f.max(1) - f.min(1))[:, None]
    tol = np.abs(rw) * U * (2 * (D + E / 32 + 12) + k + 4) + 1e-37
    got = w.t.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - rw) <= tol), float(np.max(np.abs(got - rw) - tol))


@pytest.mark.parametrize("T,E,k,G,TG,top,scores,bias,renorm", ROUTE)
def test_group_route(M, T, E, k, G, TG, top, scores, bias, renorm):
    rng = np.random.default_rng([200, T, E, k, G])
    lg = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
    check_route(M, lg, k, dict(bias=b, n_group=G, topk_group=TG, group_top=top, scores=scores, renormalize=renorm))


@pytest.mark.parametrize("G,TG,top", [(1, 1, 2), (8, 4, 2), (8, 3, 1)])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_group_route_choices_that_32_bits_cannot_tell_apart(M, G, TG, top, scores):
    # the bias undoes the score up to its own rounding: every choice value of a
    # row lies within 2^-25 of every other
    rng = np.random.default_rng([201, G, top, scores == "sigmoid"])
    E = 64
    row = rng.standard_normal(E).astype(np.float32)
    z = row.astype(np.float64)
    s = 1 / (1 + np.exp(-z)) if scores == "sigmoid" else np.exp(z) / np.exp(z).sum()
    b = (0.9 - s).astype(np.float32)
    lg = np.repeat(row[None], 5, 0)
    lg[1] += rng.standard_normal(E).astype(np.float32) * 1e-6
    lg[3] = rng.standard_normal(E)
    check_route(M, lg, 6, dict(bias=b, n_group=G, topk_group=TG, group_top=top, scores=scores))


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,G,TG,k", [(64, 1, 1, 8), (256, 8, 4, 8), (256, 8, 4, 24), (96, 6, 2, 5)])
def test_group_route_ties_and_rows_without_numbers(M, scores, bias, E, G, TG, k):
    rng = np.random.default_rng([202, E, k])
    lg = rng.integers(-2, 3, (10, E)).astype(np.float32)   # many equal logits
    lg[1] = 0.0
    lg[2] = np.where(np.arange(E) % 2, 0.0, -0.0)
    lg[3] = -np.inf                                        # a row that leaves nothing
    lg[4] = np.nan
    lg[5, ::3] = -np.inf
    lg[6, 1::2] = np.nan
    lg[7] = np.finfo(np.float32).min                       # masks of the type's lowest value
    lg[7, 5] = 1.0
    lg[8, 7] = np.inf
    b = None
    if bias:
        b = (rng.integers(-2, 3, E) / 8).astype(np.float32)
        b[3::7] = -np.inf                                  # experts taken out
        b[11] = np.nan
    for renorm in (True, False):
        check_route(M, lg, k, dict(bias=b, n_group=G, topk_group=TG, group_top=2, scores=scores, renormalize=renorm))


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,TG", [(4, 1, 1), (5, 1, 1), (31, 1, 1), (33, 1, 1), (36, 4, 2), (65, 1, 1), (96, 6, 4),
                                    (129, 1, 1), (260, 1, 1), (260, 13, 4)])
def test_group_route_biases_of_any_size_and_all_experts_chosen(M, scores, E, G, TG):
    # choice values below 0 and infinite ones, with fewer experts than lanes hold; k up to every live expert
    rng = np.random.default_rng([204, E, G])
    lg = rng.standard_normal((9, E)).astype(np.float32)
    lg[5] = -np.inf
    lg[6, ::2] = np.inf
    most = min(32, E // G * TG)
    some = np.where(np.arange(E) % 3 == 0, np.inf, rng.standard_normal(E)).astype(np.float32)
    for b in (rng.standard_normal(E).astype(np.float32) - 3, np.full(E, np.inf, np.float32), np.full(E, -np.inf, np.float32),
              some, -some, np.full(E, 3e38, np.float32), np.full(E, -3e38, np.float32)):
        for k in sorted({1, (most + 1) // 2, most}):
            for top in (1, 2):
                check_route(M, lg, k, dict(bias=b, n_group=G, topk_group=TG, group_top=top, scores=scores))


def test_group_route_equals_the_topk_route(M):
    lg = devn(np.random.default_rng(203).standard_normal((50, 256)).astype(np.float32))
    ids, w = M.moe_group_topk_route(lg, 8, 2.5, scores="softmax")
    rids, rw = M.moe_topk_route(lg, 8, 2.5)
    assert torch.equal(ids, rids) and torch.allclose(w, rw, rtol=1e-5, atol=0)


# ---------------------------------------------------------------------------
# the expert map
# ---------------------------------------------------------------------------

MAP = [  # T, E, k, block, what
    (1, 256, 8, 1, ""), (64, 256, 8, 1, "drop"), (64, 256, 8, 16, "drop"), (37, 168, 6, 128, ""), (5, 1, 1, 4, ""),
    (300, 1024, 32, 1, ""), (300, 1024, 32, 8, "drop"), (3, 1000, 2, 4096, ""), (1, 4, 1, 1, "drop"),
    (2000, 64, 4, 1, "one"), (700, 8, 8, 64, "same"), (20000, 256, 8, 128, ""), (4097, 40, 3, 1, "outside"),
    (33, 2, 32, 1, "same"), (9000, 1024, 8, 1, "drop"),
]


def map_ids(rng, T, E, k, what):
    if what == "one":                                     # every slot the same expert
        return np.full((T, k), E // 2, np.int32)
    if what == "same":                                    # an expert more than once in a token
        return rng.integers(0, E, (T, k)).astype(np.int32)
    ids = (rng.random((T, E)).argsort(1)[:, :k] if E * T < 3e7 else rng.integers(0, E, (T, k))).astype(np.int32)
    if what == "drop":
        ids[T - max(1, T // 5):] = -1
    if what == "outside":
        ids[::3, 0], ids[1::5, 1], ids[2::7, 2] = E, -7, 2 ** 31 - 1
    return ids


@pytest.mark.parametrize("T,E,k,block,what", MAP)
def test_expert_map(M, T, E, k, block, what):
    ids = map_ids(np.random.default_rng([210, T, E, k]), T, E, k, what)
    n = M.moe_expert_rows(T, E, k, block)
    for extra in (0, 37):
        g = dict(row_map=Guarded((T, k), torch.int32, fill=77), row_token=Guarded((n + extra,), torch.int32, fill=77),
                 offsets=Guarded((E + 1,), torch.int32, fill=77), counts=Guarded((E,), torch.int32, fill=77))
        M.moe_expert_map(devn(ids), E, block=block, **{name: v.t for name, v in g.items()})
        check_all(**g)
        for v, want in zip(g.values(), O.expert_map(ids, E, block, n + extra)):
            assert np.array_equal(v.t.cpu().numpy(), want)


def test_expert_map_of_an_empty_batch(M):
    ids = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    off, cnt = Guarded((9,), torch.int32, fill=5), Guarded((8,), torch.int32, fill=5)
    row_map, row_token, _, _ = M.moe_expert_map(ids, 8, offsets=off.t, counts=cnt.t)
    check_all(off=off, cnt=cnt)
    assert row_map.shape == (0, 4) and row_token.shape == (0,)
    assert not off.t.any() and not cnt.t.any()


# ---------------------------------------------------------------------------
# the experts' products
# ---------------------------------------------------------------------------

def draw_layer(seed, T, E, k, K, N, block=1, gather=True, hot=None):
    rng = np.random.default_rng([220, seed, T, E, k, K, N])
    ids = rng.random((T, E)).argsort(1)[:, :k].astype(np.int32)
    if hot is not None:
        ids[:, 0] = hot                                   # (a second slot may hold it too)
    row_map, row_token, offsets, counts = O.expert_map(ids, E, block)
    x = draw_bf16(rng, (T if gather else len(row_token), K), 1.0)
    w = draw_bf16(rng, (E, N, K), 0.05)
    return dict(ids=ids, row_map=row_map, row_token=row_token, offsets=offsets, counts=counts, x=x, w=w)


def run_expert(M, c, act, gather, fill=3.0, **kw):
    n = len(c["row_token"])
    N = c["w"].shape[1]
    out = Guarded((n, N // 2 if act else N), torch.bfloat16, fill=fill)
    flag = Guarded((1,), torch.int32, fill=0)
    M.moe_expert_linear(dev(c["x"]), dev(c["w"]), devn(c["offsets"]), devn(c["counts"]),
                        row_token=devn(c["row_token"]) if gather else None, act=act, out=out.t, err_flag=flag.t, **kw)
    check_all(out=out, flag=flag)
    return out.t, int(flag.t.item())


def check_expert(M, c, act, gather, what, flag=0):
    out, f = run_expert(M, c, act, gather)
    assert f == flag
    K = c["x"].shape[1]
    want = O.expert_linear(c["x"], c["w"], c["offsets"], c["counts"], c["row_token"] if gather else None, act,
                           rel_sum(K))
    got = values(out)
    rows = sorted(want)
    if rows:
        check_rows(got[rows], np.stack([want[r][0] for r in rows]), np.stack([want[r][1] for r in rows]), what)
    rest = np.setdiff1d(np.arange(len(got)), rows)
    assert np.all(got[rest] == 3.0), f"{what}: rows of no segment were written"


EXPERT = [  # T, E, k, K, N, block, gather, hot
    (1, 8, 8, 6144, 256, 1, True, None), (1, 4, 1, 64, 16, 1, True, None), (1, 64, 8, 256, 4096, 1, True, None),
    (3, 16, 4, 1032, 2064, 1, True, None), (64, 40, 8, 512, 256, 1, True, None), (5, 8, 2, 8, 16, 1, True, None),
    (64, 40, 8, 72, 272, 16, True, None), (37, 24, 6, 1032, 528, 1, False, None), (130, 8, 3, 200, 144, 128, False, 2),
    (700, 6, 2, 128, 256, 1, True, 3), (513, 3, 3, 320, 272, 8, False, None), (300, 1, 1, 136, 384, 1, True, None),
    (40, 1024, 8, 64, 32, 1, True, None), (2000, 16, 4, 256, 512, 1, True, None), (2500, 2, 1, 1024, 128, 1, True, 1),
    (257, 1, 1, 4096, 1024, 1, False, None), (600, 5, 2, 136, 336, 1, True, 4), (600, 5, 2, 136, 336, 8, False, 4),
    (820, 3, 1, 136, 528, 1, True, 1), (820, 3, 1, 264, 272, 1, False, 1), (1400, 8, 2, 520, 272, 1, True, 5), (1024, 2, 1, 64, 512, 1, True, 0),
    (1500, 4, 2, 1032, 528, 1, True, None), (1500, 4, 2, 1032, 512, 1, False, 0), (9, 200, 4, 2048, 64, 1, False, None),
]


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("T,E,k,K,N,block,gather,hot", EXPERT)
def test_expert_linear(M, T, E, k, K, N, block, gather, hot, act):
    c = draw_layer(1, T, E, k, K, N, block, gather, hot)
    check_expert(M, c, act, gather, f"T={T} E={E} k={k} K={K} N={N}")


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
def test_expert_linear_segment_lengths(M, rows):
    # one expert of each length beside an empty one and one of a single row
    rng = np.random.default_rng([221, rows])
    K, N = 136, 272
    counts = np.array([0, rows, 0, 1, 0], np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    c = dict(x=draw_bf16(rng, (9, K), 1.0), w=draw_bf16(rng, (5, N, K), 0.1), offsets=offsets, counts=counts,
             row_token=rng.integers(0, 9, rows + 1).astype(np.int32))
    for act in (None, "swiglu"):
        check_expert(M, c, act, True, f"rows={rows}")


def test_expert_linear_of_no_rows_writes_nothing(M):
    c = draw_layer(2, 20, 8, 2, 64, 32)
    c["counts"] = np.zeros_like(c["counts"])
    check_expert(M, c, None, True, "no rows")
    assert M.moe_expert_linear(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), dev(c["w"]), devn(c["offsets"]),
                               devn(c["counts"])).shape == (0, 32)


def test_expert_linear_bad_tokens_and_segments(M):
    c = draw_layer(3, 50, 8, 3, 256, 48)
    bad = c["row_token"].copy()
    at = [0, 17, 149]
    bad[at] = [-1, 50, 2 ** 31 - 1]
    out, flag = run_expert(M, {**c, "row_token": bad}, None, True)
    assert flag == L.MOE_FLAG_BAD_INDEX
    assert np.all(values(out)[at] == 0)
    clean, _ = run_expert(M, c, None, True)
    keep = np.setdiff1d(np.arange(150), at)
    assert np.array_equal(host16(out)[keep], host16(clean)[keep])
    # an expert whose segment leaves the rows is skipped
    for off, cnt in [(-1, 4), (149, 2), (0, -3), (2 ** 31 - 1, 2 ** 31 - 1), (151, 1)]:
        d = {**c, "offsets": c["offsets"].copy(), "counts": c["counts"].copy()}
        lo, n = int(c["offsets"][2]), int(c["counts"][2])
        d["offsets"][2], d["counts"][2] = off, cnt
        out, flag = run_expert(M, d, None, True)
        assert flag == L.MOE_FLAG_BAD_INDEX
        got, ref = host16(out), host16(clean)
        mine = np.zeros(150, bool)
        mine[lo:lo + n] = True
        assert np.array_equal(got[~mine], ref[~mine]) and np.all(values(out)[mine] == 3.0)


def test_expert_linear_infinities_stay_in_their_rows(M):
    c = draw_layer(4, 40, 6, 2, 512, 64, block=16, gather=False)
    free = np.nonzero(c["row_token"] < 0)[0]
    x = c["x"].copy()
    x[free] = 0x7FC0                                       # NaN in the padding rows
    clean, _ = run_expert(M, c, "swiglu", False)
    out, _ = run_expert(M, {**c, "x": x}, "swiglu", False)
    assert np.array_equal(host16(out), host16(clean))
    row = int(c["row_map"][7, 1])
    x[row, 100] = 0x7F80                                   # one infinite element in a live row
    out, _ = run_expert(M, {**c, "x": x}, None, False)
    plain, _ = run_expert(M, c, None, False)
    got, keep = values(out), np.arange(len(x)) != row
    assert np.array_equal(host16(out)[keep], host16(plain)[keep])
    assert not np.isfinite(got[row]).any()


@pytest.mark.parametrize("T,E,k", [(2, 12, 3), (90, 12, 3), (900, 4, 2)])
def test_expert_linear_same_bits_again(M, T, E, k):
    c = draw_layer(5, T, E, k, 1032, 272)
    a, _ = run_expert(M, c, "swiglu", True)
    for _ in range(3):
        b, _ = run_expert(M, c, "swiglu", True)
        assert torch.equal(a, b)


def ints(seed, *shape):
    """Small integers: sums of up to 28 products are whole numbers that BF16 holds."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)


@pytest.mark.parametrize("E,rows", [(80, 1), (80, 96)])
def test_expert_linear_more_pieces_than_a_walker_keeps(M, E, rows):
    # 512 (pairs: 256) weight tiles an expert: over 256 tiles a CTA or pair
    N, K = 65536, 8
    x, w = ints(1, E * rows, K), ints(2, E, N, K)
    off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * rows
    out = M.moe_expert_linear(x, w, off, torch.full((E,), rows, device="cuda", dtype=torch.int32))
    for e in range(E):
        want = (x[e * rows:(e + 1) * rows].float() @ w[e].float().T).to(torch.bfloat16)
        assert torch.equal(out[e * rows:(e + 1) * rows], want), e


def test_expert_linear_offsets_beyond_31_bits(M):
    # outputs, then rows of x, whose offsets in elements pass 2^31 and 2^32
    n, N, K = 70000, 65536, 8
    x, w = ints(3, n, K), ints(4, 1, N, K)
    seg = torch.tensor([0, n], device="cuda", dtype=torch.int32)
    out = M.moe_expert_linear(x, w, seg, seg[1:])
    at = torch.tensor([0, 1, 32767, 32768, 65535, 65536, n - 1], device="cuda")
    assert torch.equal(out[at], (x[at].float() @ w[0].float().T).to(torch.bfloat16))
    del out
    n, K, N = 70000, 65536, 16
    x = torch.zeros(n, K, dtype=torch.bfloat16, device="cuda")
    w = ints(5, 1, N, K)
    x[:, 40000:40008] = ints(6, n, 8)
    want = (x[:, 40000:40008].float() @ w[0, :, 40000:40008].float().T).to(torch.bfloat16)
    seg = torch.tensor([0, n], device="cuda", dtype=torch.int32)
    back = torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.int32)
    for tok, ref in ((None, want), (back, want.flip(0))):
        assert torch.equal(M.moe_expert_linear(x, w, seg, seg[1:], row_token=tok), ref)
    few = torch.tensor([n - 1, 0, 65536, 32768], device="cuda", dtype=torch.int32)
    four = torch.tensor([0, 4], device="cuda", dtype=torch.int32)
    assert torch.equal(M.moe_expert_linear(x, w, four, four[1:], row_token=few), want[few.long()])


def test_expert_linear_without_any_token(M):
    # no rows of x at all: every named token is outside, its row is zeros
    w = ints(7, 2, 32, 64)
    tok = torch.tensor([0, -1, 5], device="cuda", dtype=torch.int32)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    out = M.moe_expert_linear(x, w, torch.tensor([0, 2, 3], device="cuda", dtype=torch.int32),
                              torch.tensor([2, 1], device="cuda", dtype=torch.int32), row_token=tok, err_flag=flag)
    assert not out.any() and int(flag.item()) == L.MOE_FLAG_BAD_INDEX


def test_expert_linear_overlapping_segments_take_nothing(M):
    c = draw_layer(8, 40, 4, 2, 64, 32)
    c["counts"] = np.full(4, 60, np.int32)
    c["offsets"] = np.array([0, 5, 10, 15], np.int32)
    out, flag = run_expert(M, c, None, True)
    assert flag == L.MOE_FLAG_BAD_INDEX and np.all(values(out) == 3.0)


@pytest.mark.parametrize("T,gather", [(2, True), (300, False)])
def test_expert_linear_wait_runs_out_and_the_next_launch_is_clean(M, T, gather):
    c = draw_layer(6, T, 4, 2, 1024, 4096, gather=gather)
    want, flag = run_expert(M, c, None, gather)
    assert flag == 0
    M.moe_debug_withhold_expert_stage(2)
    _, flag = run_expert(M, c, None, gather)
    assert flag & L.MOE_FLAG_TIMEOUT
    again, flag = run_expert(M, c, None, gather)
    assert flag == 0 and torch.equal(again, want)
    with pytest.raises(M.MoeTailError):
        M.moe_debug_withhold_expert_stage(-2)


# ---------------------------------------------------------------------------
# the projection with adapters
# ---------------------------------------------------------------------------

ADAPTER = [  # T, N, K, R, L, ids
    (1, 4096, 6144, 16, 16, "one"), (1, 256, 64, 8, 1, "none"), (2, 528, 1032, 24, 3, "mix"), (7, 272, 256, 64, 5, "mix"),
    (64, 1024, 2048, 16, 64, "each"), (64, 256, 512, 256, 6, "mix"), (65, 144, 136, 8, 70, "each"),
    (200, 272, 320, 32, 4, "runs"), (300, 512, 512, 64, 9, "mix"), (1000, 256, 264, 16, 8, "runs"),
    (513, 16, 8, 8, 2, "mix"), (128, 512, 256, 128, 1, "one"), (1100, 272, 192, 72, 300, "mix"), (33, 64, 64, 16, 1024, "each"),
    (2100, 128, 128, 40, 12, "runs"), (260, 128, 256, 136, 3, "none"),
    (2048, 272, 136, 8, 40, "mix"), (2049, 272, 136, 8, 40, "mix"), (1400, 144, 264, 16, 7, "mix"), (8, 272, 256, 256, 3, "mix"),
    (1, 64, 64, 256, 2, "one"), (9, 272, 264, 256, 3, "mix"), (200, 272, 320, 104, 4, "runs"), (130, 65536, 64, 8, 3, "mix"),
]


def draw_adapter(T, N, K, R, L_, what):
    rng = np.random.default_rng([230, T, N, K, R, L_])
    ids = {"one": np.full(T, L_ - 1), "none": np.full(T, -1), "each": np.arange(T) % L_,
           "mix": rng.integers(-1, L_, T), "runs": np.sort(rng.integers(-1, L_, T))}[what].astype(np.int32)
    return dict(x=draw_bf16(rng, (T, K), 1.0), w=draw_bf16(rng, (N, K), 0.05), a=draw_bf16(rng, (L_, R, K), 0.05),
                b=draw_bf16(rng, (L_, N, R), 0.1), ids=ids, scale=rng.uniform(0.5, 2.0, L_).astype(np.float32))


def run_adapter(M, c, act, **kw):
    T, N = len(c["x"]), len(c["w"])
    out, flag = Guarded((T, N // 2 if act else N), torch.bfloat16, fill=3.0), Guarded((1,), torch.int32, fill=0)
    M.moe_adapter_linear(dev(c["x"]), dev(c["w"]), dev(c["a"]), dev(c["b"]), devn(c["ids"]), devn(c["scale"]), act=act,
                         out=out.t, err_flag=flag.t, **kw)
    check_all(out=out, flag=flag)
    return out.t, int(flag.t.item())


def check_adapter(c, got, act, what):
    want, err = O.adapter_linear(c["x"], c["w"], c["a"], c["b"], c["ids"], c["scale"], act,
                                 rel_sum(c["x"].shape[1] + c["a"].shape[1]), 2.0 ** -16)
    check_rows(got, want, err, what)


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("T,N,K,R,L_,ids", ADAPTER)
def test_adapter_linear(M, T, N, K, R, L_, ids, act):
    c = draw_adapter(T, N, K, R, L_, ids)
    out, flag = run_adapter(M, c, act)
    assert flag == 0
    check_adapter(c, values(out), act, f"T={T} N={N} K={K} R={R} L={L_} {ids}")


@pytest.mark.parametrize("T", [5, 90, 400, 1100])
def test_adapter_linear_ids_outside(M, T):
    c = draw_adapter(T, 144, 136, 16, 4, "mix")
    c["ids"][1], c["ids"][-1], c["ids"][2] = 4, 2 ** 31 - 1, -2 ** 31
    out, flag = run_adapter(M, c, None)
    assert flag == L.MOE_FLAG_BAD_INDEX
    check_adapter(c, values(out), None, "outside")


@pytest.mark.parametrize("T", [3, 100, 600, 1100])
def test_adapter_of_another_token_does_not_leak(M, T):
    # NaN and infinities in one adapter, and in one token, reach the tokens they belong to only
    c = draw_adapter(T, 144, 136, 16, 3, "mix")
    c["ids"][:3] = [0, 1, 2]
    clean, _ = run_adapter(M, c, None)
    d = {**c, "a": c["a"].copy(), "b": c["b"].copy()}
    d["a"][1, 3, 5], d["b"][1, 7, 2] = 0x7FC0, 0x7F80
    out, _ = run_adapter(M, d, None)
    mine = c["ids"] == 1
    assert np.array_equal(host16(out)[~mine], host16(clean)[~mine])
    assert not np.isfinite(values(out)[mine]).any()
    x = c["x"].copy()
    x[2, 9] = 0x7F80
    out, _ = run_adapter(M, {**c, "x": x}, None)
    keep = np.arange(T) != 2
    assert np.array_equal(host16(out)[keep], host16(clean)[keep])
    assert not np.isfinite(values(out)[2]).any()


@pytest.mark.parametrize("T", [3, 700])
def test_adapter_linear_offsets_beyond_31_bits(M, T):
    # tables of more than 2^32 elements; one non-zero column each, so that every sum is a whole number
    N, K, R, n = 64, 65536, 72, 1024
    ids = torch.tensor([n - 1, 0, 700], device="cuda", dtype=torch.int32).repeat(T // 3 + 1)[:T]
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[:, 50001] = ints(1, T)
    w = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    w[:, 50001] = ints(2, N)
    a = torch.zeros(n, R, K, dtype=torch.bfloat16, device="cuda")
    a[:, 71, 50001] = 1 + (torch.arange(n, device="cuda") % 3)
    b = torch.zeros(n, N, R, dtype=torch.bfloat16, device="cuda")
    b[:, :, 71] = ints(3, n, N)
    scale = torch.full((n,), 2.0, device="cuda")
    i = ids.long()
    xv = x[:, 50001].float()[:, None]
    want = (xv * w[:, 50001].float() + 2 * xv * a[i, 71, 50001].float()[:, None] * b[i, :, 71].float()).to(torch.bfloat16)
    assert torch.equal(M.moe_adapter_linear(x, w, a, b, ids, scale), want)


@pytest.mark.parametrize("T", [1, 40, 200, 600, 1000])
def test_adapter_linear_same_bits_again_and_with_a_given_workspace(M, T):
    c = draw_adapter(T, 272, 328, 24, 7, "mix")
    a, _ = run_adapter(M, c, "swiglu")
    ws = torch.full((M.lib().moe_adapter_linear_workspace(T, 272, 328, 24, 7),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        b, _ = run_adapter(M, c, "swiglu", workspace=ws)
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 40, 300, 2100])
def test_adapter_linear_reads_what_the_kernels_before_it_wrote(M, T):
    # the weights, the tokens and an adapter's tables are outputs of calls just made on the stream
    K, N, R, n = 512, 768, 8, 3
    g = torch.Generator(device="cuda").manual_seed(T)
    draw = lambda *s: (torch.randn(*s, generator=g, device="cuda") / 16).to(torch.bfloat16)
    ids = (torch.arange(T, device="cuda") % (n + 1) - 1).int()
    scale = torch.rand(n, generator=g, device="cuda")

    def made(rows, cols, out):  # rows x cols as one expert's products
        off, cnt = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([rows], dtype=torch.int32, device="cuda")
        x, w = draw(rows, 4096), draw(1, cols, 4096)
        return lambda: M.moe_expert_linear(x, w, off, cnt, out=out)

    x, w = torch.empty(T, K, dtype=torch.bfloat16, device="cuda"), torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    a, b = (torch.empty(*s, dtype=torch.bfloat16, device="cuda") for s in ((n * R, K), (n * N, R)))
    calls = [made(T, K, x), made(n * R, K, a), made(n * N, R, b), made(N, K, w)]
    run = lambda: M.moe_adapter_linear(x, w, a.view(n, R, K), b.view(n, N, R), ids, scale, act="swiglu")
    for c in calls:
        c()
    torch.cuda.synchronize()
    want = run()
    for order in (calls, calls[::-1]):
        for t in (x, w, a, b):
            t.fill_(float("nan"))
        for c in order:
            c()
        assert torch.equal(run(), want)


def test_adapter_linear_empty_batch(M):
    c = draw_adapter(4, 64, 64, 8, 2, "mix")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    out = M.moe_adapter_linear(e, dev(c["w"]), dev(c["a"]), dev(c["b"]), torch.empty(0, dtype=torch.int32, device="cuda"),
                               devn(c["scale"]))
    assert out.shape == (0, 64)


# ---------------------------------------------------------------------------
# together: the layer
# ---------------------------------------------------------------------------

def layer(M, g, p):
    """One MoE layer: router, grouped routing, map, experts, shared expert with adapters, tail."""
    logits = M.moe_router_logits_fp32(g["x"], g["w_gate"])
    ids, w = M.moe_group_topk_route(logits, p["k"], 2.5, bias=g["bias"], n_group=4, topk_group=2)
    row_map, row_token, offsets, counts = M.moe_expert_map(ids, p["E"], block=p["block"])
    h = M.moe_expert_linear(g["x"], g["w13"], offsets, counts, row_token=row_token, act="swiglu")
    rows = M.moe_expert_linear(h, g["w2"], offsets, counts)
    sh = M.moe_adapter_linear(g["x"], g["s13"], g["a13"], g["b13"], g["adapters"], g["scale"], act="swiglu")
    shared = M.moe_adapter_linear(sh, g["s2"], g["a2"], g["b2"], g["adapters"], g["scale"])
    ro, no = M.moe_finalize_add_rmsnorm(rows, row_map, w, shared, g["residual"], g["gamma"], 1e-6)
    return dict(logits=logits, ids=ids, w=w, row_map=row_map, row_token=row_token, offsets=offsets, counts=counts, h=h,
                rows=rows, sh=sh, shared=shared, ro=ro, no=no)


def draw_whole(T, H, I, E, k, block, seed=0):
    rng = np.random.default_rng([240, seed, T, H])
    R, n = 16, 5
    c = dict(x=draw_bf16(rng, (T, H), 1.0), w_gate=draw_bf16(rng, (E, H), 0.05), w13=draw_bf16(rng, (E, 2 * I, H), 0.05),
             w2=draw_bf16(rng, (E, H, I), 0.05), s13=draw_bf16(rng, (2 * I, H), 0.05), s2=draw_bf16(rng, (H, I), 0.05),
             a13=draw_bf16(rng, (n, R, H), 0.05), b13=draw_bf16(rng, (n, 2 * I, R), 0.05),
             a2=draw_bf16(rng, (n, R, I), 0.05), b2=draw_bf16(rng, (n, H, R), 0.05), residual=draw_bf16(rng, (T, H), 1.0))
    f = dict(bias=(rng.standard_normal(E) * 0.1).astype(np.float32), scale=rng.uniform(0.5, 2, n).astype(np.float32),
             gamma=(1 + 0.1 * rng.standard_normal(H)).astype(np.float32), adapters=rng.integers(-1, n, T).astype(np.int32))
    return {**c, **f}, {**{n: dev(v) for n, v in c.items()}, **{n: devn(v) for n, v in f.items()}}, dict(E=E, k=k, block=block)


@pytest.mark.parametrize("T,H,I,E,k,block", [(1, 512, 128, 16, 4, 1), (28, 264, 136, 24, 3, 16), (300, 256, 128, 16, 4, 1),
                                               (1100, 128, 72, 16, 4, 1)])
def test_layer_step_by_step(M, T, H, I, E, k, block):
    """The operators as a layer uses them, each step against its definition on
    the GPU's own inputs of that step."""
    c, g, p = draw_whole(T, H, I, E, k, block)
    o = layer(M, g, p)
    n = {name: v.cpu().numpy() for name, v in o.items() if v.dtype != torch.bfloat16}
    rids, rw = O.group_topk_route(n["logits"], k, 2.5, bias=c["bias"], n_group=4, topk_group=2)
    assert np.array_equal(n["ids"], rids)
    assert np.all(np.abs(n["w"] - rw) <= rw * U * (2 * (E / 32 + 12) + k + 4))
    for got, want in zip((n["row_map"], n["row_token"], n["offsets"], n["counts"]), O.expert_map(rids, E, block)):
        assert np.array_equal(got, want)
    h = host16(o["h"])
    for got, x, w, tok, act in [(o["h"], c["x"], c["w13"], n["row_token"], "swiglu"), (o["rows"], h, c["w2"], None, None)]:
        want = O.expert_linear(x, w, n["offsets"], n["counts"], tok, act, rel_sum(x.shape[1]))
        r = sorted(want)
        check_rows(values(got)[r], np.stack([want[i][0] for i in r]), np.stack([want[i][1] for i in r]), "experts")
    for got, x, w, a, b, act in [(o["sh"], c["x"], c["s13"], c["a13"], c["b13"], "swiglu"),
                                 (o["shared"], host16(o["sh"]), c["s2"], c["a2"], c["b2"], None)]:
        check_adapter(dict(x=x, w=w, a=a, b=b, ids=c["adapters"], scale=c["scale"]), values(got), act, "shared")
    rows = host16(o["rows"]).copy()
    ref = O.finalize_add_rmsnorm(rows, n["row_map"], n["w"], host16(o["shared"]), None, c["residual"], c["gamma"], 1e-6)
    from _tol import check_bf16, tail_deltas
    dr, dn = tail_deltas(ref, k + 2, c["gamma"], 1e-6)
    check_bf16(f"layer T={T} residual_out", host16(o["ro"]), ref["residual_out"], ref["r"], dr)
    check_bf16(f"layer T={T} normed", host16(o["no"]), ref["normed"], ref["normed64"], dn)


@pytest.mark.parametrize("T", [1, 40, 300, 1100])
def test_layer_captured_and_replayed(M, T):
    _, g, p = draw_whole(T, 256, 128, 16, 4, 1)
    eager = layer(M, g, p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(M, g, p)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(M, g, p)
    for _ in range(3):
        for v in out.values():
            v.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for name in eager:
        assert torch.equal(eager[name], out[name]), name
    # new inputs in the same buffers, replayed
    _, g2, _ = draw_whole(T, 256, 128, 16, 4, 1, seed=1)
    for name in g:
        g[name].copy_(g2[name])
    graph.replay()
    fresh = layer(M, g2, p)
    for name in fresh:
        assert torch.equal(fresh[name], out[name]), name


@pytest.mark.parametrize("T", [2, 60, 1100])
def test_layers_on_two_streams_at_once(M, T):
    _, g, p = draw_whole(T, 512, 256, 16, 4, 1)
    want = layer(M, g, p)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append(layer(M, g, p))
    # an explicit stream argument, as a stream and as a handle
    for st in (streams[0], streams[1].cuda_stream):
        got.append({"ids": M.moe_group_topk_route(want["logits"], 4, 2.5, bias=g["bias"], n_group=4, topk_group=2, stream=st)[0],
                    "h": M.moe_expert_linear(g["x"], g["w13"], want["offsets"], want["counts"],
                                             row_token=want["row_token"], act="swiglu", stream=st),
                    "shared": M.moe_adapter_linear(want["sh"], g["s2"], g["a2"], g["b2"], g["adapters"], g["scale"],
                                                   stream=st)})
    torch.cuda.synchronize()
    for o in got:
        for name in o:
            assert torch.equal(o[name], want[name]), name


def test_workspaces_of_two_graphs_are_apart(M):
    """Two captured layers replayed at the same time on two streams."""
    _, g, p = draw_whole(50, 512, 256, 16, 4, 1)
    _, g2, _ = draw_whole(50, 512, 256, 16, 4, 1, seed=1)
    layer(M, g, p)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for inputs in (g, g2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(layer(M, inputs, p))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for inputs, out in zip((g, g2), outs):
        fresh = layer(M, inputs, p)
        for name in fresh:
            assert torch.equal(fresh[name], out[name]), name


@pytest.mark.parametrize("call", ["route", "map", "expert", "adapter"])
@pytest.mark.parametrize("T", [2, 300, 1100])
def test_refused_launch_is_reported_and_the_next_call_is_clean(M, call, T):
    _, g, p = draw_whole(T, 256, 128, 16, 4, 1)
    o = layer(M, g, p)
    run = {"route": lambda: M.moe_group_topk_route(o["logits"], 4, 2.5, bias=g["bias"], n_group=4, topk_group=2)[0],
           "map": lambda: M.moe_expert_map(o["ids"], 16)[0],
           "expert": lambda: M.moe_expert_linear(o["h"], g["w2"], o["offsets"], o["counts"]),
           "adapter": lambda: M.moe_adapter_linear(o["sh"], g["s2"], g["a2"], g["b2"], g["adapters"], g["scale"])}[call]
    M.moe_debug_fail_next_launch(True)
    try:
        with pytest.raises(M.MoeTailError) as ei:
            run()
    finally:
        M.moe_debug_fail_next_launch(False)
    assert ei.value.status == L.MOE_ERR_CUDA
    want = {"route": "ids", "map": "row_map", "expert": "rows", "adapter": "shared"}[call]
    assert torch.equal(run(), o[want])
