"""GPU tests of the expert operators where they met an edge: what runs before
a call, waits that run out, scores and sizes at the ends of their ranges.
Tolerances as in test_gpu_experts.py."""

import time

import numpy as np
import pytest
import torch

import oracle as O
from _guard import Guarded, check_all
from moe_decode_layer_logits_gb300 import _lib as L
from test_gpu_experts import (M, U, check_adapter, dev, devn, draw_adapter, draw_layer, ints, run_adapter, run_expert,  # noqa: F401
                              values)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", [None, "swiglu"])
def test_adapter_linear_behind_a_kernel_that_runs_long(M, act):
    # An expert map of 2^30 slots lets its dependents start at once and then
    # runs for longer than the probes of one bounded wait last (about 0.1 s):
    # the call behind it may be resident all that time, and must not give up.
    c = draw_adapter(3, 512, 256, 16, 2, "mix")
    T, k, E = 1 << 25, 32, 1024
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    out = Guarded((3, 256 if act else 512), torch.bfloat16, fill=3.0)
    flag = Guarded((1,), torch.int32, fill=0)
    t = [dev(c[n]) for n in ("x", "w", "a", "b")] + [devn(c["ids"]), devn(c["scale"])]
    torch.cuda.synchronize()
    start = time.perf_counter()
    _, _, _, counts = M.moe_expert_map(ids, E)
    M.moe_adapter_linear(*t, act=act, out=out.t, err_flag=flag.t)
    torch.cuda.synchronize()
    print(f"both calls took {time.perf_counter() - start:.3f} s")
    check_all(out=out, flag=flag)
    assert int(flag.t.item()) == 0 and int(counts.sum(dtype=torch.int64).item()) == T * k
    check_adapter(c, values(out.t), act, "behind a long kernel")


def wrong_where_nan(out, want):
    """Where a call that gave up left NaN; everything else is the clean call's."""
    lost = torch.isnan(out)
    assert torch.equal(out[~lost], want[~lost])
    return lost


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("T,gather", [(2, True), (2, False), (300, True), (300, False)])  # single CTAs, pairs
def test_expert_linear_leaves_nan_where_a_wait_ran_out(M, T, gather, act):
    c = draw_layer(6, T, 4, 2, 1024, 4096, gather=gather)
    want, _ = run_expert(M, c, act, gather)
    for stage in (0, 2):
        M.moe_debug_withhold_expert_stage(stage)
        out, flag = run_expert(M, c, act, gather)      # (no error flag needed to see it)
        assert flag & L.MOE_FLAG_TIMEOUT
        assert 0 < int(wrong_where_nan(out, want).sum()) < out.numel()
    again, flag = run_expert(M, c, act, gather)
    assert flag == 0 and torch.equal(again, want)


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("T,few", [(3, True), (130, True), (1100, False)])
def test_adapter_linear_leaves_nan_where_a_wait_ran_out(M, T, few, act):
    c = draw_adapter(T, 8192, 1024, 16, 4, "mix")
    want, flag = run_adapter(M, c, act)
    assert flag == 0
    M.moe_debug_withhold_expert_stage(0)
    out, flag = run_adapter(M, c, act)
    assert flag & L.MOE_FLAG_TIMEOUT
    lost = wrong_where_nan(out, want)
    assert 0 < int(lost.sum()) < out.numel()
    if not few:  # both launches gave up: whole tokens by the low-rank product, tiles by the projection
        assert lost.all(1).any() and (lost.any(1) & ~lost.all(1)).any()
        assert not lost.all(1)[torch.from_numpy(c["ids"] < 0).cuda()].any()
    again, flag = run_adapter(M, c, act)
    assert flag == 0 and torch.equal(again, want)


def check_weights(M, lg, k, kw, scale=2.5):
    """ids and weights against the 64-bit definition, relative to each weight.
    The argument of an exponential is a difference rounded by 2^-24 of its own
    size, D at most (from the row's maximum, or from the best chosen logit
    where that lies 16 below it; no difference for a sigmoid of 16 or less);
    terms more than 745 down, -inf among them, are 0 in FP32 and FP64 alike and
    have no rounding.  The rest as in test_gpu_experts.py.  1e-37: below FP32's normal numbers."""
    ids, w = M.moe_group_topk_route(devn(lg), k, scale, **{**kw, "bias": None if kw.get("bias") is None else devn(kw["bias"])})
    rids, rw = O.group_topk_route(lg, k, scale, **kw)
    assert np.array_equal(ids.cpu().numpy(), rids)
    z = np.take_along_axis(lg.astype(np.float64), rids.astype(np.int64), 1)
    top = z.max(1, keepdims=True)
    ref = lg.max(1, keepdims=True).astype(np.float64) if kw["scores"] == "softmax" else np.zeros_like(top)
    with np.errstate(invalid="ignore"):
        d = np.abs(z - np.where(top - ref < -16, top, ref))
    D = np.where(d < 745, d, 0.0).max(1, keepdims=True)
    tol = np.abs(rw) * U * (2 * (D + lg.shape[1] / 32 + 12) + k + 4) + 1e-37
    assert np.all(np.abs(w.cpu().numpy() - rw) <= tol)
    return rw


@pytest.mark.parametrize("E,G,TG,k", [(64, 1, 1, 2), (64, 8, 3, 8), (256, 8, 4, 8), (1024, 32, 5, 32)])
@pytest.mark.parametrize("bias", [False, True])
def test_group_route_renormalised_weights_of_tiny_sigmoids(M, E, G, TG, k, bias):
    rng = np.random.default_rng([301, E, k])
    lg = rng.uniform(-120, -90, (16, E)).astype(np.float32)  # every score below the smallest FP32 number, or near it
    lg[1] = -92
    lg[2] = rng.uniform(-700, -695, E)
    lg[3] = rng.uniform(-700, 0, E)
    lg[4] = rng.uniform(-100, -15, E)
    lg[5] = rng.uniform(-17, -15, E)
    lg[6] = rng.uniform(-110, -80, E)
    lg[7, ::5] = -np.inf
    lg[8] = np.finfo(np.float32).min
    lg[9, 3] = 1.0
    lg[10] = rng.uniform(-95, 0, E)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
    for top in (1, 2):
        kw = dict(bias=b, n_group=G, topk_group=TG, group_top=top, scores="sigmoid")
        rw = check_weights(M, lg, k, {**kw, "renormalize": True})
        assert np.allclose(rw[:8].sum(1), 2.5)              # (the definition has no zero rows there)
        check_weights(M, lg, k, {**kw, "renormalize": False})


@pytest.mark.parametrize("E,G,TG,k", [(64, 1, 1, 2), (64, 8, 3, 8), (256, 8, 4, 8), (512, 16, 3, 20)])
def test_group_route_renormalised_weights_of_softmax_scores_far_below_the_largest(M, E, G, TG, k):
    # the bias takes out the expert that has the mass; the chosen lie 20 to 700 below it
    rng = np.random.default_rng([302, E, k])
    lg = rng.standard_normal((12, E)).astype(np.float32)
    for t, gap in enumerate([0, 10, 15.9, 16.1, 20, 60, 87, 95, 104, 150, 400, 690]):
        lg[t, 5] = lg[t].max() + gap
    b = (rng.standard_normal(E) * 0.1).astype(np.float32)
    b[5] = -9.0
    for top in (1, 2):
        rw = check_weights(M, lg, k, dict(bias=b, n_group=G, topk_group=TG, group_top=top, scores="softmax", renormalize=True))
        assert np.allclose(rw.sum(1), 2.5)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size,G,TG,big", [(2, 8, 3, 1e4), (2, 16, 7, 3e5), (2, 4, 1, 300.0), (16, 8, 4, 1e5), (32, 8, 3, 2e6)])
def test_group_route_group_scores_whose_large_biases_cancel(M, scores, size, G, TG, big):
    # a group's two best choice values are +B + s and -B + s': each is rounded by
    # up to 2^-24 B in 32 bits, while the groups' sums differ by the scores alone
    rng = np.random.default_rng([303, size, G, int(big)])
    E = size * G
    lg = rng.standard_normal((200, E)).astype(np.float32)
    b = np.full(E, -4 * big, np.float32)
    for g in range(G):
        B = np.float32(big * rng.uniform(0.9, 1.1))
        b[g * size + rng.integers(size // 2)] = B
        b[g * size + size // 2 + rng.integers(size - size // 2)] = -B
    k = min(8, size * TG)
    kw = dict(bias=b, n_group=G, topk_group=TG, group_top=2, scores=scores, renormalize=True)
    check_weights(M, lg, k, kw)
    # groups of which some are masked by the type's lowest value, or hold nothing but it
    b[:size] = np.finfo(np.float32).min
    b[size:size + 1] = np.finfo(np.float32).min
    check_weights(M, lg, k, {**kw, "bias": b})
    b[:size] = -np.inf
    check_weights(M, lg, k, {**kw, "bias": b})


def test_expert_linear_of_the_most_rows(M):
    # 2^31 - 1 rows, nearly all of one expert: row counts next to the end of 32 bits
    n, K, N = 2 ** 31 - 1, 8, 8
    x, w = ints(8, 7, K), ints(9, 2, N, K)
    token = torch.randint(0, 7, (n,), dtype=torch.int32, device="cuda")
    seg = torch.tensor([0, 5, n], device="cuda", dtype=torch.int32)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = M.moe_expert_linear(x, w, seg, seg[1:] - seg[:2], row_token=token, err_flag=flag)
    assert int(flag.item()) == 0
    want = torch.einsum("tk,enk->etn", x.float(), w.float()).to(torch.bfloat16)
    assert torch.equal(out[:5], want[0][token[:5].long()])
    for a in range(5, n, 1 << 26):
        b = min(n, a + (1 << 26))
        assert torch.equal(out[a:b], want[1][token[a:b].long()]), a


def test_calls_without_the_short_way_to_the_stream(M, monkeypatch):
    ids = torch.tensor([[1, 0], [1, 2]], dtype=torch.int32, device="cuda")
    want = M.moe_expert_map(ids, 4)
    monkeypatch.setattr(M, "_raw_stream", None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = M.moe_expert_map(ids, 4)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,R", [(3, 16), (200, 72), (1100, 16), (1100, 72), (2100, 256)])  # few tokens, then many
def test_adapter_linear_keeps_the_low_rank_product_in_32_bits(M, T, R):
    # whole numbers: W = D - A, B = 1, so that y = D x; A x has up to 21 bits
    # (64 * 127 * 255) and has to cancel to the last
    g = torch.Generator(device="cuda").manual_seed(R)
    draw = lambda lim, *s: torch.randint(-lim, lim + 1, s, generator=g, device="cuda").to(torch.bfloat16)
    K = 64
    x, a = draw(127, T, K), draw(255, 2, R, K)
    a[1] = a[0]
    at = torch.arange(R, device="cuda") % K
    w = -a[0].float()
    keep = w[torch.arange(R, device="cuda"), at]
    w[torch.arange(R, device="cuda"), at] = torch.where(keep >= 255, keep - 1, keep + 1)
    sign = torch.where(keep >= 255, -1.0, 1.0)
    b = torch.eye(R, device="cuda", dtype=torch.bfloat16).repeat(2, 1, 1)
    ids = (torch.arange(T, device="cuda") % 2).int()
    out = M.moe_adapter_linear(x, w.to(torch.bfloat16), a, b, ids, torch.ones(2, device="cuda"))
    assert int((x.double() @ a[0].double().T).abs().max()) > 2 ** 17  # (more than two BF16 hold)
    assert torch.equal(out.float(), x.float()[:, at] * sign)


@pytest.mark.parametrize("T", [2, 1100])
def test_adapter_linear_low_rank_products_beyond_the_largest_bf16(M, T):
    # v = (2 - 2^-7 + 2^-8 + 2^-9) 2^127: finite in FP32, infinite if rounded to BF16
    K, N, R = 64, 64, 16
    x = torch.zeros(T, K, device="cuda")
    x[:, 0], x[:, 1] = torch.finfo(torch.bfloat16).max, 1.5 * 2.0 ** 119
    x[1::2] *= -1
    a = torch.zeros(1, R, K, device="cuda")
    a[0, :, :2] = 1
    b = torch.zeros(1, N, R, device="cuda")
    b[0, torch.arange(N), torch.arange(N) % R] = 2.0 ** -126
    w = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    bf = lambda t: t.to(torch.bfloat16)
    out = M.moe_adapter_linear(bf(x), w, bf(a), bf(b), torch.zeros(T, dtype=torch.int32, device="cuda"),
                               torch.ones(1, device="cuda"))
    want = torch.full((T, N), 4.0, device="cuda")           # 3.996 in BF16
    want[1::2] *= -1
    assert torch.equal(out.float(), want)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,TG,k", [(16, 1, 1, 5), (64, 4, 2, 6), (256, 1, 1, 8), (600, 1, 1, 3)])
def test_group_route_equal_experts_before_a_better_one_that_32_bits_cannot_tell(M, scores, E, G, TG, k):
    # masked experts of the same bias are equal in any precision; one among them
    # has a score that only 64 bits see, and comes first although it stands last
    rng = np.random.default_rng([304, E, k])
    lg = np.full((40, E), -np.inf, np.float32)
    b = np.full(E, 0.25, np.float32)
    size = E // G
    for t in range(len(lg)):
        live = rng.permutation(size)[:k - 1]           # fewer than k experts of any weight
        lg[t, live] = rng.standard_normal(k - 1)
        rest = np.setdiff1d(np.arange(size), live)
        some = rng.permutation(rest[1:])[:1 + t % 3]
        lg[t, some] = rng.uniform(-32, -20, len(some))  # 64 bits: 0.25 + 1e-14 .. 2e-9
    for top in (1, 2):
        check_weights(M, lg, k, dict(bias=b, n_group=G, topk_group=TG, group_top=top, scores=scores, renormalize=True))
    lg[::2] = np.where(np.isinf(lg[::2]), np.float32(np.nan), lg[::2])
    ids, _ = M.moe_group_topk_route(devn(lg), k, 1.0, bias=devn(b), n_group=G, topk_group=TG, scores=scores)
    assert np.array_equal(ids.cpu().numpy(), O.group_topk_route(lg, k, 1.0, bias=b, n_group=G, topk_group=TG,
                                                               scores=scores)[0])
