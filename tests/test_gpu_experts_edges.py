"""GPU tests of the expert operators where they met an edge: what runs before
a call, waits that run out, scores and sizes at the ends of their ranges.
Tolerances as in test_gpu_experts.py."""

import time

import numpy as np
import pytest
import torch

from _guard import Guarded, check_all
from moe_decode_layer_logits_gb300 import _lib as L
from test_gpu_experts import (M, check_adapter, dev, devn, draw_adapter, draw_layer, run_adapter, run_expert,  # noqa: F401
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
