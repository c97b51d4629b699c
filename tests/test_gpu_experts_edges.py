"""GPU tests of the expert operators where they met an edge: what runs before
a call, waits that run out, scores and sizes at the ends of their ranges.
Tolerances as in test_gpu_experts.py."""

import time

import numpy as np
import pytest
import torch

from _guard import Guarded, check_all
from moe_decode_layer_logits_gb300 import _lib as L
from test_gpu_experts import (M, check_adapter, dev, devn, draw_adapter, run_adapter, values)  # noqa: F401

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
