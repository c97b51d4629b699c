"""Host side of the expert operators at the edges, no GPU."""

import subprocess
import sys


def test_package_imports_where_torch_has_no_cuda(repo_root):
    # a torch built without CUDA has none of torch._C's CUDA names; what needs no GPU still works there
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import moe_decode_layer_logits_gb300 as M
from moe_decode_layer_logits_gb300 import inputs, sharding
assert sharding.token_shard(7, 1, 2) == (4, 7)
try:
    M.moe_expert_map(torch.zeros(2, 2, dtype=torch.int32), 4)
except TypeError as e:
    assert "CUDA" in str(e)
else:
    raise AssertionError("not refused")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=repo_root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
