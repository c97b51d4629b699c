"""Decode MoE-layer tail for one sm_103a GPU (GLM-5.x style MoE layers).

Python binding of the C ABI in ``include/moe_tail.h``: argument marshalling
only.  Every step runs in the CUDA kernels of ``libmoe_tail.so``; PyTorch
provides device memory and the stream.  Functions take CUDA tensors and
launch on ``stream`` (default: the current torch stream); output tensors are
allocated with torch when not given.

* ``moe_router_logits_fp32(x, w_gate)``      -> FP32 logits [T, E]
* ``moe_topk_route(logits, k, scale)``       -> ids [T, k] int32, weights [T, k] FP32
* ``moe_finalize_add_rmsnorm(...)``          -> (residual_out, normed) BF16 [T, H]
* ``moe_tail_fused(logits, k, scale, ...)``  -> (residual_out, normed, ids, weights)
* ``moe_group_topk_route(logits, k, scale, ...)`` -> ids [T, k] int32, weights [T, k] FP32
* ``moe_expert_map(ids, E, block)``          -> (row_map, row_token, offsets, counts) int32
* ``moe_expert_linear(x, w, offsets, counts, ...)`` -> expert rows BF16 [n_rows, N or N/2]
* ``moe_adapter_linear(x, w, a, b, ids, scale, ...)`` -> BF16 [T, N or N/2]
"""

from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib
from ._lib import MoeTailError, check, lib

__all__ = [
    "moe_debug_withhold_stream_stage",
    "moe_debug_withhold_router_stage",
    "moe_debug_withhold_expert_stage",
    "moe_debug_fail_next_launch",
    "moe_debug_router_tc_shape",
    "moe_router_logits_fp32",
    "moe_topk_route",
    "moe_finalize_add_rmsnorm",
    "moe_tail_fused",
    "moe_group_topk_route",
    "moe_expert_rows",
    "moe_expert_map",
    "moe_expert_linear",
    "moe_adapter_linear",
    "MoeTailError",
    "lib",
]


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t, dtype, name, ndim=None, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    return t.data_ptr()


def moe_router_logits_fp32(x, w_gate, logits_out=None, err_flag=None, stream=None):
    """logits[T, E] = x[T, H] . w_gate[E, H]^T (BF16 in, FP32 accumulate and out).
    err_flag: optional int32 CUDA tensor; MOE_FLAG_TIMEOUT is OR-ed into it
    when a bounded wait of the tensor-memory kernel (T > 64) runs out (the
    affected logits are NaN either way)."""
    T, H = x.shape
    E = w_gate.shape[0]
    if logits_out is None:
        logits_out = torch.empty((T, E), dtype=torch.float32, device=x.device)
    st = lib().moe_router_logits_fp32(_ptr(x, torch.bfloat16, "x", 2), _ptr(w_gate, torch.bfloat16, "w_gate", 2),
                                      _ptr(logits_out, torch.float32, "logits_out", 2), T, H, E,
                                      _ptr(err_flag, torch.int32, "err_flag", optional=True), _stream(stream))
    check(st, "moe_router_logits_fp32")
    return logits_out


def moe_topk_route(logits, k, routed_scale, topk_ids=None, topk_w=None, stream=None):
    """Top-k experts per token (descending, ties to the lower index) and
    routed_scale * softmax over the selected logits."""
    T, E = logits.shape
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    st = lib().moe_topk_route(_ptr(logits, torch.float32, "logits", 2), _ptr(topk_ids, torch.int32, "topk_ids"),
                              _ptr(topk_w, torch.float32, "topk_w"), T, E, int(k), float(routed_scale),
                              _stream(stream))
    check(st, "moe_topk_route")
    return topk_ids, topk_w


def moe_finalize_add_rmsnorm(rows, row_map, topk_w, shared, residual, gamma, eps, partials=None,
                             residual_out=None, normed_out=None, err_flag=None, stream=None):
    """The fused tail: sum_j w_j rows[map_j] + shared + sum_r partials[r] + residual,
    then RMSNorm * gamma; both outputs rounded to BF16 once."""
    T, H = residual.shape
    k = 0 if row_map is None else int(row_map.shape[1])
    R = 0 if partials is None else int(partials.shape[0])
    n_rows = 0 if rows is None else int(rows.shape[0])
    if residual_out is None:
        residual_out = torch.empty_like(residual)
    if normed_out is None:
        normed_out = torch.empty_like(residual)
    st = lib().moe_finalize_add_rmsnorm(
        _ptr(rows, torch.bfloat16, "rows", 2, optional=True), n_rows,
        _ptr(row_map, torch.int32, "row_map", 2, optional=True),
        _ptr(topk_w, torch.float32, "topk_w", 2, optional=True), k,
        _ptr(shared, torch.bfloat16, "shared", 2, optional=True),
        _ptr(partials, torch.bfloat16, "partials", 3, optional=True), R,
        _ptr(residual, torch.bfloat16, "residual", 2), _ptr(gamma, torch.float32, "gamma", 1), float(eps),
        _ptr(residual_out, torch.bfloat16, "residual_out", 2), _ptr(normed_out, torch.bfloat16, "normed_out", 2),
        T, H, _ptr(err_flag, torch.int32, "err_flag", optional=True), _stream(stream))
    check(st, "moe_finalize_add_rmsnorm")
    return residual_out, normed_out


def moe_tail_fused(logits, k, routed_scale, rows, row_map, shared, residual, gamma, eps,
                   residual_out=None, normed_out=None, topk_ids=None, topk_w=None, want_route=True,
                   err_flag=None, stream=None):
    """Router-less fused tail: route from FP32 logits, then the fused tail."""
    T, H = residual.shape
    E = logits.shape[1]
    if residual_out is None:
        residual_out = torch.empty_like(residual)
    if normed_out is None:
        normed_out = torch.empty_like(residual)
    if want_route and topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=residual.device)
    if want_route and topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=residual.device)
    st = lib().moe_tail_fused(
        _ptr(logits, torch.float32, "logits", 2), E, int(k), float(routed_scale),
        _ptr(rows, torch.bfloat16, "rows", 2), int(rows.shape[0]), _ptr(row_map, torch.int32, "row_map", 2),
        _ptr(shared, torch.bfloat16, "shared", 2, optional=True), _ptr(residual, torch.bfloat16, "residual", 2),
        _ptr(gamma, torch.float32, "gamma", 1), float(eps),
        _ptr(residual_out, torch.bfloat16, "residual_out", 2), _ptr(normed_out, torch.bfloat16, "normed_out", 2),
        _ptr(topk_ids, torch.int32, "topk_ids", optional=True), _ptr(topk_w, torch.float32, "topk_w", optional=True),
        T, H, _ptr(err_flag, torch.int32, "err_flag", optional=True), _stream(stream))
    check(st, "moe_tail_fused")
    return residual_out, normed_out, topk_ids, topk_w


_SCORES = {"softmax": _lib.MOE_SCORE_SOFTMAX, "sigmoid": _lib.MOE_SCORE_SIGMOID}
_ACTS = {None: _lib.MOE_ACT_NONE, "none": _lib.MOE_ACT_NONE, "swiglu": _lib.MOE_ACT_SWIGLU}


def _choice(table, value, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(str(v) for v in table)}, got {value!r}")
    return table[value]


# the current stream's handle, without a Stream object; None in a torch built without CUDA
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _enter(device, stream):
    """(stream handle, context to close or None) of a launch on `device`:
    until the context is closed the device is current and what is allocated
    belongs to the launching stream (so that no other stream's work can still
    hold it).  A launch on the current device and stream, the usual case, needs
    no context."""
    if device.type != "cuda":
        raise TypeError("the tensors must be CUDA tensors (there is no CPU path)")
    if stream is None and _raw_stream is not None and device.index == torch.cuda.current_device():
        return _raw_stream(device.index), None
    with contextlib.ExitStack() as on:
        on.enter_context(torch.cuda.device(device))
        if stream is None:
            stream = torch.cuda.current_stream(device)
        elif isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"the stream must be on {device}, got {stream.device}")
        on.enter_context(torch.cuda.stream(stream))
        return stream.cuda_stream, on.pop_all()


def _arg(t, dtype, name, shape, device):
    """Pointer of a tensor of this type, shape and device."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {list(shape)}, got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _opt(t, dtype, name, shape, device):
    return None if t is None else _arg(t, dtype, name, shape, device)


def _out(t, dtype, name, shape, device):
    """An output and its pointer: the one given, checked, or a new one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _arg(t, dtype, name, shape, device)


def _flag(t, device):
    return None if t is None else _arg(t, torch.int32, "err_flag", t.shape, device)


def moe_group_topk_route(logits, k, routed_scale, bias=None, n_group=1, topk_group=1, group_top=2, scores="sigmoid",
                         renormalize=True, topk_ids=None, topk_w=None, stream=None):
    """Top-k experts per token by sigmoid or softmax scores plus a bias, inside
    the topk_group best of n_group expert groups (a group counts by the sum of
    its group_top best); the weights are the scores without the bias, divided
    by their sum if renormalize, times routed_scale."""
    if logits.dim() != 2:
        raise ValueError("logits must have 2 dimensions")
    (T, E), k, device = logits.shape, int(k), logits.device
    if k < 0:
        raise ValueError(f"k cannot be {k}")
    lg, bs = _arg(logits, torch.float32, "logits", (T, E), device), _opt(bias, torch.float32, "bias", (E,), device)
    score_fn = _choice(_SCORES, scores, "scores")
    handle, on = _enter(device, stream)
    try:
        topk_ids, ids = _out(topk_ids, torch.int32, "topk_ids", (T, k), device)
        topk_w, wts = _out(topk_w, torch.float32, "topk_w", (T, k), device)
        st = lib().moe_group_topk_route(lg, bs, ids, wts, T, E, k, int(n_group), int(topk_group), int(group_top), score_fn,
                                        1 if renormalize else 0, float(routed_scale), handle)
    finally:
        if on is not None:
            on.close()
    check(st, "moe_group_topk_route")
    return topk_ids, topk_w


def moe_expert_rows(T, E, k, block=1):
    """Rows moe_expert_map may need for any ids (host only)."""
    n = lib().moe_expert_rows(int(T), int(E), int(k), int(block))
    if n < 0:
        raise ValueError("sizes out of range")
    return n


def moe_expert_map(topk_ids, E, block=1, n_rows=None, row_map=None, row_token=None, offsets=None, counts=None,
                   stream=None):
    """The expert-sorted row layout of topk_ids [T, k]: (row_map [T, k],
    row_token [n_rows], offsets [E + 1], counts [E]), every expert's rows
    starting on a multiple of block; ids outside [0, E) get no row (-1)."""
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must have 2 dimensions")
    (T, k), E, block, device = topk_ids.shape, int(E), int(block), topk_ids.device
    if n_rows is None:
        n_rows = moe_expert_rows(T, E, k, block) if row_token is None else row_token.numel()
    if n_rows < 0 or E < 0:
        raise ValueError(f"n_rows and E cannot be {n_rows} and {E}")
    ids = _arg(topk_ids, torch.int32, "topk_ids", (T, k), device)
    handle, on = _enter(device, stream)
    try:
        # (four allocations: views of one take longer to make than they save)
        row_map, rm = _out(row_map, torch.int32, "row_map", (T, k), device)
        row_token, tok = _out(row_token, torch.int32, "row_token", (n_rows,), device)
        offsets, off = _out(offsets, torch.int32, "offsets", (E + 1,), device)
        counts, cnt = _out(counts, torch.int32, "counts", (E,), device)
        st = lib().moe_expert_map(ids, rm, tok, off, cnt, n_rows, T, E, k, block, handle)
    finally:
        if on is not None:
            on.close()
    check(st, "moe_expert_map")
    return row_map, row_token, offsets, counts


def _workspace(given, nbytes, device):
    """(tensor, pointer, bytes) of a call's workspace."""
    if nbytes < 0:
        raise ValueError("sizes out of range")
    if given is None:
        if nbytes == 0:
            return None, None, 0
        given = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return given, given.data_ptr(), nbytes
    return given, _arg(given, torch.uint8, "workspace", given.shape, device), given.numel()


def moe_expert_linear(x, w, offsets, counts, row_token=None, act=None, out=None, workspace=None, err_flag=None,
                      stream=None):
    """The experts' products out[r] = act(w[e] @ x[src]) for the rows r of each
    expert's segment [offsets[e], offsets[e] + counts[e]); src = row_token[r],
    or r without row_token.  x [n, K], w [E, N, K] BF16; act None or "swiglu"
    (gate rows of w first; N/2 outputs).  Rows in no segment are not written.
    workspace: a uint8 tensor to use instead of one allocated by the call."""
    if x.dim() != 2 or w.dim() != 3 or x.shape[1] != w.shape[2]:
        raise ValueError("x must be [n, K] and w [E, N, K]")
    (E, N, K), (n_x, _), device = w.shape, x.shape, x.device
    n_rows = n_x if row_token is None else row_token.numel()
    act = _choice(_ACTS, act, "act")
    n_out = N // 2 if act == _lib.MOE_ACT_SWIGLU else N
    if offsets.dim() != 1 or offsets.shape[0] not in (E, E + 1):
        raise ValueError("offsets must have E or E + 1 entries")
    args = (_arg(x, torch.bfloat16, "x", (n_x, K), device), n_x,
            _opt(row_token, torch.int32, "row_token", (n_rows,), device), _arg(w, torch.bfloat16, "w", (E, N, K), device),
            _arg(offsets, torch.int32, "offsets", offsets.shape, device),
            _arg(counts, torch.int32, "counts", (E,), device))
    L = lib()
    handle, on = _enter(device, stream)
    try:
        out, out_ptr = _out(out, torch.bfloat16, "out", (n_rows, n_out), device)
        ws, ws_ptr, nbytes = _workspace(workspace, L.moe_expert_linear_workspace(n_rows, E, N, K), device)
        st = L.moe_expert_linear(*args, out_ptr, n_rows, E, N, K, act, ws_ptr, nbytes,
                                 _flag(err_flag, device), handle)
    finally:
        if on is not None:
            on.close()
    check(st, "moe_expert_linear")
    return out


def moe_adapter_linear(x, w, adapter_a, adapter_b, adapter_ids, adapter_scale, act=None, out=None, workspace=None,
                       err_flag=None, stream=None):
    """One projection for all tokens with each token's low-rank adapter beside
    it: act(w @ x[t] + scale[a] * b[a] @ (a[a] @ x[t])), a = adapter_ids[t]
    (negative: none).  x [T, K], w [N, K], adapter_a [L, R, K], adapter_b
    [L, N, R] BF16, adapter_ids [T] int32, adapter_scale [L] FP32;
    workspace as in moe_expert_linear."""
    if x.dim() != 2 or w.dim() != 2 or adapter_a.dim() != 3 or adapter_b.dim() != 3:
        raise ValueError("x must be [T, K], w [N, K], adapter_a [L, R, K] and adapter_b [L, N, R]")
    (T, K), N, (L, R, _), device = x.shape, w.shape[0], adapter_a.shape, x.device
    act = _choice(_ACTS, act, "act")
    n_out = N // 2 if act == _lib.MOE_ACT_SWIGLU else N
    args = (_arg(x, torch.bfloat16, "x", (T, K), device), _arg(w, torch.bfloat16, "w", (N, K), device),
            _arg(adapter_a, torch.bfloat16, "adapter_a", (L, R, K), device),
            _arg(adapter_b, torch.bfloat16, "adapter_b", (L, N, R), device),
            _arg(adapter_ids, torch.int32, "adapter_ids", (T,), device),
            _arg(adapter_scale, torch.float32, "adapter_scale", (L,), device))
    so = lib()
    handle, on = _enter(device, stream)
    try:
        out, out_ptr = _out(out, torch.bfloat16, "out", (T, n_out), device)
        ws, ws_ptr, nbytes = _workspace(workspace, so.moe_adapter_linear_workspace(T, N, K, R, L), device)
        st = so.moe_adapter_linear(*args, out_ptr, T, N, K, R, L, act, ws_ptr, nbytes,
                                   _flag(err_flag, device), handle)
    finally:
        if on is not None:
            on.close()
    check(st, "moe_adapter_linear")
    return out


def moe_debug_withhold_stream_stage(stage):
    """Test hook of the bounded waits: the next persistent-kernel launch
    leaves stage `stage` of its first CTA uncopied, so that CTA's wait runs
    out and MOE_FLAG_TIMEOUT is set; -1 cancels the request."""
    check(lib().moe_debug_withhold_stream_stage(int(stage)), "moe_debug_withhold_stream_stage")


def moe_debug_withhold_router_stage(kb):
    """Test hook of the router's bounded waits: the next tensor-memory router
    launch issues no loads for K block `kb` in its first CTA, so that CTA's
    wait runs out, its tile is written as NaN and MOE_FLAG_TIMEOUT is set;
    -1 cancels the request."""
    check(lib().moe_debug_withhold_router_stage(int(kb)), "moe_debug_withhold_router_stage")


def moe_debug_withhold_expert_stage(stage):
    """Test hook of the bounded waits: the product launches of the next
    moe_expert_linear or moe_adapter_linear call issue no loads for K block
    `stage` of their first thread block, so that its wait runs out, what it
    had left to compute is NaN and MOE_FLAG_TIMEOUT is set; -1 cancels the
    request."""
    check(lib().moe_debug_withhold_expert_stage(int(stage)), "moe_debug_withhold_expert_stage")


def moe_debug_fail_next_launch(on=True):
    """Test hook of the launch-error path: the next kernel launch of any entry
    point is refused by the CUDA runtime (oversized shared-memory request),
    so that call raises MoeTailError with MOE_ERR_CUDA; on=False cancels."""
    check(lib().moe_debug_fail_next_launch(1 if on else 0), "moe_debug_fail_next_launch")


def moe_debug_router_tc_shape(T, H, E, nsm, mc2, mc4, mc8):
    """Test hook (host only): the (token tile, split-K cluster size) the
    tensor-memory router would take for T x H x E on a device with `nsm` SMs
    that holds mc2 / mc4 / mc8 clusters of 2 / 4 / 8 router CTAs at once."""
    bnt, split_k = ctypes.c_int32(), ctypes.c_int32()
    check(lib().moe_debug_router_tc_shape(int(T), int(H), int(E), int(nsm), int(mc2), int(mc4), int(mc8),
                                          ctypes.byref(bnt), ctypes.byref(split_k)), "moe_debug_router_tc_shape")
    return bnt.value, split_k.value
