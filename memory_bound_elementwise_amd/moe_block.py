"""Python binding of ``libmoe_block.so`` (C ABI in ``include/block/moe_block.h``): layer norm,
a matrix product with bias, activation and residual in its epilogue, the router, and a whole
expert layer for a few tokens.

Argument marshalling only: tensors are checked for device, dtype, shape and contiguity and
their device pointers, which the C functions want at 16 bytes, and a HIP stream are handed over
(``LayerNorm`` alone copies what lies otherwise). No CPU or PyTorch fallback.

Every call runs on the tensors' own device and on ``stream`` (a ``torch.cuda.Stream`` or a
raw handle; default: the current stream of that device). Where the C function needs a
workspace it is taken from ``workspace`` (uint8, at least ``*_workspace`` bytes) or, without
one, allocated on that stream, so that its memory is not reused before the work has run.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import build as _build

BLOCK_BF16, BLOCK_FP16, BLOCK_FP32 = 0, 1, 2
_TORCH = {torch.bfloat16: BLOCK_BF16, torch.float16: BLOCK_FP16, torch.float32: BLOCK_FP32}
ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "gelu": 2, "squared_relu": 3}
EXPERT_ACTIVATIONS = {"squared_relu": 3, "swiglu": 4}
SCORES = {"softmax": 0, "sigmoid": 1}

_lock = threading.Lock()
_lib = None
_vp, _i64, _int, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_SIGS = {
    "block_layer_norm_fwd": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _f32, _int, _int, _vp],
    "block_layer_norm_bwd_workspace": [_i64, _i64],
    "block_layer_norm_bwd": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _int, _vp, _i64, _vp],
    "block_linear_act_workspace": [_i64, _i64, _i64],
    "block_linear_act": [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _vp, _i64, _vp],
    "block_moe_route_workspace": [_i64, _i64, _int],
    "block_moe_route": [_vp, _vp, _int, _vp, _vp, _i64, _i64, _int, _int, _int, _vp, _vp, _i64, _vp],
    "block_moe_experts_workspace": [_i64, _i64, _i64, _int, _int],
    "block_moe_experts": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _i64, _i64, _i64, _int, _int, _int, _f32, _vp,
                          _vp, _i64, _vp],
    "block_moe_layer_workspace": [_i64, _i64, _i64, _int, _int],
    "block_moe_layer": [_vp, _vp, _int, _vp, _vp, _vp, _vp, _int, _vp, _vp, _i64, _i64, _i64, _int, _int, _int,
                        _int, _f32, _vp, _vp, _i64, _vp],
    "block_moe_gate_fwd": [_vp, _int, _vp, _vp, _vp, _i64, _int, _int, _int, _int, _int, _int, _int, _f32, _vp, _vp],
    "block_moe_gate_bwd": [_vp, _int, _vp, _vp, _vp, _i64, _int, _int, _int, _int, _f32, _vp, _vp],
    "block_moe_route_gated": [_vp, _vp, _int, _vp, _vp, _vp, _i64, _i64, _int, _int, _int, _int, _int, _int, _int,
                              _f32, _vp, _vp, _i64, _vp],
    "block_fp4_codes_bytes": [_i64, _i64],
    "block_fp4_scales_bytes": [_i64, _i64],
    "block_fp4_quantize": [_vp, _int, _vp, _vp, _i64, _i64, _i64, _vp],
    "block_fp4_pack": [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp],
    "block_fp4_dequantize": [_vp, _vp, _vp, _i64, _i64, _i64, _vp],
    "block_linear_act_fp4_workspace": [_i64, _i64, _i64],
    "block_linear_act_fp4": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, _i64, _vp],
    "block_moe_experts_fp4_workspace": [_i64, _i64, _i64, _int, _int],
    "block_moe_experts_fp4": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _i64, _i64, _i64, _int, _int, _int,
                              _f32, _vp, _vp, _i64, _vp],
    "moe_block_status_string": [_int],
    "moe_block_last_hip_error": [],
    "moe_block_abi_version": [],
}


class MoeBlockError(RuntimeError):
    def __init__(self, fn: str, status: int, hip_error: int = 0):
        self.status, self.hip_error = status, hip_error
        msg = load_library().moe_block_status_string(status).decode()
        super().__init__(f"{fn} failed: {msg} (status {status}" +
                         (f", hipError {hip_error})" if status == 3 else ")"))


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load (building it first if nothing is built) the HIP library; cached."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or _build.lib_path("moe_block")
        if not os.path.exists(p):
            _build.build_lib("moe_block")
        lib = ctypes.CDLL(p)
        for name, args in _SIGS.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = (ctypes.c_char_p if name == "moe_block_status_string" else
                         _i64 if name.endswith(("_workspace", "_bytes")) else _int)
        if lib.moe_block_abi_version() != 1:
            raise RuntimeError("libmoe_block.so ABI version mismatch")
        if path is None:
            _lib = lib
        return lib


_by_size = functools.lru_cache(maxsize=1024)  # workspace sizes, functions of sizes alone


def _tensor(t, name, dtype, shape, dev):
    """Address of a tensor that is checked against one dtype, shape and device (None for an
    absent one). The checks are one expression: a decoding step's launches take a few
    microseconds each, and so would as many separate ones here."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        raise ValueError("tensors must live on one device")
    return t.data_ptr()


def _kind(t, name, dtypes):
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    return t.dtype


def _call(fn, x, stream, args, workspace=None, need=None):
    """Runs one C function on the device of x, and on ``stream``; `need` None: it takes no
    workspace."""
    if not x.is_cuda:
        raise ValueError("tensors must live on the GPU")
    index = x.get_device()
    if index != _current_device():
        with torch.cuda.device(index):
            return _call(fn, x, stream, args, workspace, need)
    if stream is None:
        handle = _current_stream(index)
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device.index != index:
            raise ValueError("the stream belongs to another device")
        handle = stream.cuda_stream
    else:
        handle = int(stream)
    if need is not None:
        if workspace is not None:
            if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != index:
                raise ValueError("workspace must be a contiguous uint8 tensor on the tensors' device")
            if workspace.numel() < need:
                raise ValueError(f"workspace must hold at least {need} bytes, got {workspace.numel()}")
        elif need > 0:
            if stream is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
            else:
                own = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(handle, device=index)
                with torch.cuda.stream(own):
                    workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        args += (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    lib = _lib or load_library()
    st = getattr(lib, fn)(*args, handle)
    if st:
        raise MoeBlockError(fn, st, lib.moe_block_last_hip_error())


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):  # the same handle without a Stream object
    _current_stream = torch._C._cuda_getCurrentRawStream
# x is a GPU tensor by then, so torch.cuda is initialised
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _rows(x, name):
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    return shape


_ANY = tuple(_TORCH)
_HALF = (torch.bfloat16, torch.float16)
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------
def layer_norm_fwd(x, weight, bias, y, mean=None, rstd=None, *, eps=1e-5, stream=None):
    """y = (x - mean) * rstd * weight + bias per row of x [rows, cols] (bf16, fp16 or fp32), in
    fp32 with one rounding. ``weight`` and ``bias``: [cols] of x's dtype or fp32 (one dtype for
    both), or None. ``mean`` and ``rstd`` (fp32 [rows], both or neither) take the statistics
    that the backward needs. Nothing is recorded for autograd, whatever the inputs require: the
    gradients come from ``layer_norm_bwd``, or from ``LayerNorm``, which calls both."""
    shape = rows, cols = _rows(x, "x")
    dev, kind = x.get_device(), _kind(x, "x", _ANY)
    first = weight if weight is not None else bias
    wkind = kind if first is None else _kind(first, "weight and bias", (kind, _F32))
    if (mean is None) != (rstd is None):
        raise ValueError("mean and rstd go together")
    _call("block_layer_norm_fwd", x, stream,
          (_tensor(x, "x", kind, shape, dev), _tensor(weight, "weight", wkind, (cols,), dev),
           _tensor(bias, "bias", wkind, (cols,), dev), _tensor(y, "y", kind, shape, dev),
           _tensor(mean, "mean", _F32, (rows,), dev), _tensor(rstd, "rstd", _F32, (rows,), dev), rows, cols, eps,
           _TORCH[kind], _TORCH[wkind]))
    return y


@_by_size
def layer_norm_bwd_workspace(rows: int, cols: int) -> int:
    return (_lib or load_library()).block_layer_norm_bwd_workspace(rows, cols)


def layer_norm_bwd(grad_y, x, weight, mean, rstd, grad_x, grad_weight=None, grad_bias=None, *, workspace=None,
                   stream=None):
    """Gradients of ``layer_norm_fwd``: grad_x in x's dtype, grad_weight and grad_bias in the
    weight's (the same bits on every call); any of the three may be None. With ``weight`` None
    (a norm without scale) grad_weight and grad_bias are x's dtype or fp32."""
    shape = rows, cols = _rows(x, "x")
    dev, kind = x.get_device(), _kind(x, "x", _ANY)
    first = weight if weight is not None else grad_weight if grad_weight is not None else grad_bias
    wkind = kind if first is None else _kind(first, "weight", (kind, _F32))
    vec, st = (cols,), (rows,)
    args = (_tensor(grad_y, "grad_y", kind, shape, dev), _tensor(x, "x", kind, shape, dev),
            _tensor(weight, "weight", wkind, vec, dev), _tensor(mean, "mean", _F32, st, dev),
            _tensor(rstd, "rstd", _F32, st, dev), _tensor(grad_x, "grad_x", kind, shape, dev),
            _tensor(grad_weight, "grad_weight", wkind, vec, dev), _tensor(grad_bias, "grad_bias", wkind, vec, dev),
            rows, cols, _TORCH[kind], _TORCH[wkind])
    need = layer_norm_bwd_workspace(rows, cols) if grad_weight is not None or grad_bias is not None else 0
    _call("block_layer_norm_bwd", x, stream, args, workspace, need)
    return grad_x, grad_weight, grad_bias


def _aligned(t):
    """t, or a copy of it where it is not contiguous or does not start at 16 bytes, as the kernels
    want it (a slice of a tensor whose rows have an odd length may start anywhere)."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class LayerNorm(torch.autograd.Function):
    """Layer norm over the last axis, saving x and its fp32 statistics. Any strides and offsets.

    Its backward is not captured into a HIP graph when it ends in leaves (parameters): autograd
    hands a leaf's gradient over on the stream on which the leaf was first used, and where an
    eager graph of the same leaf is alive that stream is drawn into the capture, which then
    ends the process. A captured step calls ``layer_norm_fwd`` and ``layer_norm_bwd``."""

    @staticmethod
    def forward(ctx, x, weight=None, bias=None, eps=1e-5):
        flat = _aligned(x).view(-1, x.shape[-1])
        weight, bias = _aligned(weight), _aligned(bias)
        mean = torch.empty(flat.shape[0], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        y = layer_norm_fwd(flat, weight, bias, torch.empty_like(flat), mean, rstd, eps=eps)
        ctx.save_for_backward(flat, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        if torch.cuda.is_current_stream_capturing() and any(
                type(node).__name__ == "AccumulateGrad" for node, _ in ctx.next_functions):
            raise RuntimeError("LayerNorm's backward into leaf tensors cannot be captured into a graph: call "
                               "layer_norm_fwd and layer_norm_bwd in the captured step")
        flat, weight, mean, rstd = ctx.saved_tensors
        grad_x = torch.empty_like(flat) if ctx.needs_input_grad[0] else None
        grad_weight = torch.empty_like(weight) if ctx.needs_input_grad[1] else None
        grad_bias = (torch.empty(flat.shape[1], dtype=ctx.bias_dtype, device=flat.device)
                     if ctx.needs_input_grad[2] else None)
        layer_norm_bwd(_aligned(grad_y).view(flat.shape), flat, weight, mean, rstd, grad_x, grad_weight, grad_bias)
        return None if grad_x is None else grad_x.view(grad_y.shape), grad_weight, grad_bias, None


# ---------------------------------------------------------------------------
# Matrix product with an epilogue
# ---------------------------------------------------------------------------
@_by_size
def linear_act_workspace(m: int, n: int, k: int) -> int:
    return (_lib or load_library()).block_linear_act_workspace(m, n, k)


def linear_act(x, weight, y, *, bias=None, activation=None, residual=None, workspace=None, stream=None):
    """y = act(x @ weight.T + bias) + residual; x [m, k], weight [n, k], bias [n], residual and y
    [m, n], all bf16 or all fp16, summed and finished in fp32 with one rounding. ``activation``:
    None, "silu", "gelu" (tanh form) or "squared_relu". n and k are multiples of 8. Forward
    only: inputs that require a gradient are refused while gradients are recorded."""
    m, k = _rows(x, "x")
    n = _rows(weight, "weight")[0]
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    _forward_only("linear_act", x, weight, bias, residual)
    dev, kind = x.get_device(), _kind(x, "x", _HALF)
    args = (_tensor(x, "x", kind, (m, k), dev), _tensor(weight, "weight", kind, (n, k), dev),
            _tensor(bias, "bias", kind, (n,), dev), _tensor(residual, "residual", kind, (m, n), dev),
            _tensor(y, "y", kind, (m, n), dev), m, n, k, ACTIVATIONS[activation], _TORCH[kind])
    _call("block_linear_act", x, stream, args, workspace, linear_act_workspace(m, n, k))
    return y


def _forward_only(name, *tensors):
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise RuntimeError(f"{name} has no backward pass: call it under torch.no_grad()")


# ---------------------------------------------------------------------------
# Router and experts
# ---------------------------------------------------------------------------
@_by_size
def moe_route_workspace(tokens: int, hidden: int, experts: int) -> int:
    return (_lib or load_library()).block_moe_route_workspace(tokens, hidden, experts)


@_by_size
def moe_experts_workspace(tokens: int, hidden: int, inter: int, experts: int, top_k: int) -> int:
    return (_lib or load_library()).block_moe_experts_workspace(tokens, hidden, inter, experts, top_k)


@_by_size
def moe_layer_workspace(tokens: int, hidden: int, inter: int, experts: int, top_k: int) -> int:
    return (_lib or load_library()).block_moe_layer_workspace(tokens, hidden, inter, experts, top_k)


def _scalar(valid_tokens, dev):
    return None if valid_tokens is None else _tensor(valid_tokens.reshape(-1), "valid_tokens", _I32, (1,), dev)


def _scores(scores):
    if scores not in SCORES:
        raise ValueError(f"unknown scores {scores!r}")
    return SCORES[scores]


def _gate_rule(scores, groups, top_groups, group_top, renormalize, scale):
    """The gate's arguments as the C functions take them in a row."""
    return (SCORES[scores] if scores in SCORES else _scores(scores), groups,
            groups if top_groups is None else top_groups, group_top, bool(renormalize), scale)


def moe_route(x, router_weight, ids, probs, *, renormalize=False, scores="softmax", bias=None, groups=1,
              top_groups=None, group_top=1, scale=1.0, valid_tokens=None, workspace=None, stream=None):
    """The top experts of each token of x (bf16 [tokens, hidden]) and their weights: logits = x @
    router_weight.T (bf16 or fp32 [experts, hidden]) in fp64, the ids.shape[1] largest scores in
    descending order with ties to the lower expert into ``ids`` (int32 [tokens, top_k]) and their
    weights, of all experts' or (``renormalize``) of the chosen ones', into ``probs`` (fp32).
    ``scores``, ``bias``, ``groups``, ``top_groups``, ``group_top`` and ``scale``: the gate's, as
    for ``moe_gate_fwd``. Rows at or past ``valid_tokens`` (device int32) are left as they were."""
    tokens, hidden = _rows(x, "x")
    experts = _rows(router_weight, "router_weight")[0]
    top_k = _rows(ids, "ids")[1]
    _forward_only("moe_route", x, router_weight)
    dev, rkind = x.get_device(), _kind(router_weight, "router_weight", (_BF16, _F32))
    px, pr = (_tensor(x, "x", _BF16, (tokens, hidden), dev),
              _tensor(router_weight, "router_weight", rkind, (experts, hidden), dev))
    to = (_tensor(ids, "ids", _I32, (tokens, top_k), dev), _tensor(probs, "probs", _F32, (tokens, top_k), dev), tokens,
          hidden, experts, top_k)
    need = moe_route_workspace(tokens, hidden, experts)
    if (scores == "softmax" and bias is None and scale == 1.0 and groups == 1 and top_groups in (None, 1) and
            group_top == 1):  # the logits' own order
        _call("block_moe_route", x, stream, (px, pr, _TORCH[rkind], *to, bool(renormalize), _scalar(valid_tokens, dev)),
              workspace, need)
    else:
        _call("block_moe_route_gated", x, stream,
              (px, pr, _TORCH[rkind], None if bias is None else _tensor(bias, "bias", _F32, (experts,), dev), *to,
               *_gate_rule(scores, groups, top_groups, group_top, renormalize, scale),
               None if valid_tokens is None else _scalar(valid_tokens, dev)), workspace, need)
    return ids, probs


def _expert_args(x, w_up, w_down, activation, limit, dev):
    tokens, hidden = _rows(x, "x")
    if activation not in EXPERT_ACTIVATIONS:
        raise ValueError(f"unknown expert activation {activation!r}")
    if w_down.dim() != 3:
        raise ValueError("w_down must be [experts, hidden, inter]")
    experts, _, inter = w_down.shape
    ups = 2 * inter if activation == "swiglu" else inter
    if activation == "swiglu" and not limit > 0:
        raise ValueError("limit must be positive (inf for none)")
    return (tokens, hidden, inter, experts, _tensor(x, "x", _BF16, (tokens, hidden), dev),
            _tensor(w_up, "w_up", _BF16, (experts, ups, hidden), dev),
            _tensor(w_down, "w_down", _BF16, (experts, hidden, inter), dev))


def moe_experts(x, w_up, w_down, ids, probs, y, *, activation="swiglu", limit=math.inf, residual=None,
                valid_tokens=None, workspace=None, stream=None):
    """y[t] = residual[t] + sum over j of (act(x[t] @ w_up[e].T) * probs[t, j]) @ w_down[e].T, e =
    ids[t, j], for a few tokens (tokens * top_k <= 1024): each chosen expert's weights are read
    once. ``activation``: "swiglu" (w_up [experts, 2 inter, hidden], gate rows first, clamped
    at ``limit``) or "squared_relu" (w_up [experts, inter, hidden]). An id outside the experts
    contributes nothing. x, weights and residual bf16; y bf16 or fp32; rows of y at or past
    ``valid_tokens`` are left as they were."""
    dev = x.get_device()
    tokens, hidden, inter, experts, px, pu, pd = _expert_args(x, w_up, w_down, activation, limit, dev)
    top_k = _rows(ids, "ids")[1]
    _forward_only("moe_experts", x, w_up, w_down, probs, residual)
    ykind = _kind(y, "y", (_BF16, _F32))
    args = (px, pu, pd, _tensor(ids, "ids", _I32, (tokens, top_k), dev),
            _tensor(probs, "probs", _F32, (tokens, top_k), dev),
            _tensor(residual, "residual", _BF16, (tokens, hidden), dev), _tensor(y, "y", ykind, (tokens, hidden), dev),
            _TORCH[ykind], tokens, hidden, inter, experts, top_k, EXPERT_ACTIVATIONS[activation], limit,
            _scalar(valid_tokens, dev))
    _call("block_moe_experts", x, stream, args, workspace, moe_experts_workspace(tokens, hidden, inter, experts, top_k))
    return y


def moe_layer(x, router_weight, w_up, w_down, y, ids, probs, *, activation="swiglu", limit=math.inf,
              renormalize=False, residual=None, valid_tokens=None, workspace=None, stream=None):
    """``moe_route`` into ids and probs, then ``moe_experts`` with them into y, in one call."""
    dev = x.get_device()
    tokens, hidden, inter, experts, px, pu, pd = _expert_args(x, w_up, w_down, activation, limit, dev)
    top_k = _rows(ids, "ids")[1]
    _forward_only("moe_layer", x, router_weight, w_up, w_down, residual)
    rkind, ykind = _kind(router_weight, "router_weight", (_BF16, _F32)), _kind(y, "y", (_BF16, _F32))
    args = (px, _tensor(router_weight, "router_weight", rkind, (experts, hidden), dev), _TORCH[rkind], pu, pd,
            _tensor(residual, "residual", _BF16, (tokens, hidden), dev), _tensor(y, "y", ykind, (tokens, hidden), dev),
            _TORCH[ykind], _tensor(ids, "ids", _I32, (tokens, top_k), dev),
            _tensor(probs, "probs", _F32, (tokens, top_k), dev), tokens, hidden, inter, experts, top_k,
            bool(renormalize), EXPERT_ACTIVATIONS[activation], limit, _scalar(valid_tokens, dev))
    _call("block_moe_layer", x, stream, args, workspace, moe_layer_workspace(tokens, hidden, inter, experts, top_k))
    return y
