"""Python binding of the operators of ``libmoe_block.so`` on weights in 4 bits with group scales (C
ABI in ``include/block/moe_block.h``): quantising, packing and reading them back, the product with
bias, activation and residual, and the expert layer for a few tokens.

A matrix [n, k] is held as two uint8 tensors, codes and scales, of ``fp4_shapes(n, k)``; several
(the experts of a layer) have an axis in front. Argument marshalling as in ``moe_block``; no
CPU or PyTorch fallback.
"""
from __future__ import annotations

import math

import torch

from .moe_block import (_ANY, _BF16, _F32, _I32, _TORCH, ACTIVATIONS, EXPERT_ACTIVATIONS, _by_size, _call,
                        _forward_only, _kind, _rows, _scalar, _tensor)
from . import moe_block as _block

_U8 = torch.uint8


@_by_size
def fp4_shapes(n: int, k: int):
    """Shapes of the codes and the scales of one matrix [n, k]: tiles of 16 rows x 128 k."""
    if n < 1 or k < 32 or k % 32:
        raise ValueError(f"a matrix in 4 bits needs n >= 1 and k a multiple of 32, got {n} x {k}")
    tiles = -(-n // 16), -(-k // 128)
    return (*tiles, 1024), (*tiles, 64)


def _pair(codes, scales, name, lead, n, k, dev):
    shapes = fp4_shapes(n, k)
    return (_tensor(codes, f"{name}codes", _U8, lead + shapes[0], dev),
            _tensor(scales, f"{name}scales", _U8, lead + shapes[1], dev))


def _matrices(t, name):
    """Leading axis, matrices, rows and columns of [n, k] or [matrices, n, k]."""
    shape = tuple(t.shape)
    if len(shape) not in (2, 3):
        raise ValueError(f"{name} must be 2-D or 3-D")
    return (shape[:-2], *((1,) + shape)[-3:])


def fp4_quantize(weight, codes, scales, *, stream=None):
    """``weight`` ([n, k] or [matrices, n, k]; bf16, fp16 or fp32) to 4 bits: each 32 neighbours of
    a row share the smallest power of two for which 6, the largest element, is the nearest one to
    all of them; each becomes the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times it, ties to the even
    code. A group that holds an infinity or a NaN becomes NaN. (A tool that takes the largest power up to
    a quarter of the largest magnitude instead gives other codes where that magnitude is from 7 to 8
    of those powers; ``fp4_pack`` takes both.)"""
    lead, matrices, n, k = _matrices(weight, "weight")
    dev, kind = weight.get_device(), _kind(weight, "weight", _ANY)
    to = _pair(codes, scales, "", lead, n, k, dev)
    _call("block_fp4_quantize", weight, stream,
          (_tensor(weight, "weight", kind, weight.shape, dev), _TORCH[kind], *to, matrices, n, k))
    return codes, scales


def fp4_pack(elements, exponents, codes, scales, *, stream=None):
    """Lays weights out that a checkpoint holds row by row: ``elements`` uint8 [.., n, k / 2], two
    a byte, the first in its lower half, ``exponents`` uint8 [.., n, k / 32], each a power of two
    plus 127."""
    lead, matrices, n, half = _matrices(elements, "elements")
    k, dev = 2 * half, elements.get_device()
    to = _pair(codes, scales, "", lead, n, k, dev)
    _call("block_fp4_pack", elements, stream,
          (_tensor(elements, "elements", _U8, elements.shape, dev),
           _tensor(exponents, "exponents", _U8, lead + (n, k // 32), dev), *to, matrices, n, k))
    return codes, scales


def fp4_dequantize(codes, scales, weight, *, stream=None):
    """The bf16 values of the weights into ``weight`` [n, k] or [matrices, n, k], exactly."""
    lead, matrices, n, k = _matrices(weight, "weight")
    dev = weight.get_device()
    of = _pair(codes, scales, "", lead, n, k, dev)
    _call("block_fp4_dequantize", weight, stream,
          (*of, _tensor(weight, "weight", _BF16, weight.shape, dev), matrices, n, k))
    return weight


@_by_size
def linear_act_fp4_workspace(m: int, n: int, k: int) -> int:
    return _block.load_library().block_linear_act_fp4_workspace(m, n, k)


def linear_act_fp4(x, codes, scales, y, *, bias=None, activation=None, residual=None, workspace=None, stream=None):
    """``linear_act`` with the weight [n, k] in 4 bits: y = act(x @ weight.T + bias) + residual; x
    [m, k], bias [n], residual and y [m, n] bf16, products exact, sums and epilogue fp32, one
    rounding. n a multiple of 8, k of 32. Forward only."""
    xs, ys = _rows(x, "x"), _rows(y, "y")
    (m, k), n = xs, ys[1]
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    _forward_only("linear_act_fp4", x, bias, residual)
    dev, out = x.get_device(), (m, n)
    c, s = fp4_shapes(n, k)
    args = (_tensor(x, "x", _BF16, xs, dev), _tensor(codes, "codes", _U8, c, dev), _tensor(scales, "scales", _U8, s, dev),
            None if bias is None else _tensor(bias, "bias", _BF16, (n,), dev),
            None if residual is None else _tensor(residual, "residual", _BF16, out, dev),
            _tensor(y, "y", _BF16, out, dev), m, n, k, ACTIVATIONS[activation])
    _call("block_linear_act_fp4", x, stream, args, workspace, linear_act_fp4_workspace(m, n, k))
    return y


@_by_size
def moe_experts_fp4_workspace(tokens: int, hidden: int, inter: int, experts: int, top_k: int) -> int:
    return _block.load_library().block_moe_experts_fp4_workspace(tokens, hidden, inter, experts, top_k)


@_by_size
def _expert_shapes(experts, ups, hidden, inter):
    return tuple(tuple((experts, *shape) for shape in fp4_shapes(*size)) for size in ((ups, hidden), (hidden, inter)))


def moe_experts_fp4(x, up_codes, up_scales, down_codes, down_scales, ids, probs, y, *, activation="swiglu",
                    limit=math.inf, residual=None, valid_tokens=None, workspace=None, stream=None):
    """``moe_experts`` with the experts' weights in 4 bits: up_* hold [experts, 2 inter, hidden]
    ("swiglu", gate rows first, clamped at ``limit``) or [experts, inter, hidden]
    ("squared_relu"), down_* [experts, hidden, inter]. hidden and inter are multiples of 32; inter is
    told by the rows of up_codes."""
    xs = tokens, hidden = _rows(x, "x")
    chosen = (tokens, _rows(ids, "ids")[1])
    if activation not in EXPERT_ACTIVATIONS:
        raise ValueError(f"unknown expert activation {activation!r}")
    gated = activation == "swiglu"
    if gated and not limit > 0:
        raise ValueError("limit must be positive (inf for none)")
    if up_codes.dim() != 4:
        raise ValueError("up_codes must have shape [experts, rows / 16, hidden / 128, 1024]")
    experts, blocks = up_codes.shape[:2]
    inter = blocks * 8 if gated else blocks * 16
    _forward_only("moe_experts_fp4", x, probs, residual)
    dev, ykind, top_k = x.get_device(), _kind(y, "y", (_BF16, _F32)), chosen[1]
    up, down = _expert_shapes(experts, 2 * inter if gated else inter, hidden, inter)
    args = (_tensor(x, "x", _BF16, xs, dev), _tensor(up_codes, "up_codes", _U8, up[0], dev),
            _tensor(up_scales, "up_scales", _U8, up[1], dev), _tensor(down_codes, "down_codes", _U8, down[0], dev),
            _tensor(down_scales, "down_scales", _U8, down[1], dev), _tensor(ids, "ids", _I32, chosen, dev),
            _tensor(probs, "probs", _F32, chosen, dev),
            None if residual is None else _tensor(residual, "residual", _BF16, xs, dev), _tensor(y, "y", ykind, xs, dev),
            _TORCH[ykind], tokens, hidden, inter, experts, top_k, EXPERT_ACTIVATIONS[activation], limit,
            None if valid_tokens is None else _scalar(valid_tokens, dev))
    _call("block_moe_experts_fp4", x, stream, args, workspace,
          moe_experts_fp4_workspace(tokens, hidden, inter, experts, top_k))
    return y
