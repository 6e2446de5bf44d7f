"""Python binding of the gate of ``libmoe_block.so`` (C ABI in ``include/block/moe_block.h``):
softmax or sigmoid scores, a bias for balance, groups of experts, top-k and renormalised weights
from given logits, and the gradient of the logits. ``moe_block.moe_route`` runs the same gate
behind the router's product.

Argument marshalling as in ``moe_block``; no CPU or PyTorch fallback. Logits and gradients start at 16
bytes, as all tensors of the C functions do; ``MoeGate`` copies a slice that does not.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from .moe_block import (_ANY, _F32, _I32, _TORCH, SCORES, _aligned, _call, _gate_rule, _kind, _rows, _scalar, _scores,
                        _tensor)


def _logits(logits, ids):
    """What both directions take from the logits, and the slots a token."""
    shape, code, chosen = logits.shape, _TORCH.get(logits.dtype), ids.shape
    if len(shape) != 2 or code is None or len(chosen) != 2 or not logits.is_contiguous():
        _rows(logits, "logits")
        _rows(ids, "ids")
        _tensor(logits, "logits", _kind(logits, "logits", _ANY), shape, logits.get_device())
    return logits.data_ptr(), code, *shape, chosen[1], logits.get_device()


def moe_gate_fwd(logits, ids, probs, *, scores="softmax", bias=None, groups=1, top_groups=None, group_top=1,
                 renormalize=False, scale=1.0, valid_tokens=None, stream=None):
    """The chosen experts of each row of ``logits`` ([tokens, experts], bf16, fp16 or fp32) into
    ``ids`` (int32 [tokens, top_k]) and their weights into ``probs`` (fp32).

    ``scores``: "softmax" or "sigmoid" of the logits. Experts are ranked by score plus ``bias``
    (fp32 [experts]; None: by their logits, the same order as the scores'); with ``groups`` > 1 only
    those of the ``top_groups`` groups (None: all) whose ``group_top`` (1 or 2) largest ranks sum to
    most. The weights are the scores without the bias, divided by their sum over the chosen ones
    (``renormalize``), times ``scale``. A logit of -inf masks its expert: weight 0, chosen only where
    too few others are left. Ties go to the lower expert. Rows at or past ``valid_tokens`` (device int32) are left as they were.
    Nothing is recorded for autograd: the gradient comes from ``moe_gate_bwd``, or from
    ``MoeGate``, which calls both."""
    pl, code, tokens, experts, top_k, dev = _logits(logits, ids)
    chosen = (tokens, top_k)
    _call("block_moe_gate_fwd", logits, stream,
          (pl, code, None if bias is None else _tensor(bias, "bias", _F32, (experts,), dev),
           _tensor(ids, "ids", _I32, chosen, dev), _tensor(probs, "probs", _F32, chosen, dev), tokens, experts, top_k,
           *_gate_rule(scores, groups, top_groups, group_top, renormalize, scale),
           None if valid_tokens is None else _scalar(valid_tokens, dev)))
    return ids, probs


def moe_gate_bwd(logits, ids, grad_probs, grad_logits, *, scores="softmax", renormalize=False, scale=1.0,
                 valid_tokens=None, stream=None):
    """``grad_logits`` (logits' dtype and shape, every element written) from ``grad_probs`` (fp32
    [tokens, top_k]) and the forward's ``logits`` and ``ids``; the choice itself and the bias
    have no gradient. Rows at or past ``valid_tokens`` are left as they were."""
    pl, code, tokens, experts, top_k, dev = _logits(logits, ids)
    chosen = (tokens, top_k)
    _call("block_moe_gate_bwd", logits, stream,
          (pl, code, _tensor(ids, "ids", _I32, chosen, dev), _tensor(grad_probs, "grad_probs", _F32, chosen, dev),
           _tensor(grad_logits, "grad_logits", logits.dtype, logits.shape, dev), tokens, experts, top_k,
           SCORES[scores] if scores in SCORES else _scores(scores), bool(renormalize), scale,
           None if valid_tokens is None else _scalar(valid_tokens, dev)))
    return grad_logits


class MoeGate(torch.autograd.Function):
    """(probs, ids) of logits [..., experts]; the gradient of probs flows back to the logits. Any
    strides and offsets. Saves the logits and ids.

    As for ``LayerNorm``, a backward that ends in leaves is not captured into a HIP graph; a
    captured step calls ``moe_gate_fwd`` and ``moe_gate_bwd``."""

    @staticmethod
    def forward(ctx, logits, top_k, bias=None, scores="softmax", groups=1, top_groups=None, group_top=1,
                renormalize=False, scale=1.0):
        flat = _aligned(logits).view(-1, logits.shape[-1])
        ids = torch.empty(flat.shape[0], top_k, dtype=torch.int32, device=logits.device)
        probs = torch.empty(flat.shape[0], top_k, dtype=torch.float32, device=logits.device)
        moe_gate_fwd(flat, ids, probs, scores=scores, bias=_aligned(bias), groups=groups, top_groups=top_groups,
                     group_top=group_top, renormalize=renormalize, scale=scale)
        ctx.save_for_backward(flat, ids)
        ctx.how = dict(scores=scores, renormalize=renormalize, scale=scale)
        ids = ids.view(*logits.shape[:-1], top_k)
        ctx.mark_non_differentiable(ids)
        return probs.view(*logits.shape[:-1], top_k), ids

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_probs, _):
        if torch.cuda.is_current_stream_capturing() and any(
                type(node).__name__ == "AccumulateGrad" for node, _ in ctx.next_functions):
            raise RuntimeError("MoeGate's backward into leaf tensors cannot be captured into a graph: call "
                               "moe_gate_fwd and moe_gate_bwd in the captured step")
        flat, ids = ctx.saved_tensors
        grad = moe_gate_bwd(flat, ids, _aligned(grad_probs).view(ids.shape), torch.empty_like(flat), **ctx.how)
        return (grad.view(*grad_probs.shape[:-1], flat.shape[1]),) + (None,) * 8
