"""Routing to experts: a row's top experts with their weights, how many rows
chose each expert, the balance loss, and the gradients (argreduce_route and
argreduce_route_backward in include/argreduce.h, where the semantics stand).

``logits`` is a CUDA tensor [..., experts] of float32, float16 or bfloat16, its
strides as in ``token_logprobs``. Where a gradient is asked for, ``route_topk`` takes part in
automatic differentiation: weights, lse and balance have gradients to the logits.
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib, _stream_ptr
from ._lib import ARGR_OK, ArgreduceError
from .logits import _arg, _grad_out, _rows, _side, _under

_LIB = _lib.load()  # looked up once: these calls are short
_F32, _I64, _BOOL = torch.float32, torch.int64, torch.bool
_empty = torch.empty


class Route(NamedTuple):
    weights: torch.Tensor           #: [..., top_k] float32, 0 where nothing was chosen
    ids: torch.Tensor               #: [..., top_k] int64, the likeliest expert first; -1: nothing was chosen
    lse: torch.Tensor               #: [...] log sum exp(logits), -inf for rows that do not take part
    counts: Optional[torch.Tensor]  #: [experts] int64, rows that chose each expert; None unless asked for
    rows: Optional[torch.Tensor]    #: int64, one value: rows that take part; None unless asked for
    balance: Optional[torch.Tensor] #: float32, one value: the balance loss; None unless asked for


def _shape_of(x, dtype):
    rows, experts, stride, code = _rows(x, dtype)
    if experts > _lib.ROUTE_MAX_EXPERTS:
        raise ValueError(f"at most {_lib.ROUTE_MAX_EXPERTS} experts, got {experts}")
    return rows, experts, stride, code


@functools.lru_cache(maxsize=1024)
def _scratch_bytes(device, rows, experts):
    """What the library's plan for counts of such a route on the current device, `device`, asks for (kept: the call into it takes 1 us)."""
    return _LIB.argreduce_route_scratch_bytes(rows, experts)


def _forward(x, top_k, valid, normalize, counts, balance, dtype):
    rows, experts, stride, code = _shape_of(x, dtype)
    lead, dev = x.shape[:-1], x.device
    if not 1 <= top_k <= min(experts, _lib.ROUTE_MAX_TOP):
        raise ValueError(f"top_k must be in [1, {min(experts, _lib.ROUTE_MAX_TOP)}], got {top_k}")
    p_valid = _arg(valid, "valid", _BOOL, lead, dev)
    weights = _empty((*lead, top_k), dtype=_F32, device=dev)
    ids = _empty((*lead, top_k), dtype=_I64, device=dev)
    lse = _empty(lead, dtype=_F32, device=dev)
    n = taken = loss = p_n = p_taken = p_loss = None
    if counts or balance:
        n, taken = _empty(experts, dtype=_I64, device=dev), _empty((), dtype=_I64, device=dev)
        p_n, p_taken = n.data_ptr(), taken.data_ptr()
        if balance:
            loss = _empty((), dtype=_F32, device=dev)
            p_loss = loss.data_ptr()
    args = (x.data_ptr(), code, rows, experts, stride, top_k, bool(normalize), p_valid, weights.data_ptr(), ids.data_ptr(),
            lse.data_ptr(), p_n, p_taken, p_loss)
    handle = _stream_ptr(None, dev.index) or None
    # many rows need scratch for the counts; it is this call's own: torch keeps it until the stream has passed the call
    nbytes = _scratch_bytes(dev.index, rows, experts) if n is not None else 0
    scratch = _empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    st = _LIB.argreduce_route(*args, scratch.data_ptr() if nbytes else None, nbytes, handle)
    if st != ARGR_OK:
        raise ArgreduceError(st, "argreduce_route")
    return weights, ids, lse, n, taken, loss


class _RouteFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, top_k, valid, normalize, counts, balance, dtype):
        out = _forward(x, top_k, valid, normalize, counts, balance, dtype)
        weights, ids, lse, n, taken, _ = out
        ctx.save_for_backward(x, weights, ids, lse, n, taken)
        ctx.normalize, ctx.dtype = normalize, dtype
        ctx.mark_non_differentiable(*(t for t in (ids, n, taken) if t is not None))
        ctx.set_materialize_grads(False)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_weights, _ids, grad_lse, _counts, _rows, grad_balance):
        if grad_weights is None and grad_lse is None and grad_balance is None:
            return (None,) * 7
        given = [None if g is None else g.contiguous() for g in (grad_weights, grad_lse, grad_balance)]
        return (route_topk_backward(*ctx.saved_tensors, grad_weights=given[0], grad_lse=given[1], grad_balance=given[2],
                                    normalize=ctx.normalize, dtype=ctx.dtype),) + (None,) * 6


def route_topk(logits, top_k: int, *, valid=None, normalize: bool = True, counts: bool = False, balance: bool = False,
               dtype: Optional[str] = None, stream=None) -> Route:
    """For each row of logits (at most 1024 experts) its ``top_k`` (at most 32)
    likeliest experts, ties to the lowest index, with their softmax weights, over the
    chosen ones (``normalize``) or over all, and the row's log-sum-exp (what a loss on the logits' size is made
    from). ``counts``: also how many rows chose each expert, and how many rows took part. ``balance``: also
    experts * sum_e (share of the choices that are e) * (mean softmax of e), 1 when all is even; its
    gradient goes through the softmax, the choices are held fixed.

    ``valid`` (bool, [...]): rows where it is false are padding; they are not looked at and, like rows of
    -inf alone, hold id -1, weight 0, lse -inf and gradient 0. A logit of -inf is never chosen (id -1, weight 0
    where fewer than top_k are left). Runs on ``stream`` as ``token_logprobs`` does."""
    if stream is not None and (side := _side(stream, logits)) is not None:
        return Route(*_under(side, (logits, valid), route_topk, logits, top_k, valid=valid, normalize=normalize,
                             counts=counts, balance=balance, dtype=dtype))
    if torch.is_grad_enabled() and logits.requires_grad:
        return Route(*_RouteFunction.apply(logits, top_k, valid, normalize, counts, balance, dtype))
    return Route(*_forward(logits, top_k, valid, normalize, counts, balance, dtype))


def route_topk_backward(logits, weights, ids, lse, counts=None, rows=None, *, grad_weights=None, grad_lse=None,
                        grad_balance=None, normalize: bool = True, grad=None, dtype: Optional[str] = None, stream=None):
    """The gradient of sum(grad_weights * weights) + sum(grad_lse * lse) + grad_balance *
    balance to the logits; weights, ids, lse, counts and rows from ``route_topk`` of the same logits
    (counts and rows are needed with grad_balance alone). ``grad`` as in ``token_logprobs_backward``."""
    if stream is not None and (side := _side(stream, logits)) is not None:
        return _under(side, (logits, weights, ids, lse, counts, rows, grad_weights, grad_lse, grad_balance, grad),
                      route_topk_backward, logits, weights, ids, lse, counts, rows, grad_weights=grad_weights,
                      grad_lse=grad_lse, grad_balance=grad_balance, normalize=normalize, grad=grad, dtype=dtype)
    n, experts, stride, code = _shape_of(logits, dtype)
    lead, dev = logits.shape[:-1], logits.device
    top_k = ids.shape[-1] if ids.dim() else 0
    if not 1 <= top_k <= min(experts, _lib.ROUTE_MAX_TOP):
        raise ValueError(f"ids must name between 1 and {min(experts, _lib.ROUTE_MAX_TOP)} experts for each row, got {top_k}")
    if lse is None:
        raise TypeError("lse must be a tensor: what route_topk gave for these logits")
    if grad_balance is not None and (counts is None or rows is None):
        raise ValueError("grad_balance needs counts and rows")
    args = (_arg(weights, "weights", _F32, (*lead, top_k), dev), _arg(ids, "ids", _I64, (*lead, top_k), dev),
            _arg(lse, "lse", _F32, lead, dev), _arg(counts, "counts", _I64, (experts,), dev),
            _arg(rows, "rows", _I64, (), dev), _arg(grad_weights, "grad_weights", _F32, (*lead, top_k), dev),
            _arg(grad_lse, "grad_lse", _F32, lead, dev), _arg(grad_balance, "grad_balance", _F32, (), dev))
    if grad_weights is not None and weights is None:
        raise ValueError("grad_weights needs weights")
    grad, grad_stride = _grad_out(logits, grad)
    st = _LIB.argreduce_route_backward(logits.data_ptr(), code, n, experts, stride, top_k, bool(normalize), *args,
                                       grad.data_ptr(), grad_stride, _stream_ptr(None, dev.index) or None)
    if st != ARGR_OK:
        raise ArgreduceError(st, "argreduce_route_backward")
    return grad
