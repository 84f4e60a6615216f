"""Vocabulary rows: log probabilities of given tokens with entropy and top
alternatives, a distillation loss from a teacher's top logits, and the
gradients of both (argreduce_logprobs, argreduce_distill and their gradients in
include/argreduce.h, where the semantics stand).

``logits`` is a CUDA tensor [..., vocab] of float32, float16 or bfloat16, its
last dimension contiguous and its leading ones evenly spaced (a vocabulary cut
from padded rows will do). Where gradients are asked for, ``token_logprobs`` and
``distill_topk`` take part in automatic differentiation: the first gives the
gradients of logprob, entropy and lse, the second that of the loss, each to the
logits alone.

A teacher's ``token_logprobs(..., top_k=K)`` gives what ``distill_topk`` takes:
``top_ids`` as the slots' ids and ``top_logprobs`` as the teacher's values.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib, _stream_ptr, dtype_code
from ._lib import ARGR_OK, ArgreduceError

_LIB = _lib.load()  # looked up once: these calls are short
_F32, _I64 = torch.float32, torch.int64
_empty = torch.empty


def _current_device():
    return torch.cuda.current_device()


class TokenLogprobs(NamedTuple):
    logprob: Optional[torch.Tensor]  #: [...] log p of the given token, 0 where it is negative; None without tokens
    entropy: torch.Tensor            #: [...] -sum p log p, in nats
    lse: torch.Tensor                #: [...] log sum exp(logits / temperature)
    top_ids: Optional[torch.Tensor]  #: [..., top_k] int64, the largest logits first, ties to the lowest index
    top_logprobs: Optional[torch.Tensor]  #: [..., top_k] their log p
    stats: Optional[torch.Tensor]    #: [..., 4] what the backward pass needs: row maximum, log sum, entropy, 0; None unless asked for


class DistillLoss(NamedTuple):
    loss: torch.Tensor   #: [...]
    stats: Optional[torch.Tensor]  #: [..., 4] what the backward pass needs: row maximum, log sum, log sum of the tail, 0


_CODES = {torch.float32: _lib.ARGR_F32, torch.float16: _lib.ARGR_F16, torch.bfloat16: _lib.ARGR_BF16}


def _no_tangent(t):
    if forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None:
        raise NotImplementedError("forward-mode differentiation of operators over rows of scores (the tangent would be lost)")


def _rows(x, dtype):
    """(rows, cols, row stride, type code) of logits."""
    if not x.is_cuda:
        raise ValueError("logits must be a CUDA tensor (the library has no CPU path)")
    if x.get_device() != _current_device():
        raise ValueError(f"logits are on cuda:{x.get_device()}, but the current device is cuda:{_current_device()} "
                         "(the library plans and launches there: enter torch.cuda.device(logits.device))")
    _no_tangent(x)
    code = _CODES.get(x.dtype) if dtype is None else dtype_code(x, dtype)
    if code is None or code > _lib.ARGR_BF16:
        raise TypeError("logits must be float32, float16 or bfloat16")
    shape, stride = x.shape, x.stride()
    n = len(shape)
    if n == 0:
        raise ValueError("logits must have at least one dimension")
    cols = shape[-1]
    if cols == 0:
        raise ValueError("logits must have a vocabulary of at least one")
    if stride[-1] != 1 and cols > 1:
        raise ValueError("the last dimension of logits must be contiguous")
    if n == 2:
        return shape[0], cols, stride[0] if shape[0] > 1 else cols, code
    if n == 1:
        return 1, cols, cols, code
    if n == 3 and stride[0] == shape[1] * stride[1] and shape[1] > 1:  # evenly spaced, without a view
        return shape[0] * shape[1], cols, stride[1], code
    try:
        x = x.view(-1, cols)
    except RuntimeError:
        raise ValueError("the leading dimensions of logits must be evenly spaced (make it contiguous)") from None
    return x.shape[0], cols, x.stride(0) if x.shape[0] > 1 else cols, code


def _arg(t, what, dtype, shape, device):
    """Data pointer of an argument that must be a contiguous tensor of this type and shape on the logits' device."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        if dtype is _F32:
            _no_tangent(t)
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{what} must be a contiguous tensor on {device}")


def _side(stream, x):
    """`stream` (a torch stream or a raw handle) as a torch stream, None where it is the current one."""
    if not x.is_cuda:
        return None
    dev = x.get_device()
    handle = _stream_ptr(stream, dev)
    if handle == _stream_ptr(None, dev):
        return None
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(handle, dev) if handle else torch.cuda.default_stream(dev)
    if stream.device != x.device:
        raise ValueError(f"stream must be of {x.device}, got one of {stream.device}")
    return stream


def _under(side, given, call, *args, **kw):
    """`call` with `side` as torch's current stream: what it allocates belongs to that stream, and automatic
    differentiation runs the backward pass there, ordered with the streams that it takes gradients from and
    gives them to. What was given is kept until that stream is done with it, what it returns until the present one is."""
    here = torch.cuda.current_stream(side.device)
    with torch.cuda.stream(side):
        out = call(*args, **kw)
    for t in given:
        if t is not None:
            t.record_stream(side)
    for t in (out,) if isinstance(out, torch.Tensor) else out:
        if t is not None:
            t.record_stream(here)
    return out


def _plan(plan):
    return ctypes.byref(plan) if plan is not None else None


def _check(st, what):
    if st != ARGR_OK:
        raise ArgreduceError(st, what)


def _grad_out(x, grad):
    """The gradient's tensor and its row stride."""
    if grad is None:
        grad = _empty(x.shape, dtype=x.dtype, device=x.device)
        return grad, x.shape[-1]
    if grad.shape != x.shape or grad.dtype is not x.dtype or grad.device != x.device:
        raise ValueError("grad must have the shape, type and device of logits")
    _, _, stride, _ = _rows(grad, "f32" if grad.element_size() == 4 else "bf16")
    if not grad.is_inference():
        torch.autograd.graph.increment_version(grad)  # written through its pointer: graphs that saved it have to know
    return grad, stride


def _forward_logprobs(x, tokens, top_k, temperature, with_stats, dtype, plan):
    rows, cols, stride, code = _rows(x, dtype)
    lead, dev = x.shape[:-1], x.device
    tok = _arg(tokens, "tokens", _I64, lead, dev)
    if not 0 <= top_k <= min(cols, _lib.LOGITS_MAX_TOP):
        raise ValueError(f"top_k must be in [0, {min(cols, _lib.LOGITS_MAX_TOP)}], got {top_k}")
    entropy = _empty(lead, dtype=_F32, device=dev)
    lse = _empty(lead, dtype=_F32, device=dev)
    logprob = ids = top = stats = p_logprob = p_ids = p_top = p_stats = None
    if with_stats:
        stats = _empty((*lead, 4), dtype=_F32, device=dev)
        p_stats = stats.data_ptr()
    if tok is not None:
        logprob = _empty(lead, dtype=_F32, device=dev)
        p_logprob = logprob.data_ptr()
    if top_k:
        ids = _empty((*lead, top_k), dtype=_I64, device=dev)
        top = _empty((*lead, top_k), dtype=_F32, device=dev)
        p_ids, p_top = ids.data_ptr(), top.data_ptr()
    st = _LIB.argreduce_logprobs(x.data_ptr(), code, rows, cols, stride, temperature, tok, top_k, p_logprob,
                                 entropy.data_ptr(), lse.data_ptr(), p_ids, p_top, p_stats, _plan(plan),
                                 _stream_ptr(None, dev.index) or None)
    if st != ARGR_OK:
        raise ArgreduceError(st, "argreduce_logprobs")
    return logprob, entropy, lse, ids, top, stats


class _TokenLogprobsFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, tokens, top_k, temperature, dtype, plan):
        out = _forward_logprobs(x, tokens, top_k, temperature, True, dtype, plan)
        ctx.save_for_backward(x, tokens, out[5])
        ctx.temperature, ctx.dtype = temperature, dtype
        ctx.mark_non_differentiable(*(t for t in out[3:] if t is not None))
        ctx.set_materialize_grads(False)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_logprob, grad_entropy, grad_lse, *_):
        x, tokens, stats = ctx.saved_tensors
        if grad_logprob is None and grad_entropy is None and grad_lse is None:
            return (None,) * 6
        given = [None if g is None else g.contiguous() for g in (grad_logprob, grad_entropy, grad_lse)]
        return (token_logprobs_backward(x, tokens, stats, *given, temperature=ctx.temperature,
                                        dtype=ctx.dtype),) + (None,) * 5


def token_logprobs(logits, tokens=None, top_k: int = 0, *, temperature: float = 1.0, with_stats: bool = False,
                   dtype: Optional[str] = None, plan=None, stream=None) -> TokenLogprobs:
    """For each row of logits: log p of its token (``tokens``, int64 of the
    leading shape; negative: none), the entropy, the log of the sum of
    exponentials, and the ``top_k`` (at most 128) likeliest tokens with their
    log p. ``with_stats``: also what ``token_logprobs_backward`` needs (always there
    where the logits require a gradient). Runs on ``stream`` (default: torch's current stream) without
    synchronising, as if called with that stream as the current one."""
    if stream is not None and (side := _side(stream, logits)) is not None:
        return _under(side, (logits, tokens), token_logprobs, logits, tokens, top_k, temperature=temperature,
                      with_stats=with_stats, dtype=dtype, plan=plan)
    if torch.is_grad_enabled() and logits.requires_grad:
        return TokenLogprobs(*_TokenLogprobsFunction.apply(logits, tokens, top_k, temperature, dtype, plan))
    return TokenLogprobs(*_forward_logprobs(logits, tokens, top_k, temperature, with_stats, dtype, plan))


def token_logprobs_backward(logits, tokens, stats, grad_logprob=None, grad_entropy=None, grad_lse=None, *,
                            temperature: float = 1.0, grad=None, dtype: Optional[str] = None, plan=None, stream=None):
    """The gradient of sum(grad_logprob * logprob + grad_entropy * entropy +
    grad_lse * lse) to the logits; ``stats`` from ``token_logprobs(...,
    with_stats=True)`` of the same logits and temperature. ``grad``: a tensor for the result, which may be
    ``logits`` itself (then overwritten)."""
    if stream is not None and (side := _side(stream, logits)) is not None:
        return _under(side, (logits, tokens, stats, grad_logprob, grad_entropy, grad_lse, grad), token_logprobs_backward,
                      logits, tokens, stats, grad_logprob, grad_entropy, grad_lse, temperature=temperature, grad=grad,
                      dtype=dtype, plan=plan)
    rows, cols, stride, code = _rows(logits, dtype)
    lead, dev = logits.shape[:-1], logits.device
    tok = _arg(tokens, "tokens", _I64, lead, dev)
    if tok is None and grad_logprob is not None:
        raise ValueError("grad_logprob needs tokens")
    args = (tok, _arg(stats, "stats", _F32, (*lead, 4), dev), _arg(grad_logprob, "grad_logprob", _F32, lead, dev),
            _arg(grad_entropy, "grad_entropy", _F32, lead, dev), _arg(grad_lse, "grad_lse", _F32, lead, dev))
    grad, grad_stride = _grad_out(logits, grad)
    _check(_LIB.argreduce_logprobs_backward(logits.data_ptr(), code, rows, cols, stride, temperature, *args,
                                            grad.data_ptr(), grad_stride, _plan(plan),
                                            _stream_ptr(None, logits.get_device()) or None), "argreduce_logprobs_backward")
    return grad


def _slots(x, ids, teacher):
    """(ids, teacher, slots) of the C calls."""
    lead = x.shape[:-1]
    if ids.dim() != x.dim() or ids.shape[:-1] != lead:
        raise ValueError(f"ids must have shape {tuple(lead)} + (slots,), got {tuple(ids.shape)}")
    slots = ids.shape[-1]
    if slots > _lib.LOGITS_MAX_SLOTS:
        raise ValueError(f"at most {_lib.LOGITS_MAX_SLOTS} slots, got {slots}")
    return _arg(ids, "ids", _I64, ids.shape, x.device), _arg(teacher, "teacher", _F32, ids.shape, x.device), slots


def _forward_distill(x, ids, teacher, temperature, tail, with_stats, dtype, plan):
    rows, cols, stride, code = _rows(x, dtype)
    i, t, slots = _slots(x, ids, teacher)
    loss = _empty(x.shape[:-1], dtype=_F32, device=x.device)
    stats = _empty((*x.shape[:-1], 4), dtype=_F32, device=x.device) if with_stats else None
    _check(_LIB.argreduce_distill(x.data_ptr(), code, rows, cols, stride, temperature, i, t, slots, bool(tail),
                                  loss.data_ptr(), stats.data_ptr() if with_stats else None, _plan(plan),
                                  _stream_ptr(None, x.get_device()) or None), "argreduce_distill")
    return loss, stats


class _DistillFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, ids, teacher, temperature, tail, dtype, plan):
        loss, stats = _forward_distill(x, ids, teacher, temperature, tail, True, dtype, plan)
        ctx.save_for_backward(x, ids, teacher, stats)
        ctx.given = dict(temperature=temperature, tail=tail, dtype=dtype)
        ctx.mark_non_differentiable(stats)
        return loss, stats

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss, _):
        x, ids, teacher, stats = ctx.saved_tensors
        return (distill_topk_backward(x, ids, teacher, stats, grad_loss.contiguous(), **ctx.given),) + (None,) * 6


def distill_topk(logits, ids, teacher, *, temperature: float = 1.0, tail: bool = False, with_stats: bool = False,
                 dtype: Optional[str] = None, plan=None, stream=None) -> DistillLoss:
    """Loss of a student's logits against a teacher's top ones, for each row:
    ``ids`` [..., slots] int64 names distinct tokens (negative: an empty slot; places that
    are left over take a negative id too, not a token named already),
    ``teacher`` [..., slots] float32 holds the teacher's logits for them, whose
    softmax (at ``temperature``) over the slots is taught, or, with ``tail``,
    the teacher's log probabilities, taught together with what they leave of 1
    as one more outcome. Sums over rows, and a factor of temperature ** 2 where
    one is wanted, are the caller's. ``with_stats`` and ``stream`` as in ``token_logprobs``."""
    if stream is not None and (side := _side(stream, logits)) is not None:
        return _under(side, (logits, ids, teacher), distill_topk, logits, ids, teacher, temperature=temperature, tail=tail,
                      with_stats=with_stats, dtype=dtype, plan=plan)
    if torch.is_grad_enabled() and logits.requires_grad:
        return DistillLoss(*_DistillFunction.apply(logits, ids, teacher, temperature, tail, dtype, plan))
    return DistillLoss(*_forward_distill(logits, ids, teacher, temperature, tail, with_stats, dtype, plan))


def distill_topk_backward(logits, ids, teacher, stats, grad_loss, *, temperature: float = 1.0, tail: bool = False,
                          grad=None, dtype: Optional[str] = None, plan=None, stream=None):
    """The gradient of sum(grad_loss * loss) to the logits; ``stats`` from
    ``distill_topk(..., with_stats=True)`` with the same arguments. ``grad`` as in
    ``token_logprobs_backward``."""
    if stream is not None and (side := _side(stream, logits)) is not None:
        return _under(side, (logits, ids, teacher, stats, grad_loss, grad), distill_topk_backward, logits, ids, teacher,
                      stats, grad_loss, temperature=temperature, tail=tail, grad=grad, dtype=dtype, plan=plan)
    rows, cols, stride, code = _rows(logits, dtype)
    lead = logits.shape[:-1]
    i, t, slots = _slots(logits, ids, teacher)
    st = _arg(stats, "stats", _F32, (*lead, 4), logits.device)
    g = _arg(grad_loss, "grad_loss", _F32, lead, logits.device)
    grad, grad_stride = _grad_out(logits, grad)
    _check(_LIB.argreduce_distill_backward(logits.data_ptr(), code, rows, cols, stride, temperature, i, t,
                                           slots, bool(tail), st, g, grad.data_ptr(), grad_stride,
                                           _plan(plan), _stream_ptr(None, logits.get_device()) or None),
           "argreduce_distill_backward")
    return grad


def distill_topk_step(logits, ids, teacher, grad_loss, *, temperature: float = 1.0, tail: bool = False, grad=None,
                      dtype: Optional[str] = None, plan=None, stream=None):
    """(loss, gradient) in one call, for a training step that knows each row's
    weight ``grad_loss`` beforehand: what ``distill_topk`` and
    ``distill_topk_backward`` would give."""
    if stream is not None and (side := _side(stream, logits)) is not None:
        return _under(side, (logits, ids, teacher, grad_loss, grad), distill_topk_step, logits, ids, teacher, grad_loss,
                      temperature=temperature, tail=tail, grad=grad, dtype=dtype, plan=plan)
    rows, cols, stride, code = _rows(logits, dtype)
    lead = logits.shape[:-1]
    i, t, slots = _slots(logits, ids, teacher)
    g = _arg(grad_loss, "grad_loss", _F32, lead, logits.device)
    grad, grad_stride = _grad_out(logits, grad)
    loss = _empty(lead, dtype=_F32, device=logits.device)
    stats = _empty((*lead, 4), dtype=_F32, device=logits.device)
    _check(_LIB.argreduce_distill_step(logits.data_ptr(), code, rows, cols, stride, temperature, i, t, slots,
                                       bool(tail), g, loss.data_ptr(), stats.data_ptr(), grad.data_ptr(),
                                       grad_stride, _plan(plan), _stream_ptr(None, logits.get_device()) or None),
           "argreduce_distill_step")
    return loss, grad
