"""Beam search: the step from an item's beams and their logits to the best
continuations, and the reordering of what the beams keep
(argreduce_beam_select, argreduce_beam_reorder in include/argreduce.h, where the
semantics stand).

    chosen = beam_select(logits, totals, 2 * beams)        # [batch, beams, vocab], [batch, beams]
    ...                                                    # the caller's rules: which of them go on
    beam_reorder(caches + [histories], parents, lengths, dim=2)
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad

from . import _lib, _stream_ptr
from ._lib import ARGR_OK, ArgreduceError
from .logits import _arg, _current_device, _rows, _side, _under

_LIB = _lib.load()  # looked up once: these calls are short
_F32, _I64, _BOOL = torch.float32, torch.int64, torch.bool
_empty = torch.empty
_MAX_BEAMS, _MAX_COUNT = _lib.BEAM_MAX_BEAMS, _lib.LOGITS_MAX_TOP


class BeamSelection(NamedTuple):
    tokens: torch.Tensor   #: [..., count] int64, the best continuation first; -1: none was left
    parents: torch.Tensor  #: [..., count] int64, the beam that it continues; -1: none was left
    scores: torch.Tensor   #: [..., count] float32, its total; NaN: see beam_select


def _no_gradient(what, *tensors):
    if not torch.is_grad_enabled():
        return
    for t in tensors:
        if t is None or not t.requires_grad:
            continue
        raise RuntimeError(f"{what} has no gradient: call it under torch.no_grad(), or on detached tensors")


@functools.lru_cache(maxsize=1024)
def _scratch_bytes(device, items, beams, cols, code, count):
    """What the library's plan for such a step on the current device, `device`, asks for (kept: the call into it takes 1 us)."""
    return _LIB.argreduce_beam_scratch_bytes(items, beams, cols, code, count)


def beam_select(logits, scores, count: int, *, ended=None, end_token: int = 0, scale=None, temperature: float = 1.0,
                dtype: Optional[str] = None, stream=None) -> BeamSelection:
    """The ``count`` (at most 128) best continuations of each item's beams:
    ``logits`` [..., beams, vocab] (strides as in ``token_logprobs``, at most 64
    beams), ``scores`` [..., beams] float32 the beams' totals of log
    probabilities so far. A continuation's total is its beam's and the token's log
    probability; beams with ``ended`` (bool) have one continuation, ``end_token``, with their
    own total. ``scale`` (float32, positive) multiplies a beam's totals where they are compared, a penalty for
    length, but not in the scores that are returned. Ties go to the lowest (beam, token).

    A beam with the total -inf has no continuation, and its logits are not looked
    at (a first step: one beam has begun); neither are an ended beam's. Places that no
    continuation above -inf is left for hold -1, -1 and -inf (a total below float32's range is -inf too, beside its
    token and parent). An item with a NaN (or +inf) in what is looked at
    holds -1, -1 and NaN. Totals of different beams that differ by less than about 1e-6 may come in
    either order (within a beam the order is exact). Runs on ``stream`` as ``token_logprobs`` does. There is no gradient."""
    if stream is not None and (side := _side(stream, logits)) is not None:
        return BeamSelection(*_under(side, (logits, scores, ended, scale), beam_select, logits, scores, count, ended=ended,
                                     end_token=end_token, scale=scale, temperature=temperature, dtype=dtype))
    _no_gradient("beam_select", logits, scores, scale)
    rows, cols, stride, code = _rows(logits, dtype)
    lead, dev = logits.shape[:-1], logits.device
    if not lead:
        raise ValueError("logits must have the dimensions [..., beams, vocab]")
    beams = lead[-1]
    if not 1 <= beams <= _MAX_BEAMS:
        raise ValueError(f"between 1 and {_MAX_BEAMS} beams, got {beams}")
    if not 1 <= count <= min(beams * cols, _MAX_COUNT):
        raise ValueError(f"count must be in [1, {min(beams * cols, _MAX_COUNT)}], got {count}")
    if scores is None:
        raise TypeError("scores must be a tensor of the beams' totals")
    out = (*lead[:-1], count)
    tokens, parents = _empty(out, dtype=_I64, device=dev), _empty(out, dtype=_I64, device=dev)
    totals = _empty(out, dtype=_F32, device=dev)
    args = (logits.data_ptr(), code, rows // beams, beams, cols, stride, temperature, _arg(scores, "scores", _F32, lead, dev),
            _arg(ended, "ended", _BOOL, lead, dev), end_token, _arg(scale, "scale", _F32, lead, dev), count,
            tokens.data_ptr(), parents.data_ptr(), totals.data_ptr())
    handle = _stream_ptr(None, dev.index) or None
    # many rows need scratch; it is this call's own: torch keeps it until the stream has passed the call
    nbytes = _scratch_bytes(dev.index, rows // beams, beams, cols, code, count)
    scratch = _empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    st = _LIB.argreduce_beam_select(*args, scratch.data_ptr() if nbytes else None, nbytes, handle)
    if st != ARGR_OK:
        raise ArgreduceError(st, "argreduce_beam_select")
    return BeamSelection(tokens, parents, totals)


def _even(shape, stride):
    """(count, stride) of evenly spaced dimensions as one, None where they are not."""
    count, step = 1, 0
    for n, s in zip(reversed(shape), reversed(stride)):
        if n == 1:
            continue
        if count == 1:
            step = s
        elif s != count * step:
            return None
        count *= n
    return count, step


def _geometry(t, items, beams, dim):
    """(item stride, beam stride, segments, their stride, positions, bytes of one) of a state, strides in bytes."""
    shape, stride, es = t.shape, t.stride(), t.element_size()
    if len(shape) >= 1 and shape[0] == items * beams:
        lead, strides = 1, (beams * stride[0], stride[0])
    elif len(shape) >= 2 and shape[0] == items and shape[1] == beams:
        lead, strides = 2, (stride[0] if items > 1 else beams * stride[1], stride[1])
    else:
        raise ValueError(f"a state must have the leading dimensions [{items}, {beams}] or [{items * beams}], got {tuple(shape)}")
    if dim is not None:
        at = dim + len(shape) if dim < 0 else dim
        if not lead <= at < len(shape):
            raise ValueError(f"dim {dim} is not a dimension of a beam's state of shape {tuple(shape[lead:])}")
    else:
        at = len(shape)  # the longest contiguous end
        size = 1
        while at > lead and (shape[at - 1] == 1 or stride[at - 1] == size):
            size *= shape[at - 1]
            at -= 1
    if t.numel() == 0:
        return (0, 0, 0, 0, 0, es)
    inner = _even(shape[at + (dim is not None):], stride[at + (dim is not None):])
    outer = _even(shape[lead:at], stride[lead:at])
    if inner is None or outer is None or (inner[0] > 1 and inner[1] != 1):
        raise ValueError("a beam's state must be evenly spaced segments of contiguous positions (make it contiguous)")
    positions = shape[at] if dim is not None else 1
    if positions > 1 and stride[at] != inner[0]:
        raise ValueError("the positions of a state must be contiguous (make it contiguous)")
    return (strides[0] * es, strides[1] * es, outer[0], outer[1] * es, positions, inner[0] * es)


def _span(g, items, beams):
    """Bytes from a state's first to past its last."""
    return (items - 1) * g[0] + (beams - 1) * g[1] + (g[2] - 1) * g[3] + g[4] * g[5]


def _apart(a, ga, b, gb, items, beams):
    """Whether two states of different geometry, at the addresses a <= b, certainly share no byte:
    one ends before the other begins, or they are columns of the same rows, a beam's or the segments'."""
    if a + _span(ga, items, beams) <= b:
        return True
    if ga[:2] != gb[:2]:
        return False
    for row, na, nb, fit in ((ga[1], _span(ga, 1, 1), _span(gb, 1, 1), True),
                             (ga[3], ga[4] * ga[5], gb[4] * gb[5], ga[3] == gb[3] and ga[3] and ga[1] % ga[3] == 0)):
        if fit and row and ga[0] % row == 0 and (b - a) % row >= na and (b - a) % row + nb <= row:
            return True
    return False


def _reordered(st):
    if st != ARGR_OK:
        raise ArgreduceError(st, "argreduce_beam_reorder (do states overlap, themselves or one another?)")


def beam_reorder(states, parents, lengths=None, *, dim: Optional[int] = None, stream=None):
    """Reorder what beams keep, in place: in each of ``states`` (a tensor or a
    list of them: caches, token histories, recurrent states, of any types and sizes) beam j of
    item i takes over what beam ``parents[i, j]`` had. ``parents`` is int64 [batch, beams] (at most 64
    beams); a state is [batch, beams, ...] or [batch * beams, ...], a view if need be. A parent outside
    [0, beams), as beam_select gives where nothing was left, leaves the beam's own state.

    ``lengths`` int64 [batch] with ``dim``, the dimension of the positions (of every state): only the first
    ``lengths[i]`` positions are moved, later ones stay as they are. Positions and what is within them must be
    contiguous, the dimensions before evenly spaced; states may not overlap. Returns ``states``."""
    group = [states] if isinstance(states, torch.Tensor) else list(states)
    if stream is not None and group and (side := _side(stream, group[0])) is not None:
        _under(side, (*group, parents, lengths), lambda: [beam_reorder(group, parents, lengths, dim=dim)][1:])
        return states
    if parents is None or parents.dim() != 2:
        raise ValueError("parents must have the dimensions [batch, beams]")
    items, beams = parents.shape
    dev = parents.device
    if not parents.is_cuda:
        raise ValueError("parents must be a CUDA tensor (the library has no CPU path)")
    if parents.get_device() != _current_device():
        raise ValueError(f"parents are on cuda:{parents.get_device()}, but the current device is cuda:{_current_device()} "
                         "(the library launches there: enter torch.cuda.device(parents.device))")
    if not 1 <= beams <= _MAX_BEAMS:
        raise ValueError(f"between 1 and {_MAX_BEAMS} beams, got {beams}")
    if lengths is not None and dim is None:
        raise ValueError("lengths need dim, the dimension of the positions")
    p_parents = _arg(parents, "parents", _I64, parents.shape, dev)
    p_lengths = _arg(lengths, "lengths", _I64, (items,), dev)
    _no_gradient("beam_reorder", *group)
    plans = {}  # geometry: pointers
    shape = stride = kind = pointers = None  # of the state before: a list's are mostly alike
    tangents = forward_ad._current_level >= 0
    for t in group:
        if t.shape != shape or t.stride() != stride or t.dtype is not kind:
            shape, stride, kind = t.shape, t.stride(), t.dtype
            if t.is_sparse or t.is_conj() or t.is_neg():
                raise ValueError("states must be plain tensors")
            g = _geometry(t, items, beams, dim if lengths is not None else None)
            if lengths is None and dim is not None:
                _geometry(t, items, beams, dim)  # refuses what it would refuse with lengths
            pointers = plans.setdefault(g, []) if t.numel() else []  # (nothing moves in an empty one)
        if t.device != dev:
            raise ValueError(f"states must be on {dev}, got one on {t.device}")
        if tangents and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError("forward-mode differentiation of beam_reorder (the tangent would be lost)")
        pointers.append(t.data_ptr())
    if items == 0 or not plans:
        return states
    calls = []
    for g, pointers in plans.items():
        if len(pointers) > _lib.REORDER_MAX_STATES:
            raise ValueError(f"at most {_lib.REORDER_MAX_STATES} states of a kind, got {len(pointers)}")
        calls.append(((ctypes.c_void_p * len(pointers))(*pointers), len(pointers), items, beams, *g, p_parents, p_lengths))
    if len(calls) > 1:  # every check before the first launch
        spans = sorted((p, g) for g, pointers in plans.items() for p in pointers)
        longest = max(_span(g, items, beams) for g in plans)
        for i, (p, g) in enumerate(spans):
            for q, h in spans[i + 1:]:
                if q >= p + longest:
                    break
                if h != g and not _apart(p, g, q, h, items, beams):
                    raise ValueError("states must not overlap")
        for call in calls:
            _reordered(_LIB.argreduce_beam_reorder_check(*call))
    handle = _stream_ptr(None, dev.index) or None
    for call in calls:
        _reordered(_LIB.argreduce_beam_reorder(*call, handle))
    # written through their pointers: graphs that saved them have to know
    torch.autograd.graph.increment_version([t for t in group if not t.is_inference()])
    return states
