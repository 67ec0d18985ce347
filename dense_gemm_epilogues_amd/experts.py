"""Rows of a sparse (mixture-of-experts) layer: tokens routed and sorted by expert, and back, with gradients.

    ids, weights = expert_route(logits, topk)             # (T, k) each, of a router's logits (T, E)
    order = expert_order(ids, experts, align=128)         # ids (T, k): each token's experts
    rows = expert_dispatch(x, order)                      # (capacity, h), or quantize=True: (q, scale)
    ...                                                   # grouped products over order.offsets
    y = expert_combine(rows, order, weights)              # (T, h)
    drows, dweights = expert_combine_backward(dy, rows, order, weights)
    dx = expert_combine(drows, order)                     # the gradient of expert_dispatch
    dlogits = expert_route_backward(dweights, logits, ids)

Every function only enqueues kernels (libep.so, `ep_expert_*` in include/ep.h) on torch's current stream,
or on `stream`, as under torch.cuda.stream(stream).  All are outside autograd: results carry no gradient, the gradients
are the functions above, and a call that autograd would be expected to follow warns.
"""
import ctypes
from functools import lru_cache
from typing import NamedTuple

import torch

from . import _check, lib
from ._operators import (E4M3, ELT, blocks, check, check_out, contiguous, current_stream, empty, matrix, no_gradient,
                         on_device, streamed, unit_columns, vector)

__all__ = ["ExpertOrder", "expert_route", "expert_route_backward", "expert_order", "expert_dispatch", "expert_combine", "expert_combine_backward"]


class ExpertOrder(NamedTuple):
    """pos (T, k) int32: the row of each (token, choice), -1 where dropped; src (capacity,) int32: the flat
    (token, choice) of each row, -1 for padding; offsets (E + 1,) int32: each expert's first row."""
    pos: torch.Tensor
    src: torch.Tensor
    offsets: torch.Tensor


_SCORES = {"softmax": 0, "sigmoid": 1}


def _score(score):
    if score not in _SCORES:
        raise ValueError(f"score must be softmax or sigmoid, got {score}")
    return _SCORES[score]


@streamed
def expert_route(logits, topk, bias=None, score="softmax", groups=1, topk_groups=None, group_top=2, renormalize=True, scale=1.0):
    """(ids (T, topk) int32, weights (T, topk) float32) of a router's logits (T x E; float16, bfloat16 or float32): the topk experts
    with the highest keys, in falling order, the lowest index first among equal ones.

    An expert's key is its logit or, with a bias (E; float32) or groups, its score (softmax or sigmoid of the token's logits) plus
    the bias, in double.  With groups > 1, groups of E / groups neighbouring experts, only the topk_groups (default: all) groups with
    the greatest sum of their group_top (1 or 2) highest keys take part.  weights: scale times the chosen ones' scores (without bias), with
    renormalize over their sum.  An expert with a logit or key of -infinity or NaN is never chosen; where fewer than topk can be,
    the others' ids are -1 (which expert_order drops) with weight 0.  At most 1024 experts, 64 choices, 64 groups."""
    ld = matrix("logits", logits, ELT, (None, None))
    t, e = logits.shape
    kind = _score(score)
    if not isinstance(topk, int) or topk < 1:
        raise ValueError(f"topk must be a whole number of at least 1, got {topk}")
    if bias is not None:
        vector("bias", bias, (torch.float32,), e, logits.device)
    no_gradient("expert_route", logits, bias)
    on_device(logits)
    dev = logits.device
    ids, weights = empty((t, topk), torch.int32, dev), empty((t, topk), torch.float32, dev)
    _check(lib().ep_expert_route(logits.data_ptr(), t, e, ld, ELT[logits.dtype], None if bias is None else bias.data_ptr(), kind, groups,
                                 groups if topk_groups is None else topk_groups, group_top, topk, int(bool(renormalize)), scale,
                                 ids.data_ptr(), weights.data_ptr(), current_stream(logits)))
    return ids, weights


@streamed
def expert_route_backward(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0):
    """The gradient (T x E, the logits' type) of expert_route's logits for the gradient dweights (T, topk; float32) of its weights: ids
    are its choice, which is constant (a bias has no gradient)."""
    ldw = matrix("dweights", dweights, (torch.float32,), (None, None))
    t, k = dweights.shape
    dev = dweights.device
    ld = matrix("logits", logits, ELT, (t, None), dev)
    check("ids", ids, torch.int32, (t, k), dev)
    contiguous("ids", ids)
    kind = _score(score)
    no_gradient("expert_route_backward", dweights, logits)
    on_device(dweights)
    e = logits.shape[1]
    dlogits = empty((t, e), logits.dtype, dev)
    _check(lib().ep_expert_route_backward(dweights.data_ptr(), ldw, t, k, logits.data_ptr(), e, ld, ELT[logits.dtype], ids.data_ptr(),
                                          kind, int(bool(renormalize)), scale, dlogits.data_ptr(), e, current_stream(logits)))
    return dlogits


@lru_cache(maxsize=256)
def _order_sizes(slots, experts, align):
    """(capacity, workspace bytes): whole numbers that depend on these alone."""
    capacity, need = ctypes.c_int64(), ctypes.c_size_t()
    _check(lib().ep_expert_order_sizes(slots, experts, align, ctypes.byref(capacity), ctypes.byref(need)))
    return capacity.value, need.value


@streamed
def expert_order(ids, experts, align=1):
    """The ExpertOrder of ids (T, k; int32 or int64, contiguous): slots sorted by expert, in (token, choice)
    order within one, each expert's rows padded to a multiple of align.  An id below 0 or not below
    `experts` (at most 1024) drops its slot.  capacity = T k + min(E, T k) (align - 1), up to a multiple of
    align: as many rows as any ids can need."""
    check("ids", ids, (torch.int32, torch.int64), (None, None))
    contiguous("ids", ids)
    on_device(ids)
    t, k = ids.shape
    capacity, need = _order_sizes(t * k, experts, align)
    dev = ids.device
    pos = torch.empty((t, k), dtype=torch.int32, device=dev)
    src = torch.empty((capacity,), dtype=torch.int32, device=dev)
    offsets = torch.empty((experts + 1,), dtype=torch.int32, device=dev)
    ws = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
    _check(lib().ep_expert_order(ids.data_ptr(), ids.element_size(), t * k, experts, align, pos.data_ptr(), src.data_ptr(),
                                 offsets.data_ptr(), ws.data_ptr() if need else None, need, current_stream(ids)))
    return ExpertOrder(pos, src, offsets)


def _order(order, tokens, device):
    if not isinstance(order, ExpertOrder):
        raise ValueError(f"order must be an ExpertOrder, got {type(order).__name__}")
    check("order.pos", order.pos, torch.int32, (tokens, None), device)
    check("order.src", order.src, torch.int32, (None,), device)
    contiguous("order.pos", order.pos)
    contiguous("order.src", order.src)
    if order.pos.shape[1] < 1:
        raise ValueError("order.pos must have at least one choice a token")
    return order.pos.shape[1], order.src.shape[0]


def _weights(w, tokens, k, device):
    if w is None:
        return None, 0
    check("weights", w, torch.float32, (tokens, k), device)
    return w.data_ptr(), unit_columns("weights", w)


@streamed
def expert_dispatch(x, order, quantize=False, out=None):
    """Rows of x (T x h; float16, bfloat16 or float32) in the order's places: (capacity, h) with zeros in
    padding rows; or with quantize (q, scale), each row as quantize_fp8 quantises it, (capacity, h) e4m3 and
    (capacity, ceil(h / 128)) scales, features outermost in memory."""
    check("x", x, ELT, (None, None))
    t, h = x.shape
    k, rows = _order(order, t, x.device)
    no_gradient("expert_dispatch", x)
    ldx = unit_columns("x", x)
    on_device(x)
    dtype = E4M3 if quantize else x.dtype
    if out is None:
        out, ldo = torch.empty((rows, h), dtype=dtype, device=x.device), h
    else:
        ldo = check_out(out, dtype, (rows, h), x.device, (x, order.pos, order.src))
    scale = torch.empty((blocks(h), rows), dtype=torch.float32, device=x.device) if quantize else None
    if rows and h:
        _check(lib().ep_expert_dispatch(x.data_ptr(), t, h, ldx, ELT[x.dtype], order.pos.data_ptr(), k, order.src.data_ptr(),
                                        rows, out.data_ptr(), ldo, scale.data_ptr() if quantize else None,
                                        current_stream(x)))
    return (out, scale.t()) if quantize else out


@streamed
def expert_combine(y, order, weights=None, out=None):
    """(T, h): for each token the sum over its kept choices of weights (T, k; float32) times its row of y
    (capacity x h), in fp32, rounded once; a token with none gets zeros.  Without weights they are ones:
    the gradient of expert_dispatch."""
    check("y", y, ELT, (None, None))
    rows, h = y.shape
    t = order.pos.shape[0] if isinstance(order, ExpertOrder) else None
    k, cap = _order(order, t, y.device)
    if cap != rows:
        raise ValueError(f"y must have the order's {cap} rows, got {rows}")
    ldy = unit_columns("y", y)
    w, ldw = _weights(weights, t, k, y.device)
    no_gradient("expert_combine", y, weights)
    on_device(y)
    if out is None:
        out, ldo = torch.empty((t, h), dtype=y.dtype, device=y.device), h
    else:
        ldo = check_out(out, y.dtype, (t, h), y.device, (y, order.pos) + (() if weights is None else (weights,)))
    if t and h:
        _check(lib().ep_expert_combine(y.data_ptr(), rows, h, ldy, ELT[y.dtype], order.pos.data_ptr(), t, k, w, ldw,
                                       out.data_ptr(), ldo, current_stream(y)))
    return out


@streamed
def expert_combine_backward(dout, y, order, weights=None):
    """(dy, dweights) of expert_combine for the gradient dout (T x h) of its output: dy (capacity x h, y's
    type) with zeros in padding rows, dweights (T, k) float32 with zeros for dropped choices."""
    check("dout", dout, ELT, (None, None))
    t, h = dout.shape
    check("y", y, dout.dtype, (None, h), dout.device)
    k, rows = _order(order, t, y.device)
    if y.shape[0] != rows:
        raise ValueError(f"y must have the order's {rows} rows, got {y.shape[0]}")
    ldy, ldo = unit_columns("y", y), unit_columns("dout", dout)
    w, ldw = _weights(weights, t, k, y.device)
    no_gradient("expert_combine_backward", dout, y, weights)
    on_device(y)
    dy = torch.empty((rows, h), dtype=y.dtype, device=y.device)
    dw = torch.empty((t, k), dtype=torch.float32, device=y.device)
    if not h:
        return dy, dw.zero_()
    _check(lib().ep_expert_combine_backward(dout.data_ptr(), t, h, ldo, ELT[y.dtype], y.data_ptr(), rows, ldy,
                                            order.pos.data_ptr(), k, order.src.data_ptr(), w, ldw, dy.data_ptr(), h,
                                            dw.data_ptr(), current_stream(y)))
    return dy, dw
