"""Mixture-of-experts calls: tokens routed, their slots sorted by expert, and
token rows carried to their sorted places and back.

T tokens choose k of E experts each; slot s = t * k + j is choice j of token t.

    w, e = rs.route_topk(logits, k)                       # (T, k) weights, experts
    order, position, offsets = rs.sort_experts(e, E)      # slots by expert
    rows = rs.dispatch_rows(x, position)                  # (T * k, H), expert by expert
    # expert i works on rows[offsets[i]:offsets[i + 1]]
    out = rs.combine_rows(rows, position, w)              # (T, H)

Each call only marshals arguments to the C ABI (include/rs.h, which states the
results in full).  Gradients are calls of their own (`*_backward`), as every
call here is one or two kernel launches on the caller's stream: all of them
can be captured into a graph.  They do not record for autograd, and refuse
tensors that require a gradient while gradients are enabled (call them inside
a torch.autograd.Function, or under torch.no_grad()) or that carry a
forward-mode tangent (inside a torch.autograd.Function).

`stream` works as if the call were made under torch.cuda.stream(stream):
outputs and temp storage that a call allocates belong to that stream, and
inputs are kept from reuse until its work is done; ordering the streams is the
caller's.
"""
from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional, Tuple, Union

import torch
import torch.autograd.forward_ad as _forward

from . import _lib

__all__ = [
    "MAX_EXPERTS", "MAX_CHOICES", "ExpertOrder", "route_topk", "route_topk_backward", "temp_bytes_experts",
    "sort_experts", "dispatch_rows", "dispatch_rows_backward", "combine_rows", "combine_rows_backward",
]

MAX_EXPERTS = 1024      # RS_MAX_EXPERTS in include/rs.h
MAX_CHOICES = 64        # RS_MAX_CHOICES

_ROW_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}      # rs_dtype
_GATES = {"softmax": 0, "sigmoid": 1}                                      # rs_gate
_Tensor = torch.Tensor
_I32, _F32 = torch.int32, torch.float32
_SORT_FN = {torch.int32: "rs_sort_experts_i32", torch.int64: "rs_sort_experts_i64"}


class ExpertOrder(NamedTuple):
    """Slots sorted by expert: order[p] is the slot at place p, position[t, j]
    the place of slot (t, j) (~place where it is dropped), and expert e holds
    the places offsets[e] .. offsets[e + 1] - 1."""
    order: torch.Tensor
    position: torch.Tensor
    offsets: torch.Tensor


def _refuse(t, name, dtypes, dim, device, shape, rows) -> None:
    """Raises what is wrong with a tensor that failed the checks below."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if t.dtype not in dtypes:
        names = ", ".join(str(d).replace("torch.", "") for d in dtypes)
        raise TypeError(f"{name} must be one of {names} (got {t.dtype})")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions (got {t.dim()})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which this call does not record: use it in a "
                         "torch.autograd.Function or under torch.no_grad()")
    if rows:
        if t.shape[1] > 1 and t.stride(1) != 1 and t.shape[0]:
            raise ValueError(f"{name} must have consecutive elements in each row")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# The checks of the usual tensor in one expression; the rest is _refuse's.
def _rows(t, name, device=None, dtypes=_ROW_DTYPES, shape=None) -> None:
    """Checks a 2-D float tensor with consecutive elements in a row, any row
    stride."""
    if not (type(t) is _Tensor and t.dtype in dtypes and t.dim() == 2 and t.is_contiguous() and not t.requires_grad
            and (t.is_cuda if device is None else t.get_device() == device.index)
            and (shape is None or t.shape == shape)):
        _refuse(t, name, dtypes, 2, device, shape, True)


def _flat(t, name, dtype, device, shape) -> None:
    """Checks a contiguous tensor of a shape."""
    if not (type(t) is _Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and not t.requires_grad and t.get_device() == device.index):
        _refuse(t, name, (dtype,), None, device, shape, False)


def _places(position, weights, device, name="position") -> Tuple[int, int]:
    """(tokens, k) of a call's places, with its weights checked against them."""
    if not (type(position) is _Tensor and position.dtype is _I32 and position.dim() == 2 and position.is_contiguous()
            and position.get_device() == device.index):
        _refuse(position, name, (_I32,), 2, device, None, False)
    shape = position.shape
    if weights is not None:
        _flat(weights, "weights", _F32, device, shape)
    return shape


def _refuse_tangents(**tensors) -> None:
    """Refuses tensors that carry a forward-mode tangent; called while such a
    level is entered.  (None does where forward gradients are off.)"""
    for name, t in tensors.items():
        if t is not None and _forward.unpack_dual(t).tangent is not None:
            raise ValueError(f"{name} carries a tangent, which this call does not record: use it in a "
                             "torch.autograd.Function")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# The current stream's handle of a device, without making a Stream of it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


# The current device; a call asks only once it has a device tensor.
_current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


@contextlib.contextmanager
def _on(device, stream, *tensors):
    """Makes device, and stream if given, current, so that what a call
    allocates belongs to them, and keeps the call's tensors from reuse until
    the stream is done with them."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream must belong to {device} (got {stream.device})")
    with torch.cuda.device(device):
        if stream is None or stream == torch.cuda.current_stream():
            yield
            return
        with torch.cuda.stream(stream):
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
            yield


def _fail(code: int, name: str) -> None:
    from . import RadixSortError
    raise RadixSortError(code, name)


def _refuse_mode(mode) -> None:
    raise ValueError(f"mode must be one of {', '.join(_GATES)} (got {mode!r})")


def _refuse_k(k, experts) -> None:
    raise ValueError(f"k must be between 1 and min(experts, {MAX_CHOICES}) (got {k} of {experts} experts)")


def route_topk(logits: torch.Tensor, k: int, mode: str = "softmax", renormalize: bool = False, scale: float = 1.0,
               weights_out: Optional[torch.Tensor] = None, experts_out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The k largest logits of each row of a (T, E) tensor (float32, float16
    or bfloat16), ties to the lowest index, and the weights of those experts.

    mode "softmax" takes the softmax over the whole row, "sigmoid" each
    logit's own sigmoid; renormalize divides by the sum of the chosen ones
    (with "softmax": the softmax of the chosen logits); scale multiplies.
    Returns (weights float32, experts int32), both (T, k).  A logit of -inf
    bars the row from an expert; slots without one get expert -1, weight 0."""
    _rows(logits, "logits")
    tokens, experts = logits.shape
    device = logits.device
    if not 1 <= k <= experts or k > MAX_CHOICES:
        _refuse_k(k, experts)
    if mode not in _GATES:
        _refuse_mode(mode)
    if weights_out is not None:
        _flat(weights_out, "weights_out", _F32, device, (tokens, k))
    if experts_out is not None:
        _flat(experts_out, "experts_out", _I32, device, (tokens, k))
    if _forward._current_level >= 0:
        _refuse_tangents(logits=logits, weights_out=weights_out)
    if stream is not None or device.index != _current():
        with _on(device, stream, logits, weights_out, experts_out):
            return route_topk(logits, k, mode, renormalize, scale, weights_out, experts_out)
    w = torch.empty(tokens, k, dtype=torch.float32, device=device) if weights_out is None else weights_out
    e = torch.empty(tokens, k, dtype=torch.int32, device=device) if experts_out is None else experts_out
    code = _lib.load().rs_route_topk(logits.data_ptr(), _ROW_DTYPES[logits.dtype], tokens, experts, logits.stride(0),
                                     k, _GATES[mode], 1 if renormalize else 0, scale, w.data_ptr(), e.data_ptr(),
                                     _raw_stream(device.index))
    if code:
        _fail(code, "rs_route_topk")
    return w, e


def route_topk_backward(logits: torch.Tensor, experts: torch.Tensor, grad_weights: torch.Tensor,
                        mode: str = "softmax", renormalize: bool = False, scale: float = 1.0,
                        out: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The gradient of route_topk's logits, (T, E) in their dtype, from that
    of its weights; experts, mode, renormalize and scale are the forward
    call's."""
    _rows(logits, "logits")
    tokens, count = logits.shape
    device = logits.device
    rows, k = _places(experts, None, device, "experts")
    if not 1 <= k <= count or k > MAX_CHOICES:
        _refuse_k(k, count)
    if mode not in _GATES:
        _refuse_mode(mode)
    if rows != tokens:
        raise ValueError("experts must have a row for each row of logits")
    _flat(grad_weights, "grad_weights", _F32, device, (tokens, k))
    if out is not None:
        _rows(out, "out", device, (logits.dtype,), (tokens, count))
    if _forward._current_level >= 0:
        _refuse_tangents(logits=logits, grad_weights=grad_weights, out=out)
    if stream is not None or device.index != _current():
        with _on(device, stream, logits, experts, grad_weights, out):
            return route_topk_backward(logits, experts, grad_weights, mode, renormalize, scale, out)
    grad = logits.new_empty(tokens, count) if out is None else out
    code = _lib.load().rs_route_topk_backward(logits.data_ptr(), _ROW_DTYPES[logits.dtype], tokens, count,
                                              logits.stride(0), experts.data_ptr(), grad_weights.data_ptr(), k,
                                              _GATES[mode], 1 if renormalize else 0, scale, grad.data_ptr(), grad.stride(0),
                                              _raw_stream(device.index))
    if code:
        _fail(code, "rs_route_topk_backward")
    return grad


def temp_bytes_experts(n: int, num_experts: int) -> int:
    """Temp bytes of sort_experts on n slots."""
    return int(_lib.load().rs_temp_bytes_experts(n, num_experts))


def sort_experts(experts: torch.Tensor, num_experts: int, first_expert: int = 0,
                 order_out: Optional[torch.Tensor] = None, position_out: Optional[torch.Tensor] = None,
                 offsets_out: Optional[torch.Tensor] = None, temp: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> ExpertOrder:
    """Stable sort of the slots of a contiguous int32 or int64 tensor of
    expert numbers (any shape) by expert.

    Experts first_expert .. first_expert + num_experts - 1 are counted; slots
    of any other number are dropped: they sort last, and position holds ~place
    for them.  Returns ExpertOrder(order (n,), position (the shape of experts),
    offsets (num_experts + 1,)), all int32."""
    if not (type(experts) is _Tensor and experts.dtype in _SORT_FN and experts.is_cuda and experts.is_contiguous()):
        _refuse(experts, "experts", _SORT_FN, None, None, None, False)
    n, device, num = experts.numel(), experts.device, int(num_experts)
    if not 1 <= num <= MAX_EXPERTS:
        raise ValueError(f"num_experts must be between 1 and {MAX_EXPERTS} (got {num})")
    first = int(first_expert)
    if not 0 <= first <= 2**31 - num:
        raise ValueError(f"first_expert must be between 0 and 2^31 - num_experts (got {first})")
    if order_out is not None:
        _flat(order_out, "order_out", _I32, device, (n,))
    if position_out is not None:
        _flat(position_out, "position_out", _I32, device, experts.shape)
    if offsets_out is not None:
        _flat(offsets_out, "offsets_out", _I32, device, (num + 1,))
    if temp is not None:
        _flat(temp, "temp", torch.uint8, device, getattr(temp, "shape", None))
    if stream is not None or device.index != _current():
        with _on(device, stream, experts, order_out, position_out, offsets_out, temp):
            return sort_experts(experts, num, first_expert, order_out, position_out, offsets_out, temp)
    lib = _lib.load()
    order = torch.empty(n, dtype=torch.int32, device=device) if order_out is None else order_out
    position = torch.empty_like(experts, dtype=torch.int32) if position_out is None else position_out
    offsets = torch.empty(num + 1, dtype=torch.int32, device=device) if offsets_out is None else offsets_out
    if temp is None:
        need = lib.rs_temp_bytes_experts(n, num)
        temp = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    name = _SORT_FN[experts.dtype]
    code = getattr(lib, name)(experts.data_ptr(), n, first, num, order.data_ptr(), position.data_ptr(),
                              offsets.data_ptr(), _ptr(temp), 0 if temp is None else temp.numel(),
                              _raw_stream(device.index))
    if code:
        _fail(code, name)
    return ExpertOrder(order, position, offsets)


def dispatch_rows(x: torch.Tensor, position: torch.Tensor, weights: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Token rows carried to their sorted places: out[position[t, j]] = x[t],
    times weights[t, j] if given, and zeros at the place of a dropped slot.

    x (T, H) float32, float16 or bfloat16; position (T, k) int32 as
    sort_experts gives it; weights (T, k) float32.  out (rows, H) defaults to
    a new (T * k, H) tensor, which sort_experts's positions fill: without `out`
    the places have to be such, each row named by a slot.  Rows of a given `out`
    that no slot names are left as they were, and places beyond it are skipped.
    A row that several slots name gets each element from any of them."""
    _rows(x, "x")
    device = x.device
    tokens, k = _places(position, weights, device)
    count, width = x.shape
    if count != tokens:
        raise ValueError("position must have a row for each row of x")
    if out is not None:
        _rows(out, "out", device, (x.dtype,))
        if out.shape[1] != width:
            raise ValueError("out must have the width of x")
    if _forward._current_level >= 0:
        _refuse_tangents(x=x, weights=weights, out=out)
    if stream is not None or device.index != _current():
        with _on(device, stream, x, position, weights, out):
            return dispatch_rows(x, position, weights, out)
    rows = x.new_empty(tokens * k, width) if out is None else out
    code = _lib.load().rs_dispatch_rows(x.data_ptr(), _ROW_DTYPES[x.dtype], tokens, width, x.stride(0),
                                        position.data_ptr(), _ptr(weights), k, rows.data_ptr(), rows.shape[0],
                                        rows.stride(0), _raw_stream(device.index))
    if code:
        _fail(code, "rs_dispatch_rows")
    return rows


def dispatch_rows_backward(grad_rows: torch.Tensor, position: torch.Tensor, x: Optional[torch.Tensor] = None,
                           weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                           grad_weights_out: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None
                           ) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """The gradients of dispatch_rows from that of its rows: grad_x (T, H), and
    with x given also grad_weights (T, k) float32, as a pair.  weights are the
    forward call's."""
    _rows(grad_rows, "grad_rows")
    device = grad_rows.device
    count, width = grad_rows.shape
    tokens, k = _places(position, weights, device)
    if x is not None:
        _rows(x, "x", device, (grad_rows.dtype,), (tokens, width))
    elif grad_weights_out is not None:
        raise ValueError("grad_weights_out needs x")
    if out is not None:
        _rows(out, "out", device, (grad_rows.dtype,), (tokens, width))
    if grad_weights_out is not None:
        _flat(grad_weights_out, "grad_weights_out", _F32, device, (tokens, k))
    if _forward._current_level >= 0:
        _refuse_tangents(grad_rows=grad_rows, x=x, weights=weights, out=out, grad_weights_out=grad_weights_out)
    if stream is not None or device.index != _current():
        with _on(device, stream, grad_rows, position, x, weights, out, grad_weights_out):
            return dispatch_rows_backward(grad_rows, position, x, weights, out, grad_weights_out)
    grad = grad_rows.new_empty(tokens, width) if out is None else out
    dots = grad_weights_out
    if x is not None and dots is None:
        dots = torch.empty(tokens, k, dtype=torch.float32, device=device)
    code = _lib.load().rs_dispatch_rows_backward(
        grad_rows.data_ptr(), _ROW_DTYPES[grad_rows.dtype], count, grad_rows.stride(0), position.data_ptr(),
        _ptr(weights), k, _ptr(x), 0 if x is None else x.stride(0), grad.data_ptr(), grad.stride(0), _ptr(dots),
        tokens, width, _raw_stream(device.index))
    if code:
        _fail(code, "rs_dispatch_rows_backward")
    return grad if x is None else (grad, dots)


def combine_rows(rows: torch.Tensor, position: torch.Tensor, weights: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Sorted rows joined back to their tokens: out[t] = the sum over j of
    rows[position[t, j]], times weights[t, j] if given, without the dropped
    slots; zeros for a token that has no other.

    rows (n, H) float32, float16 or bfloat16, position (T, k) int32, weights
    (T, k) float32; out (T, H) in the dtype of rows, summed in float32."""
    _rows(rows, "rows")
    device = rows.device
    count, width = rows.shape
    tokens, k = _places(position, weights, device)
    if out is not None:
        _rows(out, "out", device, (rows.dtype,), (tokens, width))
    if _forward._current_level >= 0:
        _refuse_tangents(rows=rows, weights=weights, out=out)
    if stream is not None or device.index != _current():
        with _on(device, stream, rows, position, weights, out):
            return combine_rows(rows, position, weights, out)
    res = rows.new_empty(tokens, width) if out is None else out
    code = _lib.load().rs_combine_rows(rows.data_ptr(), _ROW_DTYPES[rows.dtype], count, rows.stride(0),
                                       position.data_ptr(), _ptr(weights), k, res.data_ptr(), tokens, width,
                                       res.stride(0), _raw_stream(device.index))
    if code:
        _fail(code, "rs_combine_rows")
    return res


def combine_rows_backward(grad_out: torch.Tensor, position: torch.Tensor, rows: Optional[torch.Tensor] = None,
                          weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                          grad_weights_out: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None
                          ) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """The gradients of combine_rows from that of its result: grad_rows, and
    with rows given also grad_weights (T, k) float32, as a pair.  weights are
    the forward call's.  grad_rows has the shape of rows, or (T * k, H) without
    them.  The rows of dropped slots are zeros, and so are the rows that no slot
    names; a given `out` keeps those as they were, as in dispatch_rows.  The
    places have to differ, as sort_experts's do: a row that several slots name
    gets the gradient of one of them, not their sum."""
    _rows(grad_out, "grad_out")
    device, width = grad_out.device, grad_out.shape[1]
    tokens, k = _places(position, weights, device)
    if grad_out.shape[0] != tokens:
        raise ValueError("position must have a row for each row of grad_out")
    if rows is not None:
        _rows(rows, "rows", device, (grad_out.dtype,))
        if rows.shape[1] != width:
            raise ValueError("rows must have the width of grad_out")
    elif grad_weights_out is not None:
        raise ValueError("grad_weights_out needs rows")
    if out is not None:
        _rows(out, "out", device, (grad_out.dtype,), None if rows is None else rows.shape)
        if out.shape[1] != width:
            raise ValueError("out must have the width of grad_out")
    like = out if rows is None else rows
    count = tokens * k if like is None else like.shape[0]
    if grad_weights_out is not None:
        _flat(grad_weights_out, "grad_weights_out", _F32, device, (tokens, k))
    if _forward._current_level >= 0:
        _refuse_tangents(grad_out=grad_out, rows=rows, weights=weights, out=out, grad_weights_out=grad_weights_out)
    if stream is not None or device.index != _current():
        with _on(device, stream, grad_out, position, rows, weights, out, grad_weights_out):
            return combine_rows_backward(grad_out, position, rows, weights, out, grad_weights_out)
    grad = grad_out.new_empty(count, width) if out is None else out
    dots = grad_weights_out
    if rows is not None and dots is None:
        dots = torch.empty(tokens, k, dtype=torch.float32, device=device)
    name = "rs_combine_rows_backward_all" if out is None else "rs_combine_rows_backward"
    code = getattr(_lib.load(), name)(
        grad_out.data_ptr(), _ROW_DTYPES[grad_out.dtype], tokens, width, grad_out.stride(0), position.data_ptr(),
        _ptr(weights), k, _ptr(rows), 0 if rows is None else rows.stride(0), grad.data_ptr(), grad.stride(0), count,
        _ptr(dots), _raw_stream(device.index))
    if code:
        _fail(code, name)
    return grad if rows is None else (grad, dots)
