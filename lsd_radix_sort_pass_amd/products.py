"""The experts' own work in a mixture-of-experts layer: matrix products of rows
that stand sorted by expert, in 16 and 32 bits or with 8-bit operands, their
gradients, and the gated activation between two products.

    order, position, offsets = rs.sort_experts(experts, E)
    rows = rs.dispatch_rows(x, position)                  # (n, H), expert by expert
    up = rs.expert_products(rows, offsets, w_up)          # w_up (E, 2 F, H): (n, 2 F)
    h = rs.gate_rows(up, offsets)                         # silu(first half) * second half: (n, F)
    down = rs.expert_products(h, offsets, w_down)         # w_down (E, H, F): (n, H)
    out = rs.combine_rows(down, position, w)

and with 8-bit operands, the weights laid out once by quantize_weights:

    q, s = rs.quantize_rows(rows, offsets)
    up = rs.expert_products_fp8(q, s, offsets, *w_up8)
    q, s = rs.gate_quantize_rows(up, offsets)
    down = rs.expert_products_fp8(q, s, offsets, *w_down8)

offsets (E + 1 int32 values on the device, ascending, as sort_experts gives them):
expert e has rows offsets[e] .. offsets[e + 1] - 1.  None: the one expert has all
rows, a plain product.  Rows of no expert (before the first offset, behind the
last: those of dropped slots) are not read; a result that the call allocates has
zeros there, a given `out` keeps what it had.

Everything else (streams, gradients as calls of their own, tensors that are
refused) is as for the calls in experts.py; include/rs.h states the results in
full.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple, Union

import torch
import torch.autograd.forward_ad as _forward

from . import _lib
from .experts import (MAX_EXPERTS, _I32, _F32, _ROW_DTYPES, _Tensor, _current, _fail, _flat, _on, _ptr, _raw_stream,
                      _refuse_tangents, _rows)

__all__ = [
    "SCALE_BLOCK", "Quantized", "expert_products", "expert_products_backward", "expert_products_fp8", "quantize_rows",
    "quantize_weights", "gate_rows", "gate_rows_backward", "gate_quantize_rows",
]

SCALE_BLOCK = 128      # RS_SCALE_BLOCK in include/rs.h

_FP8 = torch.float8_e4m3fn
_FP8_DTYPES = {_FP8: 0}
_ACTS = {"silu": 0, "gelu": 1}      # rs_act
_MAX_WIDTH = 1 << 20                # RS_MAX_ROW_WIDTH


class Quantized(NamedTuple):
    """e4m3 values with the scales of their blocks."""
    values: torch.Tensor
    scales: torch.Tensor


def _blocks(width: int) -> int:
    return (width + SCALE_BLOCK - 1) // SCALE_BLOCK


def _refuse_matrices(t, name, dtypes, device) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {', '.join(str(d).replace('torch.', '') for d in dtypes)} (got {t.dtype})")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dimensions (got {t.dim()})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if not 1 <= t.shape[0] <= MAX_EXPERTS:
        raise ValueError(f"{name} must hold 1 to {MAX_EXPERTS} experts (got {t.shape[0]})")
    if not (1 <= t.shape[1] <= _MAX_WIDTH and 1 <= t.shape[2] <= _MAX_WIDTH):
        raise ValueError(f"{name} must have widths between 1 and {_MAX_WIDTH} (got {tuple(t.shape[1:])})")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which this call does not record: use it in a "
                         "torch.autograd.Function or under torch.no_grad()")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have consecutive elements in each row")


def _matrices(t, name, device=None, dtypes=_ROW_DTYPES) -> None:
    """Checks an (experts, out, in) tensor with consecutive elements in a row."""
    if not (type(t) is _Tensor and t.dtype in dtypes and t.dim() == 3 and t.is_contiguous() and not t.requires_grad
            and (t.is_cuda if device is None else t.get_device() == device.index)
            and 1 <= t.shape[0] <= MAX_EXPERTS and 1 <= t.shape[1] <= _MAX_WIDTH and 1 <= t.shape[2] <= _MAX_WIDTH):
        _refuse_matrices(t, name, dtypes, device)


def _groups(offsets, experts, device) -> None:
    """Checks the offsets of `experts` experts."""
    if offsets is not None:
        _flat(offsets, "offsets", _I32, device, (experts + 1,))
    elif experts != 1:
        raise ValueError(f"offsets are needed for {experts} experts")


def _any_groups(offsets, device) -> int:
    """Checks offsets of any number of experts and returns that."""
    if offsets is None:
        return 1
    shape = getattr(offsets, "shape", (0,))
    if len(shape) != 1 or not 2 <= shape[0] <= MAX_EXPERTS + 1:
        if isinstance(offsets, torch.Tensor):
            raise ValueError(f"offsets must hold 2 to {MAX_EXPERTS + 1} values in one dimension (got {tuple(shape)})")
    _flat(offsets, "offsets", _I32, device, shape)
    return shape[0] - 1


def _width(name, width, most=_MAX_WIDTH) -> None:
    if not 1 <= width <= most:
        raise ValueError(f"{name} must have a width between 1 and {most} (got {width})")


def expert_products(rows: torch.Tensor, offsets: Optional[torch.Tensor], weights: torch.Tensor,
                    out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Each row times the matrix of its expert: out[r] = weights[e] @ rows[r].

    rows (n, K) and weights (E, N, K) float32, float16 or bfloat16, one type;
    out (n, N) in that type, summed in float32."""
    _rows(rows, "rows")
    device, dtype = rows.device, rows.dtype
    _matrices(weights, "weights", device, (dtype,))
    count, width = rows.shape
    experts, wide, inner = weights.shape
    if inner != width:
        raise ValueError(f"weights must take rows of width {width} (got {inner})")
    _groups(offsets, experts, device)
    if out is not None:
        _rows(out, "out", device, (dtype,), (count, wide))
    if _forward._current_level >= 0:
        _refuse_tangents(rows=rows, weights=weights, out=out)
    if stream is not None or device.index != _current():
        with _on(device, stream, rows, offsets, weights, out):
            return expert_products(rows, offsets, weights, out)
    res = rows.new_empty(count, wide) if out is None else out
    code = _lib.load().rs_expert_products(
        rows.data_ptr(), _ROW_DTYPES[dtype], count, width, rows.stride(0), _ptr(offsets), experts, weights.data_ptr(), wide,
        weights.stride(1), weights.stride(0), res.data_ptr(), res.stride(0), 1 if out is None else 0,
        _raw_stream(device.index))
    if code:
        _fail(code, "rs_expert_products")
    return res


def expert_products_backward(grad_out: torch.Tensor, offsets: Optional[torch.Tensor],
                             weights: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                             out: Optional[torch.Tensor] = None, grad_weights_out: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None
                             ) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """The gradients of expert_products from that of its result (n, N): with
    weights given grad_rows (n, K), with rows given grad_weights (E, N, K), with
    both given the two as a pair, all in the one type.  An expert without rows
    gets zeros.  Without weights E is the number of offsets less one."""
    _rows(grad_out, "grad_out")
    device, dtype = grad_out.device, grad_out.dtype
    count, wide = grad_out.shape
    _width("grad_out", wide)
    if weights is not None:
        _matrices(weights, "weights", device, (dtype,))
        experts, rows_of, inner = weights.shape
        if rows_of != wide:
            raise ValueError(f"weights must give rows of width {wide} (got {rows_of})")
        _groups(offsets, experts, device)
    elif out is not None:
        raise ValueError("out needs weights")
    if rows is not None:
        _rows(rows, "rows", device, (dtype,))
        if rows.shape[0] != count:
            raise ValueError("rows must have a row for each row of grad_out")
        if weights is None:
            experts, inner = _any_groups(offsets, device), rows.shape[1]
            _width("rows", inner)
        elif rows.shape[1] != inner:
            raise ValueError(f"rows must have the width {inner} that weights take (got {rows.shape[1]})")
    elif weights is None:
        raise ValueError("weights, rows or both are needed")
    elif grad_weights_out is not None:
        raise ValueError("grad_weights_out needs rows")
    if out is not None:
        _rows(out, "out", device, (dtype,), (count, inner))
    if grad_weights_out is not None:
        _flat(grad_weights_out, "grad_weights_out", dtype, device, (experts, wide, inner))
    if _forward._current_level >= 0:
        _refuse_tangents(grad_out=grad_out, weights=weights, rows=rows, out=out, grad_weights_out=grad_weights_out)
    if stream is not None or device.index != _current():
        with _on(device, stream, grad_out, offsets, weights, rows, out, grad_weights_out):
            return expert_products_backward(grad_out, offsets, weights, rows, out, grad_weights_out)
    grad_rows, grad_weights = out, grad_weights_out
    if weights is not None and out is None:
        grad_rows = grad_out.new_empty(count, inner)
    if rows is not None and grad_weights is None:
        grad_weights = grad_out.new_empty(experts, wide, inner)
    code = _lib.load().rs_expert_products_backward(
        grad_out.data_ptr(), _ROW_DTYPES[dtype], count, wide, grad_out.stride(0), _ptr(offsets), experts, _ptr(weights),
        0 if weights is None else weights.stride(1), 0 if weights is None else weights.stride(0), _ptr(rows),
        0 if rows is None else rows.stride(0), inner, _ptr(grad_rows), 0 if grad_rows is None else grad_rows.stride(0),
        _ptr(grad_weights), 1 if out is None else 0, _raw_stream(device.index))
    if code:
        _fail(code, "rs_expert_products_backward")
    if weights is None:
        return grad_weights
    return grad_rows if rows is None else (grad_rows, grad_weights)


def expert_products_fp8(rows: torch.Tensor, row_scales: torch.Tensor, offsets: Optional[torch.Tensor],
                        weights: torch.Tensor, weight_scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                        out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """expert_products of operands in 8 bits with scales, as quantize_rows and
    quantize_weights give them.

    rows (n, K) and weights (E, N, K) float8_e4m3fn; row_scales (ceil(K / 128), n)
    and weight_scales (E, ceil(N / 128), ceil(K / 128)) float32, the product of two
    that meet a normal number (or less, where elements are zeros); out (n, N) in
    dtype (or that of a given `out`), summed in float32, for bfloat16 with the
    products of each 128 cut 2^-18 below the largest of them."""
    _rows(rows, "rows", None, _FP8_DTYPES)
    device = rows.device
    _matrices(weights, "weights", device, _FP8_DTYPES)
    count, width = rows.shape
    experts, wide, inner = weights.shape
    if inner != width:
        raise ValueError(f"weights must take rows of width {width} (got {inner})")
    _groups(offsets, experts, device)
    _flat(row_scales, "row_scales", _F32, device, (_blocks(width), count))
    _flat(weight_scales, "weight_scales", _F32, device, (experts, _blocks(wide), _blocks(width)))
    if out is not None:
        _rows(out, "out", device, _ROW_DTYPES, (count, wide))
        dtype = out.dtype
    elif dtype not in _ROW_DTYPES:
        raise TypeError(f"dtype must be one of float32, float16, bfloat16 (got {dtype})")
    if _forward._current_level >= 0:
        _refuse_tangents(rows=rows, row_scales=row_scales, weights=weights, weight_scales=weight_scales, out=out)
    if stream is not None or device.index != _current():
        with _on(device, stream, rows, row_scales, offsets, weights, weight_scales, out):
            return expert_products_fp8(rows, row_scales, offsets, weights, weight_scales, dtype, out)
    res = torch.empty(count, wide, dtype=dtype, device=device) if out is None else out
    code = _lib.load().rs_expert_products_fp8(
        rows.data_ptr(), row_scales.data_ptr(), count, width, rows.stride(0), _ptr(offsets), experts, weights.data_ptr(),
        weight_scales.data_ptr(), wide, weights.stride(1), weights.stride(0), res.data_ptr(), _ROW_DTYPES[dtype],
        res.stride(0), 1 if out is None else 0, _raw_stream(device.index))
    if code:
        _fail(code, "rs_expert_products_fp8")
    return res


def _to_8_bits(name, rows, offsets, act, out, scales_out, stream):
    """quantize_rows (act None) and gate_quantize_rows."""
    _rows(rows, "rows")
    device = rows.device
    count, width = rows.shape
    if act is not None:
        width = _half(rows, act)
    else:
        _width("rows", width)
    experts = _any_groups(offsets, device)
    if out is not None:
        _rows(out, "out", device, _FP8_DTYPES, (count, width))
    if scales_out is not None:
        _flat(scales_out, "scales_out", _F32, device, (_blocks(width), count))
    if (out is None) != (scales_out is None):
        raise ValueError("out and scales_out are given together")
    if _forward._current_level >= 0:
        _refuse_tangents(rows=rows, out=out, scales_out=scales_out)
    if stream is not None or device.index != _current():
        with _on(device, stream, rows, offsets, out, scales_out):
            return _to_8_bits(name, rows, offsets, act, out, scales_out, None)
    q, s = out, scales_out
    if out is None:
        q = torch.empty(count, width, dtype=_FP8, device=device)
        s = torch.empty(_blocks(width), count, dtype=_F32, device=device)
    to = (q.data_ptr(), q.stride(0), s.data_ptr(), 1 if out is None else 0, _raw_stream(device.index))
    of = (rows.data_ptr(), _ROW_DTYPES[rows.dtype], count, width, rows.stride(0), _ptr(offsets), experts)
    lib = _lib.load()
    code = lib.rs_quantize_rows(*of, *to) if act is None else lib.rs_gate_quantize_rows(*of, _ACTS[act], *to)
    if code:
        _fail(code, name)
    return Quantized(q, s)


def quantize_rows(rows: torch.Tensor, offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  scales_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> Quantized:
    """Rows (n, K) float32, float16 or bfloat16 as e4m3 values (n, K) and the
    float32 scales (ceil(K / 128), n) of each row's blocks of 128: a scale is
    the largest size in its block (of what is finite, and at least 2^-100) /
    448, and values stand for themselves times it.  NaN and infinities become
    NaN.  Rows of no expert become zeros."""
    return _to_8_bits("rs_quantize_rows", rows, offsets, None, out, scales_out, stream)


def quantize_weights(weights: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> Quantized:
    """Weights (E, N, K) as e4m3 values, contiguous, and float32 scales
    (E, ceil(N / 128), ceil(K / 128)), one for each 128 x 128, as quantize_rows."""
    _matrices(weights, "weights")
    device = weights.device
    if _forward._current_level >= 0:
        _refuse_tangents(weights=weights)
    if stream is not None or device.index != _current():
        with _on(device, stream, weights):
            return quantize_weights(weights)
    experts, wide, inner = weights.shape
    q = torch.empty(experts, wide, inner, dtype=_FP8, device=device)
    s = torch.empty(experts, _blocks(wide), _blocks(inner), dtype=_F32, device=device)
    code = _lib.load().rs_quantize_weights(weights.data_ptr(), _ROW_DTYPES[weights.dtype], experts, wide, inner,
                                           weights.stride(1), weights.stride(0), q.data_ptr(), s.data_ptr(),
                                           _raw_stream(device.index))
    if code:
        _fail(code, "rs_quantize_weights")
    return Quantized(q, s)


def _half(rows, act) -> int:
    """Half the width of gated rows."""
    if act not in _ACTS:
        raise ValueError(f"act must be one of {', '.join(_ACTS)} (got {act!r})")
    width = rows.shape[1]
    if width % 2:
        raise ValueError(f"rows must have an even width (got {width})")
    _width("half a row", width // 2, _MAX_WIDTH // 2)
    return width // 2


def gate_rows(rows: torch.Tensor, offsets: Optional[torch.Tensor] = None, act: str = "silu",
              out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gated rows (n, F) of rows (n, 2 F): act of the first half of a row times
    the second.  act "silu": x / (1 + exp(-x)), "gelu": x times the normal
    distribution at x."""
    _rows(rows, "rows")
    device, dtype = rows.device, rows.dtype
    count, width = rows.shape[0], _half(rows, act)
    experts = _any_groups(offsets, device)
    if out is not None:
        _rows(out, "out", device, (dtype,), (count, width))
    if _forward._current_level >= 0:
        _refuse_tangents(rows=rows, out=out)
    if stream is not None or device.index != _current():
        with _on(device, stream, rows, offsets, out):
            return gate_rows(rows, offsets, act, out)
    res = rows.new_empty(count, width) if out is None else out
    code = _lib.load().rs_gate_rows(rows.data_ptr(), _ROW_DTYPES[dtype], count, width, rows.stride(0), _ptr(offsets),
                                    experts, _ACTS[act], res.data_ptr(), res.stride(0), 1 if out is None else 0,
                                    _raw_stream(device.index))
    if code:
        _fail(code, "rs_gate_rows")
    return res


def gate_rows_backward(grad_out: torch.Tensor, rows: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                       act: str = "silu", out: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The gradient of gate_rows's rows, (n, 2 F), from that of its result (n, F);
    rows, offsets and act are the forward call's."""
    _rows(rows, "rows")
    device, dtype = rows.device, rows.dtype
    count, width = rows.shape[0], _half(rows, act)
    _rows(grad_out, "grad_out", device, (dtype,), (count, width))
    experts = _any_groups(offsets, device)
    if out is not None:
        _rows(out, "out", device, (dtype,), (count, 2 * width))
    if _forward._current_level >= 0:
        _refuse_tangents(grad_out=grad_out, rows=rows, out=out)
    if stream is not None or device.index != _current():
        with _on(device, stream, grad_out, rows, offsets, out):
            return gate_rows_backward(grad_out, rows, offsets, act, out)
    grad = rows.new_empty(count, 2 * width) if out is None else out
    code = _lib.load().rs_gate_rows_backward(grad_out.data_ptr(), grad_out.stride(0), rows.data_ptr(), _ROW_DTYPES[dtype],
                                             count, width, rows.stride(0), _ptr(offsets), experts, _ACTS[act],
                                             grad.data_ptr(), grad.stride(0), 1 if out is None else 0,
                                             _raw_stream(device.index))
    if code:
        _fail(code, "rs_gate_rows_backward")
    return grad


def gate_quantize_rows(rows: torch.Tensor, offsets: Optional[torch.Tensor] = None, act: str = "silu",
                       out: Optional[torch.Tensor] = None, scales_out: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> Quantized:
    """gate_rows in 8 bits: e4m3 values (n, F) and scales (ceil(F / 128), n), as
    quantize_rows gives them of the gated rows, in one pass and without rounding
    those to the rows' type first."""
    return _to_8_bits("rs_gate_quantize_rows", rows, offsets, act, out, scales_out, stream)
