"""Torch-facing operators beside the MoE layer (marshalling only).

Norms before and after a block, fused with its gate and residual scale, and
matrix products in 8-bit floating point (e4m3) with a scale for each block of
128. Every operator is one launch of the sm_103a library through the C ABI
(include/epoch.h states the formulas); it allocates its outputs where none are
given and keeps nothing between calls. Results carry no gradient history. All
tensors of a call are on the current CUDA device, and an output that overlaps an
input is refused but where a function allows it. ``stream`` (default: torch's
current stream) orders the launch and the outputs allocated for it; tensors that
another stream produced are the caller's to order.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional, Tuple, Union

import torch

from . import binding as B

_CODE = {torch.float32: B.EPOCH_F32, torch.bfloat16: B.EPOCH_BF16}
BLOCK = 128  # columns (and, for weights, rows) that share a scale
_E4M3 = torch.float8_e4m3fn
_MOST = 2 ** 31 - 1  # rows and columns are 32-bit in the ABI


def _stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _empty(shape, dtype, dev, stream) -> torch.Tensor:
    """An output, from the pool of the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _device(t: torch.Tensor, what: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what} must be a CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{what} is on cuda:{dev}, which is not the current device")
    return dev


def _code(t: torch.Tensor, what: str) -> int:
    code = _CODE.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be float32 or bfloat16, not {t.dtype}")
    return code


def _rows(t: torch.Tensor, dev: int, shape, what: str) -> int:
    """Elements between the rows of a tensor of that shape (n, h) whose rows are contiguous."""
    if t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{what} must be a {list(shape)} tensor on cuda:{dev}")
    n, h = shape
    if n > _MOST or h > _MOST:
        raise ValueError(f"{what} has more than 2^31 - 1 rows or columns")
    row, col = t.stride()
    if n <= 1:
        row = h
    if (col != 1 and h > 1) or row < h:
        raise ValueError(f"rows of {what} must be contiguous and must not overlap")
    return row


def _vector(t: torch.Tensor, dev: int, h: int, par: Optional[torch.dtype], what: str) -> int:
    """Pointer of a [h] parameter; every parameter of a call has one dtype (par, where one came before)."""
    if t.shape != (h,) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous [{h}] tensor on cuda:{dev}")
    if par is not None and t.dtype != par:
        raise ValueError(f"{what} has dtype {t.dtype}, the other parameters {par}")
    return t.data_ptr()


def norm_before(x: torch.Tensor, weight: torch.Tensor, *, eps: float = 1e-6, out: Optional[torch.Tensor] = None,
                out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """RMS norm of the rows of x [n, H]: x / sqrt(mean(x^2) + eps) * weight.

    x, weight [H] and the result are float32 or bfloat16 each; ``out`` (which
    may be x) or ``out_dtype`` names the result's dtype (default: x's)."""
    dev = _device(x, "x")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [n, H]")
    n, h = shape
    w, xs = _vector(weight, dev, h, None, "weight"), _rows(x, dev, shape, "x")
    if out is None:
        out, ys = _empty(shape, out_dtype or x.dtype, x.device, stream), h
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out has dtype {out.dtype}, not {out_dtype}")
    else:
        ys = _rows(out, dev, shape, "out")
    B.check(B.lib().epoch_norm_before(x.data_ptr(), xs, _code(x, "x"), w, _code(weight, "weight"), n, h, eps,
                                      out.data_ptr(), ys, _code(out, "out"), _stream(stream, dev)), "epoch_norm_before")
    return out


def norm_after(block: torch.Tensor, residual: torch.Tensor, weight: Optional[torch.Tensor] = None, *,
               gate: Optional[torch.Tensor] = None, gate_sigmoid: bool = False,
               residual_scale: Union[float, torch.Tensor] = 1.0, next_weight: Optional[torch.Tensor] = None,
               eps: float = 1e-6, out: Optional[torch.Tensor] = None, next_out: Optional[torch.Tensor] = None,
               stream=None) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """r' = residual_scale * residual + gate * rms(block) * weight and, with
    ``next_weight``, h' = rms(r') * next_weight of the unrounded r' as well.

    block, a per-element gate and h' are [n, H] of one dtype, residual and r'
    [n, H] of another or the same; weight, next_weight, a per-channel gate and a
    tensor ``residual_scale`` are [H] of one dtype (float32 or bfloat16 each).
    weight None leaves the block's output as it is; gate_sigmoid puts the gate
    through the logistic function. ``out`` and ``next_out`` may each be block,
    residual or a per-element gate of their dtype and strides.
    Returns r', or (r', h') with next_weight."""
    dev = _device(block, "block")
    shape = block.shape
    if len(shape) != 2:
        raise ValueError("block must be [n, H]")
    n, h = shape
    dtype, res_dtype = block.dtype, residual.dtype
    par, w, nw, scale, number = None, 0, 0, 0, 1.0
    if weight is not None:
        w, par = _vector(weight, dev, h, None, "weight"), weight.dtype
    if next_weight is not None:
        nw, par = _vector(next_weight, dev, h, par, "next_weight"), next_weight.dtype
    if isinstance(residual_scale, torch.Tensor):
        scale, par = _vector(residual_scale, dev, h, par, "residual_scale"), residual_scale.dtype
    else:
        number = residual_scale
    kind, gp, gs = B.EPOCH_GATE_NONE, 0, 0
    if gate is not None:
        if gate.dim() == 1:
            kind, gp, par = B.EPOCH_GATE_CHANNEL, _vector(gate, dev, h, par, "gate"), gate.dtype
        else:
            kind, gp, gs = B.EPOCH_GATE_FULL, gate.data_ptr(), _rows(gate, dev, shape, "gate")
            if gate.dtype != dtype:
                raise ValueError(f"gate has dtype {gate.dtype}, block {dtype}")
    elif gate_sigmoid:
        raise ValueError("gate_sigmoid without a gate")
    bs, rs = _rows(block, dev, shape, "block"), _rows(residual, dev, shape, "residual")
    if out is None:
        out, ys = _empty(shape, res_dtype, block.device, stream), h
    elif out.dtype != res_dtype:
        raise ValueError(f"out has dtype {out.dtype}, residual {res_dtype}")
    else:
        ys = _rows(out, dev, shape, "out")
    np_, ns = 0, 0
    if next_weight is not None:
        if next_out is None:
            next_out, ns = _empty(shape, dtype, block.device, stream), h
        elif next_out.dtype != dtype:
            raise ValueError(f"next_out has dtype {next_out.dtype}, block {dtype}")
        else:
            ns = _rows(next_out, dev, shape, "next_out")
        np_ = next_out.data_ptr()
    elif next_out is not None:
        raise ValueError("next_out without next_weight")
    code = B.EPOCH_F32
    if par is not None:
        code = _CODE.get(par)
        if code is None:
            raise ValueError(f"parameters must be float32 or bfloat16, not {par}")
    args = B.NORM_AFTER_ARGS.pack(
        block.data_ptr(), residual.data_ptr(), w, gp, scale, nw, out.data_ptr(), np_, bs, rs, gs, ys, ns, n, h,
        _code(block, "block"), _code(residual, "residual"), code, kind, 1 if gate_sigmoid else 0, number, eps)
    B.check(B.lib().epoch_norm_after(args, _stream(stream, dev)), "epoch_norm_after")
    return out if next_weight is None else (out, next_out)


def _bytes(t: torch.Tensor, dev: int, shape, what: str) -> int:
    if t.dtype != _E4M3 or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float8_e4m3fn tensor {list(shape)} on cuda:{dev}")
    if shape[-1] > _MOST or shape[-2] > _MOST:
        raise ValueError(f"{what} has more than 2^31 - 1 rows or columns")
    return t.data_ptr()


def _scales(t: torch.Tensor, dev: int, shape, what: str) -> int:
    if t.dtype != torch.float32 or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 tensor {list(shape)} on cuda:{dev}")
    return t.data_ptr()


def _index(t: Optional[torch.Tensor], dev: int, what: str) -> Optional[int]:
    if t is None:
        return None
    if t.dtype != torch.int32 or t.dim() != 1 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 vector on cuda:{dev}")
    return t.data_ptr()


def fp8_quantize(x: torch.Tensor, *, rows: Optional[torch.Tensor] = None, swiglu: bool = False,
                 q: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(q, scales): the rows of x [n, K] (float32 or bfloat16) in e4m3, with a
    float32 scale for each 128 columns, [n, ceil(K / 128)].

    rows (int32) gathers: row i of the result is row rows[i] of x, as the
    positions of an expert-sorted worklist; an index out of range gives NaN
    scales. swiglu: x is [n, 2 K] and silu(x[:, :K]) * x[:, K:] is quantised."""
    dev = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [n, K]" if not swiglu else "x must be [n, 2 K]")
    src, k = x.shape
    if swiglu:
        if k % 2:
            raise ValueError("swiglu needs an even number of columns")
        k //= 2
    rp = _index(rows, dev, "rows")
    n = src if rows is None else rows.shape[0]
    xs = _rows(x, dev, x.shape, "x")
    kb = -(-k // BLOCK)
    if n > _MOST:
        raise ValueError("rows has more than 2^31 - 1 entries")
    if q is None:
        q = _empty((n, k), _E4M3, x.device, stream)
    else:
        _bytes(q, dev, (n, k), "q")
    if scales is None:
        scales = _empty((n, kb), torch.float32, x.device, stream)
    else:
        _scales(scales, dev, (n, kb), "scales")
    B.check(B.lib().epoch_fp8_quantize(x.data_ptr(), xs, _code(x, "x"), rp, n, src, k, 1 if swiglu else 0, q.data_ptr(),
                                       scales.data_ptr(), _stream(stream, dev)), "epoch_fp8_quantize")
    return q, scales


def fp8_quantize_weight(w: torch.Tensor, *, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(q, scales) of a weight matrix [N, K] or a stack of them [E, N, K] (float32
    or bfloat16, contiguous), with a scale for each block of 128 x 128:
    [(E,) ceil(N / 128), ceil(K / 128)]."""
    dev = _device(w, "w")
    if w.dim() not in (2, 3) or not w.is_contiguous():
        raise ValueError("w must be a contiguous [N, K] or [E, N, K] tensor")
    n, k = w.shape[-2:]
    if max(w.shape) > _MOST:
        raise ValueError("w has more than 2^31 - 1 matrices, rows or columns")
    mats = w.shape[0] if w.dim() == 3 else 1
    q = _empty(tuple(w.shape), _E4M3, w.device, stream)
    scales = _empty(tuple(w.shape[:-2]) + (-(-n // BLOCK), -(-k // BLOCK)), torch.float32, w.device, stream)
    B.check(B.lib().epoch_fp8_quantize_weight(w.data_ptr(), _code(w, "w"), mats, n, k, q.data_ptr(), scales.data_ptr(),
                                              _stream(stream, dev)), "epoch_fp8_quantize_weight")
    return q, scales


def fp8_matmul(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor, *,
               offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """Scaled product of e4m3 rows a [m, K] with e4m3 weights.

    Dense: b [N, K], y = a b^T. Grouped (``offsets`` [E + 1] int32 on the device,
    as an expert-sorted worklist has them): b [E, N, K], and rows offsets[e] ..
    offsets[e + 1] - 1 are multiplied by b[e]; rows outside keep what ``out``
    holds (a fresh result leaves them undefined). Scales as fp8_quantize and
    fp8_quantize_weight give them. K must be a multiple of 16. The result is
    bfloat16 (default) or float32, accumulated in float32 and rounded once."""
    dev = _device(a, "a")
    if a.dim() != 2 or b.dim() != (2 if offsets is None else 3):
        raise ValueError("a must be [m, K]; b [N, K], or [E, N, K] with offsets")
    m, k = a.shape
    n = b.shape[-2]
    groups = 1 if offsets is None else b.shape[0]
    kb, nb = -(-k // BLOCK), -(-n // BLOCK)
    lead = () if offsets is None else (groups,)
    op = _index(offsets, dev, "offsets")
    if offsets is not None and offsets.shape[0] != groups + 1:
        raise ValueError(f"offsets must have {groups + 1} entries")
    ap, asp = _bytes(a, dev, (m, k), "a"), _scales(a_scales, dev, (m, kb), "a_scales")
    bp, bsp = _bytes(b, dev, lead + (n, k), "b"), _scales(b_scales, dev, lead + (nb, kb), "b_scales")
    if out is None:
        out, ys = _empty((m, n), out_dtype or torch.bfloat16, a.device, stream), n
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out has dtype {out.dtype}, not {out_dtype}")
    else:
        ys = _rows(out, dev, (m, n), "out")
    B.check(B.lib().epoch_fp8_matmul(ap, asp, bp, bsp, op, groups, m, n, k, out.data_ptr(), ys, _code(out, "out"),
                                     _stream(stream, dev)), "epoch_fp8_matmul")
    return out


def status(clear: bool = False, stream=None):
    """(status, error word) of the operators on the current device; synchronises."""
    word = C.c_uint32(0)
    code = B.lib().epoch_ops_status(1 if clear else 0, _stream(stream, torch.cuda.current_device()), C.byref(word))
    return code, word.value
