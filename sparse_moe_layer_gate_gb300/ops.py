"""Torch-facing operators beside the MoE layer (marshalling only).

Norms before and after a block, fused with its gate and residual scale; matrix
products in 8-bit floating point (e4m3) with a scale for each block of 128; and a
layer's experts by themselves: the router, products grouped by expert on float32,
bfloat16 or 4-bit (e2m1) operands, and the sum of a position's edges. Every operator
is a launch of the sm_103a library (the router of many positions two, the 4-bit
quantiser of weights up to three) through the C ABI (include/epoch.h states the
formulas); it allocates its outputs where none are given and keeps nothing between calls. Results carry no gradient history. All
tensors of a call are on the current CUDA device, and an output that overlaps an
input is refused but where a function allows it. ``stream`` (default: torch's
current stream) orders the launch and the outputs allocated for it; tensors that
another stream produced are the caller's to order.
"""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple, Optional, Tuple, Union

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


class Routing(NamedTuple):
    """What ``route`` gives: experts [T, k] int32 in order of selection (-1: none), their weights [T, k] float32, the
    expert-sorted worklist's positions [T * k] int32 (-1 behind offsets[-1]) and offsets [E + 1] int32, and each
    selection's row of the worklist [T, k] int32 (-1: none)."""
    sel: torch.Tensor
    weights: torch.Tensor
    positions: torch.Tensor
    offsets: torch.Tensor
    slots: torch.Tensor


_ROUTERS = {"softmax": B.EPOCH_ROUTER_SOFTMAX, "sigmoid_group": B.EPOCH_ROUTER_SIGMOID_GROUP}


def _of(t: torch.Tensor, dev: int, dtype, shape, what: str) -> int:
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {list(shape)} on cuda:{dev}")
    return t.data_ptr()


def _flags(t: Optional[torch.Tensor], dev: int, n: int, what: str) -> int:
    if t is None:
        return 0
    if t.dtype not in (torch.uint8, torch.bool):
        raise ValueError(f"{what} must be uint8 or bool, not {t.dtype}")
    return _of(t, dev, t.dtype, (n,), what)


def route(logits: torch.Tensor, top_k: int, *, router: str = "softmax", bias: Optional[torch.Tensor] = None,
          n_group: int = 1, topk_group: int = 1, raw_weights: bool = False, live: Optional[torch.Tensor] = None,
          eligible: Optional[torch.Tensor] = None, out: Optional[Routing] = None, stream=None) -> Routing:
    """Routes positions from their router logits [T, E] (float32 or bfloat16) without running an expert: what
    grouped_matmul, fp8_quantize, fp4_quantize (positions as ``rows``), the grouped products (offsets) and combine
    (slots, weights) take.

    router "softmax" selects the largest logits (any bias included in them), "sigmoid_group" the largest sigmoid +
    bias [E] float32 under the layer's group rule; equal ones by lower id. raw_weights keeps the router's own scores
    (softmax: probabilities among all E) instead of weights that sum to 1. live [T] and eligible [E] (uint8 or bool)
    leave out positions and experts, as does a logit of -inf; a NaN logit makes its position's weights NaN."""
    dev = _device(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    n, e = logits.shape
    kind = _ROUTERS.get(router)
    if kind is None:
        raise ValueError(f"router must be one of {sorted(_ROUTERS)}, not {router!r}")
    if not 1 <= top_k <= min(16, e):
        raise ValueError(f"top_k must be in [1, {min(16, e)}], not {top_k}")
    ls = _rows(logits, dev, logits.shape, "logits")
    code = _code(logits, "logits")
    bp = 0
    if bias is not None:
        if kind == B.EPOCH_ROUTER_SOFTMAX:
            raise ValueError("a softmax router's bias is part of its logits")
        bp = _of(bias, dev, torch.float32, (e,), "bias")
    lp, ep = _flags(live, dev, n, "live"), _flags(eligible, dev, e, "eligible")
    if n * top_k > _MOST - 256:
        raise ValueError("more than 2^31 - 257 edges")
    i32, at = torch.int32, logits.device
    if out is None:
        out = Routing(_empty((n, top_k), i32, at, stream), _empty((n, top_k), torch.float32, at, stream),
                      _empty((n * top_k,), i32, at, stream), _empty((e + 1,), i32, at, stream), _empty((n, top_k), i32, at, stream))
    else:
        for t, d, shape, what in ((out.sel, i32, (n, top_k), "out.sel"), (out.weights, torch.float32, (n, top_k), "out.weights"),
                                  (out.positions, i32, (n * top_k,), "out.positions"), (out.offsets, i32, (e + 1,), "out.offsets"),
                                  (out.slots, i32, (n, top_k), "out.slots")):
            _of(t, dev, d, shape, what)
    lib, ws = B.lib(), 0
    need = lib.epoch_route_workspace_bytes(n, e)
    if need:
        work = _empty((need,), torch.uint8, at, stream)
        ws = work.data_ptr()
    sel, weights, positions, offsets, slots = out
    args = B.ROUTE_ARGS.pack(logits.data_ptr(), bp, lp, ep, sel.data_ptr(), weights.data_ptr(), positions.data_ptr(), offsets.data_ptr(),
                             slots.data_ptr(), ws, need, ls, n, e, top_k, code, kind, n_group, topk_group, 1 if raw_weights else 0)
    B.check(B.lib().epoch_route(args, _stream(stream, dev)), "epoch_route")
    return out


def combine(edges: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor, *, shared: Optional[torch.Tensor] = None,
            residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] * edges[slots[t, j]] (+ shared[t]) (+ residual[t]), summed in float32.

    edges [n, H] and shared [T, H] (the shared experts' output) are of one dtype, residual [T, H] and the result (default:
    residual's dtype, else edges') of another or the same; slots [T, k] int32 and weights [T, k] float32 as ``route``
    gives them. A negative slot adds nothing, one past the last edge makes its row NaN. ``out`` may be shared or
    residual of its dtype and strides."""
    dev = _device(edges, "edges")
    if edges.dim() != 2 or slots.dim() != 2:
        raise ValueError("edges must be [n, H], slots [T, k]")
    m, h = edges.shape
    n, k = slots.shape
    shape = (n, h)
    if n > _MOST or not 1 <= k <= 64:
        raise ValueError("slots must have at most 2^31 - 1 rows and 1 to 64 columns")
    sp, wp = _of(slots, dev, torch.int32, (n, k), "slots"), _of(weights, dev, torch.float32, (n, k), "weights")
    es = _rows(edges, dev, edges.shape, "edges")
    hp = hs = rp = rs = 0
    if shared is not None:
        hp, hs = shared.data_ptr(), _rows(shared, dev, shape, "shared")
        if shared.dtype != edges.dtype:
            raise ValueError(f"shared has dtype {shared.dtype}, edges {edges.dtype}")
    code = res = _code(edges, "edges")
    if residual is not None:
        rp, rs, res = residual.data_ptr(), _rows(residual, dev, shape, "residual"), _code(residual, "residual")
    if out is None:
        dtype = out_dtype or (edges.dtype if residual is None else residual.dtype)
        out, ys = _empty(shape, dtype, edges.device, stream), h
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out has dtype {out.dtype}, not {out_dtype}")
    else:
        ys = _rows(out, dev, shape, "out")
    args = B.COMBINE_ARGS.pack(edges.data_ptr(), hp, rp, sp, wp, out.data_ptr(), es, hs, rs, ys, n, m, h, k, code, res,
                               _code(out, "out"))
    B.check(B.lib().epoch_combine(args, _stream(stream, dev)), "epoch_combine")
    return out


def _expert(kind, x, xp, w, wp, sa, sb, offsets, rows, scale, swiglu, out, out_dtype, m, n_src, k, x_stride, dev, stream):
    """The product of experts, its operands checked: offsets, factors, output and the call."""
    shape = w.shape
    if offsets is None:
        groups, op = 1, 0
        if len(shape) != 2:
            raise ValueError("weights must be [N, K], or [E, N, K] with offsets")
    else:
        groups, op = shape[0], _index(offsets, dev, "offsets")
        if len(shape) != 3:
            raise ValueError("weights must be [N, K], or [E, N, K] with offsets")
        if offsets.shape[0] != groups + 1:
            raise ValueError(f"offsets must have {groups + 1} entries")
    n = shape[-2]
    width = n
    if swiglu:
        if n % 2:
            raise ValueError("swiglu needs an even number of rows of weights")
        width = n // 2
    number, fp = 1.0, 0
    if isinstance(scale, torch.Tensor):
        fp = _of(scale, dev, torch.float32, (groups,), "scale")
    else:
        number = scale
    if out is None:
        out, ys = _empty((m, width), out_dtype or (torch.float32 if kind == B.EPOCH_EXPERT_F32 else torch.bfloat16), x.device,
                         stream), width
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out has dtype {out.dtype}, not {out_dtype}")
    else:
        ys = _rows(out, dev, (m, width), "out")
    args = B.EXPERT_ARGS.pack(xp, wp, sa, sb, op, rows, fp, out.data_ptr(), x_stride, ys, number, groups, m, n_src, n, k, kind,
                              1 if swiglu else 0, _code(out, "out"))
    B.check(B.lib().epoch_expert_matmul(args, _stream(stream, dev)), "epoch_expert_matmul")
    return out


def grouped_matmul(x: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor], *, rows: Optional[torch.Tensor] = None,
                   swiglu: bool = False, out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                   stream=None) -> torch.Tensor:
    """Rows of x [m, K] times their expert's weights: rows offsets[e] .. offsets[e + 1] - 1 by w[e] (w [E, N, K], offsets
    [E + 1] int32 on the device, as a worklist has them; None: every row by w [N, K]).

    x and w are float32 or bfloat16 together; rows of x start on 16-byte boundaries. rows (int32, [m]) gathers: row i
    of the product is row rows[i] of x, as the positions of a worklist; an index out of range gives a row of NaN.
    swiglu: w's rows are gate | up and the result is silu(y[:, :N / 2]) * y[:, N / 2:]. Accumulated in float32 and
    rounded once (default: x's dtype); rows outside the offsets keep what ``out`` holds (a fresh result leaves them
    undefined)."""
    dev = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [m, K]")
    src, k = x.shape
    code = _code(x, "x")
    if w.dtype != x.dtype or w.get_device() != dev or not w.is_contiguous() or w.shape[-1] != k or max(w.shape) > _MOST:
        raise ValueError(f"w must be a contiguous {x.dtype} tensor [(E,) N, {k}] on cuda:{dev}")
    xs = _rows(x, dev, x.shape, "x")
    rp = _index(rows, dev, "rows") or 0
    m = src if rows is None else rows.shape[0]
    if m > _MOST:
        raise ValueError("rows has more than 2^31 - 1 entries")
    if out is None and out_dtype is None:
        out_dtype = x.dtype
    return _expert(B.EPOCH_EXPERT_BF16 if code == B.EPOCH_BF16 else B.EPOCH_EXPERT_F32, x, x.data_ptr(), w, w.data_ptr(), 0, 0,
                   offsets, rp, 1.0, swiglu, out, out_dtype, m, src, k, xs, dev, stream)


# format: (code, columns that share a scale, the scales' dtype, the product's kind)
_FP4 = {"nvfp4": (B.EPOCH_FP4_NVFP4, 16, torch.float8_e4m3fn, B.EPOCH_EXPERT_NVFP4),
        "mxfp4": (B.EPOCH_FP4_MXFP4, 32, torch.float8_e8m0fnu, B.EPOCH_EXPERT_MXFP4)}
_FP4_OF = {v[2]: v for v in _FP4.values()}


def _fp4(form: str):
    f = _FP4.get(form)
    if f is None:
        raise ValueError(f"form must be one of {sorted(_FP4)}, not {form!r}")
    return f


def _fp4_operand(q: torch.Tensor, scales: torch.Tensor, dev: int, what: str):
    """(pointers of values and scales, K, the format) of a packed operand [n, K / 2] or [E, n, K / 2]."""
    f = _FP4_OF.get(scales.dtype)
    if f is None:
        raise ValueError(f"{what}_scales must be float8_e4m3fn (nvfp4) or float8_e8m0fnu (mxfp4), not {scales.dtype}")
    shape = q.shape
    dims = len(shape)
    if dims not in (2, 3) or q.dtype != torch.uint8 or q.get_device() != dev or not q.is_contiguous():
        raise ValueError(f"{what} must be a contiguous uint8 tensor [(E,) n, K / 2] on cuda:{dev}")
    n, half = shape[-2], shape[-1]
    if half > _MOST // 2 or n > _MOST or shape[0] > _MOST:
        raise ValueError(f"{what} has more than 2^31 - 1 matrices, rows or columns")
    want = (-(-half // 128), n, 256 // f[1])
    if dims == 3:
        want = (shape[0], *want)
    if scales.shape != want or scales.get_device() != dev or not scales.is_contiguous():
        raise ValueError(f"{what}_scales must be a contiguous tensor {list(want)} on cuda:{dev}")
    return q.data_ptr(), scales.data_ptr(), 2 * half, f


def fp4_quantize(x: torch.Tensor, *, form: str = "nvfp4", rows: Optional[torch.Tensor] = None, swiglu: bool = False,
                 tensor_scale: float = 1.0, q: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(q, scales): the rows of x [n, K] (float32 or bfloat16) in e2m1, q [n, K / 2] uint8 with the even column in a
    byte's low half, and scales [ceil(K / 256), n, 256 / block].

    form "nvfp4": blocks of 16 columns with float8_e4m3fn scales of x / tensor_scale; "mxfp4": blocks of 32 with
    float8_e8m0fnu scales (powers of two). A value is q * scale (* tensor_scale, which the product's ``scale`` has
    to bring back); a tensor_scale that is a power of two rounds nothing. rows and swiglu as for fp8_quantize. K must
    be a multiple of 32."""
    dev = _device(x, "x")
    code, block, dtype, _ = _fp4(form)
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
    if n > _MOST:
        raise ValueError("rows has more than 2^31 - 1 entries")
    if q is None:
        q = _empty((n, k // 2), torch.uint8, x.device, stream)
    else:
        _of(q, dev, torch.uint8, (n, k // 2), "q")
    shape = (-(-k // 256), n, 256 // block)
    if scales is None:
        scales = _empty(shape, dtype, x.device, stream)
    else:
        _of(scales, dev, dtype, shape, "scales")
    B.check(B.lib().epoch_fp4_quantize(x.data_ptr(), xs, _code(x, "x"), rp, n, src, k, 1 if swiglu else 0, code, tensor_scale,
                                       q.data_ptr(), scales.data_ptr(), _stream(stream, dev)), "epoch_fp4_quantize")
    return q, scales


def fp4_quantize_weight(w: torch.Tensor, *, form: str = "nvfp4", stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(q, scales, tensor_scales) of a weight matrix [N, K] or a stack of them [E, N, K] (float32 or bfloat16,
    contiguous): q [(E,) N, K / 2], scales [(E,) ceil(K / 256), N, 256 / block] and a factor for each matrix, [E] float32
    ([1] for one): nvfp4: the power of two that keeps the blocks' scales within e4m3, mxfp4: 1. Together with an
    activation's tensor_scale they are fp4_matmul's ``scale``."""
    dev = _device(w, "w")
    code, block, dtype, _ = _fp4(form)
    if w.dim() not in (2, 3) or not w.is_contiguous():
        raise ValueError("w must be a contiguous [N, K] or [E, N, K] tensor")
    n, k = w.shape[-2:]
    if max(w.shape) > _MOST:
        raise ValueError("w has more than 2^31 - 1 matrices, rows or columns")
    lead = tuple(w.shape[:-2])
    mats = w.shape[0] if w.dim() == 3 else 1
    q = _empty(lead + (n, k // 2), torch.uint8, w.device, stream)
    scales = _empty(lead + (-(-k // 256), n, 256 // block), dtype, w.device, stream)
    factors = _empty((mats,), torch.float32, w.device, stream)
    B.check(B.lib().epoch_fp4_quantize_weight(w.data_ptr(), _code(w, "w"), mats, n, k, code, q.data_ptr(), scales.data_ptr(),
                                              factors.data_ptr(), _stream(stream, dev)), "epoch_fp4_quantize_weight")
    return q, scales, factors


def fp4_dequantize(q: torch.Tensor, scales: torch.Tensor, *, tensor_scale: Union[float, torch.Tensor] = 1.0,
                   out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """The values [.., n, K] that rows or a stack of weights in e2m1 stand for, times tensor_scale (a number, or a
    factor for each matrix of the stack, [E] float32), bfloat16 (default) or float32."""
    dev = _device(q, "q")
    if q.dim() not in (2, 3):
        raise ValueError("q must be [n, K / 2] or [E, n, K / 2]")
    qp, sp, k, f = _fp4_operand(q, scales, dev, "q")
    mats, n = (q.shape[0] if q.dim() == 3 else 1), q.shape[-2]
    number, fp = 1.0, None
    if isinstance(tensor_scale, torch.Tensor):
        fp = _of(tensor_scale, dev, torch.float32, (mats,), "tensor_scale")
    else:
        number = tensor_scale
    shape = tuple(q.shape[:-1]) + (k,)
    if out is None:
        out, ys = _empty(shape, out_dtype or torch.bfloat16, q.device, stream), k
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out has dtype {out.dtype}, not {out_dtype}")
    elif q.dim() == 2:
        ys = _rows(out, dev, shape, "out")
    else:
        _of(out, dev, out.dtype, shape, "out")
        ys = k
    B.check(B.lib().epoch_fp4_dequantize(qp, sp, f[0], mats, n, k, number, fp, out.data_ptr(), ys, _code(out, "out"),
                                         _stream(stream, dev)), "epoch_fp4_dequantize")
    return out


def fp4_matmul(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor, *,
               offsets: Optional[torch.Tensor] = None, scale: Union[float, torch.Tensor] = 1.0, swiglu: bool = False,
               out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """Product of e2m1 rows a [m, K / 2] with e2m1 weights of the same format, both with their scales as fp4_quantize
    and fp4_quantize_weight give them.

    Dense: b [N, K / 2], y = scale * a b^T. Grouped (``offsets``): b [E, N, K / 2], as grouped_matmul. scale: a number,
    or a factor for each matrix of b ([E] float32; dense [1]). swiglu as for grouped_matmul. The result is bfloat16
    (default) or float32, accumulated in float32 and rounded once."""
    dev = _device(a, "a")
    if a.dim() != 2:
        raise ValueError("a must be [m, K / 2]")
    ap, asp, k, f = _fp4_operand(a, a_scales, dev, "a")
    bp, bsp, kb, fb = _fp4_operand(b, b_scales, dev, "b")
    if kb != k or fb is not f:
        raise ValueError("a and b must have the same K and the same format")
    m = a.shape[0]
    return _expert(f[3], a, ap, b, bp, asp, bsp, offsets, 0, scale, swiglu, out, out_dtype, m, m, k, k // 2, dev, stream)


def status(clear: bool = False, stream=None):
    """(status, error word) of the operators on the current device; synchronises."""
    word = C.c_uint32(0)
    code = B.lib().epoch_ops_status(1 if clear else 0, _stream(stream, torch.cuda.current_device()), C.byref(word))
    return code, word.value
