"""Operators beside the layer: norms around a block, e4m3 quantisation and the
scaled e4m3 product, each against its formula in 64 bits, and their refusals.

Tolerances count roundings: u is half a step of fp32 (2^-24) and _half(t) half a
step of the result's type, both relative. They are derived at each test."""
import ctypes as C
import math

import pytest
import torch

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
TINY = 2.0 ** -126


def _half(t):
    return torch.finfo(t).eps / 2


@pytest.fixture(scope="module")
def ops():
    from sparse_moe_layer_gate_gb300 import builder, ops as o
    if builder.is_stale():
        builder.build()
    return o


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rnd(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _rms64(x, w, eps):
    k = 1.0 / torch.sqrt(x.square().mean(1, keepdim=True) + eps)
    return k, x * k * w


def _within(got, want, bound, what=""):
    d = (got.double() - want).abs()
    over = d > bound
    assert not bool(over.any()), (what, int(over.sum()), float((d / bound.clamp(min=1e-300)).max()))


def _norm_units(h):
    """Roundings of rms's factor: a thread adds at most 32 squares (or h / 512 where the row is longer) one after
    another, then 5 + 16 sums across threads; half of that through the root, plus root, mean and products."""
    return (max(32, h / 512) + 21) / 2 + 12


# ------------------------------------------------------------------------------------- norm before
@pytest.mark.gpu
@pytest.mark.parametrize("n,h", [(1, 1), (1, 2048), (3, 8), (5, 7), (33, 64), (17, 513), (2, 2047), (9, 4096),
                                 (4, 8200), (2, 16384), (3, 16392), (2, 20001)])
@pytest.mark.parametrize("xt,ot,pt", [(BF16, BF16, F32), (F32, BF16, BF16), (BF16, F32, BF16), (F32, F32, F32)])
def test_norm_before(ops, n, h, xt, ot, pt):
    g = _gen(n * 7919 + h)
    x, w = _rnd(g, n, h, std=3.0, dtype=xt), (1 + _rnd(g, h, std=0.2)).to(pt)
    got = ops.norm_before(x, w, eps=1e-5, out_dtype=ot)
    assert got.dtype == ot and got.shape == (n, h)
    _, want = _rms64(x.double(), w.double(), float(torch.tensor(1e-5)))
    _within(got, want, want.abs() * (_norm_units(h) * U + _half(ot) * (ot == BF16)) + 1e-30)


@pytest.mark.gpu
@pytest.mark.parametrize("case", ["stride", "offset", "alias", "zero_rows", "zeros", "nan_row", "far_rows"])
def test_norm_before_layouts(ops, case):
    g = _gen(5)
    n, h = 6, 256
    w = 1 + _rnd(g, h, std=0.2)
    if case == "zero_rows":
        got = ops.norm_before(torch.empty(0, h, device="cuda", dtype=BF16), w)
        assert got.shape == (0, h)
        return
    x = _rnd(g, n, h, dtype=BF16)
    want = _rms64(x.double(), w.double(), 1e-6)[1]
    bound = want.abs() * (_norm_units(h) * U + _half(BF16)) + 1e-30
    if case == "stride":  # rows apart, on and off 16-byte boundaries
        for pad in (8, 3):
            v = torch.full((n, h + pad), 99.0, device="cuda", dtype=BF16)
            v[:, :h] = x
            o = torch.full((n, h + pad + 1), -7.0, device="cuda", dtype=BF16)
            got = ops.norm_before(v[:, :h], w, out=o[:, 1:h + 1])
            _within(got, want, bound)
            assert bool((o[:, 0] == -7).all()) and bool((o[:, h + 1:] == -7).all())
    elif case == "offset":  # a base that is aligned to its element alone
        v = torch.empty(n * h + 1, device="cuda", dtype=BF16)[1:].view(n, h)
        v.copy_(x)
        _within(ops.norm_before(v, w), want, bound)
    elif case == "alias":
        v = x.clone()
        assert ops.norm_before(v, w, out=v) is v
        _within(v, want, bound)
    elif case == "zeros":  # a row of zeros is a row of zeros
        x[2] = 0
        got = ops.norm_before(x, w)
        assert bool((got[2] == 0).all()) and bool(got.isfinite().all())
    elif case == "nan_row":  # a bad row stays alone
        x[3, 17] = math.nan
        got = ops.norm_before(x, w)
        assert bool(got[3].isnan().all())
        keep = [0, 1, 2, 4, 5]
        _within(got[keep], want[keep], bound[keep])
    else:  # rows whose offsets pass 32 bits
        far = (1 << 31) // 2 + 24
        base = torch.empty(2 * far + h, device="cuda", dtype=BF16)
        v = base.as_strided((3, h), (far, 1))
        v.copy_(x[:3])
        got = ops.norm_before(v, w, out=v)
        _within(got, want[:3], bound[:3])


# -------------------------------------------------------------------------------------- norm after
def _after64(b, r, w, gate, sig, scale, nw, eps):
    """r', h' in 64 bits and the bounds of both in fp32, before their last rounding."""
    b, r = b.double(), r.double()
    h = b.shape[1]
    z = b if w is None else _rms64(b, w.double(), eps)[1]
    if gate is not None:
        gate = gate.double()
        z = z * (torch.sigmoid(gate) if sig else gate)
    sr = r * (scale.double() if isinstance(scale, torch.Tensor) else scale)
    out = sr + z
    size = sr.abs() + z.abs()
    e_out = size * (_norm_units(h) + 10) * U  # the factor, the gate (exp, sum, quotient), two products and a sum
    if nw is None:
        return out, e_out, None, None
    k, nxt = _rms64(out, nw.double(), eps)
    rel = e_out.square().mean(1, keepdim=True).sqrt() * k + _norm_units(h) * U
    return out, e_out, nxt, (e_out + out.abs() * rel) * k * nw.double().abs()


@pytest.mark.gpu
@pytest.mark.parametrize("n,h", [(1, 1), (1, 2048), (7, 40), (19, 1001), (5, 4096), (3, 8192), (2, 16400), (3, 17001)])
@pytest.mark.parametrize("at,rt,pt", [(BF16, BF16, F32), (BF16, F32, BF16), (F32, BF16, F32), (F32, F32, BF16)])
@pytest.mark.parametrize("form", ["plain", "gate", "full", "no_weight"])
def test_norm_after(ops, n, h, at, rt, pt, form):
    g = _gen(n * 104729 + h)
    b, r = _rnd(g, n, h, dtype=at), _rnd(g, n, h, std=2.0, dtype=rt)
    w, nw = (1 + _rnd(g, h, std=0.2)).to(pt), (1 + _rnd(g, h, std=0.2)).to(pt)
    gate, sig, scale = None, False, 1.0
    if form == "gate":
        gate, scale, nw = _rnd(g, h).to(pt), (1 + _rnd(g, h, std=0.1)).to(pt), None
    elif form == "full":
        gate, sig, scale = _rnd(g, n, h, std=3.0, dtype=at), True, 0.75
    elif form == "no_weight":
        w, scale = None, -0.5
    got = ops.norm_after(b, r, w, gate=gate, gate_sigmoid=sig, residual_scale=scale, next_weight=nw, eps=1e-6)
    out, e_out, nxt, e_nxt = _after64(b, r, w, gate, sig, scale, nw, 1e-6)
    a = got if nw is None else got[0]
    assert a.dtype == rt
    _within(a, out, e_out + out.abs() * _half(rt) * (1 + 2 ** -7) + 1e-30, "r'")
    if nw is not None:
        assert got[1].dtype == at
        _within(got[1], nxt, e_nxt + nxt.abs() * _half(at) * (1 + 2 ** -7) + 1e-30, "h'")


@pytest.mark.gpu
@pytest.mark.parametrize("n,h", [(1300, 4096), (2433, 2048), (5001, 1000), (20000, 64), (9731, 8), (6011, 1088),
                                 (2600, 2816), (700, 4632), (1500, 1001), (400, 5761)])
@pytest.mark.parametrize("at,rt", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("form", ["before", "channel", "full", "no_weight"])
def test_norms_of_many_rows(ops, n, h, at, rt, form):
    g = _gen(n + h)
    b, r = _rnd(g, n, h, dtype=at), _rnd(g, n, h, std=2.0, dtype=rt)
    w, nw = 1 + _rnd(g, h, std=0.2), 1 + _rnd(g, h, std=0.2)
    if form == "before":
        want = _rms64(r.double(), w.double(), 1e-6)[1]
        _within(ops.norm_before(r, w, out_dtype=at), want, want.abs() * (_norm_units(h) * U + _half(at)) + 1e-30)
        return
    gate, sig, scale = None, False, 1.0
    if form == "channel":
        gate, sig, scale = _rnd(g, h), True, 1 + _rnd(g, h, std=0.1)
    elif form == "full":
        gate, sig, scale = _rnd(g, n, h, std=3.0, dtype=at), True, 0.75
    else:
        w = None
    got = ops.norm_after(b, r, w, gate=gate, gate_sigmoid=sig, residual_scale=scale, next_weight=nw)
    out, e_out, nxt, e_nxt = _after64(b, r, w, gate, sig, scale, nw, 1e-6)
    _within(got[0], out, e_out + out.abs() * _half(rt) * (1 + 2 ** -7) + 1e-30, "r'")
    _within(got[1], nxt, e_nxt + nxt.abs() * _half(at) * (1 + 2 ** -7) + 1e-30, "h'")
    alone = ops.norm_after(b, r, w, gate=gate, gate_sigmoid=sig, residual_scale=scale, next_weight=None)
    assert torch.equal(alone, got[0])
    assert torch.equal(ops.norm_after(b, r, w, gate=gate, gate_sigmoid=sig, residual_scale=scale, out=r), got[0])


@pytest.mark.gpu
@pytest.mark.parametrize("h", [1024, 1023, 16400])
def test_norm_after_in_place_and_strided(ops, h):
    g = _gen(11)
    n = 5
    b, r = _rnd(g, n, h, dtype=BF16), _rnd(g, n, h, dtype=F32)
    w, nw = 1 + _rnd(g, h, std=0.1), 1 + _rnd(g, h, std=0.1)
    want = ops.norm_after(b, r, w, next_weight=nw)
    bb, rr = b.clone(), r.clone()
    got = ops.norm_after(bb, rr, w, next_weight=nw, out=rr, next_out=bb)
    assert got[0] is rr and got[1] is bb
    assert torch.equal(rr, want[0]) and torch.equal(bb, want[1])
    wide_b, wide_r = torch.zeros(n, h + 16, device="cuda", dtype=BF16), torch.zeros(n, h + 5, device="cuda")
    wide_b[:, :h], wide_r[:, :h] = b, r
    got = ops.norm_after(wide_b[:, :h], wide_r[:, :h], w, next_weight=nw)
    out, e_out, nxt, e_nxt = _after64(b, r, w, None, False, 1.0, nw, 1e-6)
    _within(got[0], out, e_out + 1e-30)
    _within(got[1], nxt, e_nxt + nxt.abs() * _half(BF16) * (1 + 2 ** -7) + 1e-30)


@pytest.mark.gpu
@pytest.mark.parametrize("n,h", [(5, 64), (700, 4632), (5, 1001), (1300, 2048), (3, 16400), (2, 17001), (6, 5761)])
@pytest.mark.parametrize("at,rt", [(BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("kind", ["full", "full_sigmoid", "channel", "channel_sigmoid"])
@pytest.mark.parametrize("pad", [16, 3])
def test_norm_after_every_row_tensor_strided(ops, n, h, at, rt, kind, pad):
    """Block, residual, a gate for each element and both outputs in rows of their own distances, with the gate as it is
    and through the logistic function; what lies between the rows stays as it was."""
    g = _gen(n + h + pad)
    b, r, gate = _rnd(g, n, h, dtype=at), _rnd(g, n, h, std=2.0, dtype=rt), _rnd(g, n, h, std=3.0, dtype=at)
    w, nw, scale = 1 + _rnd(g, h, std=0.2), 1 + _rnd(g, h, std=0.2), 1 + _rnd(g, h, std=0.1)
    if kind.startswith("channel"):
        gate = _rnd(g, h)

    def apart(dtype, extra, src=None):
        v = torch.full((n, h + extra), 77.0, device="cuda", dtype=dtype)
        if src is not None:
            v[:, :h] = src
        return v

    vb, vr, vo, vn = apart(at, pad, b), apart(rt, 2 * pad, r), apart(rt, 3 * pad), apart(at, 4 * pad)
    vg = gate if gate.dim() == 1 else apart(at, 5 * pad, gate)[:, :h]
    sig = kind.endswith("sigmoid")
    got = ops.norm_after(vb[:, :h], vr[:, :h], w, gate=vg, gate_sigmoid=sig, residual_scale=scale, next_weight=nw, out=vo[:, :h],
                         next_out=vn[:, :h])
    out, e_out, nxt, e_nxt = _after64(b, r, w, gate, sig, scale, nw, 1e-6)
    _within(got[0], out, e_out + out.abs() * _half(rt) * (rt == BF16) * (1 + 2 ** -7) + 1e-30, "r'")
    _within(got[1], nxt, e_nxt + nxt.abs() * _half(at) * (1 + 2 ** -7) + 1e-30, "h'")
    assert bool((vo[:, h:] == 77).all()) and bool((vn[:, h:] == 77).all())


# ---------------------------------------------------------------------------------------- quantise
def _scale32(amax):
    """max(amax / 448, 2^-126) rounded once to fp32: a quotient of fp32 values taken in 64 bits rounds to the fp32
    quotient (torch's own division by a number multiplies by its rounded reciprocal)."""
    return (amax.double() / 448.0).float().clamp(min=TINY)


def _quant64(v):
    """Scales in fp32 as defined, values in 64 bits, blocks of 128 columns."""
    n, k = v.shape
    kb = -(-k // 128)
    p = torch.nn.functional.pad(v, (0, kb * 128 - k)).view(n, kb, 128)
    return (_scale32(p.abs().amax(2)) if v.dtype == F32 else (p.abs().amax(2) / 448.0).clamp(min=TINY)), p


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("n,k", [(1, 1), (1, 128), (1, 2048), (3, 130), (5, 1001), (64, 512), (333, 264), (2, 4096), (9000, 2048), (20011, 520), (30000, 333)])
def test_fp8_quantize_rows(ops, n, k, dt):
    x = _rnd(_gen(n + k), n, k, dtype=dt)
    x[0, : max(1, k // 2)] = 0
    q, s = ops.fp8_quantize(x)
    ws, p = _quant64(x.float())  # fp32 and the same two operations: equal bit by bit
    wq = (p * (1.0 / ws.double()).float().unsqueeze(2)).flatten(1)[:, :k].to(E4M3)
    assert torch.equal(s, ws)
    assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8))


@pytest.mark.gpu
def test_fp8_quantize_gather_strided_and_bad_rows(ops):
    g = _gen(3)
    x = _rnd(g, 9, 300, dtype=BF16)
    wide = torch.zeros(9, 308, device="cuda", dtype=BF16)
    wide[:, :300] = x
    rows = torch.tensor([8, 0, 0, 3, 9, -1, 7], device="cuda", dtype=torch.int32)
    q, s = ops.fp8_quantize(wide[:, :300], rows=rows)
    good = [0, 1, 2, 3, 6]
    wq, ws = ops.fp8_quantize(x[rows[good].long()].contiguous())
    assert torch.equal(q[good].view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s[good], ws)
    assert bool(s[[4, 5]].isnan().all())
    e, es = ops.fp8_quantize(x, rows=rows[:0])
    assert e.shape == (0, 300) and es.shape == (0, 3)
    e, es = ops.fp8_quantize(x[:0], rows=rows)  # no source row: every index is out of range
    assert bool(es.isnan().all())


@pytest.mark.gpu
def test_fp8_quantize_special_values(ops):
    x = torch.zeros(5, 256, device="cuda")
    x[1, 5], x[2, 200], x[3, 0], x[4, 0] = math.nan, math.inf, 1e-40, 3e38
    q, s = ops.fp8_quantize(x)
    assert float(s[0, 0]) == TINY and bool((q[0].float() == 0).all())
    assert bool(s[1, 0].isnan()) and float(s[1, 1]) == TINY
    assert bool(s[2, 1].isinf()) and float(s[2, 0]) == TINY
    assert float(s[3, 0]) == TINY
    assert float(q[4, 0].float()) == 448.0
    b, sb = ops.fp8_quantize_weight(torch.ones(64, 256, device="cuda"))
    y = ops.fp8_matmul(q, s, b, sb)
    assert bool(y[0].eq(0).all()) and bool(y[1].isnan().all()) and bool(y[2].isnan().all())
    assert bool(y[3:].isfinite().all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("n,k", [(1, 8), (3, 512), (77, 200), (5, 333)])
def test_fp8_quantize_swiglu(ops, n, k, dt):
    x = _rnd(_gen(n * k), n, 2 * k, dtype=dt)
    q, s = ops.fp8_quantize(x, swiglu=True)
    v = torch.nn.functional.silu(x[:, :k].double()) * x[:, k:].double()
    ws, _ = _quant64(v)
    # exp (2 steps), sum, quotient and product of the SwiGLU, the quotient by 448: 8 roundings
    _within(s, ws, ws * 8 * U + 1e-300)
    sk = ws.repeat_interleave(128, 1)[:, :k]
    # half a step of e4m3 (2^-4 of the value, 2^-10 of the scale below its normal range), and 20 fp32 roundings
    _within(q.double() * s.double().repeat_interleave(128, 1)[:, :k], v,
            v.abs() * (2.0 ** -4 + 20 * U) + sk * 2.0 ** -10 * (1 + 20 * U))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (130, 300), (2, 256, 144), (3, 5, 1000)])
def test_fp8_quantize_weight(ops, shape, dt):
    w = _rnd(_gen(sum(shape)), *shape, dtype=dt)
    q, s = ops.fp8_quantize_weight(w)
    n, k = shape[-2:]
    nb, kb = -(-n // 128), -(-k // 128)
    p = torch.nn.functional.pad(w.float(), (0, kb * 128 - k, 0, nb * 128 - n)).unflatten(-1, (kb, 128)).unflatten(-3, (nb, 128))
    ws = _scale32(p.abs().amax(dim=(-3, -1)))
    assert torch.equal(s, ws)
    wide = (1.0 / ws.double()).float().repeat_interleave(128, -1).repeat_interleave(128, -2)[..., :n, :k]
    assert torch.equal(q.view(torch.uint8), (w.float() * wide).to(E4M3).view(torch.uint8))


# ----------------------------------------------------------------------------------------- product
def _operands(ops, g, m, n, k, e):
    """e4m3 operands with scales of very different sizes from block to block."""
    a = _rnd(g, m, k) * torch.exp(2 * _rnd(g, m, 1))
    b = _rnd(g, e, n, k, std=k ** -0.5) * torch.exp(_rnd(g, e, 1, 1))
    qa, sa = ops.fp8_quantize(a)
    qb, sb = ops.fp8_quantize_weight(b)
    sa = sa * torch.exp(_rnd(g, *sa.shape))
    sb = sb * torch.exp(_rnd(g, *sb.shape))
    return qa, sa.contiguous(), qb, sb.contiguous()


def _product64(qa, sa, qb, sb, offsets):
    """y in 64 bits, and the same sum over absolute values."""
    m, k = qa.shape
    e, n = qb.shape[:2]
    a = qa.double() * sa.double().repeat_interleave(128, 1)[:, :k]
    y = torch.full((m, n), math.nan, device="cuda", dtype=torch.float64)
    s = torch.zeros_like(y)
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        if hi > lo:
            w = qb[i].double() * sb[i].double().repeat_interleave(128, 1).repeat_interleave(128, 0)[:n, :k]
            y[lo:hi] = a[lo:hi] @ w.T
            s[lo:hi] = a[lo:hi].abs() @ w.abs().T
    return y, s


def _product_bound(y, s, k, out):
    """Products of e4m3 are exact in fp32. A block's 128 are summed by the tensor core (a truncating sum: 2^-23 each),
    then each block takes a product with the scale, a product of scales and a sum."""
    kb = -(-k // 128)
    return s * (128 * 2.0 ** -23 + (kb + 2) * U) + (y.abs() * _half(BF16) * (1 + 2 ** -7) if out == BF16 else 0) + 1e-30


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (1, 4096, 2048), (2, 15, 128), (7, 130, 144), (9, 33, 640), (16, 256, 48),
                                   (31, 200, 1040), (64, 129, 512), (65, 64, 128), (65, 1, 16), (128, 256, 256),
                                   (129, 300, 272), (200, 511, 1168), (257, 513, 2064), (1000, 1024, 512), (511, 584, 256),
                                   (256, 8, 400)])
def test_fp8_matmul_dense(ops, m, n, k, out):
    qa, sa, qb, sb = _operands(ops, _gen(m * n + k), m, n, k, 1)
    got = ops.fp8_matmul(qa, sa, qb[0], sb[0], out_dtype=out)
    y, s = _product64(qa, sa, qb, sb, [0, m])
    assert got.dtype == out
    _within(got, y, _product_bound(y, s, k, out))


GROUPS = {
    "one_each": [0, 1, 2, 3, 4],
    "empty_ends": [0, 0, 0, 9, 9],
    "few": [0, 5, 5, 40, 64],
    "ragged": [0, 1, 130, 130, 163, 420, 421],
    "boxes": [0, 32, 97, 161, 290, 546],
    "late_start": [3, 10, 80, 100],
    "wide": [0, 300, 301, 302, 1200],
}


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("n,k", [(64, 128), (272, 400), (513, 1040)])
@pytest.mark.parametrize("name", list(GROUPS))
def test_fp8_matmul_grouped(ops, name, n, k, out):
    offsets = GROUPS[name]
    m = offsets[-1] + 6  # rows behind the last group stay as they were
    e = len(offsets) - 1
    qa, sa, qb, sb = _operands(ops, _gen(m + n), m, n, k, e)
    buf = torch.full((m, n), 77.0, device="cuda", dtype=out)
    got = ops.fp8_matmul(qa, sa, qb, sb, offsets=torch.tensor(offsets, device="cuda", dtype=torch.int32), out=buf)
    y, s = _product64(qa, sa, qb, sb, offsets)
    lo, hi = offsets[0], offsets[-1]
    _within(got[lo:hi], y[lo:hi], _product_bound(y, s, k, out)[lo:hi])
    assert bool((got[:lo] == 77).all()) and bool((got[hi:] == 77).all())


@pytest.mark.gpu
@pytest.mark.parametrize("m", [40, 300])
def test_fp8_matmul_bad_offsets_are_read_in_range(ops, m):
    g = _gen(m)
    qa, sa, qb, sb = _operands(ops, g, m, 96, 256, 4)
    bad = torch.tensor([-5, 20, 10, m + 1000, m - 1], device="cuda", dtype=torch.int32)
    good = [0, 20, 20, m, m]
    got = ops.fp8_matmul(qa, sa, qb, sb, offsets=bad, out_dtype=F32)
    y, s = _product64(qa, sa, qb, sb, good)
    _within(got, y, _product_bound(y, s, 256, F32))
    assert ops.status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [5, 200])
def test_fp8_matmul_strided_output_and_far_rows(ops, m):
    g = _gen(m)
    n, k = 72, 256
    qa, sa, qb, sb = _operands(ops, g, m, n, k, 1)
    want = ops.fp8_matmul(qa, sa, qb[0], sb[0], out_dtype=F32)
    for pad in (8, 3):
        buf = torch.full((m, n + pad), 5.0, device="cuda")
        got = ops.fp8_matmul(qa, sa, qb[0], sb[0], out=buf[:, :n])
        assert torch.equal(got, want) and bool((buf[:, n:] == 5).all())
    stride = (1 << 31) // (m - 1) + 17  # the last rows' offsets pass 32 bits
    far = torch.empty(stride * (m - 1) + n, device="cuda", dtype=BF16).as_strided((m, n), (stride, 1))
    got = ops.fp8_matmul(qa, sa, qb[0], sb[0], out=far)
    assert torch.equal(got.contiguous(), want.to(BF16))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 48, 700])
def test_fp8_matmul_repeats_bit_by_bit(ops, m):
    """Sums are taken in a fixed order: the same operands give the same bits."""
    qa, sa, qb, sb = _operands(ops, _gen(m), m, 520, 1024, 3)
    off = torch.tensor([0, m // 3, m // 2, m], device="cuda", dtype=torch.int32)
    first = ops.fp8_matmul(qa, sa, qb, sb, offsets=off)
    for _ in range(3):
        assert torch.equal(ops.fp8_matmul(qa, sa, qb, sb, offsets=off), first)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [4128, 4176, 4256])
@pytest.mark.parametrize("k", [16, 128, 400])
def test_fp8_matmul_pairs_whose_last_columns_are_an_odd_number_of_parts(ops, n, k):
    """fp32 tiles of CTA pairs leave 32 columns at a time from two places in shared memory in turn, and a pair takes
    several tiles: with one part or three in the last columns, the next tile begins where the last store may still read."""
    m = 8192
    qa, sa, qb, sb = _operands(ops, _gen(n + k), m, n, k, 1)
    y, s = _product64(qa, sa, qb, sb, [0, m])
    bound = _product_bound(y, s, k, F32)
    first = ops.fp8_matmul(qa, sa, qb[0], sb[0], out_dtype=F32)
    _within(first, y, bound)
    for _ in range(4):
        assert torch.equal(ops.fp8_matmul(qa, sa, qb[0], sb[0], out_dtype=F32), first)
    assert ops.status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("out,n", [(BF16, 4097), (BF16, 4100), (BF16, 4104), (F32, 4098), (F32, 4100), (F32, 4199)])
def test_fp8_matmul_pairs_leave_the_columns_behind_n_alone(ops, out, n):
    """Rows of a wider buffer that start on 16-byte boundaries and end anywhere."""
    m, k, stride = 4096, 144, 4208
    qa, sa, qb, sb = _operands(ops, _gen(n), m, n, k, 1)
    buf = torch.full((m, stride), 77.0, device="cuda", dtype=out)
    got = ops.fp8_matmul(qa, sa, qb[0], sb[0], out=buf[:, :n])
    assert bool((buf[:, n:] == 77).all())
    y, s = _product64(qa, sa, qb, sb, [0, m])
    _within(got, y, _product_bound(y, s, k, out))


# Every kernel that a product can take (epoch_fp8_matmul_kernel): kernel, groups (0: dense), m, n, k. Pairs: several tiles
# each, last pairs of which one CTA has no row, edges of N inside and outside a CTA's half, K tails, ragged and empty
# groups. From 32 groups on a lane holds several offsets.
KERNELS = [(0, 0, 13, 520, 272), (0, 33, 60, 40, 400), (0, 1024, 64, 40, 144), (32, 0, 129, 511, 272), (32, 6, 421, 272, 400),
           (64, 0, 500, 2000, 400), (128, 0, 500, 2600, 1168), (128, 0, 1000, 2000, 16), (256, 0, 800, 5000, 400),
           (256, 40, 3000, 2100, 272), (256, 200, 2000, 1500, 144), (256, 1024, 5000, 136, 48), (256, 64, 1500, 520, 1040),
           (512, 0, 8191, 4100, 272), (512, 0, 4097, 4104, 16), (512, 0, 8065, 4191, 144), (512, 0, 1290, 5000, 1168),
           (512, 0, 4500, 2300, 2064), (512, 0, 6216, 1600, 400), (512, 5, 6000, 4104, 272), (512, 3, 2500, 6001, 128),
           (512, 7, 9001, 4096, 400)]


def test_every_kernel_of_the_product_has_a_shape_below(lib):
    for kernel, e, m, n, _ in KERNELS:
        assert lib.epoch_fp8_matmul_kernel(e, m, n, 152) == kernel, (e, m, n)
    assert {c[0] for c in KERNELS} == {0, 32, 64, 128, 256, 512}
    for bad in ((-1, 4, 4, 152), (1025, 4, 4, 152), (0, -1, 4, 152), (0, 4, 0, 152), (0, 4, 4, -1)):
        assert lib.epoch_fp8_matmul_kernel(*bad) == -1
    for sms in (1, 2, 3):  # small devices have a kernel for every size too
        assert all(lib.epoch_fp8_matmul_kernel(e, m, n, sms) in (0, 32, 64, 128, 256, 512) for _, e, m, n, _ in KERNELS)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("apart", ["whole", "wide", "odd"])
@pytest.mark.parametrize("case", KERNELS, ids=str)
def test_fp8_matmul_by_every_kernel(ops, lib, case, apart, out):
    """Rows of the output that follow one another, lie apart on 32-byte boundaries (the stores of wide pieces), or start
    anywhere (single elements); columns and rows that are not the product's stay as they were."""
    kernel, e, m, n, k = case
    assert lib.epoch_fp8_matmul_kernel(e, m, n, 0) == kernel
    g = _gen(m + n + k)
    qa, sa, qb, sb = _operands(ops, g, m, n, k, max(e, 1))
    if e:  # ragged groups, some of them empty, three rows before the first and five behind the last
        cuts = torch.randint(3, m - 4, (e + 1,), generator=torch.Generator().manual_seed(m)).sort().values
        cuts[0], cuts[-1] = 3, m - 5
        cuts[e // 2] = cuts[e // 2 + 1] if e > 1 else cuts[0]
        offsets = cuts.sort().values.tolist()
        off = torch.tensor(offsets, device="cuda", dtype=torch.int32)
        args = (qa, sa, qb, sb)
    else:
        offsets, off, args = [0, m], None, (qa, sa, qb[0], sb[0])
    first, stride = {"whole": (0, n), "wide": (0, n + 16 + -n % 16), "odd": (1, n + 2 + n % 2)}[apart]
    buf = torch.full((m, stride), 77.0, device="cuda", dtype=out)
    got = ops.fp8_matmul(*args, offsets=off, out=buf[:, first:first + n])
    y, s = _product64(qa, sa, qb, sb, offsets)
    lo, hi = offsets[0], offsets[-1]
    _within(got[lo:hi], y[lo:hi], _product_bound(y, s, k, out)[lo:hi])
    assert bool((buf[:lo] == 77).all()) and bool((buf[hi:] == 77).all())
    assert bool((buf[:, :first] == 77).all()) and bool((buf[:, first + n:] == 77).all())
    again = ops.fp8_matmul(*args, offsets=off, out_dtype=out)  # rows that follow one another: other stores, the same sums
    assert torch.equal(again[lo:hi], got[lo:hi])
    assert ops.status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("case", [(32, 0, 129, 511, 272), (32, 6, 421, 272, 400), (64, 0, 500, 2000, 400), (128, 0, 500, 2600, 1168),
                                  (256, 40, 3000, 2100, 1040), (512, 0, 4500, 2300, 2064), (512, 3, 2500, 6000, 128)], ids=str)
def test_fp8_matmul_waits_that_run_out(ops, lib, case, out):
    """Operands that never come whole: the call returns after its limit, writes nothing, says so until it is asked to
    clear that, and the next product is as before."""
    kernel, e, m, n, k = case
    assert lib.epoch_fp8_matmul_kernel(e, m, n, 0) == kernel
    qa, sa, qb, sb = _operands(ops, _gen(m), m, n, k, max(e, 1))
    off = torch.arange(e + 1, device="cuda", dtype=torch.int32) * (m // e) if e else None
    args = (qa, sa, qb, sb) if e else (qa, sa, qb[0], sb[0])
    want = torch.zeros(m, n, device="cuda", dtype=out)
    ops.fp8_matmul(*args, offsets=off, out=want)
    y = torch.full((m, n), 77.0, device="cuda", dtype=out)
    raw = (qa.data_ptr(), sa.data_ptr(), qb.data_ptr(), sb.data_ptr(), off.data_ptr() if e else None, max(e, 1), m, n, k,
           y.data_ptr(), n, 1 if out == BF16 else 0)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.epoch_test_fp8_timeout(*raw, 1_000_000, stream) == 0
    assert ops.status() == (4, 2)  # EPOCH_ETIMEOUT, EPOCH_DEVERR_TIMEOUT
    assert ops.status(clear=True) == (4, 2) and ops.status() == (0, 0)
    assert bool((y == 77).all())
    got = torch.zeros(m, n, device="cuda", dtype=out)
    assert torch.equal(ops.fp8_matmul(*args, offsets=off, out=got), want) and ops.status() == (0, 0)
    assert lib.epoch_test_fp8_timeout(*raw, 999, stream) == 1  # EPOCH_EINVAL
    few = raw[:6] + (min(16, m),) + raw[7:] if not e else raw[:6] + (60,) + raw[7:]
    assert lib.epoch_test_fp8_timeout(*few, 1_000_000, stream) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("m", [20, 700])
def test_weights_whose_offsets_pass_32_bits(ops, m):
    """The last of 40 matrices of 8192 x 8192 begins behind 2^31 bytes, and its rows in bf16 behind 2^32."""
    e, n, k = 40, 8192, 8192
    g = _gen(m)
    w = torch.zeros(e, n, k, device="cuda", dtype=BF16)
    last = _rnd(g, n, k, std=k ** -0.5)
    w[-1] = last
    qb, sb = ops.fp8_quantize_weight(w)
    wq, ws = ops.fp8_quantize_weight(w[-1].contiguous())
    assert torch.equal(qb[-1].view(torch.uint8), wq.view(torch.uint8)) and torch.equal(sb[-1], ws)
    del w
    qa, sa = ops.fp8_quantize(_rnd(g, m, k))
    off = torch.zeros(e + 1, device="cuda", dtype=torch.int32)
    off[-1] = m
    got = ops.fp8_matmul(qa, sa, qb, sb, offsets=off, out_dtype=F32)
    y, s = _product64(qa, sa, wq[None], ws[None], [0, m])
    _within(got, y, _product_bound(y, s, k, F32))


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1024, 1000, 1001])
def test_fp8_quantize_rows_whose_offsets_pass_32_bits(ops, k):
    g = _gen(k)
    n, far = 3, (1 << 31) // 2 + 24
    x = _rnd(g, n, k, dtype=BF16)
    v = torch.empty(far * (n - 1) + k, device="cuda", dtype=BF16).as_strided((n, k), (far, 1))
    v.copy_(x)
    for rows in (None, torch.tensor([2, 0, 2, 1], device="cuda", dtype=torch.int32)):
        src = x if rows is None else x[rows.long()].contiguous()
        q, s = ops.fp8_quantize(v, rows=rows)
        wq, ws = ops.fp8_quantize(src)
        assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s, ws)


# ------------------------------------------------------------------------------ streams and graphs
@pytest.mark.gpu
def test_ops_on_a_stream_of_their_own_and_in_a_graph(ops):
    g = _gen(1)
    h, m = 512, 96
    x, w = _rnd(g, m, h, dtype=BF16), 1 + _rnd(g, h, std=0.1)
    wq, ws = ops.fp8_quantize_weight(_rnd(g, 300, h, std=h ** -0.5))
    ob = torch.empty(m, h, device="cuda", dtype=BF16)
    oy = torch.empty(m, 300, device="cuda", dtype=BF16)
    q, s = torch.empty(m, h, device="cuda", dtype=E4M3), torch.empty(m, 4, device="cuda")

    def step(stream=None):
        ops.norm_before(x, w, out=ob, stream=stream)
        ops.fp8_quantize(ob, q=q, scales=s, stream=stream)
        ops.fp8_matmul(q, s, wq, ws, out=oy, stream=stream)

    step()
    want = oy.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    oy.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    fresh = ops.norm_before(x, w, stream=side)
    side.synchronize()
    assert torch.equal(oy, want) and torch.equal(fresh, ob)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x2 = _rnd(g, m, h, dtype=BF16)
    for src in (x2, x.clone()):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        replayed = oy.clone()
        step()
        assert torch.equal(replayed, oy)
    assert torch.equal(oy, want)


FIRST_CALL = """
import sys
sys.path.insert(0, {root!r})
import torch
from sparse_moe_layer_gate_gb300 import ops
from sparse_moe_layer_gate_gb300.layer import EpochLayer
m, n, k = {m}, 320, 512
a = torch.randn(m, k, device="cuda", dtype=torch.bfloat16)
w = torch.ones(k, device="cuda")
qb = torch.randn(n, k, device="cuda").to(torch.float8_e4m3fn)
sb = torch.ones(3, 4, device="cuda")
d = dict(device="cuda", dtype=torch.bfloat16)
lay = EpochLayer(hidden=k, n_experts=8, inter=128, top_k=2, max_positions=16, dtype="bf16", tau=1.0, refresh_R=4,
                 weights=dict(w_router=torch.randn(8, k, **d), b_router=torch.zeros(8, device="cuda"),
                              w_gate=torch.randn(8, 128, k, **d) / 22, w_up=torch.randn(8, 128, k, **d) / 22,
                              w_down=torch.randn(8, k, 128, **d) / 11))
x = torch.randn(3, k, **d)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    h = ops.norm_before(a, w)
    q, s = ops.fp8_quantize(h)
    y = ops.fp8_matmul(q, s, qb, sb)
    f = lay.forward_few(x)
g.replay()
torch.cuda.synchronize()
h2 = ops.norm_before(a, w)
assert torch.equal(h, h2) and torch.equal(y, ops.fp8_matmul(*ops.fp8_quantize(h2), qb, sb))
assert torch.equal(f, lay.forward_few(x)) and ops.status() == (0, 0) and lay.status() == (0, 0)
print("same")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("m", [5, 100, 600])
def test_a_process_whose_first_calls_are_captured(ops, m):
    """Whatever a call sets up once per process it can set up under capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=root, m=m)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.gpu
def test_two_products_at_once(ops):
    """Calls on two streams share nothing."""
    g = _gen(9)
    sets = [_operands(ops, g, m, 512, 1024, 1) for m in (256, 40)]
    want = [ops.fp8_matmul(a, sa, b[0], sb[0]) for a, sa, b, sb in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, (a, sa, b, sb) in enumerate(sets):
            got[i].append(ops.fp8_matmul(a, sa, b[0], sb[0], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


# ---------------------------------------------------------------------------------------- refusals
P = 1 << 20  # a pointer that is never followed: every call below is refused on the host, or has no rows


@pytest.fixture(scope="module")
def lib(ops):
    from sparse_moe_layer_gate_gb300 import binding
    return binding.lib()


BEFORE = dict(x=P, x_stride=64, x_dtype=1, weight=P, par=0, n=4, h=64, eps=1e-6, out=P, out_stride=64, out_dtype=1, stream=None)
AFTER = dict(block=P, res=P, weight=P, gate=0, scale=0, nw=0, out=P, nout=0, block_stride=64, res_stride=64, gate_stride=0,
             out_stride=64, nstride=0, n=4, h=64, dtype=1, res_dtype=0, par=0, kind=0, sig=0, number=1.0, eps=1e-6)
QUANT = dict(x=P, x_stride=256, dtype=1, rows=None, n=4, src=4, cols=256, swiglu=0, q=P, s=P, stream=None)
WEIGHT = dict(w=P, dtype=1, mats=1, n=128, k=128, q=P, s=P, stream=None)
MATMUL = dict(a=P, sa=P, b=P, sb=P, offsets=None, groups=1, m=4, n=64, k=128, y=P, stride=64, out=1, stream=None)


def _refusals():
    f = math.inf
    for kw in (dict(n=-1), dict(h=0), dict(h=(1 << 20) + 1), dict(x_dtype=2), dict(par=-1), dict(out_dtype=5),
               dict(eps=-1.0), dict(eps=f), dict(eps=math.nan), dict(x=None), dict(weight=None), dict(out=None),
               dict(x=P + 1), dict(weight=P + 2), dict(x_stride=63), dict(out_stride=0)):
        yield "epoch_norm_before", BEFORE, kw
    for kw in (dict(n=-1), dict(h=0), dict(dtype=3), dict(res_dtype=3), dict(par=3), dict(kind=3), dict(kind=-1),
               dict(kind=1), dict(kind=2), dict(kind=2, gate=P, gate_stride=63), dict(block=0), dict(res=0),
               dict(out=0), dict(nw=P), dict(nout=P, nstride=64), dict(nw=P, nout=P, nstride=1),
               dict(block_stride=1), dict(res_stride=1), dict(out_stride=1), dict(res=P + 2), dict(eps=math.nan),
               dict(scale=P + 1), dict(nw=P + 1, nout=P, nstride=64)):
        yield "epoch_norm_after", AFTER, kw
    for kw in (dict(n=-1, src=-1), dict(src=3), dict(cols=0), dict(dtype=7), dict(x=None), dict(x=P + 1), dict(q=None),
               dict(s=None), dict(s=P + 2), dict(x_stride=255), dict(swiglu=1), dict(rows=P + 2),
               dict(n=1 << 30, src=1 << 30, cols=512)):
        yield "epoch_fp8_quantize", QUANT, kw
    for kw in (dict(dtype=2), dict(mats=-1), dict(mats=65536), dict(n=0), dict(k=0), dict(n=(1 << 22) + 1), dict(w=None),
               dict(q=None), dict(s=None), dict(w=P + 1)):
        yield "epoch_fp8_quantize_weight", WEIGHT, kw
    for kw in (dict(m=-1), dict(n=0), dict(k=0), dict(k=8), dict(k=136), dict(k=(1 << 30) + 16), dict(groups=0), dict(groups=2),
               dict(groups=1025, offsets=P), dict(offsets=P + 2), dict(groups=1024, offsets=P, n=1 << 22), dict(a=None),
               dict(a=P + 8), dict(b=P + 4), dict(b=None), dict(sa=None), dict(sb=P + 2), dict(y=None), dict(y=P + 1),
               dict(stride=63), dict(out=2)):
        yield "epoch_fp8_matmul", MATMUL, kw


@pytest.mark.parametrize("name,base,change", list(_refusals()), ids=lambda v: str(v)[:60] if not isinstance(v, dict) else "")
def test_refused_on_the_host(lib, name, base, change):
    assert set(change) <= set(base)
    assert _call(lib, name, {**base, **change}) == 1  # EPOCH_EINVAL, nothing enqueued


POINTERS = {"x", "weight", "out", "block", "res", "gate", "scale", "nw", "nout", "rows", "q", "s", "w", "a", "sa", "b", "sb",
            "offsets", "y"}


def _apart(base):
    """The arguments with every pointer in a place of its own."""
    return {name: (P * (16 + 16 * i) if v == P else v) for i, (name, v) in enumerate(base.items())}


@pytest.mark.parametrize("name,base,change", list(_refusals()), ids=lambda v: str(v)[:60] if not isinstance(v, dict) else "")
def test_refused_on_the_host_without_any_overlap(lib, name, base, change):
    """The same refusals, each for its own reason: no two pointers are one."""
    own = {k: P * 1024 + v if k in POINTERS and v is not None and v >= P else v for k, v in change.items()}
    assert _call(lib, name, {**_apart(base), **own}) == 1


def _overlaps():
    b = _apart(BEFORE)
    x, w = b["x"], b["weight"]
    for kw in (dict(out=x + 2), dict(out=x - 2), dict(out=x + 128), dict(out=x + 3 * 128 + 126), dict(out=x - 3 * 128),
               dict(out=x, out_dtype=0), dict(out=x, out_stride=65), dict(out=x + 64, out_stride=64), dict(out=w + 4 * 63),
               dict(out=w - 3 * 128), dict(x_stride=96, out_stride=96, out=x + 2 * 32 + 62), dict(x_stride=96, out_stride=96, out=x - 2),
               dict(x_stride=640, out_stride=320, out=x + 640 * 2 * 3 - 640 - 126), dict(n=1, x_stride=0, out_stride=0, out=x + 126)):
        yield "epoch_norm_before", b, kw
    b = {**_apart(AFTER), "nstride": 64}
    blk, res, w, out = b["block"], b["res"], b["weight"], b["out"]
    far = P * 4096
    for kw in (dict(out=blk), dict(out=res + 4), dict(out=res, out_stride=66), dict(out=w + 252), dict(nw=far, nout=out),
               dict(nw=far, nout=out + 4 * 64 * 3), dict(nw=far, nout=res), dict(nw=far, nout=blk + 128), dict(nw=far, nout=far + 4),
               dict(kind=1, gate=out + 4), dict(kind=2, gate=out, gate_stride=64), dict(scale=out), dict(nw=far, nout=w)):
        yield "epoch_norm_after", b, kw
    b = _apart(QUANT)
    x, q, s = b["x"], b["q"], b["s"]
    for kw in (dict(q=x), dict(q=x + 4 * 512 - 1), dict(s=x + 4), dict(s=q), dict(s=q + 4 * 255), dict(rows=q + 4), dict(rows=s + 4 * 7),
               dict(swiglu=1, x_stride=512, q=x + 4 * 1024 - 1), dict(q=x + 512, x_stride=512)):
        yield "epoch_fp8_quantize", b, kw
    b = _apart(WEIGHT)
    for kw in (dict(q=b["w"]), dict(q=b["w"] + 2 * 128 * 128 - 1), dict(s=b["w"] + 4), dict(s=b["q"] + 4)):
        yield "epoch_fp8_quantize_weight", b, kw
    b = _apart(MATMUL)
    for kw in (dict(y=b["a"] + 2), dict(y=b["a"] + 4 * 128 - 2), dict(y=b["b"] + 64 * 128 - 2), dict(y=b["sa"]), dict(y=b["sb"]),
               dict(y=b["a"] - 4 * 128 + 2), dict(offsets=b["y"] + 4)):
        yield "epoch_fp8_matmul", b, kw


@pytest.mark.parametrize("name,base,change", list(_overlaps()), ids=lambda v: str(v)[:60] if not isinstance(v, dict) else "")
def test_outputs_that_overlap_are_refused(lib, name, base, change):
    assert set(change) <= set(base)
    assert _call(lib, name, {**base, **change}) == 1  # EPOCH_EINVAL, nothing enqueued


@pytest.mark.gpu
def test_rows_in_turn_and_columns_side_by_side_do_not_overlap(ops):
    g = _gen(21)
    n, h = 12, 64
    w = 1 + _rnd(g, h, std=0.1)
    x = _rnd(g, n, h)
    # rows that start off a 16-byte boundary add their squares in another order: the formula's bound, not equal bits
    want = _rms64(x.double(), w.double(), 1e-6)[1]
    bound = want.abs() * _norm_units(h) * U + 1e-30
    for layout in (lambda b: (b[:n, :h], b[:n, h:2 * h]), lambda b: (b[:n, 1:h + 1], b[:n, h + 1:2 * h + 1]),
                   lambda b: (b[0:2 * n:2, :h], b[1:2 * n:2, :h]), lambda b: (b[0:4 * n:4, :h], b[1:2 * n:2, :h]),
                   lambda b: (b[1:2 * n:2, 9:h + 9], b[0:4 * n:4, 9:h + 9]), lambda b: (b[n:2 * n, :h], b[:n, :h])):
        buf = torch.full((4 * n, 3 * h), 5.0, device="cuda")
        src, dst = layout(buf)
        src.copy_(x)
        assert ops.norm_before(src, w, out=dst) is dst
        assert torch.equal(src, x)
        _within(dst, want, bound)
        assert int((buf != 5).sum()) == 2 * n * h


@pytest.mark.gpu
@pytest.mark.parametrize("n,h", [(3, 64), (3, 1001), (700, 4632), (2, 17001)])
def test_norm_after_into_any_row_input(ops, n, h):
    g = _gen(22)
    w, nw = 1 + _rnd(g, h, std=0.1), 1 + _rnd(g, h, std=0.1)
    rows = [_rnd(g, n, h) for _ in range(3)]  # block, residual, gate

    def call(t, out=None, next_out=None):
        return ops.norm_after(t[0], t[1], w, gate=t[2], gate_sigmoid=True, next_weight=nw, out=out, next_out=next_out)

    want = call(rows)
    for i in range(3):
        for j in range(3):
            if i == j:
                continue
            t = [r.clone() for r in rows]
            got = call(t, t[i], t[j])
            assert got[0] is t[i] and got[1] is t[j]
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert torch.equal(t[3 - i - j], rows[3 - i - j])


def _call(lib, name, args):
    if name == "epoch_norm_after":  # takes a struct
        from sparse_moe_layer_gate_gb300 import binding
        return lib.epoch_norm_after(binding.NORM_AFTER_ARGS.pack(*args.values()), None)
    return getattr(lib, name)(*args.values())


def test_norm_after_without_arguments(lib):
    assert lib.epoch_norm_after(None, None) == 1


def test_no_rows_enqueue_nothing(lib):
    for name, base, kw in (("epoch_norm_before", BEFORE, dict(n=0, x=None, out=None)),
                           ("epoch_norm_after", AFTER, dict(n=0, block=0, res=0, out=0)),
                           ("epoch_fp8_quantize", QUANT, dict(n=0, src=0, x=None, q=None, s=None)),
                           ("epoch_fp8_quantize_weight", WEIGHT, dict(mats=0, w=None)),
                           ("epoch_fp8_matmul", MATMUL, dict(m=0, a=None, y=None))):
        assert _call(lib, name, {**base, **kw}) == 0


def test_cpu_tensors_are_refused(ops):
    x = torch.zeros(2, 64)
    for call in (lambda: ops.norm_before(x, x[0]), lambda: ops.norm_after(x, x, x[0]), lambda: ops.fp8_quantize(x),
                 lambda: ops.fp8_quantize_weight(x), lambda: ops.fp8_matmul(x.to(E4M3), x, x.to(E4M3), x)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_tensors_are_checked(ops):
    c = dict(device="cuda")
    x, w = torch.zeros(4, 64, **c), torch.zeros(64, **c)
    q, s = ops.fp8_quantize(torch.zeros(4, 128, **c))
    b, sb = ops.fp8_quantize_weight(torch.zeros(64, 128, **c))
    off = torch.zeros(3, dtype=torch.int32, **c)
    for call in (lambda: ops.norm_before(x.half(), w), lambda: ops.norm_before(x, w[:63]), lambda: ops.norm_before(x, w.cpu()),
                 lambda: ops.norm_before(x.T, w[:4]), lambda: ops.norm_before(x, w, out=x[:3]),
                 lambda: ops.norm_before(x[0].expand(4, 64), w), lambda: ops.norm_before(x, w, eps=-1.0),
                 lambda: ops.norm_before(x, w, out=x, out_dtype=BF16), lambda: ops.norm_after(x, x[:3], w),
                 lambda: ops.norm_after(x, x, w, gate=x.to(BF16)), lambda: ops.norm_after(x, x, w, gate_sigmoid=True),
                 lambda: ops.norm_after(x, x, w, next_weight=w.to(BF16)), lambda: ops.norm_after(x, x, w, next_out=x),
                 lambda: ops.norm_after(x, x, w, out=x.to(BF16)), lambda: ops.fp8_quantize(x[:, :63], swiglu=True),
                 lambda: ops.fp8_quantize(x, rows=torch.zeros(2, dtype=torch.int64, **c)),
                 lambda: ops.fp8_quantize(x, q=torch.zeros(4, 64, **c)), lambda: ops.fp8_quantize_weight(x.T),
                 lambda: ops.fp8_matmul(q, s, b[:, :64], sb), lambda: ops.fp8_matmul(q, s[:, :0], b, sb),
                 lambda: ops.fp8_matmul(q, s, b[None], sb[None], offsets=off), lambda: ops.fp8_matmul(q, s, b, sb, offsets=off),
                 lambda: ops.fp8_matmul(q, s, b, sb, out_dtype=torch.float16)):
        with pytest.raises((ValueError, RuntimeError)):
            call()


@pytest.mark.gpu
def test_more_rows_than_the_abi_counts_are_refused(ops):
    n, c = 2 ** 31, dict(device="cuda")
    one, far = torch.ones(1, **c), torch.empty(n, 1, dtype=BF16, **c)
    for call in (lambda: ops.norm_before(far, one), lambda: ops.norm_after(far, far, one, out=far),
                 lambda: ops.fp8_quantize(far.view(1, n)), lambda: ops.fp8_quantize_weight(far)):
        with pytest.raises(ValueError):
            call()
