"""Edges of the experts' operators that their own sizes pass over, against forms in 64 bits."""
import math

import numpy as np
import pytest
import torch

from test_experts import BF16, E4M3, F32, F64, FORMS, GRID, I32, U, U8, _gen, _half, _rnd, _within, check_codes, check_route, ops, route64  # noqa: F401


# ------------------------------------------------------------------------------------------- router
@pytest.mark.gpu
@pytest.mark.parametrize("E,groups,top", [(64, 4, 2), (256, 8, 4), (512, 16, 3), (96, 6, 2), (144, 8, 3)])
@pytest.mark.parametrize("size", [32.0, 100.0, 1e4])
def test_route_groups_whose_biases_cancel(ops, E, groups, top, size):
    """A group's two best have biases of +-size, so its score is near 1 and each of its terms is rounded to fp32 at `size`:
    the order of groups a few 1e-7 apart is that of 64 bits. Without an eligible mask and with one that leaves groups
    uneven (more of them are then searched, best first)."""
    g = _gen(E + int(size))
    T, k, n = 400, 8, E // groups
    x = _rnd(g, T, E)
    best = 0.3 + 0.5 * torch.rand(T, 1, 2, generator=g, device="cuda")
    far = int(40 + size)  # steps of 6e-8
    steps = torch.randint(-far, far + 1, (T, groups, 2), generator=g, device="cuda", dtype=I32)
    x.view(T, groups, n)[:, :, [1, n - 1]] = (best.expand(T, groups, 2).contiguous().view(torch.int32) + steps).view(F32)
    bias = torch.full((groups, n), -2 * size, device="cuda")
    bias[:, 1], bias[:, n - 1] = size, -size
    bias = bias.flatten()
    some = torch.rand(E, generator=g, device="cuda") < 0.6
    some.view(groups, n)[:, [1, n - 1]] = True
    for eligible, kk in ((None, k), (some, min(16, E))):
        for tops in {top, 1}:
            kw = dict(bias=bias, n_group=groups, topk_group=tops, eligible=eligible)
            check_route(ops.route(x, kk, router="sigmoid_group", **kw), route64(x, kk, True, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [12, 300])
def test_route_sigmoids_below_the_range(ops, T):
    """Selected logits so low that their sigmoids are subnormal or nothing in fp32: the weights, their quotients, are not.
    Both where every logit is low and where a mask leaves only such experts."""
    E, k = 48, 6
    g = _gen(T)
    x = _rnd(g, T, E)
    low = torch.tensor([-16.5, -17.5, -30.0, -80.0, -87.0, -88.5, -89.0, -95.0, -103.0, -110.0, -200.0, -600.0], device="cuda")
    x[:, ::3] += low[torch.arange(T, device="cuda") % 12][:, None]
    only = torch.zeros(E, dtype=torch.bool, device="cuda")
    only[::3] = True
    y = x.clone()
    y[:, 1::3] = y[:, 2::3] = -700.0
    y[::5, 0] = -16.0   # and an ordinary one among them
    y[1::5, 3] = 2.0
    for logits, eligible in ((x, only), (y, None), (y, only), (x.to(BF16), only)):
        for groups, top in ((1, 1), (4, 2)):
            for raw in (False, True):
                kw = dict(n_group=groups, topk_group=top, eligible=eligible)
                want = route64(logits, k, True, raw=raw, **kw)
                assert np.isfinite(want[1]).all()
                check_route(ops.route(logits, k, router="sigmoid_group", raw_weights=raw, **kw), want)


# ------------------------------------------------------------------------------------ 4-bit quantiser
def _borders(s):
    """Rows [scales, 32] of two blocks whose scale is s: every border between two codes times s, and a step to both sides."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    at = (s.unsqueeze(1) * mids).unsqueeze(2).view(torch.int32) + torch.tensor([-1, 0, 1], device="cuda", dtype=I32)
    at = at.view(F32).reshape(-1, 21)
    x = torch.zeros(s.numel(), 32, device="cuda")
    x[:, :11], x[:, 16:26] = at[:, :11], at[:, 11:]
    x[:, 15] = x[:, 31] = 6 * s
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 200])  # rows of every scale: few blocks, and many
def test_fp4_quotients_on_both_sides_of_every_border(ops, n):
    s = torch.arange(1, 127, device="cuda", dtype=U8).view(E4M3).float()
    x = _borders(s).repeat(n, 1)
    for y in (x, -x, torch.where(torch.arange(32, device="cuda") % 2 == 0, x, -x)):
        q, sc = ops.fp4_quantize(y)
        assert torch.equal(sc.view(U8)[0, :, :2], torch.arange(1, 127, device="cuda", dtype=U8).repeat(n)[:, None].expand(-1, 2))
        check_codes(q, sc, y, "nvfp4")
        q, sc = ops.fp4_quantize(y, tensor_scale=0.25)
        check_codes(q, sc, y, "nvfp4", 0.25)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("n", [5, 3000])
def test_fp4_quantize_by_any_tensor_scale(ops, dt, n):
    """v' = v * (1 / tensor_scale), each rounded to fp32; the codes are those of v'."""
    x = _rnd(_gen(n), n, 288, std=3.0, dtype=dt)
    for t in (0.3, 1.7, 1e-5, 12345.0):
        v = x.float() * (torch.ones((), device="cuda") / torch.tensor(t, device="cuda"))
        q, s = ops.fp4_quantize(x, tensor_scale=t)
        check_codes(q, s, v, "nvfp4")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("n", [2, 3000])
@pytest.mark.parametrize("t", [2.0 ** -20, 2.0 ** -110, 3e-7])
def test_fp4_quantize_beyond_the_largest_quotient(ops, dt, n, t):
    """Finite values whose quotient by the tensor scale is beyond fp32's range saturate, as those beyond e4m3's do; only a
    NaN or an infinity of x makes a block NaN."""
    x = torch.zeros(n, 64, device="cuda")
    x[:, :8] = torch.tensor([3e38, -3e38, 1e37, -1e30, 2e33, 1.0, -1e-30, 0.0], device="cuda")
    x[:, 16:20] = torch.tensor([-3.3e38, 3.3e38, 0.0, 1e38], device="cuda")
    x[:, 33] = math.inf
    x[:, 50] = math.nan
    x = x.to(dt)
    q, s = ops.fp4_quantize(x, tensor_scale=t)
    byte = s.view(U8)[0, :, :4]
    assert torch.equal(byte, torch.tensor([0x7E, 0x7E, 0x7F, 0x7F], device="cuda", dtype=U8).expand(n, -1))
    fine = x[:, :32].contiguous()
    q, s = ops.fp4_quantize(fine, tensor_scale=t)
    check_codes(q, s, fine, "nvfp4", t)
    # silu(30) is 30 in fp32, and so the product with u is what is quantised
    both = torch.cat([torch.full_like(fine, 30.0), fine / 32], 1)
    q, s = ops.fp4_quantize(both, tensor_scale=t, swiglu=True)
    check_codes(q, s, fine.float() / 32 * 30, "nvfp4", t)


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("n", [3, 3000])
@pytest.mark.parametrize("ot", [F32, BF16])
def test_fp4_dequantize_by_any_factor(ops, form, n, ot):
    """Every code with every finite scale, times factors that are no powers of two and such as meet the ends of fp32's
    range: the bits of the exact product (q * s has six bits and a factor 24, so 64 bits hold it) rounded to fp32 and from
    there to the result; a zero stays zero."""
    block, dtype = FORMS[form]
    g = _gen(n)
    top = 127 if form == "nvfp4" else 255
    code = (torch.arange(256, device="cuda") + torch.arange(n, device="cuda")[:, None]) % 16
    byte = torch.randint(0, top, (n, 256 // block), generator=g, device="cuda").to(U8)
    byte[0, 0], byte[0, 1], byte[1, 0] = top - 1, 0, top - 2
    q = (code[:, 0::2] | code[:, 1::2] << 4).to(U8)
    s = byte.view(1, n, -1).view(dtype)
    wide = byte.view(E4M3).double() if form == "nvfp4" else torch.exp2(byte.double() - 127)
    v = torch.tensor(GRID + [-x for x in GRID], device="cuda", dtype=F64)[code] * wide.repeat_interleave(block, 1)
    for f in (0.1, 1 / 3, -1.1, 0.875, 2.0, 8.0, 1e5, 1e30, 1e36, 3e38, 1e-5, 1e-30, 1e-40, 0.0):
        f32 = torch.tensor([f], device="cuda")
        want = (v * f32.double()).float().to(ot)
        for factor in (f, f32):
            got = ops.fp4_dequantize(q, s, tensor_scale=factor, out_dtype=ot)
            assert got.dtype == ot and torch.equal(got, want) and torch.equal(torch.signbit(got), torch.signbit(want)), f


# ---------------------------------------------------------------------------------- products of long K
@pytest.mark.gpu
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("m", [16, 17, 300, 1100])
def test_fp4_matmul_sums_of_many_columns(ops, form, m):
    """fp32 results over K = 65536 columns of one sign, where sums that truncate drift: an accumulator of the tensor core
    holds 32 products at most, each off by at most a step (two roundings) of what it holds, and K / 2048 of them are
    summed in fp32. With few rows and with tiles alike."""
    k, n = 65536, 512
    g = _gen(m)
    a, sa = ops.fp4_quantize(_rnd(g, m, k).abs(), form=form)
    b, sb, t = ops.fp4_quantize_weight(_rnd(g, n, k).abs(), form=form)
    y = ops.fp4_dequantize(a, sa, out_dtype=F32).double() @ ops.fp4_dequantize(b, sb, out_dtype=F32).double().T
    got = ops.fp4_matmul(a, sa, b, sb, out_dtype=F32)
    _within(got, y, y * (2 * 32 + k / 2048 + 4) * U)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(512, 256), (17, 5120), (3000, 512)])
@pytest.mark.parametrize("gather", [False, True])
def test_bf16_results_of_many_columns_do_not_drift(ops, m, n, gather):
    """bf16 results over K = 65536 columns of one sign: accumulators of 256 products at most, a step each, so that beside the
    result's own rounding, which averages out, the sums stay within 512 roundings of fp32 and those of K / 4096 fp32 sums."""
    k = 65536
    g = _gen(m)
    x, w = _rnd(g, m, k).abs().to(BF16), _rnd(g, n, k).abs().to(BF16)
    rows = torch.arange(m, device="cuda", dtype=I32).flip(0).contiguous() if gather else None
    y = x.double() @ w.double().T
    y = y.flip(0) if gather else y
    got = ops.grouped_matmul(x, w, None, rows=rows)
    off = (got.double() - y) / y
    drift = (512 + k / 4096 + 4) * U
    assert float(off.abs().max()) <= _half(BF16) * (1 + 2 ** -7) + drift
    # the mean of m n roundings, each spread over +-2^-8 at most: five standard deviations
    assert abs(float(off.mean())) <= drift + 5 * _half(BF16) / math.sqrt(3 * m * n)
