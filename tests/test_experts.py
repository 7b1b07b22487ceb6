"""A layer's experts by themselves: the router, products grouped by expert on fp32, bf16 and
4-bit operands, the 4-bit quantiser and the sum of a position's edges, each against its
formula in 64 bits, and their refusals.

Tolerances count roundings: U is half a step of fp32 (2^-24), _half(t) half a step of the
result's type. They are derived at each test."""
import math

import numpy as np
import pytest
import torch

BF16, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
U = 2.0 ** -24
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
FORMS = {"nvfp4": (16, E4M3), "mxfp4": (32, E8M0)}


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


def _within(got, want, bound, what=""):
    d = (got.double() - want).abs()
    over = ~(d <= bound)
    assert not bool(over.any()), (what, int(over.sum()), float((d / bound.clamp(min=1e-300)).max()))


# -------------------------------------------------------------------------------------------- route
def route64(logits, k, sigmoid=False, bias=None, n_group=1, topk_group=1, raw=False, live=None, eligible=None):
    """(sel, weights, positions, offsets, slots) by the definition, one position at a time, in 64 bits."""
    g = logits.double().cpu().numpy()
    T, E = g.shape
    b = np.zeros(E) if bias is None else bias.double().cpu().numpy()
    can = np.ones(E, bool) if eligible is None else eligible.cpu().numpy().astype(bool)
    on = np.ones(T, bool) if live is None else live.cpu().numpy().astype(bool)
    sel, w, slots = np.full((T, k), -1), np.zeros((T, k)), np.full((T, k), -1)
    for t in np.nonzero(on)[0]:
        nan = np.isnan(g[t])
        with np.errstate(over="ignore"):
            score = 1 / (1 + np.exp(-g[t])) if sigmoid else g[t]
        pick = np.where(nan, -np.inf, score + b if sigmoid else score)
        open_ = [e for e in range(E) if can[e] and not g[t, e] == -np.inf]
        if sigmoid and topk_group < n_group:
            size, best = E // n_group, []
            for i in range(n_group):
                mine = sorted((pick[e] for e in open_ if e // size == i), reverse=True)
                if mine:
                    best.append((-sum(mine[:2]), i, len(mine)))
            held, groups = 0, set()
            for rank, (_, i, n) in enumerate(sorted(best)):
                if rank < topk_group or held < k:
                    groups.add(i)
                held += n
            open_ = [e for e in open_ if e // size in groups]
        order = sorted(open_, key=lambda e: (-pick[e], e))[:k]
        sel[t, :len(order)] = order
        with np.errstate(invalid="ignore", over="ignore"):
            if sigmoid:
                v = score[order]
                total = 1.0 if raw else v.sum()
            else:
                top = np.nanmax(g[t]) if raw else (g[t, order[0]] if order else 0.0)
                v = np.exp(g[t, order] - top)
                total = np.exp(g[t] - top).sum() if raw else v.sum()
            w[t, :len(order)] = np.nan if nan.any() else v / total
    edges = sorted((sel[t, j], t, j) for t in range(T) for j in range(k) if sel[t, j] >= 0)
    positions = np.full(T * k, -1)
    for i, (_, t, j) in enumerate(edges):
        positions[i], slots[t, j] = t, i
    offsets = np.searchsorted([e for e, _, _ in edges], np.arange(E + 1))
    return sel, w, positions, offsets, slots


def check_route(r, want, what=""):
    for got, x, name in ((r.sel, want[0], "sel"), (r.offsets, want[3], "offsets"), (r.positions, want[2], "positions"), (r.slots, want[4], "slots")):
        assert got.dtype == I32 and np.array_equal(got.cpu().numpy(), x), (name, what)
    # exp and sigmoid 4 roundings of 2^-23, up to 1024 terms summed as 32 and 5 levels of them, a quotient
    w, x = r.weights.double().cpu().numpy(), want[1]
    nan = np.isnan(x)
    assert r.weights.dtype == F32 and np.array_equal(np.isnan(w), nan), what
    assert (np.abs(w - x)[~nan] <= x[~nan] * (2 * 8 + 40) * U + 1e-37).all(), what


ROUTE_SIZES = [(1, 256, 8), (1, 1, 1), (2, 2, 2), (5, 37, 3), (31, 64, 4), (32, 65, 8), (33, 256, 8), (64, 256, 16), (65, 8, 8),
               (127, 128, 1), (128, 257, 7), (129, 256, 8), (1000, 64, 6), (700, 1024, 16), (5000, 48, 2),
               (19457, 16, 3), (45000, 33, 4), (300, 512, 8), (40, 400, 16), (500, 100, 5)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", ROUTE_SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("raw", [False, True])
def test_route_softmax(ops, T, E, k, dtype, raw):
    x = _rnd(_gen(T + E), T, E, std=2.0, dtype=dtype)  # bf16: many equal logits
    check_route(ops.route(x, k, raw_weights=raw), route64(x, k, raw=raw))


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,groups,top", [(1, 256, 8, 8, 4), (1, 4, 4, 4, 1), (7, 24, 5, 6, 2), (90, 512, 8, 16, 4), (90, 128, 8, 8, 3), (64, 320, 9, 5, 2), (33, 256, 8, 1, 1), (130, 64, 16, 32, 3),
                                              (200, 1024, 8, 32, 4), (1500, 256, 8, 8, 4), (300, 512, 16, 16, 1), (40, 30, 16, 2, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("form", ["bias", "no_bias", "raw", "masks"])
def test_route_sigmoid_groups(ops, T, E, k, groups, top, dtype, form):
    g = _gen(T * 31 + E)
    x = _rnd(g, T, E, dtype=dtype)
    kw = dict(n_group=groups, topk_group=top, bias=None if form == "no_bias" else _rnd(g, E, std=0.1), raw=form == "raw")
    if form == "masks":
        kw |= dict(live=torch.rand(T, generator=g, device="cuda") < 0.7, eligible=torch.rand(E, generator=g, device="cuda") < 0.4)
    want = route64(x, k, True, **kw)
    kw["raw_weights"] = kw.pop("raw")
    check_route(ops.route(x, k, router="sigmoid_group", **kw), want)


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups", [(64, 1), (256, 8), (300, 1), (128, 4), (512, 8)])
def test_route_scores_that_fp32_cannot_tell_apart(ops, E, groups):
    """Logits a step or two apart, where sigmoid + bias round to the same fp32 value or to the wrong order: the order
    is that of exact arithmetic."""
    g = _gen(E)
    T, k = 200, 8
    base = torch.rand(T, 1, generator=g, device="cuda") * 6
    steps = torch.randint(0, 5, (T, E), generator=g, device="cuda")
    x = (base.view(torch.int32) + steps.to(I32)).view(F32)
    bias = torch.zeros(E, device="cuda")
    bias[::3] = 2.0 ** -26
    for b in (None, bias):
        for top in {1, max(1, groups // 2)}:
            check_route(ops.route(x, k, router="sigmoid_group", bias=b, n_group=groups, topk_group=top),
                        route64(x, k, True, bias=b, n_group=groups, topk_group=top))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 129, 2000])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_masks_and_values(ops, T, sigmoid):
    g = _gen(T)
    E, k = 40, 6
    kw = dict(router="sigmoid_group") if sigmoid else {}
    x = _rnd(g, T, E)
    low = torch.finfo(F32).min
    x[0] = 0.0                       # all equal: the lowest ids
    x[1, 3:] = -math.inf             # fewer than k left
    x[2] = -math.inf                 # none left
    if T > 3:
        x[3] = low                   # the type's lowest value is a number
        x[4, 5:] = low
        x[5, ::2] = -0.0             # equals 0
        x[5, 1::2] = 0.0
        x[6, 7] = math.nan           # spoils its weights, ranks last
        x[7] = math.nan
        x[8, 2] = 80.0
        x[9] = 40.0 + torch.arange(E, device="cuda") / 64  # sigmoids of 1
        x[10, 1:] = -200.0           # sigmoids of 0 in fp32 and not in 64 bits
    check_route(ops.route(x, k, **kw), route64(x, k, sigmoid))
    live = torch.zeros(T, dtype=U8, device="cuda")
    r = ops.route(x, k, live=live, **kw)  # no position at all
    assert bool((r.sel == -1).all()) and bool((r.slots == -1).all()) and bool((r.weights == 0).all())
    assert bool((r.positions == -1).all()) and bool((r.offsets == 0).all())
    live[T // 2] = 7
    some = torch.zeros(E, dtype=U8, device="cuda")
    some[[3, 11, 39]] = 1
    check_route(ops.route(x, k, live=live, eligible=some, **kw), route64(x, k, sigmoid, live=live, eligible=some))
    none = ops.route(x, k, eligible=torch.zeros(E, dtype=torch.bool, device="cuda"), **kw)
    assert bool((none.sel == -1).all()) and int(none.offsets[-1]) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_strides_reuse_and_no_positions(ops, dtype):
    g = _gen(4)
    T, E, k = 300, 64, 4
    for pad, first in ((0, 0), (8, 0), (5, 3)):
        wide = _rnd(g, T, E + pad, dtype=dtype)
        x = wide[:, first:first + E]
        want = route64(x, k)
        r = ops.route(x, k)
        check_route(r, want)
        again = ops.Routing(*(torch.full_like(t, 77) for t in r))
        assert ops.route(x, k, out=again) is again
        check_route(again, want)
    r = ops.route(torch.empty(0, E, device="cuda", dtype=dtype), k)
    assert r.sel.shape == (0, k) and r.positions.shape == (0,) and bool((r.offsets == 0).all())


@pytest.mark.gpu
def test_route_of_many_positions(ops):
    """Several passes of every CTA; against torch's sort, which is stable on equal logits."""
    T, E, k = 60000, 256, 8
    x = _rnd(_gen(1), T, E, dtype=BF16)
    live = torch.rand(T, generator=_gen(2), device="cuda") < 0.9
    r = ops.route(x, k, live=live)
    place = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k]
    sel = torch.where(live.unsqueeze(1), place, -1)
    assert torch.equal(r.sel.long(), sel)
    key, order = torch.sort(torch.where(sel < 0, E, sel).reshape(-1), stable=True)
    n = int((key < E).sum())
    assert torch.equal(r.positions[:n].long(), (order // k)[:n]) and bool((r.positions[n:] == -1).all())
    assert torch.equal(r.offsets.long(), torch.searchsorted(key, torch.arange(E + 1, device="cuda")))
    on = sel.reshape(-1) >= 0
    slots = r.slots.reshape(-1)
    assert bool((slots[~on] == -1).all()) and torch.equal(slots[order[:n]].long(), torch.arange(n, device="cuda"))
    w = torch.softmax(x.double().gather(1, place), 1)
    _within(r.weights, torch.where(live.unsqueeze(1), w, 0.0), w * 40 * U)


# ------------------------------------------------------------------------------------------ combine
def combine64(edges, slots, w, *more):
    at = slots.long()
    rows = torch.where((at >= 0).unsqueeze(2), edges.double()[at.clamp(0, edges.shape[0] - 1)], 0.0)
    terms = rows * torch.where(at >= 0, w.double(), 0.0).unsqueeze(2)
    y, size = terms.sum(1), terms.abs().sum(1)
    for m in more:
        if m is not None:
            y, size = y + m.double(), size + m.double().abs()
    return y, size


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 8, 2048), (5, 3, 7), (32, 8, 2048), (33, 9, 1000), (3, 64, 129), (200, 2, 4096), (7, 4, 8200)])
@pytest.mark.parametrize("dt,rt,ot", [(BF16, None, BF16), (BF16, F32, F32), (F32, BF16, BF16), (F32, F32, F32)])
def test_combine(ops, T, k, H, dt, rt, ot):
    g = _gen(T + H)
    n = T * k + 3
    edges, w = _rnd(g, n, H, dtype=dt), torch.rand(T, k, generator=g, device="cuda")
    slots = torch.randperm(n, generator=g, device="cuda")[:T * k].view(T, k).to(I32)
    slots[T // 2, :] = -1
    slots[0, 0] = -5 if T > 1 else 0
    shared = _rnd(g, T, H, dtype=dt) if rt is not None else None
    res = _rnd(g, T, H, dtype=rt) if rt is not None else None
    got = ops.combine(edges, slots, w, shared=shared, residual=res, out_dtype=ot)
    y, size = combine64(edges, slots, w, shared, res)
    assert got.dtype == ot and got.shape == (T, H)
    _within(got, y, size * (k + 3) * U + y.abs() * _half(ot) * (ot == BF16) * (1 + 2 ** -7) + 1e-38)


@pytest.mark.gpu
def test_combine_layouts(ops):
    g = _gen(3)
    T, k, H = 6, 3, 64
    for pad, first in ((0, 0), (8, 0), (3, 1)):
        edges, w = _rnd(g, 20, H + pad, dtype=BF16)[:, first:first + H], torch.rand(T, k, generator=g, device="cuda")
        slots = torch.randint(0, 20, (T, k), generator=g, device="cuda", dtype=I32)  # one edge may serve two positions
        res = _rnd(g, T, H + pad)[:, first:first + H]
        y, size = combine64(edges, slots, w, res)
        o = torch.full((T, H + pad), -7.0, device="cuda")
        ops.combine(edges, slots, w, residual=res, out=o[:, first:first + H])
        _within(o[:, first:first + H], y, size * 8 * U + 1e-38)
        assert bool((o[:, :first] == -7).all()) and bool((o[:, first + H:] == -7).all())
        r = res.clone() if pad == 0 else res  # in place on the residual stream
        assert ops.combine(edges, slots, w, residual=r, out=r) is r
        _within(r, y, size * 8 * U + 1e-38)
        slots[2, 1] = 20  # one past the last: not followed, and seen
        got = ops.combine(edges, slots, w)
        assert bool(got[2].isnan().all()) and int(got.isnan().any(1).sum()) == 1
    edges[4, 5] = math.inf
    slots = torch.tensor([[4], [5]], device="cuda", dtype=I32)
    got = ops.combine(edges, slots, torch.ones(2, 1, device="cuda"))
    assert bool(got[0, 5] == math.inf) and bool(got[1].isfinite().all())
    assert ops.combine(edges, slots[:0], torch.ones(0, 1, device="cuda")).shape == (0, H)
    none = torch.full((2, 1), -1, device="cuda", dtype=I32)
    assert bool((ops.combine(edges[:0], none, torch.ones(2, 1, device="cuda")) == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1, 6, 16, 77, 1032])
@pytest.mark.parametrize("rt,ot", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_combine_rows_from_any_boundary(ops, H, rt, ot):
    """Rows of each tensor that start on every 2-byte (4-byte) boundary, with NaN beside them; results stay in their row."""
    g = _gen(H)
    T, k, n = 9, 5, 40

    def rows(count, dtype, first, pad):
        flat = torch.full((first + count * (H + pad) + 1,), math.nan, device="cuda", dtype=dtype)
        view = flat[first:first + count * (H + pad)].view(count, H + pad)[:, :H]
        return flat, view.copy_(_rnd(g, count, H, dtype=dtype))

    slots = torch.randint(-1, n, (T, k), generator=g, device="cuda", dtype=I32)
    w = torch.rand(T, k, generator=g, device="cuda")
    for first in range(8):
        for pad in (first, 3 - first % 3):
            _, edges = rows(n, BF16, first, pad)
            _, shared = rows(T, BF16, (3 * first + 1) % 8, pad)
            _, res = rows(T, rt, (first + 5) % 8, pad + 1)
            flat, out = rows(T, ot, 7 - first, pad + 2)
            y, size = combine64(edges, slots, w, shared, res)
            bound = size * (k + 3) * U + y.abs() * _half(ot) * (ot == BF16) * (1 + 2 ** -7) + 1e-38
            assert ops.combine(edges, slots, w, shared=shared, residual=res, out=out) is out
            _within(out, y, bound)
            assert int(flat.isnan().sum()) == flat.numel() - T * H
            if ot == BF16:  # in place on the shared experts' output
                assert ops.combine(edges, slots, w, shared=shared, residual=res, out=shared) is shared
                assert torch.equal(shared, out)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1024, 1001])
def test_combine_offsets_pass_32_bits(ops, H):
    far = (1 << 31) // 2 + 24
    g = _gen(H)
    edges = torch.empty(2 * far + H, device="cuda", dtype=BF16).as_strided((3, H), (far, 1))
    edges.copy_(_rnd(g, 3, H, dtype=BF16))
    slots, w = torch.tensor([[2, 0], [1, 2]], device="cuda", dtype=I32), torch.rand(2, 2, generator=g, device="cuda")
    got = ops.combine(edges, slots, w, out_dtype=F32)
    y, size = combine64(edges.contiguous(), slots, w)
    _within(got, y, size * 8 * U)


# ---------------------------------------------------------------------------------- grouped products
def _offsets(r, e, m, first=0, last=None):
    """Ascending offsets with empty groups; rows before `first` and from `last` on are in none."""
    last = m if last is None else last
    cut = np.sort(r.randint(first, last + 1, e - 1)) if e > 1 else np.zeros(0, int)
    if e > 3:
        cut[e // 2] = cut[e // 2 - 1]
    return torch.tensor(np.concatenate([[first], np.sort(cut), [last]]).astype(np.int32), device="cuda")


def product64(a, b, off, swiglu=False, scale=None):
    """(y, the sum of its terms' magnitudes) of rows a and b [E, N, K] in 64 bits; swiglu: of what its product gives,
    with the size that errors of gate and up sums reach in it."""
    n = b.shape[1]
    y = torch.zeros(a.shape[0], n, device="cuda", dtype=F64)
    size = torch.zeros_like(y)
    for e in range(b.shape[0]):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            f = 1.0 if scale is None else float(scale[e])
            y[lo:hi], size[lo:hi] = a[lo:hi] @ b[e].T * f, a[lo:hi].abs() @ b[e].abs().T * abs(f)
    if not swiglu:
        return y, size
    gate, up = y.chunk(2, 1)
    sg, su = size.chunk(2, 1)
    s = torch.sigmoid(gate)
    # |silu'| <= 1.1: errors of the gate's sum times up, of the up sum times silu
    return gate * s * up, 1.1 * sg * up.abs() + su * (gate * s).abs()


def product_bound(y, size, steps, ot, swiglu):
    """steps: additions to an fp32 sum, each off by at most two roundings of what it holds; the factors' and, with
    swiglu, the silu's (exp's 2^-21 relative to its argument's size, quotient, products)."""
    b = size * (2 * steps + 8) * U + y.abs() * 4 * U
    if swiglu:
        b = b + y.abs() * 2.0 ** -19
    return b + (y.abs() * _half(ot) * (1 + 2 ** -7) if ot == BF16 else 0) + 1e-30


GROUPED = [(1, 1, 1, 8), (1, 8, 64, 64), (3, 2, 40, 72), (17, 5, 130, 200), (64, 64, 32, 128), (100, 3, 256, 512), (129, 1, 257, 1000),
           (200, 130, 96, 256), (300, 4, 520, 264), (1000, 3, 768, 192), (2050, 2, 1024, 128), (700, 1, 2000, 64),
           (1000, 1, 4096, 64), (900, 2, 4000, 192), (1100, 1, 4096, 136),
           (5, 1, 4900, 72), (40, 1, 2600, 200), (60, 3, 1700, 136), (11, 2, 100, 4104), (16, 1, 2048, 2048), (1200, 3, 600, 512), (2100, 2, 1030, 264)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,e,n,k", GROUPED)
@pytest.mark.parametrize("form", ["plain", "gather", "swiglu", "gather_swiglu"])
@pytest.mark.parametrize("dt,ot", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_grouped_matmul(ops, m, e, n, k, form, dt, ot):
    g, r = _gen(m + n), np.random.RandomState(m)
    gather, swiglu = "gather" in form, "swiglu" in form
    n += n % 2 if swiglu else 0
    src = max(1, m // 3) if gather else m
    x, w = _rnd(g, src, k, dtype=dt), _rnd(g, e, n, k, std=k ** -0.5, dtype=dt)
    rows = torch.randint(0, src, (m,), generator=g, device="cuda", dtype=I32) if gather else None
    off = _offsets(r, e, m)
    got = ops.grouped_matmul(x, w, off, rows=rows, swiglu=swiglu, out_dtype=ot)
    a = x.double() if rows is None else x.double()[rows.long()]
    y, size = product64(a, w.double(), off, swiglu)
    assert got.dtype == ot and got.shape == y.shape
    _within(got, y, product_bound(y, size, k if dt == F32 else k / 16 + 16, ot, swiglu))
    assert ops.status() == (0, 0)
    if e == 1:
        assert torch.equal(ops.grouped_matmul(x, w[0], None, rows=rows, swiglu=swiglu, out_dtype=ot), got)


@pytest.mark.gpu
@pytest.mark.parametrize("m,e,n", [(400, 2, 75), (1000, 3, 334), (700, 1, 2001), (1000, 3, 767), (1000, 1, 4095), (1100, 1, 4093), (700, 64, 1021)])
@pytest.mark.parametrize("ot", [BF16, F32])
@pytest.mark.parametrize("form", ["bf16", "nvfp4"])
def test_products_outputs_from_any_boundary(ops, m, e, n, ot, form):
    """Output rows that start on every boundary of their type have the bits of aligned ones, and their neighbours stay."""
    k, g = 64, _gen(m)
    off = _offsets(np.random.RandomState(n), e, m)
    x, w = _rnd(g, m, k, dtype=BF16), _rnd(g, e, n, k, dtype=BF16)
    if form == "nvfp4":
        (x, sx), (w, sw, _) = ops.fp4_quantize(x), ops.fp4_quantize_weight(w)

    def run(out):
        if form == "bf16":
            return ops.grouped_matmul(x, w, off, out=out)
        return ops.fp4_matmul(x, sx, w, sw, offsets=off, out=out)

    want = run(torch.empty(m, (n + 15) // 16 * 16, device="cuda", dtype=ot)[:, :n])
    for first in range(8):
        for pad in (0, first + 1, 8):
            flat = torch.full((first + m * (n + pad) + 3,), -7.0, device="cuda", dtype=ot)
            out = run(flat[first:first + m * (n + pad)].view(m, n + pad)[:, :n])
            assert torch.equal(out, want)
            assert int((flat == -7).sum()) - int((want == -7).sum()) == flat.numel() - m * n


@pytest.mark.gpu
def test_grouped_matmul_longest_rows(ops):
    """Rows of 2^31 bytes: every place that is not zero counts, behind the last 32-bit offset too."""
    k = 1 << 30
    x, w = torch.zeros(1, k, device="cuda", dtype=BF16), torch.zeros(2, k, device="cuda", dtype=BF16)
    for i, at in enumerate((0, 7, k // 2 - 1, k // 2, k - 8, k - 1)):
        x[0, at] = 1.0
        w[0, at] = 2.0 ** i
        w[1, at] = -(2.0 ** (5 - i))
    got = ops.grouped_matmul(x, w, None, out_dtype=F32)
    assert got.tolist() == [[63.0, -63.0]]
    assert ops.status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(40, 96, 64), (600, 520, 128), (1100, 512, 64)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_grouped_matmul_rows_outside_bad_rows_and_strides(ops, m, n, k, dt):
    g, e = _gen(m), 3
    x, w = _rnd(g, m, k, dtype=dt), _rnd(g, e, n, k, std=k ** -0.5, dtype=dt)
    off = torch.tensor([5, 5, m // 2, m - 4], device="cuda", dtype=I32)
    out = torch.full((m, n), -3.0, device="cuda", dtype=dt)
    ops.grouped_matmul(x, w, off, out=out)
    y, size = product64(x.double(), w.double(), off)
    bound = product_bound(y, size, k if dt == F32 else k / 16 + 16, dt, False)
    _within(out[5:m - 4], y[5:m - 4], bound[5:m - 4])
    assert bool((out[:5] == -3).all()) and bool((out[m - 4:] == -3).all())
    # descending and wild offsets: read as the nearest ascending values in range
    wild = torch.tensor([-9, m // 2, 4, m + 100], device="cuda", dtype=I32)
    tame = torch.tensor([0, m // 2, m // 2, m], device="cuda", dtype=I32)
    assert torch.equal(ops.grouped_matmul(x, w, wild), ops.grouped_matmul(x, w, tame))
    # rows apart, an output of odd stride and offset, the base on a 16-byte boundary alone
    pad = 8
    wide = _rnd(g, m, k + pad, dtype=dt)[:, pad:]
    for first, more in ((0, 0), (0, 16), (1, 3)):
        o = torch.full((m, n + more), -3.0, device="cuda", dtype=dt)
        got = ops.grouped_matmul(wide, w, tame, out=o[:, first:first + n])
        assert torch.equal(got, ops.grouped_matmul(wide.contiguous(), w, tame))
        assert bool((o[:, :first] == -3).all()) and bool((o[:, first + n:] == -3).all())
    # indexes out of range: not read, and seen
    rows = torch.arange(m, device="cuda", dtype=I32).flip(0).contiguous()
    want = ops.grouped_matmul(x, w, tame, rows=rows)
    bad = rows.clone()
    at = [0, 7, m // 2, m - 1]
    bad[at] = torch.tensor([-1, m, 2 ** 31 - 1, -2 ** 31], device="cuda", dtype=I32)
    got = ops.grouped_matmul(x, w, tame, rows=bad)
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[at] = False
    assert bool(got[~keep].isnan().all()) and torch.equal(got[keep], want[keep])
    # a bad value stays in its row
    x2 = x.clone()
    x2[9, 3] = math.nan
    got = ops.grouped_matmul(x2, w, tame)
    full = ops.grouped_matmul(x, w, tame)
    assert bool(got[9].isnan().all()) and torch.equal(got[10:], full[10:]) and torch.equal(got[:9], full[:9])
    assert ops.grouped_matmul(x[:0], w, torch.zeros(4, device="cuda", dtype=I32)).shape == (0, n)
    none = torch.full((5,), -1, device="cuda", dtype=I32)  # nothing to gather from
    assert bool(ops.grouped_matmul(x[:0], w, torch.tensor([0, 5, 5, 5], device="cuda", dtype=I32), rows=none).isnan().all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F32])
def test_grouped_matmul_offsets_pass_32_bits(ops, dt):
    """Rows far apart, and weights whose last matrix begins behind 2^32 bytes."""
    e, n, k, m = 35, 8192, 8192, 40
    g = _gen(2)
    w = torch.zeros(e, n, k, device="cuda", dtype=dt)
    last = _rnd(g, n, k, std=k ** -0.5, dtype=dt)
    w[-1] = last
    far = (1 << 30) + 8
    x = torch.empty(2 * far + k, device="cuda", dtype=dt).as_strided((3, k), (far, 1))
    x.copy_(_rnd(g, 3, k, dtype=dt))
    rows = torch.arange(m, device="cuda", dtype=I32) % 3
    off = torch.zeros(e + 1, device="cuda", dtype=I32)
    off[-1] = m
    got = ops.grouped_matmul(x, w, off, rows=rows, out_dtype=F32)
    y, size = product64(x.double()[rows.long()], last.double()[None], [0, m])
    _within(got, y, product_bound(y, size, k if dt == F32 else k / 16 + 16, F32, False))


# ------------------------------------------------------------------------------------ 4-bit quantiser
def fp4_64(x, form, t=1.0):
    """(codes, scales in 64 bits [n, K / block], bytes of the scales) of x in 64 bits, by comparing every distance."""
    block, dtype = FORMS[form]
    b = (x.double() / t).unflatten(-1, (-1, block))
    most = b.abs().amax(-1)
    ok = most.isfinite()
    if form == "nvfp4":
        # e4m3 of most / 6: the nearest of all its values, the even one among two
        grid = torch.arange(127, device=x.device, dtype=U8).view(E4M3).double()
        d = ((most / 6).clamp(max=448.0).unsqueeze(-1) - grid).abs()
        near = d == d.amin(-1, keepdim=True)
        byte = torch.where(near, torch.arange(127, device=x.device) % 2, 2).argmin(-1).clamp(min=1)
        s = grid[byte]
        byte = torch.where(ok, byte, 127)
    else:
        e = (torch.frexp(most).exponent - 3).clamp(-127, 127)
        e = torch.where(most > 0, e, -127)
        s = torch.exp2(e.double())
        byte = torch.where(ok, e + 127, 255)
    d = ((b / s.unsqueeze(-1)).abs().clamp(max=6.0).unsqueeze(-1) - torch.tensor(GRID, device=x.device, dtype=F64)).abs()
    near = d == d.amin(-1, keepdim=True)
    code = torch.where(near, torch.arange(8, device=x.device) % 2, 2).argmin(-1)
    return code.flatten(-2), torch.where(ok, s, math.nan), byte.to(U8)


def unpack(q):
    return torch.stack([q & 15, q >> 4], -1).flatten(-2)


def flat_scales(scales, k, block):
    """[.., kb, n, per] -> bytes [.., n, K / block]."""
    return scales.view(U8).transpose(-2, -3).flatten(-2)[..., :k // block]


def check_codes(q, scales, x, form, t=1.0):
    block, dtype = FORMS[form]
    k = x.shape[-1]
    code, s, byte = fp4_64(x, form, t)
    assert scales.dtype == dtype and torch.equal(flat_scales(scales, k, block), byte)
    pad = scales.view(U8).transpose(-2, -3).flatten(-2)[..., k // block:]
    assert bool((pad == 0).all())
    got = unpack(q)
    fine = s.isfinite().repeat_interleave(block, -1)
    sign = (torch.signbit(x) & fine).to(U8) * 8
    assert torch.equal(torch.where(fine, got, 0), torch.where(fine, code.to(U8) | sign, 0))
    v = torch.tensor(GRID, device=x.device, dtype=F64)[code] * s.repeat_interleave(block, -1) * t
    return torch.where(torch.signbit(x), -v, v)


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("n,k", [(1, 32), (3, 64), (5, 256), (7, 288), (33, 2048), (2, 8224), (1000, 96)])
def test_fp4_quantize(ops, form, dt, n, k):
    g = _gen(n + k)
    block, _ = FORMS[form]
    x = _rnd(g, n, k, std=2.0)
    x *= torch.exp2(torch.randint(-12, 9, (n, k // block), generator=g, device="cuda").float()).repeat_interleave(block, 1)
    x[0, :block] = 0
    if n > 2:  # borders between codes and between scales, hit exactly
        x[1, :block] = torch.tensor((GRID + [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0]) * (block // 16), device="cuda") * 1.125
        x[2, :block] = torch.linspace(-6, 6, block, device="cuda") * 2.0 ** -9
    x = x.to(dt)
    t = 0.25 if form == "nvfp4" else 1.0
    q, s = ops.fp4_quantize(x, form=form, tensor_scale=t)
    assert q.dtype == U8 and q.shape == (n, k // 2) and s.shape == (-(-k // 256), n, 256 // block)
    v = check_codes(q, s, x, form, t)
    for ot in (BF16, F32):
        got = ops.fp4_dequantize(q, s, tensor_scale=t, out_dtype=ot)
        assert got.dtype == ot and torch.equal(got.double(), v)  # six bits: exact
    # any alignment, rows apart, gathered
    odd = torch.empty(n, k + 3, device="cuda", dtype=dt)[:, 1:k + 1]
    odd.copy_(x)
    rows = torch.arange(n, device="cuda", dtype=I32).flip(0).contiguous()
    q2, s2 = ops.fp4_quantize(odd, form=form, tensor_scale=t, rows=rows)
    assert torch.equal(q2.flip(0), q) and torch.equal(s2.view(U8).flip(1), s.view(U8))


@pytest.mark.gpu
@pytest.mark.parametrize("k", [64, 512])
def test_fp4_quotients_next_to_a_border(ops, k):
    """fp32 values one step beside a border times the scale, whose quotient fp32 rounds onto the border, and block maxima
    beside a border of the scale."""
    s = torch.arange(1, 127, device="cuda", dtype=U8).view(E4M3).float()
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    at = (s.unsqueeze(1) * mids).unsqueeze(2).view(torch.int32) + torch.tensor([-1, 0, 1], device="cuda", dtype=I32)
    x = torch.zeros(s.numel(), k, device="cuda")
    x[:, :21] = at.view(F32).reshape(-1, 21)
    x[:, 16] = x[:, 16]
    x[:, 15] = 6 * s  # the block's scale is s; the next block's follows from its own values
    q, sc = ops.fp4_quantize(x)
    check_codes(q, sc, x, "nvfp4")
    between = (s[:-1] + s[1:]) / 2 * 6  # borders between scales
    x = torch.zeros(between.numel() * 3, k, device="cuda")
    x[:, 0] = (between.view(torch.int32).unsqueeze(1) + torch.tensor([-1, 0, 1], device="cuda", dtype=I32)).view(F32).reshape(-1)
    q, sc = ops.fp4_quantize(x)
    check_codes(q, sc, x, "nvfp4")


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
def test_fp4_quantize_values_that_end_ranges(ops, form):
    block, _ = FORMS[form]
    big = torch.finfo(F32).max
    x = torch.zeros(8, 64, device="cuda")
    x[0, 3] = math.nan
    x[1, block] = -math.inf
    x[2, :5] = big
    x[3, :5] = 1e-45
    x[4, :5] = 2.0 ** -126
    x[5, 1] = 448 * 6 * 3.0       # beyond nvfp4's largest scale: saturates
    x[6, 2] = 2.0 ** -10 * 6      # below the smallest
    q, s = ops.fp4_quantize(x, form=form)
    v = check_codes(q, s, x, form)
    got = ops.fp4_dequantize(q, s, out_dtype=F32)
    assert bool(got[0, :block].isnan().all()) and bool(got[1, block:2 * block].isnan().all())
    assert int(got.isnan().sum()) == 2 * block
    fine = v.isfinite() & (v.abs() < big)
    assert torch.equal(got[fine].double(), v[fine])
    rows = torch.tensor([5, -1, 8, 2 ** 31 - 1, 6], device="cuda", dtype=I32)
    q2, s2 = ops.fp4_quantize(x, form=form, rows=rows)
    got2 = ops.fp4_dequantize(q2, s2, out_dtype=F32)
    assert bool(got2[1:4].isnan().all()) and torch.equal(got2[[0, 4]], got[[5, 6]])
    assert ops.fp4_quantize(x[:0], form=form)[0].shape == (0, 32)
    assert ops.fp4_dequantize(*ops.fp4_quantize(x[:0], form=form)).shape == (0, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("n,k", [(1, 32), (17, 544), (333, 512)])
def test_fp4_quantize_swiglu(ops, form, dt, n, k):
    g = _gen(n)
    block, _ = FORMS[form]
    x = _rnd(g, n, 2 * k, std=2.0, dtype=dt)
    q, s = ops.fp4_quantize(x, form=form, swiglu=True)
    gate, up = x.double().chunk(2, 1)
    a = torch.nn.functional.silu(gate) * up
    e = a.abs() * 12 * U  # exp 4, its argument's size 2, sum, quotient and product
    sc = flat_scales(s, k, block)
    most, err = a.unflatten(-1, (-1, block)).abs().amax(-1), e.unflatten(-1, (-1, block)).amax(-1)
    lo, hi = fp4_64((most - err).repeat_interleave(block, 1), form)[2], fp4_64((most + err).repeat_interleave(block, 1), form)[2]
    assert bool(((sc >= lo) & (sc <= hi)).all())
    wide = (sc.view(E4M3).double() if form == "nvfp4" else torch.exp2(sc.double() - 127)).repeat_interleave(block, 1)
    got = ops.fp4_dequantize(q, s, out_dtype=F32).double()
    # off by half a step between codes (the largest is 2, from 4 to 6), or saturated at 6 (mxfp4: up to 8)
    size = a.abs() / wide
    step = torch.where(size < 2, 0.25, torch.where(size < 4, 0.5, 1.0))
    over = (size - 6).clamp(min=0)
    assert bool(((got - a).abs() <= wide * torch.maximum(step, over) + e * 2).all())


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 1, 32), (3, 130, 288), (5, 64, 1024), (0, 40, 512)])
def test_fp4_quantize_weight(ops, form, dt, shape):
    g = _gen(7)
    e, n, k = shape
    w = _rnd(g, max(e, 1), n, k, std=k ** -0.5, dtype=dt)
    if e > 1:
        w[1] = 0
        w[2] *= 1000
    w = w[:e] if e != 0 else w[0]
    q, s, t = ops.fp4_quantize_weight(w, form=form)
    stack = w if e else w[None]
    qs, ss = (q, s) if e else (q[None], s[None])
    assert t.shape == (stack.shape[0],)
    for i in range(stack.shape[0]):
        most = float(stack[i].abs().max())
        if form == "nvfp4" and most > 0:
            assert most <= 2688 * float(t[i]) and most > 1344 * float(t[i]) and math.frexp(float(t[i]))[0] == 0.5
        else:
            assert float(t[i]) == 1
        check_codes(qs[i], ss[i], stack[i], form, float(t[i]))
    v = ops.fp4_dequantize(q, s, tensor_scale=t, out_dtype=F32)
    assert v.shape == w.shape
    for i in range(stack.shape[0]):
        assert torch.equal((v if e else v[None])[i], ops.fp4_dequantize(qs[i], ss[i], tensor_scale=float(t[i]), out_dtype=F32))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F32])
def test_fp4_quantize_swiglu_of_any_gate(ops, dt):
    """Gates where the sigmoid is 1, a step from 1, subnormal or nothing, beside ordinary ones: a block of one value is off
    by half a step of e2m1 (an eighth), or by the smallest scale's."""
    gates = [1e-30, -1e-30, 3e-39, -0.0, 0.0, 0.7, -3.0, 17.0, 60.0, -60.0, -80.0, -87.0, -88.5, 90.0, 3e38, 1e30]
    x = torch.empty(len(gates) + 1, 2 * 64, device="cuda", dtype=dt)
    x[:, 64:] = 1.5
    x[:, :64] = torch.tensor(gates + [1.0], device="cuda")[:, None]
    x[-1, 3:40:8] = torch.tensor([-100.0, 1e-35, 0.0, 70.0, -69.5], device="cuda").to(dt)  # in one thread with ordinary ones
    q, s = ops.fp4_quantize(x, form="mxfp4", swiglu=True)
    got = ops.fp4_dequantize(q, s, out_dtype=F32).double()
    g64 = x[:, :64].double()
    v = 1.5 * g64 * torch.sigmoid(g64)
    top = v[-1].view(2, 32).abs().amax(1).repeat_interleave(32)  # the last row: by its blocks' scales
    # a value above 4 s is off by s at most (5 to 4 or 6), in a block whose largest lies from 4 s to 8 s (then 7.99 to 6)
    over = v.abs() > torch.finfo(F32).max  # 1.5 * 3e38 is infinite in fp32, and so its block NaN
    assert int(over.sum()) == 64 and bool(got[over].isnan().all())
    assert bool(((got - v)[:-1].abs() <= v[:-1].abs() / 4 + 2.0 ** -127)[~over[:-1]].all())
    assert bool(((got - v)[-1].abs() <= top / 4 + 2.0 ** -127).all())
    x[:, 5] = math.inf
    q, s = ops.fp4_quantize(x, form="mxfp4", swiglu=True)
    back = ops.fp4_dequantize(q, s)
    assert bool(back[:, :32].isnan().all()) and bool(back[:, 32:][~over[:, 32:]].isfinite().all())


# -------------------------------------------------------------------------------------- 4-bit products
def fp4_operand(g, form, *shape, std=1.0):
    """(q, scales, values in 64 bits), made here: any code, scales of several octaves."""
    block, dtype = FORMS[form]
    k = shape[-1]
    code = torch.randint(0, 16, shape, generator=g, device="cuda", dtype=torch.int64)
    lead = shape[:-1]
    pad = -(-k // 256) * 256 // block
    if form == "nvfp4":
        byte = torch.randint(0x28, 0x48, lead + (k // block,), generator=g, device="cuda")
        s = byte.to(U8).view(E4M3).double()
    else:
        byte = torch.randint(120, 130, lead + (k // block,), generator=g, device="cuda")
        s = torch.exp2(byte.double() - 127)
    v = torch.tensor(GRID + [-x for x in GRID], device="cuda", dtype=F64)[code] * s.repeat_interleave(block, -1)
    byte = torch.nn.functional.pad(byte.to(U8), (0, pad - k // block))
    scales = byte.unflatten(-1, (-1, 256 // block)).transpose(-2, -3).contiguous().view(dtype)
    q = (code[..., 0::2] | code[..., 1::2] << 4).to(U8)
    return q, scales, v


FP4 = [(1, 1, 1, 32), (1, 8, 64, 256), (3, 2, 40, 96), (17, 5, 130, 288), (64, 64, 32, 512), (100, 3, 256, 1024), (129, 1, 257, 800),
       (200, 130, 96, 256), (300, 4, 520, 512), (1000, 3, 768, 320), (2050, 2, 1024, 256), (700, 1, 2000, 64), (600, 1, 4096, 768),
       (700, 64, 1024, 256), (5, 1, 4900, 96), (40, 1, 300, 288), (13, 2, 100, 8224), (16, 1, 2048, 2048), (2, 500, 48, 544)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,e,n,k", FP4)
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("ot", [BF16, F32])
def test_fp4_matmul(ops, m, e, n, k, form, swiglu, ot):
    g, r = _gen(m + n), np.random.RandomState(m)
    n += n % 2 if swiglu else 0
    a, sa, va = fp4_operand(g, form, m, k)
    b, sb, vb = fp4_operand(g, form, e, n, k)
    off = _offsets(r, e, m)
    scale = torch.rand(e, generator=g, device="cuda") * k ** -0.5
    got = ops.fp4_matmul(a, sa, b, sb, offsets=off, scale=scale, swiglu=swiglu, out_dtype=ot)
    y, size = product64(va, vb, off, swiglu, scale.double())
    assert got.dtype == ot and got.shape == y.shape
    _within(got, y, product_bound(y, size, k / 64 + 16, ot, swiglu))
    assert ops.status() == (0, 0)
    if e == 1:
        assert torch.equal(ops.fp4_matmul(a, sa, b[0], sb[0], scale=scale, swiglu=swiglu, out_dtype=ot), got)
        one = ops.fp4_matmul(a, sa, b[0], sb[0], scale=float(scale[0]), swiglu=swiglu, out_dtype=ot)
        assert torch.equal(one, got)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 12, 300])  # few rows, and tiles
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
def test_fp4_matmul_scales_of_their_whole_range(ops, m, form):
    """Every finite scale of nvfp4, zero and subnormal ones among them; every one of mxfp4, 2^-127 and 2^127, in pairs whose
    products stay fp32's."""
    n, k = 136, 32 * 255
    g, (block, dtype) = _gen(m), FORMS[form]
    a, _, va = fp4_operand(g, form, m, k)
    b, _, vb = fp4_operand(g, form, 1, n, k)
    grid = torch.tensor(GRID + [-x for x in GRID], device="cuda", dtype=F64)
    lay = lambda byte: torch.nn.functional.pad(byte.to(U8), (0, -(-k // 256) * 256 // block - k // block)).unflatten(  # noqa: E731
        -1, (-1, 256 // block)).transpose(-2, -3).contiguous().view(dtype)
    value = lambda q: grid[torch.stack([q & 15, q >> 4], -1).flatten(-2).long()]  # noqa: E731
    if form == "nvfp4":
        ba, bb = (torch.randint(0, 0x7F, (r, k // block), generator=g, device="cuda") for r in (m, n))
        fa, fb = (t.to(U8).view(E4M3).double() for t in (ba, bb))
    else:
        ba = torch.randperm(255, generator=g, device="cuda").expand(m, -1)
        bb = (254 - ba[:1] + torch.randint(-1, 2, (n, 255), generator=g, device="cuda")).clamp(0, 254)
        fa, fb = (torch.exp2(t.double() - 127) for t in (ba, bb))
    va, vb = value(a) * fa.repeat_interleave(block, -1), value(b[0]) * fb.repeat_interleave(block, -1)
    off = torch.tensor([0, m], device="cuda", dtype=I32)
    y, size = product64(va, vb[None], off)
    got = ops.fp4_matmul(a, lay(ba), b[0], lay(bb), out_dtype=F32)
    _within(got, y, product_bound(y, size, k / 64 + 16, F32, False))


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("m,n,k", [(40, 96, 288), (600, 520, 512), (1100, 512, 64)])
def test_fp4_matmul_rows_outside_and_bad_blocks(ops, form, m, n, k):
    g, e = _gen(m), 3
    a, sa, va = fp4_operand(g, form, m, k)
    b, sb, vb = fp4_operand(g, form, e, n, k)
    off = torch.tensor([5, 5, m // 2, m - 4], device="cuda", dtype=I32)
    out = torch.full((m, n + 1), -3.0, device="cuda", dtype=F32)[:, 1:]
    ops.fp4_matmul(a, sa, b, sb, offsets=off, out=out)
    y, size = product64(va, vb, off)
    bound = product_bound(y, size, k / 64 + 16, F32, False)
    _within(out[5:m - 4], y[5:m - 4], bound[5:m - 4])
    assert bool((out[:5] == -3).all()) and bool((out[m - 4:] == -3).all())
    # a NaN scale spoils its row, or its column of the group, and nothing else
    bad = sa.clone()
    bad.view(U8)[0, 9, 1] = 0x7F if form == "nvfp4" else 0xFF
    full = ops.fp4_matmul(a, sa, b, sb, offsets=off, out_dtype=F32)
    got = ops.fp4_matmul(a, bad, b, sb, offsets=off, out_dtype=F32)
    assert bool(got[9].isnan().all()) and torch.equal(got[10:m - 4], full[10:m - 4]) and torch.equal(got[5:9], full[5:9])
    bad = sb.clone()
    bad.view(U8)[1, 0, 7, 0] = 0x7F if form == "nvfp4" else 0xFF
    got = ops.fp4_matmul(a, sa, b, bad, offsets=off, out_dtype=F32)
    assert bool(got[5:m // 2, 7].isnan().all()) and int(got[5:m - 4].isnan().sum()) == m // 2 - 5


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
def test_fp4_offsets_pass_32_bits(ops, form):
    """The last of 70 matrices of 8192 x 8192 begins behind 2^31 bytes of codes and 2^33 of bf16 weights."""
    e, n, k, m = 70, 8192, 8192, 150
    g = _gen(5)
    w = torch.zeros(e, n, k, device="cuda", dtype=BF16)
    w[-1] = _rnd(g, n, k, std=k ** -0.5)
    b, sb, t = ops.fp4_quantize_weight(w, form=form)
    one = ops.fp4_quantize_weight(w[-1].contiguous(), form=form)
    assert torch.equal(b[-1], one[0]) and torch.equal(sb[-1].view(U8), one[1].view(U8)) and torch.equal(t[-1:], one[2])
    del w
    a, sa = ops.fp4_quantize(_rnd(g, m, k), form=form)
    off = torch.zeros(e + 1, device="cuda", dtype=I32)
    off[-1] = m
    got = ops.fp4_matmul(a, sa, b, sb, offsets=off, scale=t, out_dtype=F32)
    va = ops.fp4_dequantize(a, sa, out_dtype=F32).double()
    vb = ops.fp4_dequantize(*one[:2], tensor_scale=one[2], out_dtype=F32).double()
    y, size = product64(va, vb[None], [0, m])
    _within(got, y, product_bound(y, size, k / 64 + 16, F32, False))


# -------------------------------------------------------------------------------------------- router
@pytest.mark.gpu
@pytest.mark.parametrize("E,groups,top", [(256, 8, 4), (64, 4, 2), (512, 16, 3), (96, 6, 2)])
def test_route_groups_that_fp32_cannot_tell_apart(ops, E, groups, top):
    """Groups whose two best add up to the same but for a step or two of a logit."""
    g = _gen(E)
    T, k, size = 150, 8, E // groups
    x = _rnd(g, T, E) - 3
    best = 1 + torch.rand(T, 1, 2, generator=g, device="cuda")
    steps = torch.randint(-2, 3, (T, groups, 2), generator=g, device="cuda", dtype=I32)
    x.view(T, groups, size)[:, :, [1, size - 1]] = (best.expand(T, groups, 2).contiguous().view(torch.int32) + steps).view(F32)
    for bias in (None, torch.zeros(E, device="cuda")):
        check_route(ops.route(x, k, router="sigmoid_group", bias=bias, n_group=groups, topk_group=top),
                    route64(x, k, True, bias=bias, n_group=groups, topk_group=top))


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups,top", [(24, 8, 1), (60, 10, 1), (96, 32, 2), (256, 32, 0)])
def test_route_more_groups_than_asked_for(ops, E, groups, top):
    """Groups that hold fewer than k: more of them are searched, best first, and so on their order it depends which, where
    some hold less than others (masks)."""
    g = _gen(E)
    T, k, size, top = 150, 8, E // groups, max(top, 1)
    x = _rnd(g, T, E) - 3
    best = 1 + torch.rand(T, 1, 2, generator=g, device="cuda")
    steps = torch.randint(-2, 3, (T, groups, 2), generator=g, device="cuda", dtype=I32)
    x.view(T, groups, size)[:, :, [1, size - 1]] = (best.expand(T, groups, 2).contiguous().view(torch.int32) + steps).view(F32)
    x[::2] = _rnd(g, T // 2, E)
    for kk in (k, min(16, E)):
        for eligible in (None, torch.rand(E, generator=g, device="cuda") < 0.7):
            check_route(ops.route(x, kk, router="sigmoid_group", n_group=groups, topk_group=top, eligible=eligible),
                        route64(x, kk, True, n_group=groups, topk_group=top, eligible=eligible))


# ------------------------------------------------------------------------------ streams and graphs
def _steps(ops, seed, T=40):
    """A run of every operator on buffers of its own: (the buffers that new inputs go to, the call, its outputs)."""
    g = _gen(seed)
    H, E, I, k = 256, 8, 128, 3
    x, logits = _rnd(g, T, H, dtype=BF16), _rnd(g, T, E)
    w13, w2 = _rnd(g, E, 2 * I, H, std=H ** -0.5, dtype=BF16), _rnd(g, E, H, I, std=I ** -0.5, dtype=BF16)
    q13, s13, t13 = ops.fp4_quantize_weight(w13)
    q2, s2, t2 = ops.fp4_quantize_weight(w2, form="mxfp4")

    def call(stream=None):
        r = ops.route(logits, k, stream=stream)
        a = ops.grouped_matmul(x, w13, r.offsets, rows=r.positions, swiglu=True, stream=stream)
        o = ops.grouped_matmul(a, w2, r.offsets, stream=stream)
        y = ops.combine(o, r.slots, r.weights, residual=x, stream=stream)
        q, s = ops.fp4_quantize(x, rows=r.positions, stream=stream)
        gu = ops.fp4_matmul(q, s, q13, s13, offsets=r.offsets, scale=t13, stream=stream)
        q, s = ops.fp4_quantize(gu, form="mxfp4", swiglu=True, stream=stream)
        o4 = ops.fp4_matmul(q, s, q2, s2, offsets=r.offsets, scale=t2, out_dtype=F32, stream=stream)
        v = ops.fp4_dequantize(q, s, stream=stream)
        y4 = ops.combine(o4, r.slots, r.weights, out_dtype=BF16, stream=stream)
        return (*r, a, o, y, v, y4)

    return (x, logits), call


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 300])
def test_operators_on_a_stream_of_their_own_and_in_a_graph(ops, T):
    inputs, call = _steps(ops, T, T)
    want = call()
    assert all(bool(t.float().isfinite().all()) for t in want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    side.synchronize()
    assert _same(got, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    g = _gen(99)
    old = [t.clone() for t in inputs]
    for turn in range(3):
        for t, o in zip(inputs, old):
            t.copy_(o if turn == 2 else _rnd(g, *t.shape, dtype=t.dtype))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in out]
        assert _same(replayed, call())
    assert _same(replayed, want)


@pytest.mark.gpu
def test_runs_on_two_streams_at_once_and_two_graphs(ops):
    sets = [_steps(ops, s, T)[1] for s, T in ((1, 200), (2, 33))]
    want = [c() for c in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, c in enumerate(sets):
            got[i].append(c(streams[i]))
    torch.cuda.synchronize()
    assert all(_same(o, want[i]) for i in range(2) for o in got[i])
    graphs, outs = [], []
    for c in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(c())
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert all(_same(outs[i], want[i]) for i in range(2))
    assert ops.status() == (0, 0)


FIRST_CALLS = """
import sys
sys.path.insert(0, {root!r})
sys.path.insert(0, {root!r} + "/tests")
import torch
from sparse_moe_layer_gate_gb300 import ops
T, H, E, I, k = {T}, 256, 8, 128, 3
d = dict(device="cuda", dtype=torch.bfloat16)
x, logits = torch.randn(T, H, **d), torch.randn(T, E, device="cuda")
w = torch.randn(E, 2 * I, H, **d) / 16
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
def call():
    qw, sw, tw = ops.fp4_quantize_weight(w)
    r = ops.route(logits, k)
    a = ops.grouped_matmul(x, w, r.offsets, rows=r.positions)
    q, s = ops.fp4_quantize(x, rows=r.positions)
    f = ops.fp4_matmul(q, s, qw, sw, offsets=r.offsets, scale=tw)
    return (*r, a, f, ops.combine(a, r.slots, r.weights), ops.fp4_dequantize(q, s), ops.grouped_matmul(x.float(), w.float(), r.offsets, rows=r.positions))
with torch.cuda.graph(g):
    out = call()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, call())) and ops.status() == (0, 0)
print("same")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 100, 2000])
def test_a_process_whose_first_calls_are_captured(ops, T):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=root, T=T)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


WIDTHS = [32, 64, 128, 256, 512]  # columns of a tile; 512: pairs


def test_every_kernel_of_the_products_is_reached(lib):
    """The sizes above take each width of tiles, pairs, and the kernel for few rows (0), on a device of 152 SMs."""
    for kind, sizes in ((1, GROUPED), (2, FP4), (3, FP4)):
        assert {lib.epoch_expert_matmul_kernel(kind, e, m, n, k, 152) for m, e, n, k in sizes} == {0, *WIDTHS}, kind
    assert lib.epoch_expert_matmul_kernel(0, 2, 10, 64, 64, 152) == 0


def _taking(lib, kind, kernel):
    """Rows, groups and columns that take the kernel here."""
    for m, e in ((40, 1), (130, 1), (300, 1), (700, 1), (1100, 1), (1500, 1), (3000, 1), (700, 64)):
        for n in (64, 256, 512, 1024, 2048, 4096):
            if lib.epoch_expert_matmul_kernel(kind, e, m, n, 1024, 0) == kernel:
                return m, e, n
    raise AssertionError((kind, kernel))


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["bf16", "bf16_gather", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("kernel", WIDTHS)
def test_waits_that_run_out(ops, lib, form, kernel):
    """Operand copies that count bytes that never come: the status, an untouched output, and the same bits afterwards."""
    from sparse_moe_layer_gate_gb300 import binding as B
    kind = {"nvfp4": B.EPOCH_EXPERT_NVFP4, "mxfp4": B.EPOCH_EXPERT_MXFP4}.get(form, B.EPOCH_EXPERT_BF16)
    m, e, n = _taking(lib, kind, kernel)
    k, g = 1024, _gen(kernel)
    off = (torch.arange(e + 1, device="cuda") * m // e).to(I32)
    y = torch.full((m, n), -3.0, device="cuda", dtype=BF16)
    rows = torch.arange(m, device="cuda", dtype=I32) if form == "bf16_gather" else None
    if kind == B.EPOCH_EXPERT_BF16:
        x, w = _rnd(g, m, k, dtype=BF16), _rnd(g, e, n, k, std=k ** -0.5, dtype=BF16)
        sx = sw = None
        want = ops.grouped_matmul(x, w, off, rows=rows)
    else:
        x, sx = ops.fp4_quantize(_rnd(g, m, k), form=form)
        w, sw, _ = ops.fp4_quantize_weight(_rnd(g, e, n, k), form=form)
        want = ops.fp4_matmul(x, sx, w, sw, offsets=off)
    ptr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    args = B.EXPERT_ARGS.pack(ptr(x), ptr(w), ptr(sx), ptr(sw), ptr(off), ptr(rows), 0, ptr(y), k, n, 1.0, e, m, m, n, k, kind,
                              0, B.EPOCH_BF16)
    stream = torch.cuda.current_stream().cuda_stream
    assert ops.status() == (0, 0)
    assert B.lib().epoch_test_expert_timeout(args, 2_000_000, stream) == 0
    code, word = ops.status(clear=True)
    assert code == B.EPOCH_ETIMEOUT and word == B.EPOCH_DEVERR_TIMEOUT
    assert bool((y == -3).all())
    assert B.lib().epoch_expert_matmul(args, stream) == 0
    assert torch.equal(y, want) and ops.status() == (0, 0)
    assert B.lib().epoch_test_expert_timeout(args, 999, stream) == 1  # EPOCH_EINVAL


# ---------------------------------------------------------------------------------------- refusals
P = 1 << 20  # a pointer that is never followed: every call below is refused on the host, or has no rows


@pytest.fixture(scope="module")
def lib(ops):
    from sparse_moe_layer_gate_gb300 import binding
    return binding.lib()


ROUTE = dict(logits=P, bias=0, live=0, eligible=0, sel=P, weights=P, positions=P, offsets=P, slots=P, ws=0, bytes=0, stride=64,
             n=4, experts=64, k=4, dtype=0, router=0, groups=1, top=1, raw=0)
COMBINE = dict(edges=P, shared=0, residual=0, slots=P, weights=P, out=P, es=64, ss=64, rs=64, os=64, n=4, edges_n=16, h=64, k=4,
               dtype=1, rd=0, od=1)
FQUANT = dict(x=P, x_stride=256, dtype=1, rows=None, n=4, src=4, cols=256, swiglu=0, form=0, t=1.0, q=P, s=P, stream=None)
FWEIGHT = dict(w=P, dtype=1, mats=1, n=128, k=128, form=0, q=P, s=P, t=P, stream=None)
FBACK = dict(q=P, s=P, form=0, mats=1, n=8, k=128, scale=1.0, factors=None, out=P, stride=128, dtype=1, stream=None)
EXPERT = dict(a=P, b=P, sa=0, sb=0, offsets=0, rows=0, factors=0, y=P, a_stride=128, stride=64, scale=1.0, groups=1, m=4, src=4, n=64,
              k=128, kind=1, swiglu=0, out=1)
EXPERT4 = dict(EXPERT, sa=P, sb=P, kind=2)


def _call(lib, name, args):
    from sparse_moe_layer_gate_gb300 import binding as B
    packed = {"epoch_route": B.ROUTE_ARGS, "epoch_combine": B.COMBINE_ARGS, "epoch_expert_matmul": B.EXPERT_ARGS}
    if name in packed:
        return getattr(lib, name)(packed[name].pack(*args.values()), None)
    return getattr(lib, name)(*args.values())


def _apart(base):
    """The arguments with every pointer in a place of its own."""
    return {name: (P * (16 + 16 * i) if v == P else v) for i, (name, v) in enumerate(base.items())}


def _refusals():
    f, far = math.inf, P * 4096
    b = _apart(ROUTE)
    for kw in (dict(n=-1), dict(experts=0), dict(experts=1025, stride=1025), dict(k=0), dict(k=17), dict(experts=3, k=4), dict(dtype=2),
               dict(router=2), dict(bias=far), dict(n=(1 << 30), k=4), dict(logits=0), dict(logits=far + 2), dict(stride=63),
               dict(sel=0), dict(weights=far + 2), dict(positions=0), dict(offsets=0), dict(offsets=far + 1), dict(slots=0),
               dict(router=1, groups=0), dict(router=1, groups=33, experts=66, stride=66), dict(router=1, groups=5),
               dict(router=1, groups=4, top=0), dict(router=1, groups=4, top=5), dict(router=1, bias=far + 2),
               dict(n=4000), dict(n=4000, ws=far, bytes=16), dict(n=4000, ws=far + 2, bytes=1 << 20),
               # outputs that overlap
               dict(sel=b["weights"]), dict(slots=b["positions"] + 60), dict(offsets=b["sel"] + 60), dict(weights=b["logits"] + 4),
               dict(live=b["sel"] + 63), dict(eligible=b["offsets"]), dict(router=1, bias=b["slots"])):
        yield "epoch_route", b, kw
    b = _apart(COMBINE)
    for kw in (dict(n=-1), dict(edges_n=-1), dict(h=0), dict(h=(1 << 20) + 1), dict(k=0), dict(k=65), dict(dtype=2), dict(rd=2),
               dict(od=-1), dict(edges=0), dict(edges=far + 1), dict(slots=0), dict(weights=far + 2), dict(out=0), dict(es=63),
               dict(os=1), dict(residual=far, rs=3), dict(shared=far, ss=63), dict(n=1 << 30, h=1 << 20, es=1 << 20, os=1 << 20),
               dict(out=b["edges"] + 64), dict(out=b["slots"] + 2), dict(out=b["weights"]), dict(residual=b["out"]),
               dict(shared=b["out"] + 2), dict(shared=b["out"], ss=65)):
        yield "epoch_combine", b, kw
    b = _apart(FQUANT)
    for kw in (dict(n=-1, src=-1), dict(src=3), dict(cols=0), dict(cols=48), dict(cols=(1 << 30) + 32), dict(dtype=7), dict(form=2),
               dict(t=0.0), dict(t=-1.0), dict(t=f), dict(t=math.nan), dict(t=1e-45), dict(form=1, t=2.0), dict(x=None),
               dict(x=far + 1), dict(q=None), dict(q=far + 8), dict(s=None), dict(s=far + 4), dict(x_stride=255), dict(swiglu=1),
               dict(rows=far + 2), dict(n=1 << 30, src=1 << 30, cols=512, x_stride=512),
               dict(q=b["x"]), dict(s=b["x"] + 16), dict(q=b["s"]), dict(rows=b["q"] + 4), dict(rows=b["s"])):
        yield "epoch_fp4_quantize", b, kw
    b = _apart(FWEIGHT)
    for kw in (dict(dtype=2), dict(form=-1), dict(mats=-1), dict(mats=65536), dict(n=0), dict(k=0), dict(k=40), dict(n=(1 << 22) + 1),
               dict(w=None), dict(q=None), dict(s=None), dict(t=None), dict(t=far + 2), dict(q=b["w"]), dict(s=b["q"]), dict(t=b["s"])):
        yield "epoch_fp4_quantize_weight", b, kw
    b = _apart(FBACK)
    for kw in (dict(dtype=2), dict(form=2), dict(mats=-1), dict(n=-1), dict(k=16), dict(k=33), dict(scale=f), dict(q=None), dict(q=far + 8),
               dict(s=None), dict(s=far + 8), dict(factors=far + 2), dict(out=None), dict(out=far + 1), dict(stride=127), dict(out=b["q"]),
               dict(out=b["s"]), dict(factors=b["out"])):
        yield "epoch_fp4_dequantize", b, kw
    for base in (EXPERT, EXPERT4):
        b = _apart(base)
        for kw in (dict(m=-1, src=-1), dict(n=0), dict(k=0), dict(k=4), dict(k=(1 << 30) + 32), dict(groups=0), dict(groups=2),
                   dict(groups=1025, offsets=far), dict(offsets=far + 2), dict(groups=1024, offsets=far, n=1 << 22), dict(kind=4),
                   dict(kind=-1), dict(a=0), dict(a=far + 8), dict(b=far + 4), dict(b=0), dict(y=0), dict(y=far + 1), dict(stride=63),
                   dict(out=2), dict(scale=f), dict(scale=math.nan), dict(swiglu=1, n=63), dict(factors=far + 2), dict(src=5),
                   dict(src=-1, rows=far), dict(y=b["a"] + 4), dict(y=b["b"] + 64), dict(offsets=b["y"]), dict(factors=b["y"] + 4)):
            yield "epoch_expert_matmul", b, kw
    b = _apart(EXPERT)
    for kw in (dict(a_stride=127), dict(a_stride=132), dict(k=12, a_stride=16), dict(rows=far + 2), dict(rows=b["y"]),
               dict(kind=0, a_stride=130), dict(kind=0, k=6, a_stride=8), dict(kind=0, a=far + 4)):
        yield "epoch_expert_matmul", b, kw
    b = _apart(EXPERT4)
    for kw in (dict(rows=far), dict(k=48), dict(sa=0), dict(sb=far + 8), dict(y=b["sa"]), dict(y=b["sb"])):
        yield "epoch_expert_matmul", b, kw


@pytest.mark.parametrize("name,base,change", list(_refusals()), ids=lambda v: str(v)[:60] if not isinstance(v, dict) else "")
def test_refused_on_the_host(lib, name, base, change):
    assert set(change) <= set(base)
    assert _call(lib, name, {**base, **change}) == 1  # EPOCH_EINVAL, nothing enqueued


def test_without_arguments(lib):
    for name in ("epoch_route", "epoch_combine", "epoch_expert_matmul"):
        assert getattr(lib, name)(None, None) == 1
    assert lib.epoch_test_expert_timeout(None, 1000, None) == 1
    assert lib.epoch_route_workspace_bytes(0, 64) == 0 and lib.epoch_route_workspace_bytes(100, 2000) == 0
    assert lib.epoch_expert_matmul_kernel(9, 0, 1, 1, 8, 152) == -1


def test_no_rows_enqueue_nothing(lib):
    for name, base, kw in (("epoch_combine", COMBINE, dict(n=0, edges=0, out=0)),
                           ("epoch_fp4_quantize", FQUANT, dict(n=0, src=0, x=None, q=None, s=None)),
                           ("epoch_fp4_quantize_weight", FWEIGHT, dict(mats=0, w=None)),
                           ("epoch_fp4_dequantize", FBACK, dict(n=0, q=None, out=None)),
                           ("epoch_expert_matmul", EXPERT, dict(m=0, src=0, a=0, y=0)),
                           ("epoch_expert_matmul", EXPERT4, dict(m=0, src=0, a=0, y=0))):
        assert _call(lib, name, {**base, **kw}) == 0


def test_cpu_tensors_are_refused(ops):
    x, q = torch.zeros(2, 64), torch.zeros(2, 32, dtype=U8)
    s, i = torch.zeros(1, 2, 16).to(E4M3), torch.zeros(2, 1, dtype=I32)
    for call in (lambda: ops.route(x, 2), lambda: ops.combine(x, i, x[:, :1]), lambda: ops.grouped_matmul(x, x, None),
                 lambda: ops.fp4_quantize(x), lambda: ops.fp4_quantize_weight(x), lambda: ops.fp4_dequantize(q, s),
                 lambda: ops.fp4_matmul(q, s, q, s)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_tensors_are_checked(ops):
    c = dict(device="cuda")
    x, w = torch.zeros(4, 64, **c), torch.zeros(64, **c)
    i = torch.zeros(4, 2, dtype=I32, **c)
    q, s = ops.fp4_quantize(x)
    qm, sm = ops.fp4_quantize(x, form="mxfp4")
    off = torch.zeros(3, dtype=I32, **c)
    r = ops.route(x, 2)
    for call in (lambda: ops.route(x.half(), 2), lambda: ops.route(x[0], 2), lambda: ops.route(x, 0), lambda: ops.route(x, 17),
                 lambda: ops.route(x, 2, router="top"), lambda: ops.route(x, 2, bias=w), lambda: ops.route(x.T, 2),
                 lambda: ops.route(x, 2, router="sigmoid_group", bias=w.to(BF16)), lambda: ops.route(x, 2, router="sigmoid_group", n_group=5),
                 lambda: ops.route(x, 2, live=w[:4]), lambda: ops.route(x, 2, live=w[:3].bool()), lambda: ops.route(x, 2, eligible=w[:4].bool()),
                 lambda: ops.route(x, 2, out=r._replace(slots=r.slots[:3])), lambda: ops.route(x, 2, out=r._replace(sel=r.slots)),
                 lambda: ops.combine(x, i.long(), x[:, :2].contiguous()), lambda: ops.combine(x, i, x[:, :2]),
                 lambda: ops.combine(x, i, x[:, :2].contiguous(), residual=x[:3]), lambda: ops.combine(x, i, x[:, :2].contiguous(), out=x),
                 lambda: ops.combine(x, i, x[:, :2].contiguous(), shared=x.to(BF16)), lambda: ops.combine(x.half(), i, x[:, :2].contiguous()),
                 lambda: ops.grouped_matmul(x, x.to(BF16), None), lambda: ops.grouped_matmul(x, x[:, :32], None),
                 lambda: ops.grouped_matmul(x, x[None], off), lambda: ops.grouped_matmul(x, x, off), lambda: ops.grouped_matmul(x, x[None], None),
                 lambda: ops.grouped_matmul(x.half(), x.half(), None), lambda: ops.grouped_matmul(x[:, 1:61], x[:, :60].contiguous(), None),
                 lambda: ops.grouped_matmul(x, x[:3].contiguous(), None, swiglu=True), lambda: ops.grouped_matmul(x, x, None, rows=off.long()),
                 lambda: ops.grouped_matmul(x, x, None, out=x), lambda: ops.grouped_matmul(x, x, None, out_dtype=torch.float16),
                 lambda: ops.fp4_quantize(x, form="fp4"), lambda: ops.fp4_quantize(x[:, :48]), lambda: ops.fp4_quantize(x[:, :63], swiglu=True),
                 lambda: ops.fp4_quantize(x, q=x), lambda: ops.fp4_quantize(x, scales=sm), lambda: ops.fp4_quantize(x, form="mxfp4", tensor_scale=0.5),
                 lambda: ops.fp4_quantize_weight(x.T), lambda: ops.fp4_dequantize(q, sm[:, :3]), lambda: ops.fp4_dequantize(q, s.view(U8)),
                 lambda: ops.fp4_dequantize(q, s, tensor_scale=w[:2]), lambda: ops.fp4_matmul(q, s, qm, sm), lambda: ops.fp4_matmul(q, s, q[:, :16], s),
                 lambda: ops.fp4_matmul(q, s, q[None], s[None]), lambda: ops.fp4_matmul(q, s, q, s, scale=w[:2]),
                 lambda: ops.fp4_matmul(q, s, q, s, out_dtype=torch.float16), lambda: ops.fp4_matmul(x, s, q, s)):
        with pytest.raises((ValueError, RuntimeError)):
            call()
