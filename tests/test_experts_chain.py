"""A layer run in parts, as a model uses the operators together: router, the experts' products over the worklist (bf16,
fp32, FP8 or 4-bit operands), the shared expert, the sum of the edges with the residual stream; against the formulas in
64 bits and against the layer itself. Bounds are the sums of the stages' roundings."""
import pytest
import torch

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24


@pytest.fixture(scope="module")
def mod():
    from sparse_moe_layer_gate_gb300 import builder
    if builder.is_stale():
        builder.build()
    from sparse_moe_layer_gate_gb300 import layer, ops
    return layer, ops


def weights(seed, H, E, I, dtype, shared=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, std: (torch.randn(*s, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
    w = dict(w_router=rnd(E, H, std=H ** -0.5), b_router=0.1 * torch.randn(E, generator=g, device="cuda"),
             w_gate=rnd(E, I, H, std=H ** -0.5), w_up=rnd(E, I, H, std=H ** -0.5), w_down=rnd(E, H, I, std=I ** -0.5))
    if shared:
        w |= dict(ws_gate=rnd(shared, I, H, std=H ** -0.5), ws_up=rnd(shared, I, H, std=H ** -0.5), ws_down=rnd(shared, H, I, std=I ** -0.5))
    return w, g


def moe64(x, w, sel, wgt):
    """Routed and shared experts of given selections in 64 bits, and the sum of the magnitudes of the down products' terms."""
    X, y, size = x.double(), torch.zeros_like(x, dtype=F64), torch.zeros_like(x, dtype=F64)
    swiglu = lambda v, a, b: torch.nn.functional.silu(v @ a.double().T) * (v @ b.double().T)  # noqa: E731
    for e in range(w["w_gate"].shape[0]):
        t, j = (sel == e).nonzero(as_tuple=True)
        if t.numel():
            a, f = swiglu(X[t], w["w_gate"][e], w["w_up"][e]), wgt[t, j].double().unsqueeze(1)
            y.index_add_(0, t, f * (a @ w["w_down"][e].double().T))
            size.index_add_(0, t, f * (a.abs() @ w["w_down"][e].double().abs().T))
    for s in range(w["ws_gate"].shape[0] if "ws_gate" in w else 0):
        a = swiglu(X, w["ws_gate"][s], w["ws_up"][s])
        y += a @ w["ws_down"][s].double().T
        size += a.abs() @ w["ws_down"][s].double().abs().T
    return y, size


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 6, 33, 700])
@pytest.mark.parametrize("router", ["softmax", "sigmoid_group"])
def test_a_layer_in_parts(mod, dtype, n, router):
    """y = x + shared(x) + sum_j w_j E_j(x), captured and replayed, with some positions dead."""
    layer, ops = mod
    H, E, I, k = 512, 32, 128, 4
    w, g = weights(n, H, E, I, dtype)
    x = torch.randn(n, H, generator=g, device="cuda").to(dtype)
    live = (torch.rand(n, generator=g, device="cuda") < 0.8).to(torch.uint8)
    w13 = torch.cat([w["w_gate"], w["w_up"]], 1).contiguous()
    s13 = torch.cat([w["ws_gate"], w["ws_up"]], 1)[0].contiguous()
    kw = dict(router=router) if router == "softmax" else dict(router=router, bias=w["b_router"], n_group=4, topk_group=2)
    logits = (x.float() @ w["w_router"].float().T + (w["b_router"] if router == "softmax" else 0.0)).contiguous()

    def run():
        r = ops.route(logits, k, live=live, **kw)
        a = ops.grouped_matmul(x, w13, r.offsets, rows=r.positions, swiglu=True)
        o = ops.grouped_matmul(a, w["w_down"], r.offsets, out_dtype=F32)
        sh = ops.grouped_matmul(ops.grouped_matmul(x, s13, None, swiglu=True), w["ws_down"][0], None, out_dtype=F32)
        return (*r, o, sh, ops.combine(o, r.slots, r.weights, shared=sh, residual=x))

    eager = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    graph.replay()
    torch.cuda.synchronize()
    edges = int(eager[3][-1])
    assert edges == k * int(live.sum()) and int(out[3][-1]) == edges
    for a, b in zip(eager[:5], out[:5]):
        assert torch.equal(a, b)
    assert torch.equal(eager[5][:edges], out[5][:edges]) and torch.equal(eager[-1], out[-1])
    assert out[-1].dtype == dtype and ops.status() == (0, 0)
    y, size = moe64(x, w, eager[0].long(), eager[1])
    half = torch.finfo(BF16).eps / 2 if dtype == BF16 else U
    # the activation's rounding and its error before it (gate and up sums of 512 columns: 64 roundings of terms that add up
    # to at most 16 times their scale) on every term, sums of 128 and of 4 + 2 terms, y's rounding
    bound = size * (half * (1 + 2 ** -7) + (16 * (512 if dtype == F32 else 64) + 300) * U) + (y + x.double()).abs() * half * (1 + 2 ** -7)
    assert bool(((out[-1].double() - x.double() - y).abs() <= bound).all())
    dead = live == 0
    if bool(dead.any()):  # nothing but the shared expert and the residual
        want = out[6][dead].double() + x[dead].double()
        size = out[6][dead].double().abs() + x[dead].double().abs()
        assert bool(((out[-1][dead].double() - want).abs() <= size * 4 * U + want.abs() * half * (1 + 2 ** -7)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 20, 64])
def test_the_parts_against_the_layers_few_tokens(mod, n):
    layer, ops = mod
    H, E, I, k = 512, 32, 128, 4
    w, g = weights(n + 7, H, E, I, BF16)
    lay = layer.EpochLayer(hidden=H, n_experts=E, inter=I, top_k=k, n_shared=1, max_positions=64, dtype="bf16", tau=1.0,
                           refresh_R=None, weights=w)
    x = torch.randn(n, H, generator=g, device="cuda").to(BF16)
    want = lay.forward_few(x).double()
    logits = (x.double() @ w["w_router"].double().T + w["b_router"].double()).float()
    r = ops.route(logits, k)
    a = ops.grouped_matmul(x, torch.cat([w["w_gate"], w["w_up"]], 1).contiguous(), r.offsets, rows=r.positions, swiglu=True, out_dtype=BF16)
    o = ops.grouped_matmul(a, w["w_down"], r.offsets, out_dtype=F32)
    sa = ops.grouped_matmul(x, torch.cat([w["ws_gate"], w["ws_up"]], 1)[0].contiguous(), None, swiglu=True)
    y = ops.combine(o, r.slots, r.weights, shared=ops.grouped_matmul(sa, w["ws_down"][0], None, out_dtype=F32), out_dtype=BF16)
    # one activation in bf16 (the layer keeps two parts): 2^-9 root mean square of independent roundings of 128 terms,
    # and both results' own rounding
    assert float((y.double() - want).norm() / want.norm()) <= 3 * 2.0 ** -9


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 33, 512])
def test_the_fp8_chain_ends_in_y(mod, n):
    layer, ops = mod
    H, E, I, k = 512, 24, 256, 3
    w, g = weights(n, H, E, I, BF16, shared=0)
    x = torch.randn(n, H, generator=g, device="cuda").to(BF16)
    logits = (x.float() @ w["w_router"].float().T + w["b_router"]).contiguous()
    r = ops.route(logits, k)
    w13, s13 = ops.fp8_quantize_weight(torch.cat([w["w_gate"], w["w_up"]], 1).contiguous())
    w2, s2 = ops.fp8_quantize_weight(w["w_down"])
    q, s = ops.fp8_quantize(x, rows=r.positions)
    q, s = ops.fp8_quantize(ops.fp8_matmul(q, s, w13, s13, offsets=r.offsets), swiglu=True)
    y = ops.combine(ops.fp8_matmul(q, s, w2, s2, offsets=r.offsets, out_dtype=F32), r.slots, r.weights)
    want, _ = moe64(x, w, r.sel.long(), r.weights)
    # e4m3's 2^-4 on each of four operands, independent
    assert float((y.double() - want).norm() / want.norm()) <= 2 * 2.0 ** -4


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("n", [1, 33, 512])
def test_four_bit_experts(mod, form, n):
    """Stage by stage in 64 bits from the values that each stage was given, and the fused SwiGLU against the quantiser's."""
    layer, ops = mod
    H, E, I, k = 512, 24, 256, 3
    w, g = weights(n, H, E, I, BF16, shared=0)
    x = torch.randn(n, H, generator=g, device="cuda").to(BF16)
    r = ops.route((x.float() @ w["w_router"].float().T + w["b_router"]).contiguous(), k)
    w13, s13, t13 = ops.fp4_quantize_weight(torch.cat([w["w_gate"], w["w_up"]], 1).contiguous(), form=form)
    w2, s2, t2 = ops.fp4_quantize_weight(w["w_down"], form=form)
    q, s = ops.fp4_quantize(x, form=form, rows=r.positions)
    assert torch.equal(q, ops.fp4_quantize(x[r.positions.long()].contiguous(), form=form)[0])
    gu = ops.fp4_matmul(q, s, w13, s13, offsets=r.offsets, scale=t13, out_dtype=F32)
    fused = ops.fp4_matmul(q, s, w13, s13, offsets=r.offsets, scale=t13, swiglu=True, out_dtype=F32)
    gate, up = gu.double().chunk(2, 1)
    act = torch.nn.functional.silu(gate) * up
    assert bool(((fused.double() - act).abs() <= act.abs() * 2.0 ** -19 + 1e-30).all())  # of the same sums: exp and quotient
    q2, sc2 = ops.fp4_quantize(fused, form=form)
    o = ops.fp4_matmul(q2, sc2, w2, s2, offsets=r.offsets, scale=t2, out_dtype=F32)
    y = ops.combine(o, r.slots, r.weights)
    off = r.offsets.tolist()
    back = lambda q, s, t=1.0: ops.fp4_dequantize(q, s, tensor_scale=t, out_dtype=F32).double()  # noqa: E731
    a1, b1, a2, b2 = back(q, s), back(w13, s13, t13), back(q2, sc2), back(w2, s2, t2)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        for got, a, b in ((gu, a1, b1), (o, a2, b2)):
            want, size = a[lo:hi] @ b[e].T, a[lo:hi].abs() @ b[e].abs().T
            assert bool(((got[lo:hi].double() - want).abs() <= size * 40 * 2.0 ** -23 + 1e-30).all())
    rows = o.double()[r.slots.long()] * r.weights.double().unsqueeze(2)
    assert bool(((y.double() - rows.sum(1)).abs() <= rows.abs().sum(1) * 6 * U).all())
    # the whole: e2m1 rounds by a quarter at most (between 1 and 1.5 a half step is 0.25), a tenth root mean square, on each of
    # four operands
    want, _ = moe64(x, w, r.sel.long(), r.weights)
    assert float((y.double() - want).norm() / want.norm()) <= 0.4
