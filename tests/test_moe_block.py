"""The operators together, as a model runs them: a decoder's MoE block for a few
tokens (norm before, the layer, norm after), and a layer's routed experts in FP8
over the worklist that the layer's own routing made. Each against the formulas in
64 bits; bounds are the sums of the stages' roundings."""
import pytest
import torch

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def mod():
    from sparse_moe_layer_gate_gb300 import builder
    if builder.is_stale():
        builder.build()
    from sparse_moe_layer_gate_gb300 import layer, ops
    return layer, ops


def build(layer, H, E, I, k, n_shared, dtype, seed, max_positions=64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = {"bf16": BF16, "f32": F32}[dtype]
    rnd = lambda *s, std: (torch.randn(*s, generator=g, device="cuda") * std).to(d)  # noqa: E731
    w = dict(w_router=rnd(E, H, std=H ** -0.5), b_router=0.1 * torch.randn(E, generator=g, device="cuda"),
             w_gate=rnd(E, I, H, std=H ** -0.5), w_up=rnd(E, I, H, std=H ** -0.5), w_down=rnd(E, H, I, std=I ** -0.5))
    if n_shared:
        w |= dict(ws_gate=rnd(n_shared, I, H, std=H ** -0.5), ws_up=rnd(n_shared, I, H, std=H ** -0.5),
                  ws_down=rnd(n_shared, H, I, std=I ** -0.5))
    return layer.EpochLayer(hidden=H, n_experts=E, inter=I, top_k=k, n_shared=n_shared, max_positions=max_positions,
                            dtype=dtype, tau=1.0, refresh_R=None, weights=w), w, g


def rms(x, w):
    return x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-6) * w


def moe64(h, w, k):
    """The layer of h in 64 bits, and the sum of its terms' magnitudes."""
    W = {n: t.double() for n, t in w.items()}
    logits = h @ W["w_router"].T + W["b_router"]
    val, sel = logits.topk(k, dim=1)
    wgt = torch.softmax(val, dim=1)
    gap = val[:, -1] - torch.where(torch.zeros_like(logits).scatter_(1, sel, 1).bool(), -float("inf"), logits).amax(1)
    y, size = torch.zeros_like(h), torch.zeros_like(h)
    for t in range(h.shape[0]):
        for j in range(k):
            e = int(sel[t, j])
            a = torch.nn.functional.silu(W["w_gate"][e] @ h[t]) * (W["w_up"][e] @ h[t])
            o = W["w_down"][e] @ a
            y[t] += wgt[t, j] * o
            size[t] += wgt[t, j] * (W["w_down"][e].abs() @ a.abs())
        for s in range(w["ws_gate"].shape[0] if "ws_gate" in w else 0):
            a = torch.nn.functional.silu(W["ws_gate"][s] @ h[t]) * (W["ws_up"][s] @ h[t])
            y[t] += W["ws_down"][s] @ a
            size[t] += W["ws_down"][s].abs() @ a.abs()
    return y, size, gap


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 6, 33])
def test_a_decoders_block(mod, dtype, n):
    """h = norm(r); b = layer(h); r' = 0.9 r + sigmoid(g) norm(b); h' = norm(r'), captured and replayed, against the
    stages in 64 bits from the rounded values that each stage was given."""
    layer, ops = mod
    H, k = 512, 4
    lay, w, g = build(layer, H, 32, 128, k, 1, dtype, seed=n)
    half = torch.finfo(BF16).eps / 2 if dtype == "bf16" else U
    d = BF16 if dtype == "bf16" else F32
    near = lambda: 1 + 0.1 * torch.randn(H, generator=g, device="cuda")  # noqa: E731
    w1, w2, w3, gate = near(), near(), near(), torch.randn(H, generator=g, device="cuda")
    r = torch.randn(n, H, generator=g, device="cuda") * 2

    def block():
        h = ops.norm_before(r, w1, out_dtype=d)
        b = lay.forward_few(h)
        return h, b, *ops.norm_after(b, r, w2, gate=gate, gate_sigmoid=True, residual_scale=0.9, next_weight=w3)

    eager = block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, b, r2, h2 = block()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(eager, (h, b, r2, h2)):
        assert torch.equal(x, y)
    want = rms(r.double(), w1.double())
    assert bool(((h.double() - want).abs() <= want.abs() * (half + 40 * U)).all())
    y, size, gap = moe64(h.double(), w, k)
    keep = gap > 1e-4  # a selection that no rounding of a logit (2e-5 here) can change
    assert int(keep.sum()) >= 0.9 * n
    # the activation's rounding on every term (bf16: to two parts), sums of 512 (2^-23 a step of 16 columns, both
    # products, the second of both parts) and y's rounding
    bound = size * ((half * half if dtype == "bf16" else U) + 300 * U) + y.abs() * half * (1 + 2 ** -7)
    # gate and up sums of an activation: 64 roundings of terms whose sizes add up to at most 16 times the sum's scale
    bound = bound + size * 16 * 64 * U
    assert bool(((b.double() - y).abs() <= bound)[keep].all()), float(((b.double() - y).abs() / bound)[keep].max())
    z = rms(b.double(), w2.double()) * torch.sigmoid(gate.double())
    want = 0.9 * r.double() + z
    size = (0.9 * r.double()).abs() + z.abs()
    assert bool(((r2.double() - want).abs() <= size * 60 * U).all())
    nxt = rms(want, w3.double())
    scale = (1 / torch.sqrt(want.square().mean(1, keepdim=True) + 1e-6)) * w3.double().abs()
    assert bool(((h2.double() - nxt).abs() <= nxt.abs() * (half + 100 * U) + size * scale * 60 * U).all())


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 7, 64, 512])
def test_routed_experts_in_fp8_over_the_layers_worklist(mod, n):
    layer, ops = mod
    H, E, I, k = 512, 24, 256, 3
    lay, w, g = build(layer, H, E, I, k, 0, "bf16", seed=n, max_positions=512)
    x = torch.randn(n, H, generator=g, device="cuda").to(BF16)
    live = torch.ones(n, dtype=torch.uint8, device="cuda")
    routed = lay.moe_iter(x, live, 1 - live, 0).double()  # no plan: every position over every expert
    positions, offsets = lay.worklist()
    edges = n * k
    assert int(offsets[-1]) == edges and positions.shape == (512 * k,)
    w13, s13 = ops.fp8_quantize_weight(torch.cat([w["w_gate"], w["w_up"]], 1))  # [E, 2 I, H]
    w2, s2 = ops.fp8_quantize_weight(w["w_down"])
    rows = positions[:edges]
    q, s = ops.fp8_quantize(x, rows=rows)
    gu = ops.fp8_matmul(q, s, w13, s13, offsets=offsets)
    qa, sa = ops.fp8_quantize(gu, swiglu=True)
    o = ops.fp8_matmul(qa, sa, w2, s2, offsets=offsets, out_dtype=F32)
    assert ops.status() == (0, 0) and lay.status() == (0, 0)
    # stage by stage in 64 bits, from the values that each stage was given
    wide = lambda t, s, r: t.double() * s.double().repeat_interleave(128, -1).repeat_interleave(r, -2)[..., :t.shape[-2], :t.shape[-1]]  # noqa: E731
    off = offsets.tolist()
    assert torch.equal(q.view(torch.uint8), ops.fp8_quantize(x[rows.long()].contiguous())[0].view(torch.uint8))
    a1, b1, a2, b2 = wide(q, s, 1), wide(w13, s13, 128), wide(qa, sa, 1), wide(w2, s2, 128)
    act = torch.nn.functional.silu(gu[:, :I].double()) * gu[:, I:].double()
    sk = sa.double().repeat_interleave(128, 1)[:, :I]
    assert bool(((a2 - act).abs() <= act.abs() * (2 ** -4 + 20 * U) + sk * 2 ** -10 * (1 + 20 * U)).all())
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        want, size = a1[lo:hi] @ b1[e].T, a1[lo:hi].abs() @ b1[e].abs().T
        assert bool(((gu[lo:hi].double() - want).abs() <= size * 140 * 2.0 ** -23 + want.abs() * 2 ** -8 * (1 + 2 ** -7) + 1e-30).all())
        want, size = a2[lo:hi] @ b2[e].T, a2[lo:hi].abs() @ b2[e].abs().T
        assert bool(((o[lo:hi].double() - want).abs() <= size * 140 * 2.0 ** -23 + 1e-30).all())
    # the whole against the bf16 layer: weighted sums of the edges, within what e4m3 (2^-4 on each of four operands,
    # independent: 2-norm) leaves of it
    logits = x.double() @ w["w_router"].double().T + w["b_router"].double()
    val, sel = logits.topk(k, dim=1)
    wgt = torch.softmax(val, dim=1)
    expert = torch.bucketize(torch.arange(edges, device="cuda"), offsets[1:].long(), right=True)
    dense = torch.zeros(n, E, device="cuda", dtype=torch.float64).scatter_(1, sel, wgt)
    y = torch.zeros(n, H, device="cuda", dtype=torch.float64)
    y.index_add_(0, rows.long(), o.double() * dense[rows.long(), expert].unsqueeze(1))
    assert float((y - routed).norm() / routed.norm()) <= 2 * 2.0 ** -4
