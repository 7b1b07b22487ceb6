"""The few-token call of a layer (EpochLayer.forward_few) against its formula in
64 bits: sizes, routers, types, exact ties, rows that are not finite, blocks in
progress, streams and graphs, and refusals.

Tolerances count roundings, from the 64-bit values: see _bound."""
import math

import numpy as np
import pytest
import torch

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def Layer():
    from sparse_moe_layer_gate_gb300 import builder
    if builder.is_stale():
        builder.build()
    from sparse_moe_layer_gate_gb300.layer import EpochLayer
    return EpochLayer


def make(Layer, H, E, I, k, dtype, n_shared=0, shared_inter=None, seed=0, max_positions=64, bias_scale=0.3, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = DT[dtype]
    rnd = lambda *s, std: (torch.randn(*s, generator=g, device="cuda") * std).to(d)  # noqa: E731
    w = dict(w_router=rnd(E, H, std=H ** -0.5), b_router=torch.randn(E, generator=g, device="cuda") * bias_scale,
             w_gate=rnd(E, I, H, std=H ** -0.5), w_up=rnd(E, I, H, std=H ** -0.5), w_down=rnd(E, H, I, std=I ** -0.5))
    if n_shared:
        si = shared_inter or I
        w |= dict(ws_gate=rnd(n_shared, si, H, std=H ** -0.5), ws_up=rnd(n_shared, si, H, std=H ** -0.5),
                  ws_down=rnd(n_shared, H, si, std=si ** -0.5))
    lay = Layer(hidden=H, n_experts=E, inter=I, top_k=k, max_positions=max_positions, dtype=dtype, tau=1.0, refresh_R=4,
                weights=w, n_shared=n_shared, shared_inter=shared_inter, **kw)
    return lay, w


def tokens(H, n, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, H, generator=g, device="cuda").to(DT[dtype])


def select64(logits, bias, c):
    """(experts, weights, margin) of one token: margin is the smallest gap that decides the selection."""
    E, k = logits.shape[0], c["top_k"]
    if c.get("router", "softmax") == "softmax":
        v = logits + bias
        order = np.argsort(-v, kind="stable")
        sel = order[:k]
        p = np.exp(v - v.max())
        wgt = p[sel] / (p.sum() if c.get("raw_weights") else p[sel].sum())
        return sel, wgt, (v[order[k - 1]] - v[order[k]] if k < E else math.inf)
    s = 1 / (1 + np.exp(-logits))
    pick, n, top = s + bias, c["n_group"], c["topk_group"]
    gs, margin = E // n, math.inf
    score = np.array([np.sort(pick[i * gs:(i + 1) * gs])[::-1][:2].sum() for i in range(n)])
    order = np.argsort(-score, kind="stable")
    take = min(n, max(top, -(-k // gs)))
    if take < n:
        margin = score[order[take - 1]] - score[order[take]]
    open_ = np.full(E, -np.inf)
    for i in order[:take]:
        open_[i * gs:(i + 1) * gs] = pick[i * gs:(i + 1) * gs]
    order = np.argsort(-open_, kind="stable")
    sel = order[:k]
    if k < take * gs:
        margin = min(margin, open_[order[k - 1]] - open_[order[k]])
    return sel, s[sel] / (1.0 if c.get("raw_weights") else s[sel].sum()), margin


def layer64(w, x, c, dtype):
    """(y, bound, sure): the layer in 64 bits, the error that its roundings allow, and the tokens whose selection no
    rounding can change."""
    H = x.shape[1]
    xd = x.double()
    W = {n: t.double() for n, t in w.items()}
    # A sum over H: a warp holds at most a quarter of it and adds a tensor-core product of 16 columns (truncated to
    # 2^-23 each) or, in fp32, four columns at a time to a thread's own; then the threads and warps meet.
    chain = (H / 64 + 24) * 2.0 ** -23
    logits = xd @ W["w_router"].T
    d_logit = (xd.abs() @ W["w_router"].abs().T).amax(1) * chain + 4 * U
    bias = W["b_router"].cpu().numpy()
    half = torch.finfo(DT[dtype]).eps / 2 if dtype == "bf16" else U

    def expert(v, g, u, d):
        a, b = v @ g.T, v @ u.T
        da, db = (v.abs() @ g.abs().T) * chain, (v.abs() @ u.abs().T) * chain
        act = torch.nn.functional.silu(a) * b
        # silu' <= 1.1; exp, sum, quotient, product: 8 roundings; bf16 layers keep a value in two bf16 parts, so what
        # is lost is half a step of what the first part leaves, itself at most half a step
        e_act = 1.1 * da * b.abs() + torch.nn.functional.silu(a).abs() * db + act.abs() * (8 * U + (U if half == U else half * half))
        # bf16: a warp's part of I (all of it below 512 columns) in products of 16 columns, twice for the two parts
        cols = d.shape[1]
        inner = ((cols / 64 if half == U else max(min(cols, 512), cols / 4) / 8) + 24) * 2.0 ** -23
        return act @ d.T, e_act @ d.abs().T + (act.abs() @ d.abs().T) * inner

    y, err = torch.zeros_like(xd), torch.zeros_like(xd)
    size = torch.zeros_like(xd)
    sure, edges = [], {}
    for t in range(x.shape[0]):
        sel, wgt, margin = select64(logits[t].cpu().numpy(), bias, c)
        if margin > 4 * float(d_logit[t]) + 8 * U or margin == 0:  # an exact tie is decided by the ids
            sure.append(t)
        for e, v in zip(sel, wgt):
            edges.setdefault(int(e), []).append((t, float(v)))
    for e, lst in edges.items():
        t = torch.tensor([i for i, _ in lst], device=x.device)
        v = torch.tensor([u for _, u in lst], device=x.device, dtype=torch.float64).unsqueeze(1)
        o, eo = expert(xd[t], W["w_gate"][e], W["w_up"][e], W["w_down"][e])
        y[t] += v * o
        size[t] += (v * o).abs()
        err[t] += v * eo + (v * o).abs() * (2 * d_logit[t].unsqueeze(1) + 40 * U)  # the weight: exp of a difference of logits
    for j in range(w["ws_gate"].shape[0] if "ws_gate" in w else 0):
        o, eo = expert(xd, W["ws_gate"][j], W["ws_up"][j], W["ws_down"][j])
        y, err, size = y + o, err + eo, size + o.abs()
    if c.get("residual"):
        y, size = y + xd, size + xd.abs()
    return y, err + size * 20 * U + y.abs() * half * (1 + 2 ** -7) + 1e-30, sure


def check(lay, w, x, c, dtype, least=0.9):
    got = lay.forward_few(x)
    y, bound, sure = layer64(w, x, c, dtype)
    assert lay.status() == (0, 0)
    assert len(sure) >= least * x.shape[0]
    d = (got.double() - y).abs()[sure]
    assert bool((d <= bound[sure]).all()), (float((d / bound[sure]).max()), int((d > bound[sure]).sum()))
    return got


BF16 = [dict(H=256, E=4, I=128, top_k=1), dict(H=256, E=16, I=128, top_k=2, n_shared=1),
        dict(H=512, E=256, I=128, top_k=8, n_shared=1), dict(H=2048, E=64, I=256, top_k=8),
        dict(H=256, E=1, I=384, top_k=1, n_shared=2, shared_inter=256), dict(H=768, E=13, I=128, top_k=13),
        dict(H=256, E=1001, I=128, top_k=16, n_shared=1, shared_inter=512), dict(H=1280, E=40, I=640, top_k=4)]
F32 = [dict(H=4, E=2, I=4, top_k=1), dict(H=256, E=16, I=128, top_k=2, n_shared=1), dict(H=100, E=30, I=36, top_k=5),
       dict(H=1020, E=48, I=388, top_k=4, n_shared=1, shared_inter=12), dict(H=68, E=1024, I=20, top_k=16)]


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64])
@pytest.mark.parametrize("i", range(len(BF16)))
def test_bf16_layers(Layer, i, n):
    c = BF16[i]
    lay, w = make(Layer, c["H"], c["E"], c["I"], c["top_k"], "bf16", c.get("n_shared", 0), c.get("shared_inter"), seed=i)
    check(lay, w, tokens(c["H"], n, "bf16", seed=n), c, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3, 8, 9, 17, 40, 64])
@pytest.mark.parametrize("i", range(len(F32)))
def test_f32_layers(Layer, i, n):
    c = F32[i]
    lay, w = make(Layer, c["H"], c["E"], c["I"], c["top_k"], "f32", c.get("n_shared", 0), c.get("shared_inter"), seed=i)
    check(lay, w, tokens(c["H"], n, "f32", seed=n), c, "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", [dict(raw_weights=True), dict(residual=True),
                               dict(router="sigmoid_group", n_group=1, topk_group=1),
                               dict(router="sigmoid_group", n_group=4, topk_group=2, raw_weights=True),
                               dict(router="sigmoid_group", n_group=8, topk_group=3, residual=True),
                               dict(router="sigmoid_group", n_group=16, topk_group=1)])  # 4 experts a group, 6 selected
def test_routers_and_options(Layer, c, dtype):
    lay, w = make(Layer, 512, 64, 128, 6, dtype, 1, seed=5, bias_scale=0.02 if "router" in c else 0.3, **c)
    for n in (1, 12, 50):
        check(lay, w, tokens(512, n, dtype, seed=n), dict(c, top_k=6), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("E,n_group,topk_group,k", [(60, 4, 2, 6), (140, 4, 1, 3), (1001, 7, 3, 8), (96, 32, 5, 8), (35, 5, 1, 7),
                                                    (12, 6, 1, 8), (250, 2, 1, 16), (21, 21, 4, 4)])
def test_groups_of_any_size(Layer, E, n_group, topk_group, k):
    c = dict(router="sigmoid_group", n_group=n_group, topk_group=topk_group)
    lay, w = make(Layer, 256, E, 128, k, "bf16", seed=E, bias_scale=0.02, **c)
    for n in (1, 16, 33):
        check(lay, w, tokens(256, n, "bf16", seed=n), dict(c, top_k=k), "bf16", least=0.8)


@pytest.mark.gpu
@pytest.mark.parametrize("router", ["softmax", "sigmoid_group"])
def test_exact_ties_go_to_the_lower_expert(Layer, router):
    """x = 0: every logit is its bias, in groups of four equal values."""
    c = dict(router=router, n_group=4, topk_group=2) if router != "softmax" else dict(router=router)
    lay, w = make(Layer, 256, 32, 128, 6, "f32", seed=3, residual=True, **c)
    w["b_router"].copy_(-torch.div(torch.arange(32, device="cuda"), 4, rounding_mode="floor").float() * 0.125)
    # experts that are selected are told apart by a gate that does not vanish at x = 0: make x tiny instead
    x = torch.zeros(5, 256, device="cuda")
    x[:, 0] = 2.0 ** -20
    w["w_router"][:, 0] = 0
    w["w_gate"][:, :, 0] *= 2.0 ** 20
    w["w_up"][:, :, 0] *= 2.0 ** 20
    check(lay, w, x, dict(c, top_k=6, residual=True), "f32", least=1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_row_that_is_not_finite_stays_alone(Layer, dtype, bad):
    lay, w = make(Layer, 256, 32, 128, 4, dtype, 1, seed=2)
    x = tokens(256, 11, dtype)
    want = lay.forward_few(x)
    x2 = x.clone()
    x2[4, 9] = bad
    got = lay.forward_few(x2)
    keep = [t for t in range(11) if t != 4]
    assert torch.equal(got[keep], want[keep])
    assert not bool(got[4].isfinite().any())
    assert torch.equal(lay.forward_few(x), want)  # nothing of it stays behind


@pytest.mark.gpu
def test_all_tokens_on_the_same_experts(Layer):
    """A bias that sends every token to one set of experts: more tokens on an expert than one pass holds."""
    for dtype in ("bf16", "f32"):
        lay, w = make(Layer, 256, 24, 128, 3, dtype, seed=8)
        w["b_router"].copy_(torch.where(torch.arange(24, device="cuda") % 7 == 2, 60.0, 0.0))
        for n in (33, 64):
            check(lay, w, tokens(256, n, dtype, seed=n), dict(top_k=3), dtype, least=0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_every_time_and_alone_or_together(Layer, dtype):
    """Sums are in a fixed order, and a token's result does not depend on its neighbours'."""
    lay, w = make(Layer, 512, 48, 128, 4, dtype, 1, seed=4)
    x = tokens(512, 29, dtype)
    first = lay.forward_few(x)
    for _ in range(4):
        assert torch.equal(lay.forward_few(x), first)
    for t in (0, 13, 28):
        assert torch.equal(lay.forward_few(x[t:t + 1].contiguous()), first[t:t + 1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_block_in_progress_is_left_alone(Layer, dtype):
    def block(few):
        lay, _ = make(Layer, 256, 16, 128, 2, dtype, 1, seed=6)
        x = tokens(256, 64, dtype)
        live = torch.ones(64, dtype=torch.uint8, device="cuda")
        dec = torch.zeros(64, dtype=torch.uint8, device="cuda")
        out = []
        lay.plan_block(x)
        for i in range(5):
            if few:
                lay.forward_few(x[:7].contiguous())
            out.append(lay.moe_iter(x, live, dec, i).clone())
            live[i * 8:(i + 1) * 8] = 0
            dec[i * 8:(i + 1) * 8] = 1
        st = lay.stats()
        counters = lay.path_counters()
        return out, st, counters

    a, b = block(False), block(True)
    assert all(torch.equal(p, q) for p, q in zip(a[0], b[0]))
    assert a[1:] == b[1:]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,tol", [("bf16", 1e-2), ("f32", 1e-5)])
def test_agrees_with_a_full_fresh_iteration(Layer, dtype, tol):
    """moe_iter without a plan runs every position over every expert: the same layer, to the tolerance of its tests."""
    lay, _ = make(Layer, 512, 32, 128, 4, dtype, 1, seed=9, residual=True)
    x = tokens(512, 32, dtype)
    few = lay.forward_few(x).float()
    live = torch.ones(32, dtype=torch.uint8, device="cuda")
    it = lay.moe_iter(x, live, 1 - live, 0).float()
    assert float((few - it).abs().max()) <= tol * float(it.abs().max())


@pytest.mark.gpu
def test_streams_graphs_and_outputs(Layer):
    lay, w = make(Layer, 512, 32, 128, 4, "bf16", 1, seed=10)
    x = tokens(512, 9, "bf16")
    want = lay.forward_few(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lay.forward_few(x, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    torch.cuda.current_stream().wait_stream(side)
    y = torch.full((11, 512), 3.0, device="cuda", dtype=torch.bfloat16)
    assert lay.forward_few(x, y=y[1:10]).data_ptr() == y[1:10].data_ptr()
    assert torch.equal(y[1:10], want) and bool((y[[0, 10]] == 3).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mid = lay.forward_few(x)
        out = lay.forward_few(mid)
    for seed in (1, 2, 3):
        x.copy_(tokens(512, 9, "bf16", seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        assert torch.equal(replayed, lay.forward_few(lay.forward_few(x)))
    assert lay.forward_few(x[:0]).shape == (0, 512)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 20])
def test_in_place(Layer, dtype, n):
    lay, _ = make(Layer, 512, 32, 128, 4, dtype, 1, seed=12, residual=True)
    x = tokens(512, n, dtype)
    want = lay.forward_few(x)
    assert lay.forward_few(x, y=x) is x
    assert torch.equal(x, want)


@pytest.mark.gpu
def test_two_layers_and_two_graphs_of_one_layer(Layer):
    """Two layers overlap on two streams; two graphs of one layer, replayed one after the other, share its workspace."""
    a, _ = make(Layer, 512, 32, 128, 4, "bf16", 1, seed=13)
    b, _ = make(Layer, 1024, 16, 256, 2, "bf16", 0, seed=14)
    xa, xb = tokens(512, 30, "bf16"), tokens(1024, 5, "bf16")
    wa, wb = a.forward_few(xa), b.forward_few(xb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ya, yb = [], []
    for _ in range(10):
        ya.append(a.forward_few(xa, stream=sa))
        yb.append(b.forward_few(xb, stream=sb))
    torch.cuda.synchronize()
    assert all(torch.equal(y, wa) for y in ya) and all(torch.equal(y, wb) for y in yb)
    assert a.status() == (0, 0) and b.status() == (0, 0)
    graphs = []
    for n in (3, 30):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = a.forward_few(xa[:n])
        graphs.append((g, y, n))
    for _ in range(3):
        for g, y, n in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, wa[:n])


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported_and_cleared(Layer):
    """A limit of a microsecond lets the grid barriers give up; the call returns, the status says so, and after
    clearing it the layer works as before."""
    lay, w = make(Layer, 2048, 64, 512, 8, "bf16", 1, seed=11)
    x = tokens(2048, 32, "bf16")
    want = lay.forward_few(x)
    lay.set_wait_timeout(1000)
    for _ in range(3):
        got = lay.forward_few(x)
        code, word = lay.status()
        assert (code, word) in ((0, 0), (4, 2))  # EPOCH_ETIMEOUT, EPOCH_DEVERR_TIMEOUT
        if code == 0:
            assert torch.equal(got, want)
        lay.clear_status()
    lay.set_wait_timeout(2_000_000_000)
    assert torch.equal(lay.forward_few(x), want)
    assert lay.status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,barriers", [(1, (0, 2, 3)), (16, (0, 2, 3)), (40, (0, 1, 2, 3))])
def test_every_barriers_wait_can_run_out(Layer, dtype, n, barriers):
    """A barrier that waits for an arrival that never comes gives up after the limit: the call returns, the status
    says so, and after clearing it the layer gives the same bits as before."""
    from sparse_moe_layer_gate_gb300 import binding as B
    lay, _ = make(Layer, 512, 32, 128, 4, dtype, 1, seed=15)
    x = tokens(512, n, dtype)
    want, y = lay.forward_few(x), torch.empty_like(x)
    assert lay.status() == (0, 0)
    stream = torch.cuda.current_stream().cuda_stream
    lay.set_wait_timeout(1_000_000)
    for b in barriers:
        assert B.lib().epoch_test_few_timeout(lay.handle, x.data_ptr(), n, y.data_ptr(), b, stream) == B.EPOCH_OK
        assert lay.status() == (4, 2)  # EPOCH_ETIMEOUT, EPOCH_DEVERR_TIMEOUT
        assert lay.status() == (4, 2)  # until it is cleared
        lay.clear_status()
        assert torch.equal(lay.forward_few(x), want)
        assert lay.status() == (0, 0)
    for b in (-1, 4) + (() if n > 16 else (1,)):
        assert B.lib().epoch_test_few_timeout(lay.handle, x.data_ptr(), n, y.data_ptr(), b, stream) == B.EPOCH_EINVAL
    assert B.lib().epoch_test_few_timeout(None, x.data_ptr(), n, y.data_ptr(), 0, stream) == B.EPOCH_EINVAL


@pytest.mark.gpu
def test_refusals(Layer):
    lay, _ = make(Layer, 256, 16, 128, 2, "bf16", max_positions=20)
    x = tokens(256, 64, "bf16")
    from sparse_moe_layer_gate_gb300 import binding as B
    for bad in (x[:21], x):  # more than max_positions
        with pytest.raises(B.EpochError):
            lay.forward_few(bad.contiguous())
    big, _ = make(Layer, 256, 16, 128, 2, "bf16", max_positions=100)
    with pytest.raises(B.EpochError):
        big.forward_few(tokens(256, 65, "bf16"))
    for bad in (x[:4].float(), x[:4, :128], x[:4].cpu(), x[:8:2], x[0]):
        with pytest.raises(ValueError):
            lay.forward_few(bad)
    with pytest.raises(ValueError):
        lay.forward_few(x[:4], y=x[4:7])
    with pytest.raises(ValueError):  # overlaps x without being x
        lay.forward_few(x[:4], y=x[3:7])
    h, L = lay.handle, B.lib()
    p = x.data_ptr()
    assert L.epoch_moe_few(None, p, 4, p + 8192, None) == B.EPOCH_EINVAL
    for args in ((None, 4, p), (p, 4, None), (p + 2, 4, p), (p, 4, p + 8), (p, -1, p)):
        assert L.epoch_moe_few(h, args[0], args[1], args[2], None) == B.EPOCH_EINVAL


@pytest.mark.gpu
def test_a_y_that_overlaps_x_is_refused_by_the_abi(Layer):
    from sparse_moe_layer_gate_gb300 import binding as B
    lay, _ = make(Layer, 256, 16, 128, 2, "bf16")
    buf = torch.zeros(20, 256, device="cuda", dtype=torch.bfloat16)
    p, row = buf.data_ptr(), 512
    for x, y in ((p, p + row), (p + 16, p), (p, p + 4 * row - 16), (p + 3 * row, p)):
        assert B.lib().epoch_moe_few(lay.handle, x, 4, y, None) == B.EPOCH_EINVAL
    for x, y in ((p, p), (p, p + 4 * row), (p + 4 * row, p)):
        assert B.lib().epoch_moe_few(lay.handle, x, 4, y, None) == B.EPOCH_OK
    torch.cuda.synchronize()
    assert lay.status() == (0, 0)


def test_a_null_layer_is_refused_on_the_host():
    from sparse_moe_layer_gate_gb300 import binding as B, builder
    if builder.is_stale():
        builder.build()
    assert B.lib().epoch_moe_few(None, 256, 1, 512, None) == B.EPOCH_EINVAL
