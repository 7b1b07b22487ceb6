"""Layers with the sigmoid router whose logits all lie where fp32's sigmoids are subnormal or nothing: the weights, quotients
of them, are ordinary numbers. The few-token call against 64 bits, an iteration of a block against that call."""
import pytest
import torch

from test_few import DT, Layer, check, make, tokens  # noqa: F401


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("low", [-30.0, -96.0, -150.0])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_layers_of_low_logits(Layer, dtype, low, groups, top):
    H, E, k, n = 256, 64, 6, 33
    c = dict(router="sigmoid_group", n_group=groups, topk_group=top)
    _, w = make(Layer, H, E, 128, k, dtype, 1, seed=3, **c)
    w["w_router"][:, 0] = low
    lay = Layer(hidden=H, n_experts=E, inter=128, top_k=k, max_positions=64, dtype=dtype, tau=1.0, refresh_R=4, weights=w, n_shared=1, **c)
    x = tokens(H, n, dtype)
    x[:, 0] = 1.0
    few = check(lay, w, x, dict(c, top_k=k), dtype, least=0.8)
    assert bool(few.isfinite().all())
    flags = torch.ones(n, dtype=torch.uint8, device="cuda")
    lay.plan_block(x)
    y = lay.moe_iter(x, flags, torch.zeros_like(flags), 0)
    lay.block_end()
    assert lay.status() == (0, 0)
    # a block's iteration: bf16 activations between its two products, and logits that another order of sums moves a little
    assert bool(((y.double() - few.double()).abs() <= (2e-2 if dtype == "bf16" else 1e-3) * few.double().abs().max()).all())
