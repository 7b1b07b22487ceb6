"""Edges of the experts' operators that their own sizes pass over, against forms in 64 bits."""
import numpy as np
import pytest
import torch

from test_experts import BF16, F32, I32, _gen, _rnd, check_route, ops, route64  # noqa: F401


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
