"""Edges of the experts' operators that their own sizes pass over, against forms in 64 bits."""
import pytest
import torch

from test_experts import F32, I32, _gen, _rnd, check_route, ops, route64  # noqa: F401


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
