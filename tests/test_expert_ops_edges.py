"""Inputs of the FP8 expert operators where a shortcut can go wrong: routing rows whose
fp32 scores do not decide, and grouping in clusters of every size.

References and tolerances as in test_expert_ops.py.
"""

import numpy as np
import pytest
import torch

import expert_ops_reference as R
from moe_decode_router_gb300 import flint_moe as F
from test_expert_ops import check_route, dev, gen, gpu

# ------------------------------------------------------------------ groups whose two best cancel


@gpu
@pytest.mark.parametrize("softmax", [False, True])
def test_route_group_sum_cancels(softmax):
    """Two keys of opposite sign leave a small sum; what fp32 lost in the keys is as large as
    the difference between the groups."""
    d = dev()
    x = torch.tensor([[-0.80, 0.58, 0.37, -0.58]], device=d)
    b = torch.tensor([1e4, -1e4, 0.0, 0.0], device=d)
    check_route(x, 2, bias=b, softmax=softmax, n_groups=2, top_groups=1, top2=True)


@gpu
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("size", [4.0, 64.0, 1e4, 1e8])
@pytest.mark.parametrize("E,G,top,k", [(16, 8, 3, 4), (256, 8, 4, 8), (160, 8, 3, 6), (96, 4, 1, 5), (64, 32, 3, 6)])
def test_route_biases_of_both_signs(softmax, size, E, G, top, k):
    """Every group has one expert forced by a large bias, one let through by its negative and
    the rest forbidden, so that each group's sum is that of two scores."""
    d = dev()
    T = 400
    g = gen(E + G)
    x = (0.02 * torch.randn(T, E, generator=g)).to(d)
    b = torch.full((G, E // G), -3 * size)
    b[:, 0], b[:, -1] = size, -size
    b = b.reshape(-1).to(d)
    check_route(x, k, bias=b, softmax=softmax, n_groups=G, top_groups=top, top2=True)
    mixed = (size * torch.randint(-1, 2, (E,), generator=g)).to(d)
    check_route(x, k, bias=mixed, softmax=softmax, n_groups=G, top_groups=top, top2=True)


@gpu
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E,G", [(16, 2), (64, 8), (160, 8)])
def test_route_group_sum_beyond_fp32(softmax, E, G):
    """Biases of the type's lowest value: the sum of two lies beyond fp32, but the group still
    has candidates and comes before one that has none."""
    d = dev()
    low = torch.finfo(torch.float32).min
    size = E // G
    x = torch.randn(6, E, generator=gen(E))
    b = torch.full((E,), low)
    x[0, :size] = -float("inf")           # group 0 has no candidate
    x[1, :(G - 1) * size] = -float("inf")  # only the last group has
    x[2, size:] = float("nan")             # only the first has
    check_route(x.to(d), 2, bias=b.to(d), softmax=softmax, n_groups=G, top_groups=1, top2=True)
    b[-size:] = low / 2 * 1.5              # the last group's sum is the larger one, both beyond fp32
    check_route(x.to(d), 2, bias=b.to(d), softmax=softmax, n_groups=G, top_groups=1, top2=True)
    check_route(x.to(d), 2, bias=-b.to(d), softmax=softmax, n_groups=G, top_groups=1, top2=True)


# ------------------------------------------------------------------ more equal candidates than lanes


@gpu
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E,odd", [(64, 40), (64, 63), (200, 33), (256, 255), (512, 300), (1024, 1023)])
def test_route_best_behind_many_equal_ones(softmax, E, odd):
    """One expert that fp32 cannot tell from the others, and that comes before them, at an index
    behind the 32 that a warp looks at; by its bias, and by its logit."""
    d = dev()
    for k in (1, 8, 16):
        x, b = torch.zeros(3, E), torch.zeros(E)
        b[odd] = 1e-9
        x[1] = 0.75
        x[2] = -3.0
        check_route(x.to(d), k, bias=b.to(d), softmax=softmax)
        check_route(x.to(torch.bfloat16).to(d), k, bias=b.to(d), softmax=softmax)
        check_route(x.to(d), k, bias=-b.to(d), softmax=softmax)
        x = torch.zeros(2, E)
        x[0, odd], x[1, odd] = 1e-9, -1e-9
        check_route(x.to(d), k, bias=torch.zeros(E, device=d), softmax=softmax)


@gpu
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("groups", [(1, 1, False), (4, 2, False), (4, 2, True), (8, 8, True)])
def test_route_few_distinct_candidates(softmax, groups):
    """Rows of a handful of values a few times 1e-9 apart, each held by dozens of experts, and
    rows that are equal throughout."""
    d = dev()
    E, T = 256, 64
    g = gen(13)
    x = 1e-9 * torch.randint(0, 3, (T, E), generator=g)
    x[::4] = 0.0
    b = 1e-9 * (torch.rand(E, generator=g) < 0.02)
    for bias in (b, torch.zeros(E), 0.5 + torch.zeros(E)):
        check_route(x.to(d), 8, bias=bias.to(d), softmax=softmax, n_groups=groups[0], top_groups=groups[1], top2=groups[2])


# ------------------------------------------------------------------ grouping by cluster size


def test_group_ctas():
    """One CTA, eight or sixteen by the number of pairs, and never more than the device places."""
    ctas = F.load_library().flint_group_pairs_ctas
    assert [ctas(n, 16) for n in (1, 2048, 2049, 8192, 8193, 1 << 24)] == [1, 1, 8, 8, 16, 16]
    assert [ctas(n, 8) for n in (1, 2048, 2049, 8192, 8193, 1 << 24)] == [1, 1, 8, 8, 8, 8]
    assert {ctas(n, 1) for n in (1, 2049, 8193, 1 << 24)} == {1}


@gpu
@pytest.mark.parametrize("E", [1, 5, 300, 1024])
@pytest.mark.parametrize("pairs", [2048, 2049, 5000, 8191, 8192, 8193, 16385])
def test_group_pairs_of_every_cluster(pairs, E):
    d = dev()
    ids = torch.randint(-1, E + 1, (pairs,), generator=gen(pairs + E), dtype=torch.int32)
    offsets = torch.full((E + 1,), -9, dtype=torch.int32, device=d)
    order, pos = (torch.full((pairs,), -9, dtype=torch.int32, device=d) for _ in range(2))
    F.group_pairs(ids.to(d), offsets, order, pos)
    torch.cuda.synchronize()
    for got, want in zip((offsets, order, pos), R.group(ids.numpy(), E)):
        assert np.array_equal(got.cpu().numpy(), want)
