"""Routing with biases that keep experts from being chosen: -10^4, -10^9, fp32's lowest number, -inf, for a
few, most or all experts of a group, beside balance biases; those left over, and those masked where fewer
than k are left, are still told apart by 64 bits."""
import pytest
import torch

from block_cases import gen
from test_gpu_route import check

pytestmark = pytest.mark.gpu
LOWEST = torch.finfo(torch.float32).min


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,n_group,topk_group", [(30, 512, 10, 1, 1), (30, 512, 10, 8, 4), (20, 1023, 16, 33, 7),
                                                      (20, 1020, 16, 17, 5), (40, 60, 4, 4, 2), (40, 7, 3, 1, 1)])
@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e30, LOWEST, -float("inf"), 1e9, -LOWEST])
def test_masks(score, T, E, k, n_group, topk_group, mask):
    g = gen(E + n_group)
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[::3] = (logits[::3] * 8).round() / 8                                    # ties
    base = torch.randint(-60, 61, (E,), generator=g, device="cuda").float() * 0.001
    per = E // n_group
    some, most, group = (torch.zeros(E, dtype=torch.bool, device="cuda") for _ in range(3))
    some[::7] = True
    most[torch.randperm(E, generator=g, device="cuda")[k - 1:]] = True             # one fewer than k are left
    group[:per] = True
    for masked in (some, most, group, ~most, torch.ones_like(most)):
        bias = torch.where(masked, torch.full_like(base, mask), base)
        for group_top in (1, 2):
            check(logits, k, bias, score=score, n_group=n_group, topk_group=topk_group, group_top=min(group_top, per))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n_group,topk_group", [(1, 1), (8, 3)])
def test_biases_of_all_sizes_and_signs(score, n_group, topk_group):
    """Large ones of both signs side by side (a group's two best may all but cancel), and neighbours of a size."""
    g = gen(31)
    T, E, k = 30, 128, 12
    logits = torch.randn(T, E, generator=g, device="cuda")
    sign = torch.randint(0, 2, (E,), generator=g, device="cuda").float() * 2 - 1
    for bias in (sign * 1e9, sign * 10.0 ** torch.randint(-6, 12, (E,), generator=g, device="cuda").float(), sign * LOWEST,
                 sign * 2.0 ** 24 + torch.randint(-2, 3, (E,), generator=g, device="cuda"),
                 1e6 + torch.randint(0, 3, (E,), generator=g, device="cuda").float() / 16):
        for group_top in (1, 2):
            check(logits, k, bias.contiguous(), score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
