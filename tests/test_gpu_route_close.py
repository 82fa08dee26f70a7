"""Choices among experts whose biased scores all lie within a few roundings of fp32 of each other: the
bias is minus a token's scores, rounded, so that only 64 bits tell them apart.  Every number of
experts a lane, 32 (groups of 31 and 60) among them."""
import numpy as np
import pytest
import torch

from block_cases import gen
from oracle import around
from test_gpu_route import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


SHAPES = [(40, 4, 1, 1), (100, 8, 1, 1), (200, 8, 4, 2), (500, 16, 1, 1), (1024, 16, 1, 1), (1020, 16, 17, 5),
          (1023, 16, 33, 7), (990, 32, 33, 33)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,n_group,topk_group", SHAPES)
@pytest.mark.parametrize("spread", [0.05, 1.0, 4.0])
def test_scores_that_a_bias_makes_equal(score, E, k, n_group, topk_group, spread):
    for seed in range(4):
        g = gen(seed + E)
        row = torch.randn(1, E, generator=g, device="cuda") * spread
        s = around.scores(row.cpu().numpy(), score)[0]
        logits = row.repeat(3, 1)
        logits[1] = row[0].flip(0)                         # (for this token the bias decides)
        for step in (0.0, 2.0 ** -24):                     # as close as roundings; and moved by single steps of 2^-24
            at = np.random.default_rng(seed).integers(-2, 3, E) * step
            bias = torch.tensor((0.5 - s + at).astype(np.float32), device="cuda")
            for group_top in (1, 2):
                check(logits, k, bias, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
