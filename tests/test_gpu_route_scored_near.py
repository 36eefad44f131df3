"""Routing by scores where many experts lie nearer together than FP32 can tell, some of them the
same: who else may be among the first k does not end with the first equal one."""
import pytest
import torch

from test_gpu_route_scored import BF, F32, gen, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(10, 3), (48, 6), (100, 8), (256, 8), (448, 30), (1024, 32)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("values", [2, 4, 40])
def test_many_equal_and_many_near(E, k, score, values):
    # logits a few units of 2^-22 apart: choice values differ by 6e-8 of the largest score, which FP64 tells apart
    T = 40
    x = 0.5 + torch.randint(0, values, (T, E), generator=gen(E + values)).float() * 2.0 ** -22
    run(x, k, score=score, bias=torch.zeros(E))
    run(x, k, score=score, bias=torch.full((E,), 0.25))
    bias = torch.randint(0, 2, (E,), generator=gen(E)).float() * 0.5
    run(x, k, score=score, bias=bias)
    if E % 4 == 0:
        for kept in (1, 3):
            for by in ("max", "top2"):
                run(x, min(k, kept * E // 4), score=score, bias=bias, groups=4, kept=kept, by=by)


@pytest.mark.parametrize("E,k", [(64, 8), (300, 20)])
def test_scores_that_bias_brings_together(E, k):
    # BF16 logits of two values, biases that make up for them but for a few units in the last place
    g = gen(E)
    x = torch.where(torch.rand(40, E, generator=g) < 0.3, 1.0, 1.0078125)
    s = torch.sigmoid(x[0].double())
    bias = (1.0 - s).float() + torch.randint(0, 3, (E,), generator=g).float() * 2.0 ** -24
    run(x, k, bias=bias, dtype=BF)
    run(x, k, bias=bias, dtype=F32)
    run(x, k, bias=bias, groups=4, kept=2, dtype=BF)


@pytest.mark.parametrize("E", [64, 256, 1000])
def test_rows_of_equal_logits(E):
    # (a padded batch: every choice value is the same, and the lowest experts are right)
    run(torch.zeros(70, E), 8, bias=torch.zeros(E))
    x = torch.zeros(70, E)
    x[::2, E - 1] = 2.0 ** -20
    run(x, 8, bias=torch.zeros(E))
    run(x, 8, score="softmax", bias=torch.zeros(E))
