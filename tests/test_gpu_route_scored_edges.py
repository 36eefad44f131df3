"""Routing by scores where a sum of two choice values lies below FP32's range."""
import pytest
import torch

from test_gpu_route_scored import BF, F32, gen, run

pytestmark = pytest.mark.gpu

LOWEST = -3.4028234663852886e38


@pytest.mark.parametrize("groups,kept", [(4, 1), (4, 2), (4, 3), (3, 2), (8, 5)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_groups_of_the_lowest_bias(groups, kept, score, dtype):
    # A bias of the type's lowest value is finite: its experts come last, but they may be chosen
    E = 24
    x = torch.randn(70, E, generator=gen(kept + groups))
    size = E // groups
    for low in (LOWEST, -1.8e38, -3.0e38):
        for first in (0, 1, groups - 1):        # from this group on all are low
            bias = 0.1 * torch.randn(E, generator=gen(first))
            bias[first * size:] = low
            run(x, min(kept * size, 20), score=score, bias=bias, groups=groups, kept=kept, dtype=dtype)
    bias = torch.full((E,), LOWEST)
    bias[::5] = torch.nextafter(torch.tensor(LOWEST), torch.tensor(0.0))
    run(x, kept * size, score=score, bias=bias, groups=groups, kept=kept, dtype=dtype)
