"""Routing at the edges of its keys, masks and sizes, on the GPU against the float64 reference."""
import pytest
import torch

from gpu_util import require_gpu
from test_gpu_route import check_route

pytestmark = pytest.mark.gpu


def test_a_chosen_expert_far_below_the_largest():
    """Rows whose last expert is chosen 20 and 30 below the row's largest logit, from the one group that stays."""
    m = require_gpu()
    a, b = torch.full((64,), -20.0), torch.full((64,), -1.0)
    a[56:] = torch.tensor([20.0, -10, -10, -10, -10, -10, -10, 0])
    b[56:] = torch.tensor([20.0, 0.1, 0.2, 0.3, 0.4, 0.5, 0.6, 1.0])
    x = torch.stack([a, b]).cuda()
    for score in ("softmax", "sigmoid"):
        ids = check_route(m, x, 4, score, groups=8, keep=1)[0].tolist()
        assert ids[0][:2] == [56, 63] and ids[1] == [56, 63, 62, 61]


@pytest.mark.parametrize("E,groups,keep,top", [(64, 8, 1, 4), (64, 8, 2, 5), (64, 4, 1, 6), (128, 8, 1, 8), (256, 16, 1, 3),
                                               (512, 64, 2, 6), (512, 32, 1, 16), (1024, 64, 1, 7), (1024, 64, 1, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_few_kept_experts_of_a_wide_spread(E, groups, keep, top, score):
    """At most 16 experts stay, the last group among them, and most lie far below the row's largest."""
    m = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(E + groups)
    size = E // groups
    for off in (15.0, 17.0, 30.0, 50.0, 200.0):
        x = torch.randn((60, E), generator=g, device="cuda")
        x[:, E - size] += off
        x[20:40] = x[20:40].masked_fill(torch.rand((20, E), generator=g, device="cuda") < 0.4, -torch.inf)
        x[40:, E - size + 1:] -= 20.0
        for bias in (None, 0.1 * torch.randn(E, generator=g, device="cuda")):
            check_route(m, x, top, score, bias, groups, keep, 1 if bias is None else 2)
