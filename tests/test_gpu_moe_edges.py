"""Edges of the mixture-of-experts calls: sums far outside the range of exponentials, scores below the normal range."""
import numpy as np
import pytest
import torch

from gpu_util import nw, step
from test_gpu_moe import route64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("experts", [16, 100])
def test_route_sums_beyond_a_billion(experts, sign):
    """Sums around 2^32 that lie an eighth apart: softmax is taken from their differences, whatever their size.

    Every sum is a multiple of 1/8 below 2^33, exact in 64 bits in any order; exp and the division are off by a few
    2^-52.  The rounding to fp32 is 2^-24 of the value: 2^-22 covers both."""
    step(f"moe route sums of {sign} 2^32, E {experts}")
    x = torch.full((3, 4096), 1024.0, dtype=torch.float16, device="cuda")
    router = torch.full((experts, 4096), sign * 1024.0, dtype=torch.float16, device="cuda")
    g = torch.Generator().manual_seed(5)
    x[:, 0], x[:, 1] = 1.0, torch.tensor([1000.0, 1.0, 1700.0]).half().cuda()
    router[:, 0] = (torch.randperm(experts, generator=g) / 8).half().cuda()
    router[:, 1] = 1.0
    rid, rw = route64(x, router, 5, renormalize=False)
    ids, weights = nw().moe_route(x, router, 5, renormalize=False)
    w = weights.cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    assert (np.abs(w - rw) <= 2.0 ** -22 * rw).all()


@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_renormalizes_scores_near_the_smallest(sigmoid):
    """A bias picks experts whose scores are around 1e-308 and below: their quotients are ordinary numbers.

    The sums are exact.  Softmax scores from exp(-721), 7e-314, on hold 33 bits; a quotient's score and its sum are off by
    less than 2^-30 each, and 2^-22 covers that and the rounding to fp32."""
    step(f"moe route tiny scores, sigmoid {sigmoid}")
    x = torch.zeros(2, 256, dtype=torch.float16, device="cuda")
    router = torch.zeros(9, 256, dtype=torch.float16, device="cuda")
    x[:, :2] = 1
    router[1:, 0] = -708 if sigmoid else -720
    router[1:, 1] = -(torch.arange(8) / (4 if sigmoid else 8)).half().cuda()
    bias = torch.linspace(3, 2, 9).cuda()
    bias[0] = -10
    for scale in (1.0, 12.0):
        rid, rw = route64(x, router, 2, bias, sigmoid, True, scale)
        ids, weights = nw().moe_route(x, router, 2, bias=bias, sigmoid=sigmoid, scale=scale)
        w = weights.cpu().numpy().astype(np.float64)
        np.testing.assert_array_equal(ids.cpu().numpy(), rid)
        assert np.isfinite(rw).all() and (np.abs(w - rw) <= 2.0 ** -22 * rw).all()


@pytest.mark.parametrize("topk", [0, -1, 9, 2 ** 32 + 2])
def test_route_refuses_topk_before_any_output(topk):
    step(f"moe route topk {topk}")
    x, router = (torch.zeros(n, 256, dtype=torch.float16, device="cuda") for n in (2, 16))
    with pytest.raises(nw().SqllmError, match="moe_route"):
        nw().moe_route(x, router, topk)
