"""The route weights of expert selection are the same number whichever kernel forms them."""

import pytest
import torch

from tests.test_gpu_around import DTYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from int4_quantised_moe_b200 import binding
    return binding


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("Q,E,bias", [(300, 64, False), (300, 384, True), (4100, 128, False), (300, 1024, True),
                                      (300, 1025, True), (20, 1025, False)])
def test_one_renormalised_expert_has_the_whole_weight(B, Q, E, bias, score, dtype):
    """k = 1: p / p is 1, whatever p rounds to."""
    g = torch.Generator().manual_seed(Q + E)
    z = (torch.randn((Q, E), generator=g) * 3 - 2).to(DTYPES[dtype]).cuda()
    b = (torch.randn(E, generator=g) * 0.1).cuda() if bias else None
    _, w = B.router_select(z, B.make_select_cfg(E, 1, score=score, scale=2.5), b)
    assert (w == 2.5).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_renormalised_weights_do_not_depend_on_the_batch(B, score, dtype):
    """2048 tokens and more have a kernel of their own; the k shares are formed in the same order."""
    g = torch.Generator().manual_seed(9)
    z = (torch.randn((2049, 100), generator=g) * 3).to(DTYPES[dtype]).cuda()
    cfg = B.make_select_cfg(100, 7, score=score, scale=1.5)
    ids, w = B.router_select(z, cfg)
    for lo in range(0, 2049, 512):
        i, v = B.router_select(z[lo:lo + 512], cfg)
        assert torch.equal(i, ids[lo:lo + 512]) and torch.equal(v, w[lo:lo + 512])
