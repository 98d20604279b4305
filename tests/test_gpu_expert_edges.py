"""GPU tests of the expert operators at the edges of their contracts: tokens
that went nowhere with logits that are no numbers, results and memory on
another stream than the current one, no tokens, no columns, segments that do
not start on whole blocks, quotients half-way between two codes."""

import math

import numpy as np
import pytest
import torch

from oracle import blocks as O
from oracle import experts as X
from tests.test_gpu_blocks import check_product, coded, matrix, of, raw

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import matrix_aware_optimizer_step_amd as m
    m._lib.load()
    return m


# ------------------------------------------------------------ the router's gradient

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,experts,k", [(6, 40, 4), (90, 300, 8)])
def test_gradient_of_masked_rows_that_are_not_numbers(mx, tokens, experts, k, dtype, renormalize, score):
    """Padding holds anything: its weights are 0, so its logits' gradient is, whatever they are."""
    z = torch.randn(tokens, experts, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    z[1] = math.nan
    z[2, 3] = math.inf
    z[3, 5] = math.nan
    z[4] = math.inf
    mask = torch.ones(tokens, dtype=torch.bool)
    mask[1:5] = False
    g = torch.randn(tokens, k, generator=torch.Generator().manual_seed(2))
    r = mx.route(z, k, score=score, renormalize=renormalize, scale=1.5, mask=mask.cuda())
    assert (r.experts[1:5] == -1).all() and not r.weights[1:5].any()
    got = mx.route_backward(z, r, g.cuda())
    assert not got[1:5].any()
    z[1:5] = 0.0  # the other rows are what they are without such padding
    assert torch.equal(got, mx.route_backward(z, mx.route(z, k, score=score, renormalize=renormalize, scale=1.5,
                                                          mask=mask.cuda()), g.cuda()))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_of_rows_that_are_not_numbers_without_a_mask(mx, renormalize, score):
    z = torch.randn(6, 40, generator=torch.Generator().manual_seed(1)).cuda()
    z[1, 3] = math.nan
    z[2] = -math.inf
    r = mx.route(z, 4, score=score, renormalize=renormalize)
    got = mx.route_backward(z, r, torch.ones(6, 4).cuda())
    assert got[1].isnan().all() and not got[2].any() and got[[0, 3, 4, 5]].isfinite().all()
