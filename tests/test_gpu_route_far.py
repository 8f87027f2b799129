"""The router's gradient where all scores are tiny."""
import pytest
import torch

import block_common as bc
import moe_common as mc
import mxfp8_block_scaled_mxgemm_amd as pkg
from gpu_common import say, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k", [(33, 64, 8), (5, 500, 20)])
@pytest.mark.parametrize("size", [1e-6, 1.0, 1e12, 1e30])
def test_normalised_sigmoids_of_far_logits(T, E, k, size):
    """Sigmoids down to e^-699 and their gradient, whose reciprocal sum times a
    large gradient leaves FP64's range.  There s = e^x to 64 bits and 1 - s = 1, so
    that the weights are a softmax over the chosen logits."""
    torch_cuda()
    g = torch.Generator().manual_seed(T)
    x = -699 + 4 * torch.rand(T, E, generator=g)
    d = size * torch.randn(T, k, generator=g)
    say(f"far logits T={T} E={E} k={k} size={size:g}")
    ids, w = pkg.route_tokens(x.cuda(), k, score="sigmoid", scale=1.5)
    got = pkg.route_tokens_backward(d.cuda(), x.cuda(), ids, score="sigmoid", scale=1.5)
    at = ids.cpu().long()
    p = torch.softmax(x.double().gather(1, at), 1)
    mc.assert_within(w, 1.5 * p, 1.5 * p * (bc.U + 2.0 ** -40), "weights")
    each = 1.5 * p * (d.double() - (p * d.double()).sum(1, keepdim=True))
    ref = torch.zeros(T, E, dtype=torch.float64).scatter_(1, at, each)
    # 64-bit arithmetic on terms up to |d| (products of 1e-6 and a score are
    # subnormal and keep 36 bits), then float32
    mc.assert_within(got, ref, 2.0 ** -34 * d.double().abs().max() + bc.U * ref.abs(), "d_logits")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(300, 64, 1), (40, 300, 1), (40, 600, 20)])
def test_the_only_choice_has_no_gradient(T, E, k, score):
    """Normalised, the weight of a token's only expert is the scale whatever its
    logit is, and the gradient zero, not what two roundings leave of it."""
    torch_cuda()
    g = torch.Generator().manual_seed(T)
    x, d = 3 * torch.randn(T, E, generator=g), torch.randn(T, k, generator=g)
    say(f"one choice T={T} E={E} k={k} {score}")
    ids, _ = pkg.route_tokens(x.cuda(), k, score=score, scale=2.5)
    ids[:, 1:] = -1
    got = pkg.route_tokens_backward(d.cuda(), x.cuda(), ids, score=score, scale=2.5)
    assert not got.any(), float(got.abs().max())
