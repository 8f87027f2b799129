"""The router under biases that FP32 cannot add up: infinite ones, pairs whose
sum leaves its range, pairs that cancel.  The choice is the one of the 64-bit
keys whatever the number of tokens."""
import math

import pytest
import torch

import block_common as bc
import mxfp8_block_scaled_mxgemm_amd as pkg
from gpu_common import say, torch_cuda

pytestmark = pytest.mark.gpu


def _same_choice(x, k, checked, **how):
    """Many tokens in one call choose as the kernel for few does, and the first
    of them as the definition says."""
    ids, w = pkg.route_tokens(x, k, **how)
    few = [pkg.route_tokens(p, k, **how) for p in x.split(4096)]
    wrong = (ids != torch.cat([i for i, _ in few])).any(1)
    assert not wrong.any(), f"{int(wrong.sum())} of {x.shape[0]} tokens, the first is {int(wrong.nonzero()[0])}"
    ref = torch.cat([v for _, v in few]).double()
    assert ((w.double() - ref).abs() <= 2 * bc.U * ref.abs()).all()
    host = {n: v.cpu() if torch.is_tensor(v) else v for n, v in how.items()}
    assert torch.equal(ids[:checked].cpu(), bc.route(x[:checked].cpu(), k, **host)[0])


def _biases(E, size, g):
    """Name and bias of each case; runs of `size` experts are one group."""
    run = torch.arange(E) // size
    normal = torch.randn(E, generator=g) * 0.2
    one = normal.clone()
    one[::size] = math.inf
    two = one.clone()
    two[1::size] = math.inf
    some = torch.where((run % 2 == 1) & (torch.arange(E) % size == 0), math.inf, normal)
    huge = (2 + torch.rand(E, generator=g)) * 1e38
    mixed = torch.where(run % 3 == 0, -huge, huge)
    mixed[2] = math.inf
    return {"infinite": one, "two infinite": two, "some infinite": some, "sums past FP32": huge,
            "sums below FP32": -huge, "both": mixed}


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top", [(32, 6, 8, 4), (256, 8, 8, 4), (128, 4, 16, 1), (64, 16, 2, 1), (16, 8, 16, 9)])
def test_infinite_and_huge_biases(E, k, groups, top, score):
    torch_cuda()
    g = torch.Generator().manual_seed(E + groups)
    x = torch.randn(4096 + 21, E, generator=g).cuda()
    for name, bias in _biases(E, max(2, E // groups), g).items():
        say(f"{name} E={E} k={k} groups={groups}/{top} {score}")
        _same_choice(x, k, 24, score=score, bias=bias.cuda(), groups=groups, top_groups=top)
        _same_choice(x, k, 24, score=score, bias=bias.cuda())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [64.0, 256.0, 1e4, 1e6])
@pytest.mark.parametrize("E,k,groups,top", [(16, 8, 8, 4), (128, 4, 8, 2)])
def test_biases_that_cancel_in_a_rank(E, k, groups, top, size, score):
    """A group's two largest keys hold a large bias and its negative: their sum is
    as small as the scores, its rounding in FP32 as large as the bias."""
    torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(E)
    T = 1 << (20 if E == 16 else 17)
    x = torch.randn(T, E, generator=g, device="cuda")
    bias = torch.full((E,), -2 * size, device="cuda")
    run = E // groups
    bias[::run], bias[1::run] = size, -size
    say(f"cancel E={E} +-{size:g} {score}")
    _same_choice(x, k, 24, score=score, bias=bias, groups=groups, top_groups=top)
