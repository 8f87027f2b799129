"""silu and its derivative in FP32, seen through the scales of blocks that hold
one value each."""
import pytest
import torch

import block_common as bc
import mxfp8_block_scaled_mxgemm_amd as pkg
from gpu_common import say, torch_cuda

pytestmark = pytest.mark.gpu
FMAX = 448.0


def _all(lo, hi):
    """Every bfloat16 number in [lo, hi)."""
    z = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    z = z[torch.isfinite(z)]
    return z[(z.double() >= lo) & (z.double() < hi)]


def _one_each(v, blocks, at):
    """Rows of `blocks` blocks of 128 columns, v's numbers one to a block, at
    column `at` of it; zeros elsewhere."""
    rows = -(-v.numel() // blocks)
    out = torch.zeros(rows * blocks, 128, dtype=v.dtype)
    out[:v.numel(), at] = v
    return out.view(rows, blocks * 128)


def _slopes(z, C, gated):
    """|silu'(z)| as the quantiser's scales give it (64-bit, one rounding past
    the kernel's), in rows of C columns."""
    blocks = -(-C // 128)
    at = 1
    zz = _one_each(z, blocks, at)[:, :C]
    d = _one_each(torch.ones(z.numel()), blocks, at)[:, :C]
    if gated:       # [d u silu'(g), d silu(g)] with u = 1
        zz = torch.cat([zz, torch.ones_like(zz)], 1)
    (_, s), _ = pkg.block_quantize_backward(d.cuda(), zz.cuda(), act="silu", gated=gated, cols=False)
    return s[:, :blocks].cpu().double().reshape(-1)[:z.numel()] * FMAX


# (gated halves are whole blocks or they would share one)
@pytest.mark.parametrize("C,gated", [(256, False), (130, False), (136, False), (128, True), (384, True)])
def test_slope_of_silu_does_not_cancel(C, gated):
    """From 8 to 20, where 1 - sigmoid is below 4e-4: 1 + exp(-z), its reciprocal,
    1 + z (1 - sigmoid), that times the sigmoid and the scale's division by 448
    are one rounding each; z (1 - sigmoid) is below 3e-3, so its own (seven) add
    less than a tenth of one."""
    torch_cuda()
    z = _all(8, 20)
    say(f"slope of silu, {z.numel()} numbers, C={C} gated={gated}")
    got, x = _slopes(z, C, gated), z.double()
    ref = torch.sigmoid(x) * (1 + x * torch.sigmoid(-x))
    assert ((got - ref).abs() <= 5.1 * bc.U * ref).all(), float(((got - ref).abs() / ref).max() / bc.U)


@pytest.mark.parametrize("C,gated", [(256, False), (130, False), (128, True)])
def test_slope_of_silu_everywhere(C, gated):
    """The sigmoid s is good to six roundings (an exponential of three, 1 + it,
    the reciprocal's one and what its Newton step leaves of the estimate's), 1 - s
    to seven of its own; then a fused multiply-add, a product and the scale's
    division.  Where |z| < 126 ln 2, past which both are 0 or 1."""
    torch_cuda()
    z = torch.cat([_all(-80, 0), _all(0, 80)])
    say(f"slope of silu, {z.numel()} numbers, C={C} gated={gated}")
    got, x = _slopes(z, C, gated), z.double()
    s, c = torch.sigmoid(x), torch.sigmoid(-x)
    ref = (s * (1 + x * c)).abs()
    bound = bc.U * s * (9 * (1 + x * c).abs() + 7 * x.abs() * c)
    # (a scale is 2^-126 at least)
    assert ((got - ref).abs() <= bound + FMAX * bc.LOW).all(), float(((got - ref).abs() / bound).max())


def test_slope_of_silu_far_out():
    """1 and 0 past what FP32's exponential holds, to the type's largest number."""
    torch_cuda()
    big = torch.finfo(torch.bfloat16).max
    z = torch.tensor([90.0, 120.0, 1e4, 2.3e38, 2.5e38, big, -120.0, -1e4, -2.5e38, -big]).bfloat16()
    for C, gated in ((256, False), (130, False), (128, True)):
        say(f"slope of silu far out, C={C} gated={gated}")
        got = _slopes(z, C, gated)
        ref = (z > 0).double()
        assert ((got - ref).abs() <= bc.U * ref + FMAX * bc.LOW).all()
