"""Refusals of the products with scales of 128 that come after their operands'
checks."""
import pytest
import torch

import mxfp8_block_scaled_mxgemm_amd as pkg
from gpu_common import say, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offsets", [None, [0, 256], 256, torch.tensor(256, dtype=torch.int32), torch.zeros(1, 2).int()])
def test_offsets_that_are_no_vector(offsets):
    torch_cuda()
    u8, f = torch.zeros(4, 256, dtype=torch.uint8, device="cuda"), torch.ones(4, 2, device="cuda")
    if isinstance(offsets, torch.Tensor):
        offsets = offsets.cuda()
    say(f"offsets {offsets}")
    kind = ValueError if isinstance(offsets, torch.Tensor) else TypeError
    with pytest.raises(kind, match="offsets"):
        pkg.block_linear_by_inner(u8, f, u8, f, offsets)
    if offsets is not None:
        with pytest.raises(kind, match="offsets"):
            pkg.block_linear(u8, f, u8[None], f[None], offsets)
    with pytest.raises(ValueError, match="precision"):
        pkg.block_linear(u8, f, u8, f, precision="fast")
