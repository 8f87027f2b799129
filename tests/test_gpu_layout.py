"""Byte transposes and operands given as transposed views."""
import pytest
import torch

import mxfp8_block_scaled_mxgemm_amd as pkg
import moe_common as mc
from gpu_common import say, torch_cuda
from mxfp8_block_scaled_mxgemm_amd import _moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,rows,cols,pad", [(1, 1, 1, 0), (1, 3, 200, 0), (2, 128, 128, 0), (3, 129, 15, 5),
                                                 (1, 1000, 257, 16), (5, 17, 640, 1)])
def test_transpose(batch, rows, cols, pad):
    torch_cuda()
    say(f"transpose {batch} x {rows} x {cols} pad {pad}")
    g = torch.Generator().manual_seed(rows + cols)
    src = torch.randint(0, 256, (batch, rows, cols + pad), generator=g, dtype=torch.uint8).cuda()[:, :, :cols]
    out = _moe._laid_out(src.transpose(1, 2))
    assert torch.equal(out.cpu(), src.cpu().transpose(1, 2))
    if rows > 1 and cols > 1:
        assert out.is_contiguous()


@pytest.mark.parametrize("by", [False, True])
def test_transposed_operands_of_linear(by):
    torch_cuda()
    M, N, K, E = 70, 96, 384, 3
    g = torch.Generator().manual_seed(1)
    a, a_s = (t.cuda() for t in mc.codes(g, (M, K), "e4m3"))
    w, w_s = (t.cuda() for t in mc.codes(g, (E, N, K) if by else (N, K), "e4m3"))
    offsets = pkg.sort_tokens(mc.ids_of(g, M, 1, E).cuda(), E).offsets if by else None
    turn = lambda t: t.transpose(-1, -2).contiguous().transpose(-1, -2)  # noqa: E731
    ref = pkg.linear(a, a_s, w, w_s, offsets=offsets)
    got = pkg.linear(turn(a), turn(a_s), turn(w), turn(w_s), offsets=offsets)
    assert not turn(w).is_contiguous() and torch.equal(ref, got)


def test_rows_strided_both_ways_are_refused():
    torch_cuda()
    a = torch.zeros(16, 512, dtype=torch.uint8, device="cuda")[:, ::2]
    a_s = torch.zeros(16, 8, dtype=torch.uint8, device="cuda")
    w, w_s = torch.zeros(32, 256, dtype=torch.uint8, device="cuda"), torch.zeros(32, 8, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        pkg.linear(a, a_s, w, w_s)
