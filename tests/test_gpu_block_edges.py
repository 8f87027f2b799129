"""Quantisation of batches whose tiles hold dropped rows only."""
import math

import pytest
import torch

import block_common as bc
import mxfp8_block_scaled_mxgemm_amd as pkg
from gpu_common import say, torch_cuda

pytestmark = pytest.mark.gpu


# widths in eights, others, and gated gradients whose halves are whole blocks
@pytest.mark.parametrize("C,act,gated", [(136, "none", False), (130, "silu", False), (128, "silu", True), (256, "gelu", True)])
@pytest.mark.parametrize("live", [0, 1, 128, 130])
@pytest.mark.parametrize("cols", [False, True])
def test_tiles_of_dropped_rows(live, C, act, gated, cols):
    """What dropped rows hold is not used, and they are zero, codes and scales;
    the rows before them are those of a batch without them."""
    torch_cuda()
    M, E = 300, 2
    g = torch.Generator().manual_seed(C + live)
    ids = torch.full((M, 1), -1, dtype=torch.int32)
    ids[:live] = 1
    sort, few = pkg.sort_tokens(ids.cuda(), E), pkg.sort_tokens(ids[:live].cuda(), E)
    x, z = torch.randn(M, 2 * C if gated else C, generator=g), torch.randn(M, 2 * C if gated else C, generator=g).bfloat16()
    d = torch.randn(M, C, generator=g).bfloat16()
    for t in (x, z, d):
        t[live:] = math.nan
    say(f"dropped tiles live={live} C={C} {act} gated={gated} cols={cols}")
    how = dict(act=act, gated=gated, cols=cols)
    plain = act == "none"
    for call, args in ((pkg.block_quantize, (x,)), (pkg.block_quantize_backward, (d, None if plain else z))):
        args = [t if t is None else t.cuda() for t in args]
        (q, s), (qt, st) = call(*args, sort=sort, **how)
        assert not q[live:].any() and not s[live:].any()
        (q1, s1), (qt1, st1) = call(*(t if t is None else t[:live] for t in args), sort=few, **how)
        assert torch.equal(q[:live], q1) and torch.equal(s[:live], s1)
        assert torch.isfinite(s).all()
        if cols:
            used = bc.up(live)
            assert torch.equal(qt[:, :used], qt1[:, :used]) and torch.equal(st[:, :used // 128], st1[:, :used // 128])
            assert not qt[:, used:].any() and not st[:, used // 128:].any()
