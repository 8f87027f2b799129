"""Router on the GPU against its definition in 64 bits."""
import math

import pytest
import torch

import block_common as bc
import moe_common as mc
import mxfp8_block_scaled_mxgemm_amd as pkg
from gpu_common import say, torch_cuda

pytestmark = pytest.mark.gpu


def _logits(g, T, E, dtype, scale=1.5):
    return ((torch.randn(T, E, generator=g) + torch.randn(E, generator=g) * 0.3) * scale).to(dtype)


def _check(logits, k, **how):
    ids, w = pkg.route_tokens(logits.cuda(), k, **{n: v.cuda() if torch.is_tensor(v) else v for n, v in how.items()})
    ref_ids, ref_w = bc.route(logits, k, **how)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert torch.equal(ids.cpu(), ref_ids)
    # 64-bit arithmetic (a few hundred roundings at most) and one rounding
    mc.assert_within(w, ref_w, ref_w.abs() * (bc.U + 2.0 ** -43) + 2.0 ** -149, "weights")
    return ids, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top,bias", [
    (1, 1, 1, 1, 1, False), (5, 4, 4, 1, 1, True), (37, 8, 2, 4, 2, True), (64, 63, 7, 3, 2, False),
    (130, 64, 8, 8, 4, True), (33, 128, 8, 1, 1, False), (33, 256, 8, 8, 4, True), (20, 200, 6, 5, 5, True),
    (9, 512, 16, 64, 7, False), (9, 1000, 10, 2, 1, True), (7, 1024, 64, 1, 1, False), (3, 100, 64, 1, 1, True),
    (4, 64, 20, 64, 20, True),
])
def test_route(T, E, k, groups, top, bias, score, normalize, dtype):
    torch_cuda()
    g = torch.Generator().manual_seed(T + E)
    say(f"route T={T} E={E} k={k} groups={groups}/{top} bias={bias} {score} {normalize} {dtype}")
    _check(_logits(g, T, E, dtype), k, score=score, bias=torch.randn(E, generator=g) * 0.2 if bias else None,
           groups=groups, top_groups=top, normalize=normalize, scale=2.5 if bias else 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top,bias", [(256, 8, 8, 4, True), (256, 8, 8, 4, False), (128, 6, 1, 1, False),
                                                 (64, 4, 4, 2, True), (40, 8, 1, 1, True), (3, 2, 1, 1, False),
                                                 (200, 16, 1, 1, True), (128, 8, 16, 3, True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tokens_choose_as_few_do(E, k, groups, top, bias, score, dtype):
    """The kernel for many tokens against the one for few (which the definition
    checks), with keys that are equal, nearly equal, masked and tiny."""
    torch_cuda()
    g = torch.Generator().manual_seed(E + k)
    T = 4096 + 37
    x = _logits(g, T, E, torch.float32)
    x[:300] = torch.round(x[:300])                      # ties
    x[300:600] *= 30                                    # scores that end near 0 and 1
    x[600:700, ::2] = -math.inf
    x[700:720] = -math.inf
    x[720:730, 1:] = math.nan
    x[730:900] = x[730:900] * 1e-6                      # keys that differ by less than an FP32 step
    x[900:1000] -= 90
    x = x.to(dtype)
    b = torch.randn(E, generator=g) * 0.2 if bias else None
    if bias:
        b[E // 3:E // 2] = 0.125
    say(f"many tokens E={E} k={k} groups={groups}/{top} bias={bias} {score} {dtype}")
    for normalize in (True, False):
        how = dict(score=score, bias=None if b is None else b.cuda(), groups=groups, top_groups=top,
                   normalize=normalize, scale=1.5)
        ids, w = pkg.route_tokens(x.cuda(), k, **how)
        few = [pkg.route_tokens(p, k, **how) for p in x.cuda().split(1500)]
        assert torch.equal(ids, torch.cat([i for i, _ in few]))
        ref = torch.cat([v for _, v in few]).double()
        assert ((w.double() - ref).abs() <= 2 * bc.U * ref.abs()).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias,groups,top", [(False, 1, 1), (True, 1, 1), (True, 4, 2), (False, 4, 2)])
def test_masked_and_unusual_logits(bias, groups, top, score):
    """Rows with few or no experts left, infinities, NaN, ties, far logits."""
    torch_cuda()
    E, k = 32, 6
    g = torch.Generator().manual_seed(3)
    x = _logits(g, 14, E, torch.float32)
    x[0] = -math.inf
    x[1, :29] = -math.inf
    x[2, 5:] = math.nan
    x[3] = 0.25                             # all equal: the lowest indexes
    x[4, 7] = math.inf
    x[5, 3], x[5, 9] = math.inf, math.inf
    x[6] = x[6] * 40
    x[7, ::2] = -math.inf
    x[8] = -200.0
    x[9, 4:28] = -math.inf
    x[10] = math.nan
    x[11] = torch.tensor([0.0, -0.0] * 16)
    x[12] = -3e38
    x[13, 1:] = -1e4
    b = None
    if bias:
        b = torch.randn(E, generator=g) * 0.2
        b[2], b[17] = -math.inf, math.nan
    say(f"masked {score} bias={bias} groups={groups}")
    if not bias or score == "softmax":
        b = b if b is None else torch.where(torch.isnan(b), -math.inf, b)
    rows = [t for t in range(14) if not (t in (4, 5, 8, 12) and groups > 1)]    # ties between sums of rounded scores
    for normalize in (True, False):
        ids, w = _check(x[rows], k, score=score, bias=b, groups=groups, top_groups=top, normalize=normalize)
        assert (ids[0] == -1).all() and not w[0].any()
    sort = pkg.sort_tokens(ids, E)          # the pairs that are left out are dropped
    assert int(sort.offsets[-1]) == int((ids >= 0).sum())


def _backward_ref(d, x, ids, score, normalize, scale):
    x = x.double().requires_grad_()
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    kept = ids >= 0
    w = torch.where(kept, s.gather(1, ids.long().clamp(min=0)), 0.0)
    if normalize:
        w = w / w.sum(1, keepdim=True)
    return torch.autograd.grad(scale * w, x, torch.where(kept, d.double(), 0.0))[0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 4, 4), (70, 64, 8), (33, 130, 6), (9, 256, 8), (5, 500, 64), (3, 1024, 2)])
def test_route_backward(T, E, k, score, normalize, dtype):
    torch_cuda()
    g = torch.Generator().manual_seed(T * E)
    x, d = _logits(g, T, E, dtype), torch.randn(T, k, generator=g)
    say(f"route backward T={T} E={E} k={k} {score} {normalize} {dtype}")
    ids, _ = pkg.route_tokens(x.cuda(), k, score=score, normalize=normalize, scale=1.5)
    if k > 2:
        ids[0, 1] = -1
    got = pkg.route_tokens_backward(d.cuda(), x.cuda(), ids, score=score, normalize=normalize, scale=1.5)
    assert got.dtype == dtype
    ref = _backward_ref(d, x, ids.cpu(), score, normalize, 1.5)
    # 64-bit arithmetic on terms up to |d|; float32, then the type
    bound = 2.0 ** -40 * d.abs().max() + mc.rounding(ref * (1 + 2 * bc.U), dtype) + bc.U * ref.abs()
    mc.assert_within(got, ref, bound, "d_logits")


def test_route_backward_against_differences():
    torch_cuda()
    g = torch.Generator().manual_seed(9)
    T, E, k = 6, 16, 4
    x, d, v = _logits(g, T, E, torch.float32), torch.randn(T, k, generator=g), torch.randn(T, E, generator=g)
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            say(f"differences {score} {normalize}")
            ids, _ = pkg.route_tokens(x.cuda(), k, score=score, normalize=normalize)
            got = pkg.route_tokens_backward(d.cuda(), x.cuda(), ids, score=score, normalize=normalize)

            def loss(y):
                s = torch.sigmoid(y) if score == "sigmoid" else torch.softmax(y, 1)
                w = s.gather(1, ids.cpu().long())
                return float((d.double() * (w / w.sum(1, keepdim=True) if normalize else w)).sum())

            h = 1e-5        # error h^2 / 6 third derivatives (below 1e2), and 1e-15 / h
            slope = (loss(x.double() + h * v.double()) - loss(x.double() - h * v.double())) / (2 * h)
            dot = float((got.cpu().double() * v.double()).sum())
            size = float((got.cpu().double() * v.double()).abs().sum())
            assert abs(dot - slope) <= 2 * bc.U * size + 1e-7


def test_route_masked_backward():
    """Masked experts get no gradient, and a row of them none at all; the same
    index twice counts twice."""
    torch_cuda()
    g = torch.Generator().manual_seed(5)
    x = _logits(g, 3, 16, torch.float32)
    x[0] = -math.inf
    x[1, 4:] = -math.inf
    d = torch.randn(3, 6, generator=g).cuda()
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            say(f"masked backward {score} {normalize}")
            ids, _ = pkg.route_tokens(x.cuda(), 6, score=score, normalize=normalize)
            assert (ids[1, 4:] == -1).all()
            got = pkg.route_tokens_backward(d, x.cuda(), ids, score=score, normalize=normalize).cpu()
            assert not got[0].any() and not got[1, 4:].any() and torch.isfinite(got).all() and got[2].any()
    twice = torch.tensor([[3, 3]], dtype=torch.int32).cuda()
    got = pkg.route_tokens_backward(torch.tensor([[1.0, 2.0]]).cuda(), x[2:].cuda(), twice, normalize=False,
                                    score="sigmoid").cpu()
    s = torch.sigmoid(x[2].double())
    ref = torch.zeros(1, 16, dtype=torch.float64)
    ref[0, 3] = 3 * s[3] * (1 - s[3])
    mc.assert_within(got, ref, 2 * bc.U * ref.abs(), "twice")


def test_route_strides_streams_and_none():
    torch_cuda()
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(40, 77, generator=g).cuda()
    view = wide[:, 5:69]
    say("strided logits")
    ids, w = pkg.route_tokens(view, 4)
    ids2, w2 = pkg.route_tokens(view.contiguous(), 4)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    d = torch.randn(40, 4, generator=g).cuda()
    assert torch.equal(pkg.route_tokens_backward(d, view, ids), pkg.route_tokens_backward(d, view.contiguous(), ids))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    ids3, w3 = pkg.route_tokens(view, 4, stream=stream)
    stream.synchronize()
    assert torch.equal(ids, ids3) and torch.equal(w, w3)
    empty = torch.empty(0, 64, device="cuda")
    ids, w = pkg.route_tokens(empty, 4)
    assert ids.shape == w.shape == (0, 4)
    assert pkg.route_tokens_backward(w, empty, ids).shape == (0, 64)


def test_route_of_many_tokens():
    """More tokens than the grid has waves."""
    torch_cuda()
    T = (1 << 22) + 5
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, 4, generator=g, device="cuda")
    say(f"route T={T}")
    ids, w = pkg.route_tokens(x, 2)
    top = x.topk(2, dim=1)
    assert torch.equal(x.gather(1, ids.long()), top.values)
    assert (w - torch.softmax(top.values.double(), 1)).abs().max() < 2 * bc.U
    d = torch.ones(T, 2, device="cuda")
    d[:, 1] = 0
    got = pkg.route_tokens_backward(d, x, ids).double()
    p = torch.softmax(top.values.double(), 1).prod(1)
    assert (got.gather(1, ids.long())[:, 0] - p).abs().max() < 2 * bc.U
    assert (got != 0).sum(1).max() <= 2
