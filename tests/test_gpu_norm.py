"""Norms between blocks, with gate and residual scale, against 64 bits."""
import pytest
import torch

import block_common as bc
import moe_common as mc
import mxfp8_block_scaled_mxgemm_amd as pkg
from gpu_common import say, torch_cuda

pytestmark = pytest.mark.gpu
EPS = 1e-5
# Every sum over a row of at most 8192 has fewer than 8 + 6 + 16 additions in
# a line, so a mean, a root and a normalised element are good to 64 roundings.
ROW = 64 * bc.U


def _inputs(g, T, H, G, dtype, residual=True, gate=True, post=True, pre=True, weight=torch.float32):
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=(r(T, H) * 3 + 0.5).to(dtype), residual=r(T, H).to(dtype) if residual else None,
                gate=r(G, H).to(dtype) if gate else None, post=(1 + 0.2 * r(H)).to(weight) if post else None,
                pre=(1 + 0.2 * r(H)).to(weight) if pre else None)


def _cuda(t):
    return None if t is None else t.cuda()


def _wide(t):
    return None if t is None else t.double()


def _norm_error(v, kind):
    """Error bound of normed(v), 64 bits against FP32: relative, and the mean's
    rounding over the row's root mean square."""
    hat = bc.normed(v, kind, EPS)
    if kind == "rms":
        return ROW * hat.abs()
    m = v - v.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(m.square().mean(1, keepdim=True) + EPS)
    shift = ROW * rstd * (v.abs().mean(1, keepdim=True) + v.abs())
    # (a shift of the mean also moves the root mean square, by less)
    return ROW * hat.abs() + shift * (1 + hat.abs())


def _check(s, kind, scale, G, grads=True, g=None):
    dtype = s["x"].dtype
    T, H = s["x"].shape
    how = dict(gate=_cuda(s["gate"]), scale=scale, post_weight=_cuda(s["post"]), pre_weight=_cuda(s["pre"]), kind=kind,
               eps=EPS)
    y, r = pkg.add_norm(s["x"].cuda(), _cuda(s["residual"]), **how)
    w = {n: _wide(t) for n, t in s.items()}
    rows = None if w["gate"] is None else w["gate"].repeat_interleave(T // G, 0)
    ref = bc.norm_r(w["x"], w["residual"], w["gate"], scale, w["post"], kind, EPS)
    one = torch.ones(1, dtype=torch.float64)
    t = (_norm_error(w["x"], kind) * w["post"].abs() if w["post"] is not None else 0 * w["x"])
    part = (ref - (0 if w["residual"] is None else w["residual"])).abs()
    t = t * abs(scale) * (one if rows is None else rows.abs()) + 4 * bc.U * part + bc.U * ref.abs()
    mc.assert_within(r, ref, t + mc.rounding(ref.abs() + t, dtype), "r")
    kept = r.cpu().double()
    if s["pre"] is None:
        assert y is None
    else:
        ref = bc.normed(kept, kind, EPS) * w["pre"]
        t = _norm_error(kept, kind) * w["pre"].abs() + 2 * bc.U * ref.abs()
        mc.assert_within(y, ref, t + mc.rounding(ref.abs() + t, dtype), "y")
    if not grads:
        return
    d_y = torch.randn(T, H, generator=g).to(dtype) if s["pre"] is not None else None
    d_r = torch.randn(T, H, generator=g).to(dtype)
    got = pkg.add_norm_backward(_cuda(d_y), d_r.cuda(), s["x"].cuda(), r, **how)
    # by the formulas, from r as it was kept
    def back(d, v):
        """(gradient through normed, bound given a bound of d and of normed)"""
        m = v - v.mean(1, keepdim=True) if kind == "layer" else v
        rstd = 1 / torch.sqrt(m.square().mean(1, keepdim=True) + EPS)
        hat = m * rstd
        ref = d - hat * (d * hat).mean(1, keepdim=True)
        if kind == "layer":
            ref = ref - d.mean(1, keepdim=True)
        return rstd * ref, hat, rstd

    def back_error(d, td, v):
        m = v - v.mean(1, keepdim=True) if kind == "layer" else v
        rstd = 1 / torch.sqrt(m.square().mean(1, keepdim=True) + EPS)
        hat, th = (m * rstd).abs(), _norm_error(v, kind)
        d = d.abs()
        dot, tdot = (d * hat).mean(1, keepdim=True), (td * hat + d * th + td * th + ROW * d * hat).mean(1, keepdim=True)
        mean, tmean = d.mean(1, keepdim=True), (td + ROW * d).mean(1, keepdim=True)
        size = d + hat * dot + (mean if kind == "layer" else 0)
        return rstd * (td + th * dot + (hat + th) * tdot + tmean + 2 * ROW * size + _shift(v) * size)

    def _shift(v):      # relative error of the root mean square
        if kind == "rms":
            return ROW
        m = v - v.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt(m.square().mean(1, keepdim=True) + EPS)
        return ROW * (1 + rstd * v.abs().mean(1, keepdim=True))

    d, td = d_r.double(), 0 * kept
    sums = T + 64       # additions in a line, at most
    if s["pre"] is not None:
        e = d_y.double() * w["pre"]
        through, hat, _ = back(e, kept)
        td = back_error(e, 2 * bc.U * e.abs(), kept)
        ref = (d_y.double() * hat).sum(0)
        size = (d_y.double().abs() * hat.abs()).sum(0)
        t = (d_y.double().abs() * _norm_error(kept, kind)).sum(0) + sums * bc.U * size
        mc.assert_within(got.d_pre_weight, ref, t, "d_pre_weight")
        d = d + through
        td = td + bc.U * (d.abs() + d_r.double().abs() + through.abs())
    else:
        assert got.d_pre_weight is None
    mc.assert_within(got.d_residual, d, td + mc.rounding(d.abs() + td, dtype), "d_residual")
    u, tu = scale * d, abs(scale) * td + 2 * bc.U * (scale * d).abs()
    x = w["x"]
    n, tn = x, 0 * x
    if s["post"] is not None:
        n = bc.normed(x, kind, EPS) * w["post"]
        tn = _norm_error(x, kind) * w["post"].abs() + 2 * bc.U * n.abs()
    if rows is not None:
        by = lambda v: v.view(G, T // G, H).sum(1)  # noqa: E731
        ref = by(u * n)
        t = by(u.abs() * tn + tu * n.abs() + tu * tn) + sums * bc.U * by((u * n).abs())
        mc.assert_within(got.d_gate.view(G, H), ref, t + mc.rounding(ref.abs() + t, s["gate"].dtype), "d_gate")
        u, tu = u * rows, tu * rows.abs() + 2 * bc.U * (u * rows).abs()
    else:
        assert got.d_gate is None
    if s["post"] is not None:
        hat, th = bc.normed(x, kind, EPS), _norm_error(x, kind)
        ref = (u * hat).sum(0)
        t = (u.abs() * th + tu * hat.abs() + tu * th).sum(0) + sums * bc.U * (u * hat).abs().sum(0)
        mc.assert_within(got.d_post_weight, ref, t, "d_post_weight")
        f, tf = u * w["post"], tu * w["post"].abs() + 2 * bc.U * (u * w["post"]).abs()
        u, tu = back(f, x)[0], back_error(f, tf, x)
    else:
        assert got.d_post_weight is None
    mc.assert_within(got.d_x, u, tu + mc.rounding(u.abs() + tu, dtype), "d_x")


SIZES = [(1, 1, 1), (3, 5, 1), (4, 64, 4), (7, 129, 1), (12, 512, 3), (5, 513, 5), (9, 1000, 1), (6, 1024, 2),
         (5, 2047, 1), (8, 2048, 8), (3, 4095, 1), (6, 4096, 2), (4, 7168, 1), (3, 8192, 3), (1, 8191, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,H,G", SIZES)
def test_norm(T, H, G, kind, dtype):
    torch_cuda()
    g = torch.Generator().manual_seed(T * H)
    say(f"norm T={T} H={H} G={G} {kind} {dtype}")
    _check(_inputs(g, T, H, G, dtype), kind, 0.5, G, g=g)


@pytest.mark.parametrize("weight", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("residual,gate,post,pre", [
    (False, False, False, True), (True, False, False, True), (True, True, False, False), (False, True, True, False),
    (True, False, True, True), (True, True, False, True), (False, False, False, False), (True, False, True, False),
])
def test_parts_left_out(residual, gate, post, pre, weight):
    torch_cuda()
    g = torch.Generator().manual_seed(8)
    say(f"norm parts {residual} {gate} {post} {pre}")
    for kind in ("rms", "layer"):
        _check(_inputs(g, 10, 200, 5, torch.bfloat16, residual, gate, post, pre, weight), kind, -1.5, 5, g=g)


@pytest.mark.parametrize("T,H,G", [(3000, 40, 1), (3000, 40, 3), (3000, 40, 1500), (3000, 40, 3000), (2100, 600, 7),
                                   (1300, 4096, 1), (1025, 130, 1025), (2048, 130, 1024), (4000, 16, 1000)])
def test_sums_over_many_rows(T, H, G):
    """Workers with many rows, several gate rows, or a share of one."""
    torch_cuda()
    g = torch.Generator().manual_seed(T + G)
    say(f"norm sums T={T} H={H} G={G}")
    _check(_inputs(g, T, H, G, torch.bfloat16), "rms", 1.0, G, g=g)


def test_norm_backward_against_differences():
    torch_cuda()
    g = torch.Generator().manual_seed(4)
    T, H, G = 6, 24, 3
    for kind in ("rms", "layer"):
        say(f"norm differences {kind}")
        s = _inputs(g, T, H, G, torch.float32)
        d_y, d_r = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)
        how = dict(gate=s["gate"].cuda(), scale=0.7, post_weight=s["post"].cuda(), pre_weight=s["pre"].cuda(),
                   kind=kind, eps=EPS)
        _, r = pkg.add_norm(s["x"].cuda(), s["residual"].cuda(), **how)
        got = pkg.add_norm_backward(d_y.cuda(), d_r.cuda(), s["x"].cuda(), r, **how)
        w = {n: t.double() for n, t in s.items()}

        def loss(v):
            r = bc.norm_r(v["x"], v["residual"], v["gate"], 0.7, v["post"], kind, EPS)
            return float((d_y.double() * bc.normed(r, kind, EPS) * v["pre"]).sum() + (d_r.double() * r).sum())

        for name, grad in (("x", got.d_x), ("residual", got.d_residual), ("gate", got.d_gate),
                           ("post", got.d_post_weight), ("pre", got.d_pre_weight)):
            v = torch.randn(s[name].shape, generator=g).double()
            h = 1e-5        # h^2 / 6 times third derivatives below 1e3; 1e-14 / h
            slope = (loss({**w, name: w[name] + h * v}) - loss({**w, name: w[name] - h * v})) / (2 * h)
            dot = grad.cpu().double() * v
            assert abs(float(dot.sum()) - slope) <= 1e-6 + 2.0 ** -15 * float(dot.abs().sum()), name


def test_rows_of_zeros_and_constants():
    """What the mean square leaves nothing of."""
    torch_cuda()
    for kind in ("rms", "layer"):
        for H in (64, 700, 5000):
            x = torch.zeros(4, H)
            x[1], x[2, 3] = 2.0, 1.0
            s = dict(x=x.bfloat16(), residual=torch.zeros(4, H).bfloat16(), gate=None, post=torch.ones(H),
                     pre=torch.ones(H))
            say(f"norm constants {kind} H={H}")
            _check(s, kind, 1.0, 1, grads=False)


@pytest.mark.parametrize("H", [130, 512, 3001])
def test_norm_strides_alignment_and_streams(H):
    """Rows apart, from odd elements on, a gate of broadcast rows, another
    stream: the same bits."""
    torch_cuda()
    g = torch.Generator().manual_seed(H)
    T = 6
    wide = lambda: torch.randn(T, H + 9, generator=g).bfloat16().cuda()[:, 3:H + 3]  # noqa: E731
    x, res, d_y, d_r = (wide() for _ in range(4))
    w = torch.randn(H + 1, generator=g).cuda()[1:]
    gate = torch.randn(1, H, generator=g).bfloat16().cuda()
    say(f"norm strides H={H}")
    how = dict(scale=0.5, post_weight=w, pre_weight=w, kind="layer", eps=EPS)
    y, r = pkg.add_norm(x, res, gate=gate, **how)
    y2, r2 = pkg.add_norm(x.contiguous(), res.contiguous(), gate=gate[0], **how)
    assert torch.equal(y, y2) and torch.equal(r, r2)
    y2, r2 = pkg.add_norm(x, res, gate=gate.expand(T, H), **how)        # stride 0
    assert torch.equal(y, y2) and torch.equal(r, r2)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    y2, r2 = pkg.add_norm(x, res, gate=gate, stream=stream, **how)
    a = pkg.add_norm_backward(d_y, d_r, x, r2, gate=gate, stream=stream, **how)
    stream.synchronize()
    assert torch.equal(y, y2) and torch.equal(r, r2)
    b = pkg.add_norm_backward(d_y.contiguous(), d_r.contiguous(), x.contiguous(), r, gate=gate[0], **how)
    assert all(torch.equal(p.view(-1), q.view(-1)) for p, q in zip(a, b))
    c = pkg.add_norm_backward(d_y, d_r, x, r, gate=gate.expand(T, H), **how)
    ref = (c.d_gate.double().sum(0) - b.d_gate.double().view(-1)).abs()
    assert (ref <= (T + 2) * mc.HALF[torch.bfloat16] * c.d_gate.double().abs().sum(0)).all()


def test_norm_without_rows_or_gradients():
    torch_cuda()
    H = 96
    x = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H, device="cuda")
    gate = torch.ones(3, H, device="cuda")
    say("norm T=0")
    how = dict(gate=gate, post_weight=w, pre_weight=w)
    y, r = pkg.add_norm(x, x, **how)
    assert y.shape == r.shape == (0, H)
    got = pkg.add_norm_backward(y, r, x, r, **how)
    assert got.d_x.shape == (0, H) and not got.d_gate.any() and not got.d_post_weight.any() and not got.d_pre_weight.any()
    x = torch.randn(5, H, device="cuda")
    y, r = pkg.add_norm(x, pre_weight=w)
    got = pkg.add_norm_backward(None, None, x, r, pre_weight=w, residual=False)
    assert not got.d_x.any() and got.d_residual is None and not got.d_pre_weight.any()
