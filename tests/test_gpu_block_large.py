"""Elements past 2^32, and outputs past 2^31: the last rows of a long input give
the bits that they give alone."""
import pytest
import torch

import mxfp8_block_scaled_mxgemm_amd as pkg
from gpu_common import say, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _freed():
    yield
    torch.cuda.empty_cache()


def _long(rows, cols, tail, dtype=torch.bfloat16, seed=0):
    """Zeros, but for random rows at both ends."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros(rows, cols, dtype=dtype, device="cuda")
    for part in (x[:tail], x[-tail:]):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    assert x.numel() > 2 ** 32
    return x


def test_norm_rows_past_32_bits():
    torch_cuda()
    T, H, n = 540000, 8192, 40
    say("norm, 540000 x 8192")
    x = _long(T, H, n)
    w = torch.linspace(0.5, 1.5, H, device="cuda")
    y, r = pkg.add_norm(x, x, scale=0.5, post_weight=w, pre_weight=w)
    for part in (slice(0, n), slice(T - n, T)):
        y1, r1 = pkg.add_norm(x[part], x[part], scale=0.5, post_weight=w, pre_weight=w)
        assert torch.equal(y[part], y1) and torch.equal(r[part], r1)
    del y
    got = pkg.add_norm_backward(x, x, x, r, scale=0.5, post_weight=w, pre_weight=w)
    for part in (slice(0, n), slice(T - n, T)):
        one = pkg.add_norm_backward(x[part], x[part], x[part], r[part], scale=0.5, post_weight=w, pre_weight=w)
        assert torch.equal(got.d_x[part], one.d_x) and torch.equal(got.d_residual[part], one.d_residual)


def test_route_rows_past_32_bits():
    torch_cuda()
    T, E, k, n = 17_000_000, 256, 4, 100
    say("route, 17000000 x 256")
    x = _long(T, E, n)
    how = dict(score="sigmoid", scale=2.0)
    bias = torch.linspace(-0.1, 0.1, E, device="cuda")
    ids, w = pkg.route_tokens(x, k, bias=bias, groups=8, top_groups=4, **how)
    d = torch.ones_like(w)
    d[:, 0] = -1.0
    got = pkg.route_tokens_backward(d, x, ids, **how)
    for part in (slice(0, n), slice(T - n, T)):
        # (enough tokens for the kernel that the long input takes)
        some = slice(0, 5000) if part.start == 0 else slice(T - 5000, T)
        keep = slice(0, n) if part.start == 0 else slice(5000 - n, 5000)
        i1, w1 = pkg.route_tokens(x[some], k, bias=bias, groups=8, top_groups=4, **how)
        assert torch.equal(ids[part], i1[keep]) and torch.equal(w[part], w1[keep])
        one = pkg.route_tokens_backward(d[some].contiguous(), x[some], i1, **how)
        assert torch.equal(got[part], one[keep])


def test_quantise_elements_past_32_bits():
    torch_cuda()
    M, C, n = 33024, 131072, 128
    say("quantise, 33024 x 131072")
    x = _long(M, C, n)
    (q, s), (qt, st) = pkg.block_quantize(x, cols=True)
    for part in (slice(0, n), slice(M - n, M)):
        (q1, s1), (qt1, st1) = pkg.block_quantize(x[part], cols=True)
        assert torch.equal(q[part], q1) and torch.equal(s[part], s1)
        assert torch.equal(qt[:, part], qt1)
        assert torch.equal(st[:, part.start // 128:part.stop // 128], st1)


@pytest.mark.parametrize("precision", ["exact", "native"])
def test_products_past_32_bits(precision):
    """Outputs of more than 2^31 elements; codes of more than 2^32 bytes."""
    torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    code = lambda *s: (torch.randn(*s, generator=g, device="cuda")).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    M, N, K, n = 66048, 33024, 128, 256
    say(f"product {M} x {N} x {K} {precision}")
    a, w = code(M, K), code(N, K)
    a_s, w_s = torch.rand(M, 1, generator=g, device="cuda"), torch.rand(N // 128, 1, generator=g, device="cuda")
    out = pkg.block_linear(a, a_s, w, w_s, precision=precision, tile_cfg=1)
    assert out.numel() > 2 ** 31
    one = pkg.block_linear(a[-n:], a_s[-n:], w, w_s, precision=precision, tile_cfg=1)
    assert torch.equal(out[-n:], one)
    del out, one
    E, N, K = 260, 4096, 4224
    say(f"product by expert, {E} of {N} x {K}")
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    assert w.numel() > 2 ** 32
    w[-1] = code(N, K)
    a = code(64, K)
    a_s, w_s = (torch.rand(*s, generator=g, device="cuda") for s in ((64, K // 128), (E, N // 128, K // 128)))
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = 64
    for cfg in (1, 3):
        got = pkg.block_linear(a, a_s, w, w_s, off, precision=precision, tile_cfg=cfg)
        one = pkg.block_linear(a, a_s, w[-1:], w_s[-1:], off[-2:], precision=precision, tile_cfg=cfg)
        assert torch.equal(got, one)
    del w
    M, N, E = 8192, 8192, 34
    say(f"product by inner, {E} x {M} x {N}")
    a, w = code(M, 128 * E), code(N, 128 * E)
    a_s, w_s = torch.rand(M, E, generator=g, device="cuda"), torch.rand(N, E, generator=g, device="cuda")
    off = (torch.arange(E + 1, device="cuda") * 128).int()
    out = pkg.block_linear_by_inner(a, a_s, w, w_s, off, precision=precision)
    assert out.numel() > 2 ** 31
    last = slice(128 * (E - 1), None)
    one = pkg.block_linear_by_inner(a[:, last].contiguous(), a_s[:, -1:].contiguous(), w[:, last].contiguous(),
                                    w_s[:, -1:].contiguous(), off[:2], precision=precision)
    assert torch.equal(out[-1], one[0])
