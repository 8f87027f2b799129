"""Quantisation to FP8 with scales of 128, and the products of such operands,
against 64 bits."""
import math

import pytest
import torch

import block_common as bc
import moe_common as mc
import mxfp8_block_scaled_mxgemm_amd as pkg
from gpu_common import say, torch_cuda

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- quantise --

def _forward(x, act, gated):
    """y and its error bound in FP32."""
    x = x.double()
    if not gated:
        y = mc.act(x, act)
        return y, (mc.ACT_ERR * x.abs() if act != "none" else 0 * y)
    h = x.shape[1] // 2
    a, u = mc.act(x[:, :h], act), x[:, h:]
    t = (mc.ACT_ERR * x[:, :h].abs() if act != "none" else 0 * a) * u.abs() + bc.U * (a * u).abs()
    return a * u, t


def _backward(d, z, act, gated):
    d, z = d.double(), z.double()
    one = lambda v: (4 * mc.ACT_ERR * (1 + v.abs()) if act != "none" else 0 * v)  # noqa: E731
    if not gated:
        s = mc.act_grad(z, act)
        return d * s, d.abs() * (one(z) + 2 * bc.U * s.abs())
    h = z.shape[1] // 2
    g, u = z[:, :h], z[:, h:]
    s, a = mc.act_grad(g, act), mc.act(g, act)
    y = torch.cat([d * u * s, d * a], 1)
    return y, torch.cat([(d * u).abs() * one(g), d.abs() * one(g)], 1) + 3 * bc.U * y.abs()


def _sorted(g, M, E, drop):
    ids = mc.ids_of(g, M, 1, E, drop)
    return pkg.sort_tokens(ids.cuda(), E), *mc.order(ids, E)[:2]


def _check_quantized(rows, cols, y, t, fmt, offsets=None, k_offsets=None, E=0):
    (q, s), (qt, st) = rows, cols
    M, C = y.shape
    live = M if offsets is None else offsets[-1]
    if q is not None:
        assert s.t().is_contiguous()
        assert not q[live:].any() and not s[live:].any()
        if live:
            bc.check_blocks(q[:live], s[:live], y[:live], t[:live], fmt, "rows")
    if qt is None:
        return
    parts, errors = [], []
    ends = [0, M] if offsets is None else offsets
    for lo, hi in zip(ends, ends[1:]):
        pad = (0, 0, 0, bc.up(hi - lo) - (hi - lo))
        parts.append(torch.nn.functional.pad(y[lo:hi], pad))
        errors.append(torch.nn.functional.pad(t[lo:hi], pad))
    wide, err = torch.cat(parts), torch.cat(errors)
    used = wide.shape[0]
    assert qt.shape == (C, bc.up(M) + 128 * E) and used == (bc.up(M) if k_offsets is None else k_offsets[-1])
    assert not qt[:, used:].any() and not st[:, used // 128:].any()
    if used:
        bc.check_blocks(qt[:, :used], st[:, :used // 128], wide.t(), err.t(), fmt, "columns")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("act,gated", [("none", False), ("silu", True), ("gelu", False), ("gelu_tanh", True),
                                       ("relu", True), ("none", True)])
@pytest.mark.parametrize("M,C,E,drop,fmt", [
    (1, 1, 0, 0, "e4m3"), (3, 130, 0, 0, "e5m2"), (128, 128, 0, 0, "e4m3"), (200, 300, 0, 0, "e4m3"),
    (257, 64, 5, 0.1, "e5m2"), (300, 257, 3, 0.5, "e4m3"), (40, 128, 2, 1.0, "e4m3"), (700, 384, 40, 0.05, "e4m3"),
])
def test_block_quantize(M, C, E, drop, fmt, act, gated, dtype):
    torch_cuda()
    g = torch.Generator().manual_seed(M * C)
    x = torch.randn(M, 2 * C if gated else C, generator=g).to(dtype)
    say(f"quantize M={M} C={C} E={E} {act} {gated} {fmt} {dtype}")
    sort = offsets = k_offsets = None
    if E:
        sort, offsets, k_offsets = _sorted(g, M, E, drop)
    y, t = _forward(x, act, gated)
    how = dict(act=act, gated=gated, sort=sort, fmt=fmt)
    both = pkg.block_quantize(x.cuda(), cols=True, **how)
    _check_quantized(*both, y, t, fmt, offsets, k_offsets, E)
    rows, none = pkg.block_quantize(x.cuda(), **how)
    assert none == (None, None) and all(torch.equal(p, q) for p, q in zip(rows, both[0]))
    none, cols = pkg.block_quantize(x.cuda(), rows=False, cols=True, **how)
    assert none == (None, None) and all(torch.equal(p, q) for p, q in zip(cols, both[1]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("act,gated", [("silu", False), ("silu", True), ("gelu", True), ("gelu_tanh", False),
                                       ("relu", True), ("none", True), ("none", False)])
@pytest.mark.parametrize("M,N,E,drop,fmt", [
    (1, 2, 0, 0, "e4m3"), (5, 34, 0, 0, "e5m2"), (128, 256, 0, 0, "e4m3"), (200, 300, 0, 0, "e4m3"),
    (257, 64, 5, 0.1, "e5m2"), (300, 258, 3, 0.5, "e4m3"), (40, 512, 2, 1.0, "e4m3"), (700, 384, 40, 0.05, "e4m3"),
])
def test_block_quantize_backward(M, N, E, drop, fmt, act, gated, dtype):
    torch_cuda()
    g = torch.Generator().manual_seed(M * N)
    d = (torch.randn(M, N // 2 if gated else N, generator=g) * 0.01).to(dtype)
    z = torch.randn(M, N, generator=g).bfloat16()
    say(f"quantize backward M={M} N={N} E={E} {act} {gated} {fmt} {dtype}")
    sort = offsets = k_offsets = None
    if E:
        sort, offsets, k_offsets = _sorted(g, M, E, drop)
    y, t = _backward(d, z, act, gated)
    rows, cols = pkg.block_quantize_backward(d.cuda(), z.cuda(), act=act, gated=gated, sort=sort, fmt=fmt)
    _check_quantized(rows, cols, y, t, fmt, offsets, k_offsets, E)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("E,N,K,fmt", [(0, 1, 128, "e4m3"), (0, 128, 128, "e5m2"), (3, 200, 384, "e4m3"),
                                       (2, 300, 130, "e4m3"), (0, 5, 3, "e4m3"), (1, 129, 257, "e5m2")])
def test_block_quantize_weight(E, N, K, fmt, dtype):
    torch_cuda()
    g = torch.Generator().manual_seed(N * K)
    lead = (E,) if E else ()
    w = torch.randn(*lead, N, K, generator=g).to(dtype)
    say(f"quantize weight E={E} N={N} K={K} {fmt} {dtype}")
    (q, s), (qt, st) = pkg.block_quantize_weight(w.cuda(), fmt=fmt, transposed=True)
    Np, Kp = bc.up(N), bc.up(K)
    assert q.shape == (*lead, N, Kp) and s.shape == (*lead, Np // 128, Kp // 128)
    assert qt.shape == (*lead, K, Np) and st.shape == (*lead, Kp // 128, Np // 128)
    assert torch.equal(st, s.transpose(-1, -2))
    assert torch.equal(qt[..., :N], q[..., :K].transpose(-1, -2)) and not qt[..., N:].any() and not q[..., K:].any()
    q2, s2 = pkg.block_quantize_weight(w.cuda(), fmt=fmt)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    wide = torch.nn.functional.pad(w.double(), (0, Kp - K, 0, Np - N))
    ref = (wide.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128)).abs().amax((-3, -1)) / bc.FMAX[fmt]).clamp(min=bc.LOW)
    mc.assert_within(s, ref, 2 * bc.U * ref, "scales")
    v = bc.square_value(q.cpu(), s.cpu(), fmt)
    each = s.cpu().double().repeat_interleave(128, -2).repeat_interleave(128, -1)[..., :N, :]
    wide = wide[..., :N, :]
    mc.assert_within(v, wide, (bc.REL[fmt] + 3 * bc.U) * wide.abs() + bc.SUB[fmt] * (1 + 4 * bc.U) * each, "codes")


def test_blocks_of_zeros_tiny_huge_and_non_finite():
    torch_cuda()
    x = torch.zeros(9, 128)
    x[1, 3] = 1e-38 * 3                 # below fmax 2^-126
    x[2] = torch.logspace(-44, -38, 128)
    x[3] = 3.4e38
    x[4, 7] = math.nan
    x[5, 9] = math.inf
    x[6, 9] = -math.inf
    x[7] = torch.linspace(-448, 448, 128)
    x[8, 0], x[8, 1] = -0.0, 1.0
    for fmt in ("e4m3", "e5m2"):
        say(f"unusual blocks {fmt}")
        (q, s), (qt, st) = pkg.block_quantize(x.cuda(), fmt=fmt, cols=True)
        fine = [0, 1, 2, 3, 7, 8]
        y = x[fine].double()
        bc.check_blocks(q[fine], s[fine], y, 0 * y, fmt, "rows")
        assert torch.isnan(s[4:7]).all() and (q[4:7] == 0x7F).all()
        bad = ~torch.isfinite(x).all(0)
        assert torch.isnan(st.cpu()[bad]).all() and (qt.cpu()[bad] == 0x7F).all()
        assert torch.isfinite(st.cpu()[~bad]).all()
        w, ws = pkg.block_quantize_weight(x.cuda(), fmt=fmt)
        assert torch.isnan(ws).all() and (w == 0x7F).all()


def test_quantize_reads_no_dropped_row_and_leaves_nothing_unwritten():
    torch_cuda()
    g = torch.Generator().manual_seed(4)
    M, C, E = 300, 80, 6
    sort, offsets, k_offsets = _sorted(g, M, E, 0.3)
    live = offsets[-1]
    x = torch.randn(M, C, generator=g)
    x[live:] = math.nan
    junk = [torch.full(s, 0xA5, dtype=torch.uint8, device="cuda") for s in ((M, 128), (C, 384 + 128 * E), (M * 4,),
                                                                           ((3 + E) * C * 4,))]
    del junk        # what allocations of these sizes hold next
    say("quantize: dropped rows of NaN")
    rows, cols = pkg.block_quantize(x.cuda(), sort=sort, cols=True)
    y = torch.where(torch.isnan(x), 0.0, x).double()
    _check_quantized(rows, cols, y, 0 * y, "e4m3", offsets, k_offsets, E)
    rows, _ = pkg.block_quantize(x.cuda(), sort=sort)
    _check_quantized(rows, (None, None), y, 0 * y, "e4m3", offsets, k_offsets, E)


def test_quantize_strides_streams_and_none():
    torch_cuda()
    g = torch.Generator().manual_seed(6)
    wide = torch.randn(90, 400, generator=g).bfloat16().cuda()
    x, z = wide[:, 3:203], wide[:, 101:301]
    say("quantize strides")
    same = lambda a, b: all(torch.equal(p, q) for m, n in zip(a, b) for p, q in zip(m, n))  # noqa: E731
    one = pkg.block_quantize(x, act="silu", gated=True, cols=True)
    assert same(one, pkg.block_quantize(x.contiguous(), act="silu", gated=True, cols=True))
    assert same(pkg.block_quantize_backward(x, z, act="gelu"),
                pkg.block_quantize_backward(x.contiguous(), z.contiguous(), act="gelu"))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    two = pkg.block_quantize(x, act="silu", gated=True, cols=True, stream=stream)
    stream.synchronize()
    assert same(one, two)
    (q, s), (qt, st) = pkg.block_quantize(x[:0], cols=True)
    assert q.shape == (0, 256) and s.shape == (0, 2) and qt.shape == (200, 0) and st.shape == (200, 0)
    sort = pkg.sort_tokens(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 3)
    (q, s), (qt, st) = pkg.block_quantize(x[:0], cols=True, sort=sort)
    assert qt.shape == (200, 384) and not qt.any() and not st.any()
    # segments where there are no rows
    bad = sort._replace(k_offsets=torch.tensor([0, 128, 128, 384], dtype=torch.int32, device="cuda"))
    for act, gated in (("none", False), ("silu", True)):
        _, (qt, st) = pkg.block_quantize(x[:0], act=act, gated=gated, cols=True, sort=bad)
        assert not qt.any() and not st.any()
    _, (qt, st) = pkg.block_quantize_backward(x[:0, :128], torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"),
                                              act="silu", gated=True, sort=bad)
    assert not qt.any() and not st.any()


# ---------------------------------------------------------------- products --

TILES = {0: (False, False), 1: (True, True), 2: (True, True), 3: (True, False), 4: (True, False)}   # exact? rows of scales?


def _operands(g, M, N, K, a_fmt, w_fmt, squares, lead=()):
    a = torch.randn(M, K, generator=g)
    a = torch.where(torch.rand(M, K, generator=g) < 0.01, a * 30, a)
    w = torch.randn(*lead, N, K, generator=g)
    return *bc.blocks(a, a_fmt), *(bc.squares(w, w_fmt) if squares else bc.blocks(w, w_fmt))


def _values(w, w_s, fmt, squares):
    return bc.square_value(w, w_s, fmt) if squares else bc.value(w, w_s, fmt)


def _check_product(out, a, w, precision, dtype, what):
    ref = a @ w.t()
    t = bc.product_error(a.abs() @ w.abs().t(), a.shape[1], precision)
    mc.assert_within(out, ref, t + mc.rounding(ref.abs() + t, dtype), what)


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("cfg", [-1, *TILES])
@pytest.mark.parametrize("squares", [True, False])
def test_block_linear(squares, cfg, precision):
    torch_cuda()
    if cfg >= 0 and (precision == "exact" and not TILES[cfg][0] or not squares and not TILES[cfg][1]):
        pytest.skip("no kernel of this tile")
    g = torch.Generator().manual_seed(cfg + 3)
    for M, N, K, a_fmt, w_fmt, dtype in ((1, 1, 128, "e4m3", "e4m3", torch.float32),
                                         (300, 264, 384, "e5m2", "e4m3", torch.float32),
                                         (37, 50, 128, "e4m3", "e5m2", torch.bfloat16),
                                         (513, 700, 640, "e4m3", "e4m3", torch.float16),
                                         (64, 130, 2176, "e4m3", "e4m3", torch.bfloat16),
                                         (17, 2051, 1024, "e5m2", "e5m2", torch.float32)):
        say(f"linear M={M} N={N} K={K} cfg={cfg} {precision} {a_fmt} {w_fmt} {dtype} squares={squares}")
        a, a_s, w, w_s = _operands(g, M, N, K, a_fmt, w_fmt, squares)
        out = pkg.block_linear(a.cuda(), a_s.cuda(), w.cuda(), w_s.cuda(), out_dtype=dtype, precision=precision,
                               a_fmt=a_fmt, w_fmt=w_fmt, tile_cfg=cfg)
        assert out.shape == (M, N) and out.dtype == dtype
        _check_product(out, bc.value(a, a_s, a_fmt), _values(w, w_s, w_fmt, squares), precision, dtype, "out")


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("cfg", [-1, *TILES])
@pytest.mark.parametrize("M,N,K,E,drop", [(1, 40, 128, 3, 0.0), (70, 200, 384, 5, 0.2), (600, 130, 1152, 3, 0.1),
                                          (50, 64, 256, 300, 0.0), (9, 64, 256, 2, 1.0)])
def test_block_linear_by_expert(M, N, K, E, drop, cfg, precision):
    torch_cuda()
    if precision == "exact" and cfg >= 0 and not TILES[cfg][0]:
        pytest.skip("no kernel of this tile")
    g = torch.Generator().manual_seed(M + N)
    for squares in (True, False):
        if not squares and cfg >= 0 and not TILES[cfg][1]:
            continue
        say(f"by expert M={M} N={N} K={K} E={E} cfg={cfg} {precision} squares={squares}")
        sort, offsets, _ = _sorted(g, M, E, drop)
        a, a_s, w, w_s = _operands(g, M, N, K, "e4m3", "e4m3", squares, (E,))
        a[offsets[-1]:], a_s[offsets[-1]:] = 0x7F, math.nan        # dropped rows are not read
        out = pkg.block_linear(a.cuda(), a_s.cuda(), w.cuda(), w_s.cuda(), offsets=sort.offsets, precision=precision,
                               out_dtype=torch.float32, tile_cfg=cfg)
        assert not out[offsets[-1]:].any()
        av, wv = bc.value(a, a_s, "e4m3"), _values(w, w_s, "e4m3", squares)
        for e in range(E):
            lo, hi = offsets[e], offsets[e + 1]
            if hi > lo:
                _check_product(out[lo:hi], av[lo:hi], wv[e], precision, torch.float32, f"expert {e}")


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("cfg", [-1, 1, 2])
def test_block_linear_by_inner(cfg, precision, out_dtype):
    """Inner ranges that are empty, a block, several and many; columns beyond
    the last range are no expert's."""
    torch_cuda()
    steps = [0, 1, 3, 0, 6, 17]
    offsets = [0]
    for n in steps:
        offsets.append(offsets[-1] + 128 * n)
    K = offsets[-1] + 256
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(cfg + 3)
    for M, N, a_fmt in ((300, 264, "e5m2"), (37, 50, "e4m3"), (1, 1, "e4m3")):
        say(f"by inner M={M} N={N} K={K} cfg={cfg} {precision} {out_dtype} {a_fmt}")
        a, a_s, w, w_s = _operands(g, M, N, K, a_fmt, "e4m3", False)
        a[:, offsets[-1]:], a_s[:, offsets[-1] // 128:] = 0x7F, math.nan        # never read
        out = pkg.block_linear_by_inner(a.cuda(), a_s.t().contiguous().t().cuda(), w.cuda(), w_s.cuda(), off,
                                        out_dtype=out_dtype, precision=precision, a_fmt=a_fmt, tile_cfg=cfg)
        assert out.shape == (len(steps), M, N) and out.dtype == out_dtype
        av, wv = bc.value(a, a_s, a_fmt), bc.value(w, w_s, "e4m3")
        for e in range(len(steps)):
            lo, hi = offsets[e], offsets[e + 1]
            if hi == lo:
                assert not out[e].any()
            else:
                _check_product(out[e], av[:, lo:hi], wv[:, lo:hi], precision, out_dtype, f"expert {e}")


@pytest.mark.parametrize("cfg", [-1, *TILES])
def test_whole_numbers_are_exact(cfg):
    """Codes and scales whose products and sums are exact in every step: the
    same numbers from every tile, precision and order."""
    torch_cuda()
    g = torch.Generator().manual_seed(11)
    M, N, K = 260, 300, 1024
    small = lambda *s: torch.randint(-3, 4, s, generator=g).float().to(torch.float8_e4m3fn)  # noqa: E731
    power = lambda *s: torch.exp2(torch.randint(-2, 3, s, generator=g).float())  # noqa: E731
    a, w, a_s, w_s = small(M, K), small(N, K), power(M, K // 128), power(3, K // 128)
    ref = (a.double() * a_s.double().repeat_interleave(128, 1)) @ \
        (w.double() * w_s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)).t()
    for precision in ("exact", "native"):
        if precision == "exact" and cfg >= 0 and not TILES[cfg][0]:
            continue
        say(f"whole numbers cfg={cfg} {precision}")
        out = pkg.block_linear(a.view(torch.uint8).cuda(), a_s.cuda(), w.view(torch.uint8).cuda(), w_s.cuda(),
                               out_dtype=torch.float32, precision=precision, tile_cfg=cfg)
        assert torch.equal(out.cpu().double(), ref)


def test_scales_of_any_strides_and_transposed_weights():
    torch_cuda()
    g = torch.Generator().manual_seed(12)
    M, N, K = 200, 256, 384
    a, a_s, w, w_s = (t.cuda() for t in _operands(g, M, N, K, "e4m3", "e4m3", True))
    say("strided scales")
    ref = pkg.block_linear(a, a_s, w, w_s)
    spread = torch.zeros(M, 3, 5, device="cuda")
    spread[:, :, 2] = a_s
    pad = torch.zeros(M, K + 64, dtype=torch.uint8, device="cuda")
    pad[:, :K] = a
    assert torch.equal(pkg.block_linear(pad[:, :K], spread[:, :, 2], w, w_s.t().contiguous().t()), ref)
    assert torch.equal(pkg.block_linear(a, a_s.t().contiguous().t(), w.t().contiguous().t(), w_s), ref)
    one = a_s[:1].expand(M, -1)             # one row's scales for all
    assert torch.equal(pkg.block_linear(a, one, w, w_s), pkg.block_linear(a, one.contiguous(), w, w_s))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = pkg.block_linear(a, a_s, w, w_s, stream=stream)
    stream.synchronize()
    assert torch.equal(out, ref)
    assert pkg.block_linear(a[:0], a_s[:0], w, w_s).shape == (0, N)


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("M,N,K,by", [(2048, 4096, 2176, 0), (3000, 2000, 1152, 0), (64, 2048, 7168, 0),
                                      (16, 4096, 4096, 0), (3000, 2048, 1024, 12), (4352, 4096, 2048, 4),
                                      (4096, 4352, 2048, 0)])
def test_block_products_repeat_bit_for_bit(M, N, K, by, precision):
    """The same inputs give the same bits on every call, with other work in
    between; and near the library's product in 64 bits."""
    torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(M)
    lead = (by,) if by else ()
    code = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.float8_e4m3fn)  # noqa: E731
    scale = lambda *s: torch.rand(*s, generator=g, device="cuda") + 0.5  # noqa: E731
    a, w, a_s, w_s = code(M, K), code(*lead, N, K), scale(M, K // 128), scale(*lead, bc.up(N) // 128, K // 128)
    offsets, ends = None, [0, M]
    if by:
        sort, ends, _ = _sorted(torch.Generator().manual_seed(M), M, by, 0.05)
        offsets = sort.offsets
    say(f"repeat M={M} N={N} K={K} by={by} {precision}")
    run = lambda x: pkg.block_linear(x.view(torch.uint8), a_s, w.view(torch.uint8), w_s, offsets=offsets,  # noqa: E731
                                     precision=precision, out_dtype=torch.float32)
    first = run(a)
    other = a.view(torch.uint8).flip(0)
    for _ in range(4):
        run(other)
        assert torch.equal(run(a), first)
    av = a.double() * a_s.double().repeat_interleave(128, 1)
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi == lo:
            continue
        we, se = (w[e], w_s[e]) if by else (w, w_s)
        wv = we.double() * se.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
        ref = torch.mm(av[lo:hi], wv.t())
        t = bc.product_error(torch.mm(av[lo:hi].abs(), wv.abs().t()), K, precision)
        assert ((first[lo:hi].double() - ref).abs() <= t + bc.U * (ref.abs() + t)).all()


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("act,gated,by", [("none", False, False), ("silu", True, False), ("silu", True, True),
                                          ("gelu", False, True)])
def test_block_linear_backward(act, gated, by, precision):
    """d_a and d_w are the products of what block_quantize_backward holds."""
    torch_cuda()
    g = torch.Generator().manual_seed(21)
    M, N, K, E = 300, 384 if gated else 200, 256, 3
    sort = _sorted(g, M, E, 0.1)[0] if by else None
    lead = (E,) if by else ()
    w = torch.randn(*lead, N, K, generator=g).cuda()
    x = torch.randn(M, K, generator=g).cuda()
    d = torch.randn(M, N // 2 if gated else N, generator=g).bfloat16().cuda()
    z = None if act == "none" and not gated else torch.randn(M, N, generator=g).bfloat16().cuda()
    _, (wt, wt_s) = pkg.block_quantize_weight(w, transposed=True)
    _, (at, at_s) = pkg.block_quantize(x, sort=sort, rows=False, cols=True)
    say(f"backward {act} gated={gated} by={by} {precision}")
    d_a, d_w = pkg.block_linear_backward(d, z, at, at_s, wt, wt_s, act=act, gated=gated, sort=sort, precision=precision,
                                         out_dtype=torch.float32)
    (q, s), (qt, st) = pkg.block_quantize_backward(d, z, act=act, gated=gated, sort=sort)
    rows, cols = bc.value(q.cpu(), s.cpu(), "e4m3"), bc.value(qt.cpu(), st.cpu(), "e4m3")
    av, wv = bc.value(at.cpu(), at_s.cpu(), "e4m3"), bc.square_value(wt.cpu(), wt_s.cpu(), "e4m3")
    ends = sort.offsets.tolist() if by else [0, M]
    blocks = sort.k_offsets.tolist() if by else [0, cols.shape[1]]
    assert d_a.shape == (M, K) and d_w.shape == (*lead, N, K)
    for e in range(len(ends) - 1):
        lo, hi = ends[e], ends[e + 1]
        _check_product(d_a[lo:hi], rows[lo:hi], wv[e] if by else wv, precision, torch.float32, "d_a")
        lo, hi = blocks[e], blocks[e + 1]
        _check_product(d_w[e] if by else d_w, cols[:, lo:hi], av[:, lo:hi], precision, torch.float32, "d_w")
    assert not d_a[ends[-1]:].any()


def test_block_linear_backward_without_tokens():
    torch_cuda()
    u8 = dict(dtype=torch.uint8, device="cuda")
    say("backward M=0")
    d = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    d_a, d_w = pkg.block_linear_backward(d, None, torch.zeros(256, 0, **u8), torch.zeros(256, 0, device="cuda"),
                                         torch.zeros(256, 128, **u8), torch.zeros(2, 1, device="cuda"))
    assert d_a.shape == (0, 256) and d_w.shape == (64, 256) and not d_w.any()
