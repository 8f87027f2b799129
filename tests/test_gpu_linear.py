"""The MXFP8 product with its fused epilogue, dense and by expert, and its
gradient on the GPU, against the definitions in 64 bits on the CPU."""
import pytest
import torch

import mxfp8_block_scaled_mxgemm_amd as pkg
import moe_common as mc
from gpu_common import say, torch_cuda

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
# tile configuration -> rows and columns of a tile, exact mode has it
TILES = {0: (256, 256, False), 1: (128, 128, True), 2: (64, 64, True), 3: (32, 32, True), 4: (16, 32, True)}


def _operands(g, M, N, K, a_fmt="e4m3", w_fmt="e4m3", lead=()):
    a, a_s = mc.codes(g, (M, K), a_fmt)
    w, w_s = mc.codes(g, (*lead, N, K), w_fmt, K ** -0.5)
    return a, a_s, w, w_s


def _cuda(*ts):
    return tuple(None if t is None else t.cuda() for t in ts)


def _check_out(out, ref, t, out_dtype, what):
    if isinstance(out_dtype, str):
        q, s = out[0], out[1]
        mc.assert_within(mc.value(q.cpu(), s.cpu(), out_dtype), ref, mc.mx_bound(ref, t, out_dtype), what)
    else:
        mc.assert_within(out, ref, t + mc.rounding(ref.abs() + t, out_dtype), what)


def _dense(M, N, K, act="none", gated=False, bias=None, residual=False, out_dtype=torch.bfloat16, preact=False,
           precision="exact", a_fmt="e4m3", w_fmt="e4m3", cfg=-1):
    say(f"linear M={M} N={N} K={K} act={act} gated={gated} bias={bias} residual={residual} out={out_dtype} "
        f"z={preact} {precision} {a_fmt} x {w_fmt} cfg={cfg}")
    g = torch.Generator().manual_seed(M * 7 + N * 3 + K)
    a, a_s, w, w_s = _operands(g, M, N, K, a_fmt, w_fmt)
    b = None if bias is None else torch.randn(N, generator=g).to(bias)
    cols = N // 2 if gated else N
    res_dtype = torch.bfloat16 if isinstance(out_dtype, str) else out_dtype
    res = torch.randn(M, cols, generator=g).to(res_dtype) if residual else None
    ca, ca_s, cw, cw_s, cb, cres = _cuda(a, a_s, w, w_s, b, res)
    out = pkg.linear(ca, ca_s, cw, cw_s, bias=cb, act=act, gated=gated, residual=cres, out_dtype=out_dtype,
                     preact=preact, precision=precision, a_fmt=a_fmt, w_fmt=w_fmt, tile_cfg=cfg)
    ref, t, z, tz = mc.linear(mc.value(a, a_s, a_fmt), mc.value(w, w_s, w_fmt), b, act, gated, res, precision)
    first = out if isinstance(out_dtype, str) else (out[0] if preact else out)
    _check_out(first, ref, t, out_dtype, "out")
    if preact:
        mc.assert_within(out[-1], z, tz + mc.rounding(z.abs() + tz, torch.bfloat16), "z")


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("cfg", sorted(TILES))
@pytest.mark.parametrize("K", [128, 384, 640, 1152])
def test_every_tile_whole_and_ragged(cfg, K, precision):
    torch_cuda()
    tm, tn, exact = TILES[cfg]
    if precision == "exact" and not exact:
        with pytest.raises(pkg.MxgemmError):
            _dense(tm, tn, K, precision=precision, cfg=cfg)
        return
    _dense(tm, 2 * tn, K, precision=precision, cfg=cfg)
    _dense(2 * tm + 5, tn + 7, K, "silu", bias=torch.float32, residual=True, preact=True, precision=precision, cfg=cfg)
    _dense(tm - 1, 2 * tn + 64, K, "gelu", gated=True, bias=torch.bfloat16, residual=True, out_dtype=torch.float32,
           preact=True, precision=precision, cfg=cfg)
    _dense(tm + 3, 2 * tn + 64, K, "gelu_tanh", gated=True, out_dtype="e4m3", precision=precision, cfg=cfg)
    _dense(tm + 3, tn + 32, K, "relu", bias=torch.float16, out_dtype="e5m2", residual=True, precision=precision,
           cfg=cfg)


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K,gated", [(1, 1, 128, False), (1, 2, 128, True), (3, 17, 256, False),
                                         (16, 130, 512, True), (100, 72, 1024, False), (129, 258, 256, True),
                                         (300, 515, 384, False)])
def test_dense_sizes(M, N, K, gated, act, precision):
    torch_cuda()
    for out_dtype in (torch.bfloat16, torch.float16, torch.float32):
        _dense(M, N, K, act, gated, torch.float32, True, out_dtype, True, precision)


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("a_fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("w_fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M", [5, 200, 600])
def test_formats(M, a_fmt, w_fmt, precision):
    torch_cuda()
    _dense(M, 384, 512, "silu", precision=precision, a_fmt=a_fmt, w_fmt=w_fmt)


@pytest.mark.parametrize("cfg", sorted(TILES))
@pytest.mark.parametrize("precision", ["exact", "native"])
def test_bit_exact_on_small_integers(cfg, precision):
    """Products and sums of small integers are exact in every step."""
    torch_cuda()
    tm, tn, exact = TILES[cfg]
    if precision == "exact" and not exact:
        pytest.skip("no exact kernel of this tile")
    M, N, K = tm + 9, tn + 40, 1280
    g = torch.Generator().manual_seed(cfg)
    av = torch.randint(-1, 2, (M, K), generator=g).float()
    wv = torch.where(torch.rand(N, K, generator=g) < 0.05, torch.randint(-2, 3, (N, K), generator=g).float(), 0.0)
    one = lambda v: (v.to(torch.float8_e4m3fn).view(torch.uint8),  # noqa: E731
                     torch.full((v.shape[0], K // 32), 127, dtype=torch.uint8))
    a, a_s = one(av)
    w, w_s = one(wv)
    out = pkg.linear(*_cuda(a, a_s, w, w_s), out_dtype=torch.float32, precision=precision, tile_cfg=cfg)
    assert torch.equal(out.cpu(), av @ wv.t())


def _grouped(ids, E, N, K, act, gated, out_dtype, precision, cfg=-1, bias=True, preact=False):
    T, k = ids.shape
    say(f"linear by expert rows={T * k} E={E} N={N} K={K} act={act} gated={gated} out={out_dtype} {precision} cfg={cfg}")
    g = torch.Generator().manual_seed(T + N)
    a, a_s, w, w_s = _operands(g, T * k, N, K, lead=(E,))
    b = torch.randn(E, N, generator=g) if bias else None
    cols = N // 2 if gated else N
    res = torch.randn(T * k, cols, generator=g).to(torch.bfloat16 if isinstance(out_dtype, str) else out_dtype)
    offsets = mc.order(ids, E)[0]
    sort = pkg.sort_tokens(ids.cuda(), E)
    live = offsets[-1]
    # rows of no expert hold NaN: they must not be read, and their outputs are zero
    a[live:], a_s[live:] = 0x7F, 0xFF
    ca, ca_s, cw, cw_s, cb, cres = _cuda(a, a_s, w, w_s, b, res)
    out = pkg.linear(ca, ca_s, cw, cw_s, bias=cb, act=act, gated=gated, residual=cres, offsets=sort.offsets,
                     out_dtype=out_dtype, preact=preact, precision=precision, tile_cfg=cfg)
    ref = torch.zeros(T * k, cols, dtype=torch.float64)
    t, z = torch.zeros_like(ref), torch.zeros(T * k, N, dtype=torch.float64)
    tz = torch.zeros_like(z)
    av = mc.value(a, a_s, "e4m3")
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            ref[lo:hi], t[lo:hi], z[lo:hi], tz[lo:hi] = mc.linear(
                av[lo:hi], mc.value(w[e], w_s[e], "e4m3"), None if b is None else b[e], act, gated, res[lo:hi],
                precision)
    first = out if isinstance(out_dtype, str) else (out[0] if preact else out)
    _check_out(first, ref, t, out_dtype, "out")
    if isinstance(out_dtype, str):
        assert not bool(first[0][live:].any()) and not bool(first[1][live:].any())
    if preact:
        mc.assert_within(out[-1], z, tz + mc.rounding(z.abs() + tz, torch.bfloat16), "z")


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("T,k,E,drop", [(1, 2, 8, 0.0), (1, 1, 1, 1.0), (9, 4, 6, 0.2), (70, 2, 3, 0.1),
                                        (301, 2, 70, 0.05), (700, 2, 4, 0.02), (64, 4, 130, 0.0)])
def test_by_expert(T, k, E, drop, precision):
    torch_cuda()
    ids = mc.ids_of(torch.Generator().manual_seed(T), T, k, E, drop)
    _grouped(ids, E, 96, 256, "none", False, torch.bfloat16, precision)
    _grouped(ids, E, 192, 384, "silu", True, torch.float32, precision, preact=True)
    _grouped(ids, E, 192, 128, "silu", True, "e4m3", precision)
    _grouped(ids, E, 160, 256, "gelu", False, "e5m2", precision, preact=True)


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("cfg", sorted(TILES))
def test_by_expert_every_tile(cfg, precision):
    torch_cuda()
    if precision == "exact" and not TILES[cfg][2]:
        pytest.skip("no exact kernel of this tile")
    # counts around a tile's height: empty, one, one below, whole, one above, several
    tm = TILES[cfg][0]
    counts = [0, 1, tm - 1, 0, tm, tm + 1, 2 * tm + 3]
    flat = torch.cat([torch.full((n,), e, dtype=torch.int32) for e, n in enumerate(counts)] +
                     [torch.full((tm + 2,), -1, dtype=torch.int32)])
    ids = flat[torch.randperm(len(flat), generator=torch.Generator().manual_seed(1))].view(-1, 1)
    _grouped(ids, 7, 128, 256, "silu", True, torch.bfloat16, precision, cfg, preact=True)
    _grouped(ids, 7, 96, 640, "none", False, "e4m3", precision, cfg, bias=False)


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("M,N,K", [(33, 64, 2048), (64, 200, 7168), (130, 515, 2176), (70, 96, 4096)])
def test_k_split_over_work_groups(M, N, K, precision):
    """Few tiles of a long K: split sums and their separate epilogue."""
    torch_cuda()
    _dense(M, N, K, precision=precision)
    _dense(M, N, K, "silu", bias=torch.float32, residual=True, preact=True, precision=precision)
    if N % 64 == 0:
        _dense(M, N, K, "gelu", gated=True, bias=torch.bfloat16, residual=True, out_dtype="e4m3", precision=precision)
        _dense(M, N, K, "relu", residual=True, out_dtype="e5m2", preact=True, precision=precision)
    if N % 2 == 0:
        _dense(M, N, K, "gelu_tanh", gated=True, residual=True, out_dtype=torch.float32, preact=True,
               precision=precision)


# ------------------------------------------------------------- non-finite ---

@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("M", [7, 70, 260])
def test_a_nan_block_reaches_its_row_only(M, precision):
    torch_cuda()
    g = torch.Generator().manual_seed(M)
    a, a_s, w, w_s = _operands(g, M, 160, 512)
    a_s[3, 5] = 0xFF
    out = pkg.linear(*_cuda(a, a_s, w, w_s), act="silu", precision=precision).cpu()
    bad = torch.isnan(out)
    assert bool(bad[3].all()) and int(bad.sum()) == 160
    q, s = pkg.linear(*_cuda(a, a_s, w, w_s), act="relu", precision=precision, out_dtype="e4m3")
    assert bool((s[3] == 255).all()) and int((s == 255).sum()) == 160 // 32 and bool((q[3] == 0x7F).all())


# --------------------------------------------------------------- gradient ---

def _dz(d, z, act, gated):
    d, z = d.double(), None if z is None else z.double()
    if gated:
        h = z.shape[1] // 2
        return torch.cat([d * z[:, h:] * mc.act_grad(z[:, :h], act), d * mc.act(z[:, :h], act)], 1)
    return d if z is None else d * mc.act_grad(z, act)


# FP32 evaluation of dz: a product or two of a slope known to a few units of
# 2^-24 of (1 + |z|), the largest term of any slope's formula
def _dz_error(d, z, gated):
    d = d.double().abs()
    if z is None:
        return d * 0
    z = z.double().abs()
    if gated:
        h = z.shape[1] // 2
        return 64 * 2.0 ** -24 * torch.cat([d * z[:, h:] * (1 + z[:, :h]), d * (1 + z[:, :h])], 1)
    return 64 * 2.0 ** -24 * d * (1 + z)


GRAD_CASES = [(1, 2, "silu", True), (1, 1, "none", False), (5, 34, "gelu", True), (130, 64, "gelu_tanh", False),
              (128, 128, "silu", True), (257, 200, "relu", False), (300, 514, "gelu", True), (64, 96, "none", False)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("by", [False, True])
@pytest.mark.parametrize("M,N,act,gated", GRAD_CASES)
def test_epilogue_backward(M, N, act, gated, by, fmt):
    torch_cuda()
    say(f"epilogue backward M={M} N={N} act={act} gated={gated} by={by} {fmt}")
    g = torch.Generator().manual_seed(M + N)
    cols = N // 2 if gated else N
    plain = act == "none" and not gated
    z = None if plain else (torch.randn(M, N, generator=g) * 2).bfloat16()
    E = 5
    sort, offsets, k_offsets = None, [0, M], [0, -(-M // 128) * 128]
    if by:
        ids = mc.ids_of(g, M, 1, E, 0.1)
        sort = pkg.sort_tokens(ids.cuda(), E)
        offsets, k_offsets = mc.order(ids, E)[:2]
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        d = torch.randn(M, cols, generator=g).to(dtype)
        (q, s), (qt, st), db = pkg.epilogue_backward(d.cuda(), None if z is None else z.cuda(), act=act, gated=gated,
                                                     sort=sort, fmt=fmt)
        dz, t = _dz(d, z, act, gated), _dz_error(d, z, gated)
        live = offsets[-1]
        Np = -(-N // 128) * 128
        assert tuple(q.shape) == (M, Np)
        pad = torch.nn.functional.pad
        ref, tr = pad(dz, (0, Np - N))[:live], pad(t, (0, Np - N))[:live]
        mc.assert_within(mc.value(q.cpu(), s.cpu(), fmt)[:live], ref, mc.mx_bound(ref, tr, fmt), "along the columns")
        assert not bool(q[:live, N:].any())
        got = mc.value(qt.cpu(), st.cpu(), fmt)
        rdb = torch.zeros(len(offsets) - 1, N, dtype=torch.float64)
        tdb = torch.zeros_like(rdb)
        for e in range(len(offsets) - 1):
            lo, hi, k0, k1 = offsets[e], offsets[e + 1], k_offsets[e], k_offsets[e + 1]
            ref, tr = (pad(x[lo:hi].t(), (0, k1 - k0 - (hi - lo))) for x in (dz, t))
            if hi > lo:
                mc.assert_within(got[:, k0:k1], ref, mc.mx_bound(ref, tr, fmt), "along the tokens")
                assert not bool(qt[:, k0 + hi - lo:k1].any())
            rdb[e] = dz[lo:hi].sum(0)
            tdb[e] = t[lo:hi].sum(0) + (hi - lo + 8) * 2.0 ** -24 * dz[lo:hi].abs().sum(0)
        mc.assert_within(db, rdb if by else rdb[0], tdb if by else tdb[0], "d_bias")


def test_epilogue_gradient_is_the_derivative():
    """Differences of the fused epilogue itself: linear with K = 128 whose
    product is zero, so z is the bias."""
    torch_cuda()
    N, h = 256, 2.0 ** -7
    zero = torch.zeros(1, 128, dtype=torch.uint8), torch.full((1, 4), 127, dtype=torch.uint8)
    w = torch.zeros(2 * N, 128, dtype=torch.uint8), torch.full((2 * N, 4), 127, dtype=torch.uint8)
    zero, w = _cuda(*zero), _cuda(*w)
    g = torch.Generator().manual_seed(3)
    z = (torch.randn(2 * N, generator=g) * 1.5).bfloat16().float()
    z = torch.where(z.abs() < 2 * h, torch.full_like(z, 0.5), z)       # away from relu's kink
    for act in ACTS:
        for gated in (False, True):
            cols = N if gated else 2 * N
            d = torch.ones(1, cols)
            _, _, db = pkg.epilogue_backward(d.cuda(), z.bfloat16().cuda().view(1, -1), act=act, gated=gated)
            f = {}
            for sign in (1, -1):
                for half in (0, 1):
                    step = torch.zeros(2 * N)
                    step[half * N:(half + 1) * N] = sign * h
                    b = (z + step).cuda()
                    f[sign, half] = pkg.linear(*zero, *w, bias=b, act=act, gated=gated,
                                               out_dtype=torch.float32).cpu().double()[0]
            for half in (0, 1):
                slope = (f[1, half] - f[-1, half]) / (2 * h)
                slope = slope if gated else slope[half * N:(half + 1) * N]
                # third derivatives are at most 2 (times |u| <= 8): h^2 / 6 of
                # that, and the FP32 rounding of two values over 2 h
                bound = 8 * 2 * h * h / 6 + 8 * 64 * 2.0 ** -24 / h
                mc.assert_within(db[half * N:(half + 1) * N], slope, bound, f"{act} gated={gated} half {half}")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ACTS)
def test_activations_of_large_values(act, gated):
    """Far out, where squares and cubes pass FP32's range: values and slopes
    stay those of the limits (z or 0, 1 or 0)."""
    torch_cuda()
    v = torch.tensor([64.0, 1e4, 1e10, 1e13, 1e19, 3e19, 1e20, 1e30, 3e38]).bfloat16().float()
    z = torch.cat([v, -v, torch.zeros(14)])
    n = z.numel()
    full = torch.cat([z, torch.ones(n)]) if gated else z
    zero = _cuda(torch.zeros(1, 128, dtype=torch.uint8), torch.full((1, 4), 127, dtype=torch.uint8))
    w = _cuda(torch.zeros(full.numel(), 128, dtype=torch.uint8), torch.full((full.numel(), 4), 127, dtype=torch.uint8))
    out = pkg.linear(*zero, *w, bias=full.cuda(), act=act, gated=gated, out_dtype=torch.float32)
    ref = mc.act(z.double(), act).view(1, -1)
    mc.assert_within(out, ref, mc.ACT_ERR * z.double().abs().view(1, -1) + 2.0 ** -126, f"{act} gated={gated}")
    for pad in (0, 1):      # whole eights, and not
        d = torch.ones(1, n + pad)
        fz = torch.cat([torch.nn.functional.pad(x, (0, pad)) for x in full.view(-1, n)]).view(1, -1).bfloat16()
        _, _, db = pkg.epilogue_backward(d.bfloat16().cuda(), fz.cuda(), act=act, gated=gated)
        slope = mc.act_grad(z.double(), act)
        mc.assert_within(db[:n], slope, 64 * 2.0 ** -24 + 0 * slope, f"{act} slope gated={gated}")
        if gated:
            mc.assert_within(db[n + pad:2 * n + pad], ref[0], 64 * 2.0 ** -24 * z.double().abs() + 2.0 ** -126,
                             f"{act} of the gate")


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("by", [False, True])
@pytest.mark.parametrize("M,N,K,act,gated", [(96, 128, 256, "none", False), (200, 162, 128, "none", False),
                                             (300, 256, 384, "silu", True), (700, 96, 256, "gelu_tanh", False)])
def test_linear_backward(M, N, K, act, gated, by, precision):
    """The products are checked against the held dz itself (as the library
    quantised it, checked above), so their bounds are the products' alone."""
    torch_cuda()
    say(f"linear backward M={M} N={N} K={K} act={act} gated={gated} by={by} {precision}")
    g = torch.Generator().manual_seed(M + N + K)
    E = 4 if by else 1
    x = torch.randn(M, K, generator=g).bfloat16()
    w = (torch.randn(E, N, K, generator=g) * K ** -0.5).bfloat16()
    z = None if act == "none" else torch.randn(M, N, generator=g).bfloat16()
    d = torch.randn(M, N // 2 if gated else N, generator=g).bfloat16()
    sort, offsets, k_offsets = None, [0, M], [0, -(-M // 128) * 128]
    if by:
        ids = mc.ids_of(g, M, 1, E, 0.1)
        ids[ids == 2] = 1                      # an expert without tokens
        sort = pkg.sort_tokens(ids.cuda(), E)
        offsets, k_offsets = mc.order(ids, E)[:2]
    at, at_s = pkg.quantize_transposed(x.cuda(), sort)
    parts = [pkg.quantize_transposed(w[e].cuda()) for e in range(E)]
    wt, wt_s = (torch.stack([p[i] for p in parts]) for i in (0, 1))
    if not by:
        wt, wt_s = wt[0], wt_s[0]
    zc = None if z is None else z.cuda()
    got = pkg.linear_backward(d.cuda(), zc, at, at_s, wt, wt_s, act=act, gated=gated, sort=sort, fmt="e5m2",
                              precision=precision)
    (q, s), (qt, st), db = pkg.epilogue_backward(d.cuda(), zc, act=act, gated=gated, sort=sort, fmt="e5m2")
    assert torch.equal(db, got.d_bias)
    live = offsets[-1]
    rows, cols = mc.value(q.cpu(), s.cpu(), "e5m2"), mc.value(qt.cpu(), st.cpu(), "e5m2")
    atv, wtv = mc.value(at.cpu(), at_s.cpu(), "e4m3"), mc.value(wt.cpu(), wt_s.cpu(), "e4m3")
    assert not bool(got.d_a[live:].any())
    for e in range(E):
        lo, hi, k0, k1 = offsets[e], offsets[e + 1], k_offsets[e], k_offsets[e + 1]
        we = wtv[e] if by else wtv
        for what, out, u, v in (("d_a", got.d_a[lo:hi], rows[lo:hi], we),
                                ("d_w", got.d_w[e] if by else got.d_w, cols[:, k0:k1], atv[:, k0:k1])):
            if out.numel():
                ref = u @ v.t()
                t = mc.product_error(u.abs() @ v.abs().t(), u.shape[1], precision)
                mc.assert_within(out, ref, t + mc.rounding(ref.abs() + t, torch.bfloat16), what)
    # and the transposed operands stand for x and w
    for e in range(E):
        lo, hi, k0 = offsets[e], offsets[e + 1], k_offsets[e]
        if by and hi > lo:
            xe = torch.nn.functional.pad(x[lo:hi].double().t(), (0, k_offsets[e + 1] - k0 - (hi - lo)))
            mc.assert_within(atv[:, k0:k_offsets[e + 1]], xe, mc.mx_bound(xe, xe.abs() * 0, "e4m3"), "at")


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("cfg", [-1, 1, 4])
@pytest.mark.parametrize("E", [256, 257, 600, 1024])
def test_by_many_experts(E, cfg, precision):
    """More experts than one round of the row tiles' list holds; most of them
    have no row."""
    torch_cuda()
    ids = mc.ids_of(torch.Generator().manual_seed(E), 150, 2, E, 0.05)
    ids[::7, 0] = E - 1
    _grouped(ids, E, 64, 128, "silu", True, torch.bfloat16, precision, cfg)


@pytest.mark.parametrize("E", [300, 1024])
def test_backward_by_many_experts(E):
    torch_cuda()
    M, N, K = 500, 64, 128
    say(f"linear backward by expert M={M} N={N} K={K} E={E}")
    g = torch.Generator().manual_seed(E)
    ids = mc.ids_of(g, M, 1, E, 0.05)
    sort = pkg.sort_tokens(ids.cuda(), E)
    offsets, k_offsets = mc.order(ids, E)[:2]
    x, d = torch.randn(M, K, generator=g).bfloat16(), torch.randn(M, N, generator=g).bfloat16()
    at, at_s = pkg.quantize_transposed(x.cuda(), sort)
    wt = torch.randint(0x30, 0x40, (E, K, 128), generator=g, dtype=torch.uint8)
    wt_s = torch.full((E, K, 4), 127, dtype=torch.uint8)
    got = pkg.linear_backward(d.cuda(), None, at, at_s, wt.cuda(), wt_s.cuda(), sort=sort)
    (q, s), (qt, st), db = pkg.epilogue_backward(d.cuda(), sort=sort)
    assert torch.equal(db, got.d_bias)
    rows, cols = mc.value(q.cpu(), s.cpu(), "e4m3"), mc.value(qt.cpu(), st.cpu(), "e4m3")
    atv, wtv = mc.value(at.cpu(), at_s.cpu(), "e4m3"), mc.value(wt, wt_s, "e4m3")
    da, ta = torch.zeros(M, K, dtype=torch.float64), torch.zeros(M, K, dtype=torch.float64)
    dw, tw = torch.zeros(E, N, K, dtype=torch.float64), torch.zeros(E, N, K, dtype=torch.float64)
    rdb, tdb = torch.zeros(E, N, dtype=torch.float64), torch.zeros(E, N, dtype=torch.float64)
    for e in range(E):
        lo, hi, k0, k1 = offsets[e], offsets[e + 1], k_offsets[e], k_offsets[e + 1]
        if hi > lo:
            for ref, t, at_, u, v in ((da, ta, slice(lo, hi), rows[lo:hi], wtv[e]),
                                      (dw, tw, e, cols[:, k0:k1], atv[:, k0:k1])):
                ref[at_] = u @ v.t()
                t[at_] = mc.product_error(u.abs() @ v.abs().t(), u.shape[1], "exact")
            rdb[e] = d[lo:hi].double().sum(0)
            tdb[e] = (hi - lo + 8) * 2.0 ** -24 * d[lo:hi].double().abs().sum(0)
    for what, out, ref, t in (("d_a", got.d_a, da, ta), ("d_w", got.d_w, dw, tw)):
        mc.assert_within(out, ref, t + mc.rounding(ref.abs() + t, torch.bfloat16), what)
    mc.assert_within(db, rdb, tdb, "d_bias")


def test_no_tokens():
    torch_cuda()
    u8 = dict(dtype=torch.uint8, device="cuda")
    w, w_s = torch.zeros(64, 128, **u8), torch.zeros(64, 4, **u8)
    assert pkg.linear(torch.empty(0, 128, **u8), torch.empty(0, 4, **u8), w, w_s).shape == (0, 64)
    got = pkg.linear_backward(torch.empty(0, 64, device="cuda"), None, torch.empty(128, 0, **u8),
                              torch.empty(128, 0, **u8), torch.zeros(128, 128, **u8), torch.zeros(128, 4, **u8))
    assert got.d_a.shape == (0, 128) and not got.d_w.any() and got.d_w.shape == (64, 128) and not got.d_bias.any()
    sort = pkg.sort_tokens(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 3)
    got = pkg.linear_backward(torch.empty(0, 64, device="cuda"), None, torch.empty(128, 384, **u8),
                              torch.empty(128, 12, **u8), torch.zeros(3, 128, 128, **u8),
                              torch.zeros(3, 128, 4, **u8), sort=sort)
    assert got.d_w.shape == (3, 64, 128) and not got.d_w.any() and not got.d_bias.any()


def test_strides_streams_and_graph():
    torch_cuda()
    M, N, K = 90, 160, 256
    g = torch.Generator().manual_seed(9)
    a, a_s, w, w_s = _cuda(*_operands(g, M, N, K))
    res = torch.randn(M, N + 3, generator=g).bfloat16().cuda()[:, 1:N + 1]
    wide = torch.zeros(M, K + 64, dtype=torch.uint8, device="cuda")
    wide[:, 16:16 + K] = a
    bias = torch.randn(N, generator=g).cuda()
    run = lambda **kw: pkg.linear(wide[:, 16:16 + K], a_s, w, w_s, bias=bias, act="silu",  # noqa: E731
                                  residual=res, **kw)
    ref = pkg.linear(a, a_s, w, w_s, bias=bias, act="silu", residual=res.contiguous())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        bias.add_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run())


def test_refusals():
    torch_cuda()
    u8 = dict(dtype=torch.uint8, device="cuda")
    a, a_s = torch.zeros(8, 256, **u8), torch.zeros(8, 8, **u8)
    w, w_s = torch.zeros(64, 256, **u8), torch.zeros(64, 8, **u8)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    ok = pkg.linear(a, a_s, w, w_s)
    assert not ok.any()
    bias = torch.zeros(64, device="cuda")
    for bad in (lambda: pkg.linear(a[:, :96], a_s[:, :3], w[:, :96], w_s[:, :3]),
                lambda: pkg.linear(a, a_s[:, :4], w, w_s), lambda: pkg.linear(a, a_s, w[:, :128], w_s[:, :4]),
                lambda: pkg.linear(a.cpu(), a_s, w, w_s), lambda: pkg.linear(a.float(), a_s, w, w_s),
                lambda: pkg.linear(a, a_s, w, w_s, bias=bias[:63]), lambda: pkg.linear(a, a_s, w, w_s, act="tanh"),
                lambda: pkg.linear(a, a_s, w, w_s, bias=bias.double()),
                lambda: pkg.linear(a, a_s, w[:63], w_s[:63], gated=True),
                lambda: pkg.linear(a, a_s, w[:40], w_s[:40], out_dtype="e4m3"),
                lambda: pkg.linear(a, a_s, w, w_s, out_dtype="e3m4"),
                lambda: pkg.linear(a, a_s, w, w_s, out_dtype=torch.float64),
                lambda: pkg.linear(a, a_s, w, w_s, residual=torch.zeros(8, 64, device="cuda")),
                lambda: pkg.linear(a, a_s, w, w_s, precision="fast"),
                lambda: pkg.linear(a, a_s, w, w_s, a_fmt="e3m4"), lambda: pkg.linear(a, a_s, w, w_s, tile_cfg=7),
                lambda: pkg.linear(a, a_s, w, w_s, offsets=off),
                lambda: pkg.linear(a, a_s, w.view(2, 32, 256), w_s.view(2, 32, 8), offsets=off.long()),
                lambda: pkg.linear(a, a_s, w.view(2, 32, 256), w_s.view(2, 32, 8), offsets=off[:2]),
                lambda: pkg.linear(torch.zeros(8, 264, **u8)[:, 8:], a_s, w, w_s),     # not 16-byte aligned
                lambda: pkg.epilogue_backward(bias.view(1, 64), act="silu"),
                lambda: pkg.epilogue_backward(bias.view(1, 64), bias.view(1, 64), act="silu"),
                lambda: pkg.linear_backward(bias.view(1, 64), None, w, w_s, w, w_s),
                lambda: pkg.quantize_transposed(bias)):
        with pytest.raises((TypeError, ValueError, pkg.MxgemmError)):
            bad()
