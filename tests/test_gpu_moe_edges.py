"""Edges of the expert layer on the GPU."""
import ctypes
import importlib.util
import os

import pytest
import torch

import mxfp8_block_scaled_mxgemm_amd as pkg
import moe_common as mc
from gpu_common import say, torch_cuda
from mxfp8_block_scaled_mxgemm_amd import _lib, _moe

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _filled(*shape):
    return torch.full(shape, 0xA5, dtype=torch.uint8, device="cuda")


def _pointer(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _grad_abi(d, z, act, gated, sort, fmt, ld_qt, rows=True, cols=True):
    """mxgemm_epilogue_backward by expert into buffers that hold 0xA5."""
    M, N = d.shape[0], d.shape[1] * (2 if gated else 1)
    E, Np = sort.offsets.numel() - 1, -(-N // 128) * 128
    q, s = (_filled(M, Np), _filled(M, Np // 32)) if rows else (None, None)
    qt, st = (_filled(N, ld_qt), _filled(N, ld_qt // 32)) if cols else (None, None)
    rc = _moe._load().mxgemm_epilogue_backward(
        _pointer(d), _moe._TYPES[d.dtype], d.shape[1], _pointer(z), N, M, N, pkg._moe.ACTIVATIONS[act], int(gated),
        _pointer(sort.offsets), _pointer(sort.k_offsets), E, pkg._moe._FMT[fmt], _pointer(q), _pointer(s),
        _pointer(qt), _pointer(st), ld_qt, None, None, 0, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0, pkg.last_error()
    torch.cuda.synchronize()
    return q, s, qt, st


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,act,gated,E,drop", [
    (1, 2, "silu", True, 5, 1.0), (5, 34, "gelu", True, 3, 0.5), (130, 64, "gelu_tanh", False, 5, 0.1),
    (300, 128, "silu", True, 4, 0.3), (700, 192, "none", False, 2, 0.9), (257, 200, "relu", False, 40, 0.2),
    (1000, 320, "silu", True, 3, 1.0), (64, 96, "none", False, 300, 0.0),
])
def test_epilogue_backward_leaves_nothing_unwritten(M, N, act, gated, E, drop, dtype):
    """By expert: rows of dropped pairs and the columns past the last segment
    are zero, in buffers that held something else, also where ld_qt leaves no
    column past it."""
    torch_cuda()
    g = torch.Generator().manual_seed(M + N)
    ids = mc.ids_of(g, M, 1, E, drop)
    sort = pkg.sort_tokens(ids.cuda(), E)
    offsets, k_offsets = mc.order(ids, E)[:2]
    live, used = offsets[-1], k_offsets[-1]
    plain = act == "none" and not gated
    z = None if plain else torch.randn(M, N, generator=g).bfloat16().cuda()
    d = torch.randn(M, N // 2 if gated else N, generator=g).to(dtype).cuda()
    wide = (-(-M // 128) + E) * 128
    say(f"epilogue backward M={M} N={N} act={act} gated={gated} E={E} live={live} used={used} {dtype}")
    (q0, s0), (qt0, st0), _ = pkg.epilogue_backward(d, z, act=act, gated=gated, sort=sort, bias=False)
    assert qt0.shape == (N, wide)
    assert not q0[live:].any() and not s0[live:].any() and not qt0[:, used:].any() and not st0[:, used // 32:].any()
    for ld_qt in sorted({used, used + 128, wide}):
        q, s, qt, st = _grad_abi(d, z, act, gated, sort, "e4m3", ld_qt)
        assert torch.equal(q, q0) and torch.equal(s, s0)
        assert torch.equal(qt[:, :used], qt0[:, :used]) and torch.equal(st[:, :used // 32], st0[:, :used // 32])
        assert not qt[:, used:].any() and not st[:, used // 32:].any()
    q, s, _, _ = _grad_abi(d, z, act, gated, sort, "e4m3", wide, cols=False)
    assert torch.equal(q, q0) and torch.equal(s, s0)
    _, _, qt, st = _grad_abi(d, z, act, gated, sort, "e4m3", wide, rows=False)
    assert torch.equal(qt, qt0) and torch.equal(st, st0)


def test_quantize_transposed_leaves_nothing_unwritten():
    torch_cuda()
    g = torch.Generator().manual_seed(4)
    ids = mc.ids_of(g, 300, 2, 6, 0.2)
    sort = pkg.sort_tokens(ids.cuda(), 6)
    used = mc.order(ids, 6)[1][-1]
    x = torch.randn(600, 80, generator=g).bfloat16().cuda()
    junk = [torch.full((80, 1408), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(8)]
    del junk        # what an allocation of this size holds next
    qt, st = pkg.quantize_transposed(x, sort)
    assert qt.shape == (80, 1408) and not qt[:, used:].any() and not st[:, used // 32:].any()


def test_combine_backward_of_many_tokens():
    """More tokens than one launch takes with a work-group of 256 threads each."""
    torch_cuda()
    T, H = (1 << 24) + 3, 8
    pair = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).contiguous()
    live = T - 5
    sort = pkg.TokenSort(torch.tensor([0, live], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
                         pair.view(T, 1), pair)
    g = torch.Generator(device="cuda").manual_seed(1)
    whole = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").bfloat16()  # noqa: E731
    rows, d, w = whole(T, H), whole(T, H), whole(T, 1).float()
    say(f"combine backward T={T}")
    d_rows, d_w = pkg.combine_tokens_backward(d, rows, sort, w)
    ref = (w * d.float()).bfloat16().flip(0)
    ref[live:] = 0
    assert torch.equal(d_rows, ref)
    rows = rows.flip(0)                     # token t's row
    rows[:T - live] = 0
    assert torch.equal(d_w, (rows.float() * d.float()).sum(1, keepdim=True))
    out = pkg.combine_tokens(d_rows, sort, w)
    assert torch.equal(out, (w * d_rows.flip(0).float()).bfloat16().masked_fill(
        (torch.arange(T, device="cuda") < T - live).unsqueeze(1), 0))


def test_more_pieces_than_one_launch():
    """Seven columns, a thread per element: over 2^32 threads."""
    torch_cuda()
    T, H = 614_000_001, 7
    assert T * H > 1 << 32
    pair = torch.arange(T, dtype=torch.int32, device="cuda")
    sort = pkg.TokenSort(torch.tensor([0, T - 1], dtype=torch.int32, device="cuda"),
                         torch.zeros(2, dtype=torch.int32, device="cuda"), pair.view(T, 1), pair)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    step = 1 << 27
    for i in range(0, T, step):
        x[i:i + step] = torch.randint(-9, 10, (min(step, T - i), H), device="cuda", dtype=torch.int8)
    say(f"dispatch and combine T={T} H={H}")
    rows = pkg.dispatch_tokens(x, sort)
    x[T - 1] = 0            # the last token's pair is dropped
    assert all(torch.equal(rows[i:i + step], x[i:i + step]) for i in range(0, T, step))
    x.zero_()
    out = pkg.combine_tokens(rows, sort, residual=x)
    assert all(torch.equal(rows[i:i + step], out[i:i + step]) for i in range(0, T, step))


def test_mx_dispatch_over_two_launches():
    """Token ranges of a launch begin at the right rows of x and row_of."""
    torch_cuda()
    T, H = (1 << 30) + 7, 32        # two threads a token: just over 2^31
    pair = torch.arange(T, dtype=torch.int32, device="cuda")
    sort = pkg.TokenSort(torch.tensor([0, T - 3], dtype=torch.int32, device="cuda"),
                         torch.zeros(2, dtype=torch.int32, device="cuda"), pair.view(T, 1), pair)
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    x[1 << 30:] = 3.0
    say(f"dispatch mx T={T} H={H}")
    q, s = pkg.dispatch_tokens_mx(x, sort)
    del x
    small = torch.tensor([[1.0] * H, [3.0] * H], device="cuda")
    rq, rs = pkg.quantize_mxfp8(small)
    step = 1 << 27
    for i in range(0, T, step):
        lo, hi = i, min(i + step, T)
        which = (pair[lo:hi] >= 1 << 30).long()
        kept = (pair[lo:hi] < T - 3).unsqueeze(1)
        assert torch.equal(s[lo:hi], rs[which] * kept) and torch.equal(q[lo:hi], rq[which] * kept)


def test_product_of_too_many_work_groups_is_refused():
    """2^26 tiles of 64 x 64 with 256 threads each: the host refuses, nothing is
    launched."""
    torch_cuda()
    n = 1 << 19
    p = torch.zeros(4096, dtype=torch.uint8, device="cuda").data_ptr()
    say("refusal of a grid of 2^34 threads")
    rc = _moe._load().mxgemm_linear(_moe.LINEAR_ARGS.pack(
        p, p, p, p, 0, 0, p, 0, 0, 0, n, n, 128, 128, 4, 128, 4, 0, 0, 0, n, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 2, 0, 0),
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == _lib.MXGEMM_EUNSUPPORTED, (rc, pkg.last_error())


@pytest.mark.parametrize("by", [False, True])
@pytest.mark.parametrize("act,gated", [("silu", False), ("gelu", False), ("silu", True), ("none", True),
                                       ("gelu_tanh", True), ("relu", False)])
def test_no_tokens_behind_an_activation(act, gated, by):
    torch_cuda()
    N, K, E = 64, 128, 3
    u8 = dict(dtype=torch.uint8, device="cuda")
    sort = pkg.sort_tokens(torch.empty(0, 2, dtype=torch.int32, device="cuda"), E) if by else None
    lead, Mp = ((E,), E * 128) if by else ((), 0)
    d = torch.empty(0, N // 2 if gated else N, dtype=torch.bfloat16, device="cuda")
    z = torch.empty(0, N, dtype=torch.bfloat16, device="cuda")
    got = pkg.linear_backward(d, z, torch.zeros(K, Mp, **u8), torch.zeros(K, Mp // 32, **u8),
                              torch.zeros(*lead, K, 128, **u8), torch.zeros(*lead, K, 4, **u8), act=act, gated=gated,
                              sort=sort)
    assert got.d_a.shape == (0, K) and got.d_w.shape == (*lead, N, K) and got.d_bias.shape == (*lead, N)
    assert not got.d_w.any() and not got.d_bias.any()
    with pytest.raises(ValueError):
        pkg.epilogue_backward(d, None, act=act, gated=gated, sort=sort)


def test_layer_without_tokens():
    """A rank that receives no token: serving and training steps of the whole
    layer."""
    torch_cuda()
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    E, H, F = 3, 256, 128
    w1, w2 = torch.randn(E, 2 * F, H, device="cuda").bfloat16(), torch.randn(E, H, F, device="cuda").bfloat16()
    layer = example.ExpertLayer(w1, w2)
    x = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    ids, weights = torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda")
    say("layer T=0")
    assert layer.forward(x, ids, weights).shape == (0, H)
    y, (d_x, d_weights, d_w1, d_w2) = layer.train_step(x, ids, weights, x)
    assert y.shape == d_x.shape == (0, H) and d_weights.shape == (0, 2)
    assert d_w1.shape == w1.shape and d_w2.shape == w2.shape and not d_w1.any() and not d_w2.any()


def test_gradient_takes_matrices_only():
    """A stack of matrices is refused, not read as one of its corners."""
    torch_cuda()
    x = torch.randn(3, 64, 128, device="cuda").bfloat16()
    for bad in (lambda: pkg.quantize_transposed(x), lambda: pkg.epilogue_backward(x),
                lambda: pkg.epilogue_backward(x, x, act="silu"), lambda: pkg.quantize_transposed(x[None])):
        with pytest.raises(ValueError):
            bad()


def test_stores_past_32_bits():
    """Outputs whose rows lie more than 2^32 elements apart."""
    torch_cuda()
    T, H, K = 3, 64, 128
    g = torch.Generator().manual_seed(7)
    ld = (1 << 32) + 64
    big = torch.zeros(2 * ld + H, dtype=torch.bfloat16, device="cuda")
    far = torch.as_strided(big, (T, H), (ld, 1))
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    lib = _moe._load()
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    sort = pkg.sort_tokens(torch.tensor([[2], [0], [1]], dtype=torch.int32, device="cuda"), 3)
    off, row_of = _pointer(sort.offsets), _pointer(sort.row_of)
    p = _pointer
    say("dispatch, combine and linear with rows 2^32 + 64 elements apart")
    assert lib.mxgemm_dispatch_tokens(p(x), H, 0, T, 1, H, off, 3, row_of, p(big), ld, stream) == 0
    assert torch.equal(far.contiguous(), pkg.dispatch_tokens(x, sort))
    far.zero_()
    assert lib.mxgemm_combine_tokens(p(x), H, 0, T, 1, H, off, 3, row_of, None, None, 0, p(big), ld, stream) == 0
    assert torch.equal(far.contiguous(), pkg.combine_tokens(x, sort))
    far.zero_()
    d_w = torch.empty(T, 1, device="cuda")
    assert lib.mxgemm_combine_tokens_backward(p(x), H, p(x), H, 0, T, 1, H, off, 3, row_of, None, p(big), ld, p(d_w),
                                              stream) == 0
    assert torch.equal(far.contiguous(), pkg.combine_tokens_backward(x, x, sort)[0])
    a, a_s, w, w_s = (t.cuda() for t in (*mc.codes(g, (T, K), "e4m3"), *mc.codes(g, (H, K), "e4m3")))
    for cfg in (1, 2, 4):
        ref, z = pkg.linear(a, a_s, w, w_s, act="silu", preact=True, tile_cfg=cfg)
        out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        for outp, ldo, zp, ldz, want in ((big, ld, out, H, ref), (out, H, big, ld, z)):
            far.zero_()
            rc = lib.mxgemm_linear(_moe.LINEAR_ARGS.pack(
                a.data_ptr(), a_s.data_ptr(), w.data_ptr(), w_s.data_ptr(), 0, 0, outp.data_ptr(), 0, zp.data_ptr(), 0,
                T, H, K, K, K // 32, K, K // 32, 0, 0, 0, ldo, 0, 0, ldz, 0, 0, 0, 0, 0, 0, 4, 0, 0, cfg, 0, 0), stream)
            assert rc == 0, pkg.last_error()
            assert torch.equal(far.contiguous(), want), cfg
    del big, far


# ---------------------------------------------------------------- products --

@pytest.mark.parametrize("stride", [0, 1, 5, 64 * 256 + 3])
def test_stride_of_the_only_expert_does_not_matter(stride):
    torch_cuda()
    M, N, K = 40, 64, 256
    g = torch.Generator().manual_seed(2)
    a, a_s, w, w_s = (t.cuda() for t in (*mc.codes(g, (M, K), "e4m3"), *mc.codes(g, (N, K), "e4m3")))
    say(f"one expert, stride {stride}")
    offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    lone = lambda t: torch.as_strided(t, (1, *t.shape), (stride, t.shape[1], 1))  # noqa: E731
    assert torch.equal(pkg.linear(a, a_s, lone(w), lone(w_s), offsets=offsets), pkg.linear(a, a_s, w, w_s))

TILES = {0: False, 1: True, 2: True, 3: True, 4: True}      # configuration: has it an exact kernel


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("cfg", [-1, *sorted(TILES)])
def test_linear_by_inner(cfg, precision, out_dtype):
    """Inner ranges that are empty, a K-step, several and many; columns beyond
    the last range are no expert's."""
    torch_cuda()
    if precision == "exact" and not TILES.get(cfg, True):
        pytest.skip("no exact kernel of this tile")
    steps = [0, 1, 3, 0, 6, 17]
    offsets = [0]
    for n in steps:
        offsets.append(offsets[-1] + 128 * n)
    K = offsets[-1] + 256
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(cfg + 3)
    for M, N, a_fmt in ((300, 264, "e5m2"), (37, 50, "e4m3")):
        say(f"by inner M={M} N={N} K={K} cfg={cfg} {precision} {out_dtype} {a_fmt}")
        a, a_s = mc.codes(g, (M, K), a_fmt)
        w, w_s = mc.codes(g, (N, K), "e4m3")
        a[:, offsets[-1]:], a_s[:, offsets[-1] // 32:] = 0x7F, 0xFF         # never read
        out = pkg.linear_by_inner(a.cuda(), a_s.cuda(), w.cuda(), w_s.cuda(), off, out_dtype=out_dtype,
                                  precision=precision, a_fmt=a_fmt, tile_cfg=cfg)
        assert out.shape == (len(steps), M, N) and out.dtype == out_dtype
        av, wv = mc.value(a, a_s, a_fmt), mc.value(w, w_s, "e4m3")
        for e in range(len(steps)):
            u, v = av[:, offsets[e]:offsets[e + 1]], wv[:, offsets[e]:offsets[e + 1]]
            ref = u @ v.t()
            t = mc.product_error(u.abs() @ v.abs().t(), u.shape[1], precision)
            mc.assert_within(out[e], ref, t + mc.rounding(ref.abs() + t, out_dtype), f"expert {e}")


def _integers(g, M, N, K, lead=()):
    """Operands whose products and sums are exact in every step."""
    one = lambda v: (v.to(torch.float8_e4m3fn).view(torch.uint8),  # noqa: E731
                     torch.full((*v.shape[:-1], K // 32), 127, dtype=torch.uint8, device="cuda"))
    av = torch.randint(-1, 2, (M, K), generator=g, device="cuda").float()
    wv = torch.randint(-2, 3, (*lead, N, K), generator=g, device="cuda").float()
    wv = torch.where(torch.rand(wv.shape, generator=g, device="cuda") < 0.05, wv, 0.0)
    return av, wv, one(av), one(wv)


@pytest.mark.parametrize("E,N", [(2, 32768), (4, 16384 - 96)])
def test_large_native_product_by_expert(E, N):
    """Rows and columns enough for the largest tile by its own rule, ragged."""
    torch_cuda()
    K, M = 2048, 1100 * E
    g = torch.Generator(device="cuda").manual_seed(E)
    av, wv, (a, a_s), (w, w_s) = _integers(g, M, N, K, (E,))
    say(f"native by expert M={M} N={N} K={K} E={E}")
    # unequal shares, some rows dropped
    offsets = [0] + [1100 * e + 37 * (e % 2) for e in range(1, E)] + [M - 60]
    out = pkg.linear(a, a_s, w, w_s, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                     out_dtype=torch.float32, precision="native")
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        assert torch.equal(out[lo:hi], torch.mm(av[lo:hi], wv[e].t())), e
    assert not out[M - 60:].any()


def _codes(g, *shape):
    """Any finite E4M3 codes under scales of 2^-9 .. 2^0, made on the GPU."""
    q = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    return (torch.where((q & 0x7F) == 0x7F, 0, q).to(torch.uint8),
            torch.randint(118, 128, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda", dtype=torch.uint8))


@pytest.mark.parametrize("precision", ["exact", "native"])
@pytest.mark.parametrize("M,N,K,by", [(4096, 4096, 2176, 0), (3000, 2000, 1152, 0), (64, 2048, 7168, 0),
                                      (16, 4096, 4096, 0), (3000, 2048, 1024, 12), (9000, 8192, 2048, 8)])
def test_products_repeat_bit_for_bit(M, N, K, by, precision):
    """The same inputs give the same bits on every call, with other work in
    between."""
    torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(M)
    (a, a_s), (w, w_s) = _codes(g, M, K), _codes(g, *((by,) if by else ()), N, K)
    offsets = None
    if by:
        offsets = pkg.sort_tokens(mc.ids_of(torch.Generator().manual_seed(M), M, 1, by, 0.05).cuda(), by).offsets
    say(f"repeat M={M} N={N} K={K} by={by} {precision}")
    run = lambda x: pkg.linear(x, a_s, w, w_s, act="silu", offsets=offsets, precision=precision)  # noqa: E731
    first = run(a)
    assert not torch.isnan(first).any()
    other = a.flip(0)
    for _ in range(6):
        run(other)
        assert torch.equal(run(a), first)


# -------------------------------------------------------------------- gelu --

def test_gelu_keeps_float32_in_its_tail():
    """gelu and its slope against 64 bits, relative to themselves: with a = z^2
    / 2, exp(-a) in float32 is good to (a 2.5 + 2) units (a's rounding, that of
    its product with log2 e, the constant's, the hardware's last place), and
    the reciprocal, the polynomial's nine steps and the products to less than
    30 more."""
    torch_cuda()
    N = 4096
    z = torch.cat([torch.linspace(-13, 13, 2 * N - 512), -torch.logspace(-8, 1, 256), torch.logspace(-8, 1, 256)])
    z = z.bfloat16().float()
    zero = torch.zeros(1, 128, dtype=torch.uint8).cuda(), torch.full((1, 4), 127, dtype=torch.uint8).cuda()
    n = z.numel()
    w = torch.zeros(n, 128, dtype=torch.uint8).cuda(), torch.full((n, 4), 127, dtype=torch.uint8).cuda()
    zd = z.double()
    units = (3 * zd * zd / 2 + 32) * 2.0 ** -24
    cdf = 0.5 * torch.special.erfc(-zd / 2 ** 0.5)
    pdf = torch.exp(-zd * zd / 2) / (2 * torch.pi) ** 0.5
    out = pkg.linear(*zero, *w, bias=z.cuda(), act="gelu", out_dtype=torch.float32).cpu().double()[0]
    # at z > 0 the tail is taken from one
    tail = torch.minimum(cdf, 1 - cdf)
    bound = zd.abs() * (units * tail + (zd > 0) * 2.0 ** -23) + 2.0 ** -126
    mc.assert_within(out, zd * cdf, bound, "gelu")
    for pad in (0, 1):      # whole eights, and not
        d = torch.ones(1, n + pad)
        fz = torch.nn.functional.pad(z, (0, pad)).view(1, -1)
        _, _, db = pkg.epilogue_backward(d.bfloat16().cuda(), fz.bfloat16().cuda(), act="gelu")
        bound = units * (tail + zd.abs() * pdf) + (zd > 0) * 2.0 ** -23 + 2.0 ** -23 * (cdf + zd * pdf).abs() + 2.0 ** -126
        mc.assert_within(db[:n], cdf + zd * pdf, bound, "slope")
