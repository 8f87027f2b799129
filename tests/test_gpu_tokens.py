"""Tokens sorted by expert and back on the GPU, against the definitions in 64
bits on the CPU."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_mxgemm_amd as pkg
import moe_common as mc
from gpu_common import say, torch_cuda

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _sorted(ids, E):
    got = pkg.sort_tokens(ids.cuda(), E)
    torch.cuda.synchronize()
    return got


@pytest.mark.parametrize("T,k,E,drop", [
    (0, 2, 4, 0.0), (1, 1, 1, 0.0), (1, 8, 128, 0.0), (3, 2, 5, 0.5), (7, 3, 1, 0.0), (64, 1, 63, 0.0),
    (65, 1, 64, 0.1), (1000, 6, 40, 0.1), (2048, 8, 256, 0.0), (2049, 8, 256, 0.02), (5001, 7, 1023, 0.0),
    (4097, 4, 1024, 0.3), (40000, 8, 8, 0.02), (300, 2, 16, 1.0),
])
@pytest.mark.parametrize("wide", [False, True])
def test_sort(T, k, E, drop, wide):
    torch_cuda()
    say(f"sort T={T} k={k} E={E} drop={drop} int64={wide}")
    ids = mc.ids_of(torch.Generator().manual_seed(T + E), T, k, E, drop)
    if wide:
        ids = ids.long()
        if T > 2:
            ids[0, 0] = 1 << 40        # out of range however it is truncated
    else:
        if T > 2:
            ids[0, 0] = E              # one past the end
    got = _sorted(ids, E)
    offsets, k_offsets, row_of, pair_of = mc.order(ids, E)
    assert got.offsets.tolist() == offsets and got.k_offsets.tolist() == k_offsets
    assert np.array_equal(got.row_of.cpu().numpy(), row_of)
    assert np.array_equal(got.pair_of.cpu().numpy(), pair_of)


def test_sort_one_expert_takes_all():
    torch_cuda()
    ids = torch.full((30000, 2), 3, dtype=torch.int32)
    got = _sorted(ids, 9)
    assert got.offsets.tolist() == [0, 0, 0, 0] + [60000] * 6
    assert torch.equal(got.pair_of.cpu(), torch.arange(60000, dtype=torch.int32))


CASES = [(1, 1, 4, 8, 0.0), (1, 8, 16, 7168, 0.0), (5, 3, 4, 1, 0.3), (9, 2, 4, 7, 0.0), (33, 4, 8, 64, 0.1),
         (130, 6, 12, 2047, 0.1), (257, 9, 16, 256, 0.0), (40, 17, 32, 130, 0.2), (20, 3, 4, 512, 1.0)]


def _setup(T, k, E, H, drop, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + T * 31 + H)
    ids = mc.ids_of(g, T, k, E, drop)
    sort = _sorted(ids, E)
    _, _, row_of, pair_of = mc.order(ids, E)
    live = int(((ids >= 0) & (ids < E)).sum())
    return g, sort, torch.from_numpy(row_of), torch.from_numpy(pair_of), live


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,drop", CASES)
def test_dispatch_and_gradient(T, k, E, H, drop, dtype):
    torch_cuda()
    say(f"dispatch T={T} k={k} E={E} H={H} drop={drop} {dtype}")
    g, sort, row_of, pair_of, live = _setup(T, k, E, H, drop, dtype)
    x = torch.randn(T, H, generator=g).to(dtype)
    rows = pkg.dispatch_tokens(x.cuda(), sort)
    ref = x[pair_of // k].clone()
    ref[live:] = 0
    assert torch.equal(rows.cpu(), ref)
    d_rows = torch.randn(T * k, H, generator=g).to(dtype)
    # values in rows of dropped pairs must not matter
    d_rows[live:] = float("nan")
    dx = pkg.dispatch_tokens_backward(d_rows.cuda(), sort)
    picked = d_rows[row_of].double()
    picked[row_of >= live] = 0
    total = picked.sum(1)
    bound = k * 2.0 ** -24 * picked.abs().sum(1)
    mc.assert_within(dx, total, bound + mc.rounding(total.abs() + bound, dtype), "dx")


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,drop", [(1, 8, 16, 7168, 0.0), (5, 3, 4, 32, 0.3), (33, 4, 8, 96, 0.1),
                                          (130, 6, 12, 2048, 0.1), (20, 3, 4, 512, 1.0)])
def test_dispatch_mx(T, k, E, H, drop, dtype, fmt):
    torch_cuda()
    say(f"dispatch mx T={T} k={k} E={E} H={H} drop={drop} {dtype} {fmt}")
    g, sort, row_of, pair_of, live = _setup(T, k, E, H, drop, dtype)
    x = (torch.randn(T, H, generator=g) * torch.exp2(torch.randint(-12, 12, (T, 1), generator=g).float())).to(dtype)
    x[0, :32] = 0
    q, s = pkg.dispatch_tokens_mx(x.cuda(), sort, fmt=fmt)
    rq, rs = mc.quantize(x, fmt)
    rq, rs = rq[pair_of // k].clone(), rs[pair_of // k].clone()
    rq[live:], rs[live:] = 0, 0
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)


def test_dispatch_mx_non_finite_is_the_quantisers():
    """NaN blocks: scale 0xFF, codes 0x7F; infinities saturate under e = 127."""
    torch_cuda()
    x = torch.ones(2, 96)
    x[0, 3], x[0, 40], x[1, 70] = float("nan"), float("inf"), float("-inf")
    sort = _sorted(torch.zeros(2, 1, dtype=torch.int32), 1)
    q, s = pkg.dispatch_tokens_mx(x.cuda(), sort)
    rq, rs = pkg.quantize_mxfp8(x.cuda())
    assert torch.equal(q, rq) and torch.equal(s, rs)
    assert s[0, 0] == 255 and bool((q[0, :32] == 0x7F).all()) and s[0, 1] == 254 and q[0, 40] == 0x7E


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_dispatch_mx_codes_are_the_quantisers(fmt):
    """Every finite bfloat16 value, beside its neighbours and beside random
    others, and random float32 bit patterns: the same codes and scales as the
    quantiser's."""
    torch_cuda()
    bits = torch.arange(1 << 16, dtype=torch.int32)
    bits = bits[(bits & 0x7F80) != 0x7F80].short()
    g = torch.Generator().manual_seed(2)
    n = bits.numel() // 32 * 32
    wild = torch.randint(-(1 << 31), 1 << 31, (1 << 20,), generator=g, dtype=torch.int64).int().view(torch.float32)
    tame = torch.randn(1 << 20, generator=g) * torch.exp2(torch.randint(-20, 20, (1 << 20,), generator=g).float())
    for x in (bits[:n].view(torch.bfloat16).float(), bits[torch.randperm(bits.numel(), generator=g)[:n]].view(
            torch.bfloat16).float(), wild, tame):
        x = x.view(-1, 128 if x.numel() % 128 == 0 else 32).cuda()
        sort = _sorted(torch.zeros(x.shape[0], 1, dtype=torch.int32), 1)
        q, s = pkg.dispatch_tokens_mx(x, sort, fmt=fmt)
        rq, rs = pkg.quantize_mxfp8(x, fmt=pkg.FMT_E5M2 if fmt == "e5m2" else pkg.FMT_E4M3)
        assert torch.equal(s, rs) and torch.equal(q, rq)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("weighted,residual", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("T,k,E,H,drop", CASES)
def test_combine(T, k, E, H, drop, weighted, residual, dtype):
    torch_cuda()
    say(f"combine T={T} k={k} E={E} H={H} drop={drop} {dtype} weighted={weighted} residual={residual}")
    g, sort, row_of, pair_of, live = _setup(T, k, E, H, drop, dtype)
    rows = torch.randn(T * k, H, generator=g).to(dtype)
    rows[live:] = float("inf")
    w = torch.softmax(torch.randn(T, k, generator=g), 1) if weighted else None
    if weighted:
        w[row_of >= live] = float("nan")
    res = torch.randn(T, H, generator=g).to(dtype) if residual else None
    out = pkg.combine_tokens(rows.cuda(), sort, None if w is None else w.cuda(),
                             residual=None if res is None else res.cuda())
    kept = (row_of < live).unsqueeze(2)
    terms = torch.where(kept, rows[row_of].double(), 0.0)
    if weighted:
        terms = torch.where(kept, w.double().unsqueeze(2) * terms, 0.0)
    ref = terms.sum(1)
    mag = terms.abs().sum(1)
    if residual:
        ref, mag = ref + res.double(), mag + res.double().abs()
    bound = (k + 2) * 2.0 ** -23 * mag      # a product and a sum rounded per term
    mc.assert_within(out, ref, bound + mc.rounding(ref.abs() + bound, dtype), "out")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,E,H,drop", CASES)
def test_combine_backward(T, k, E, H, drop, weighted, dtype):
    torch_cuda()
    say(f"combine backward T={T} k={k} E={E} H={H} drop={drop} {dtype} weighted={weighted}")
    g, sort, row_of, pair_of, live = _setup(T, k, E, H, drop, dtype)
    rows = torch.randn(T * k, H, generator=g).to(dtype)
    rows[live:] = float("nan")
    w = torch.softmax(torch.randn(T, k, generator=g), 1) if weighted else None
    d = torch.randn(T, H, generator=g).to(dtype)
    d_rows, d_w = pkg.combine_tokens_backward(d.cuda(), rows.cuda(), sort, None if w is None else w.cuda())
    one = torch.ones(T, k) if w is None else w
    ref = one.double().flatten()[pair_of].unsqueeze(1) * d.double()[pair_of // k]
    ref[live:] = 0
    mc.assert_within(d_rows, ref, mc.rounding(ref, dtype) + 2.0 ** -24 * ref.abs(), "d_rows")
    terms = torch.where((row_of < live).unsqueeze(2), rows[row_of].double(), 0.0) * d.double().unsqueeze(1)
    mc.assert_within(d_w, terms.sum(2), (H + 8) * 2.0 ** -24 * terms.abs().sum(2) + 2.0 ** -140, "d_weights")
    assert bool((d_w.cpu()[row_of >= live] == 0).all())


def test_combine_backward_is_the_derivative():
    """Differences of combine along random directions, in float32."""
    torch_cuda()
    T, k, E, H = 37, 3, 6, 72
    g, sort, row_of, pair_of, live = _setup(T, k, E, H, 0.2, torch.float32)
    rows, d = torch.randn(T * k, H, generator=g), torch.randn(T, H, generator=g)
    w = torch.rand(T, k, generator=g)
    d_rows, d_w = pkg.combine_tokens_backward(d.cuda(), rows.cuda(), sort, w.cuda())
    h = 2.0 ** -6
    for which in ("rows", "weights"):
        v = torch.randn(*(rows.shape if which == "rows" else w.shape), generator=g)
        f = []
        for sign in (1, -1):
            r2, w2 = (rows + sign * h * v, w) if which == "rows" else (rows, w + sign * h * v)
            f.append((pkg.combine_tokens(r2.cuda(), sort, w2.cuda()).cpu().double() * d.double()).sum())
        grad = d_rows if which == "rows" else d_w
        slope = float((grad.cpu().double() * v.double()).sum())
        # linear in either argument: only float32 rounding remains, of T H
        # outputs of a few units each against 2 h
        assert abs(float(f[0] - f[1]) / (2 * h) - slope) <= T * H * 16 * 2.0 ** -24 / h


def test_strided_rows_and_other_streams():
    torch_cuda()
    T, k, E, H = 50, 4, 8, 100
    g, sort, row_of, pair_of, live = _setup(T, k, E, H, 0.1, torch.bfloat16)
    wide = torch.randn(T, 3 * H + 1, generator=g).bfloat16().cuda()
    x = wide[:, 5:5 + H]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rows = pkg.dispatch_tokens(x, sort, stream=side)
    out = pkg.combine_tokens(rows, sort, stream=side, residual=wide[:, H:2 * H])
    torch.cuda.current_stream().wait_stream(side)
    a = pkg.dispatch_tokens(x.contiguous(), sort)
    assert torch.equal(rows, a)
    assert torch.equal(out, pkg.combine_tokens(a, sort, residual=wide[:, H:2 * H].contiguous()))


def test_offsets_past_32_bits():
    """Rows beyond 2^32 elements from the first are written and read."""
    torch_cuda()
    T, k, H = 2, 1, 64
    sort = _sorted(torch.tensor([[1], [0]], dtype=torch.int32), 2)
    ld = (1 << 32) + 64
    big = torch.empty(ld + H, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(T, H).bfloat16()
    rows = torch.as_strided(big, (T, H), (ld, 1))
    rows.copy_(x.cuda())
    out = pkg.combine_tokens(rows, sort)
    assert torch.equal(out.cpu(), x[[1, 0]])
    del big, rows


def test_refusals():
    torch_cuda()
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    sort = pkg.sort_tokens(ids, 3)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: pkg.sort_tokens(ids, 0), lambda: pkg.sort_tokens(ids, 1025),
                lambda: pkg.sort_tokens(ids.float(), 3), lambda: pkg.sort_tokens(ids[:, :1], 3),
                lambda: pkg.sort_tokens(ids.cpu(), 3),
                lambda: pkg.dispatch_tokens(x[:3], sort), lambda: pkg.dispatch_tokens(x.double(), sort),
                lambda: pkg.dispatch_tokens(x.t(), sort), lambda: pkg.dispatch_tokens(x.cpu(), sort),
                lambda: pkg.dispatch_tokens_mx(x[:, :40], sort), lambda: pkg.dispatch_tokens_mx(x, sort, fmt="e3m4"),
                lambda: pkg.combine_tokens(rows[:7], sort), lambda: pkg.combine_tokens(rows, sort, x),
                lambda: pkg.combine_tokens(rows, sort, torch.zeros(4, 2, device="cuda"), residual=x.float()),
                lambda: pkg.combine_tokens_backward(x.float(), rows, sort),
                lambda: pkg.combine_tokens_backward(x[:3], rows, sort)):
        with pytest.raises((TypeError, ValueError, pkg.MxgemmError)):
            bad()


def test_graph_replays_match_eager():
    torch_cuda()
    T, k, E, H = 300, 4, 16, 256
    g = torch.Generator().manual_seed(5)
    ids = mc.ids_of(g, T, k, E, 0.1).cuda()
    x = torch.randn(T, H, generator=g).bfloat16().cuda()

    def step():
        sort = pkg.sort_tokens(ids, E)
        rows = pkg.dispatch_tokens(x, sort)
        return rows, pkg.combine_tokens(rows, sort)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        ids.copy_(mc.ids_of(g, T, k, E, 0.1 * i))
        graph.replay()
        torch.cuda.synchronize()
        ref = step()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
