"""The operators with scales of 128 as a layer uses them, one on the other's
output, forward and backward: every stage against 64 bits, from what the stage
before it gave; captured into graphs and replayed; on two streams at once."""
import pytest
import torch

import block_common as bc
import moe_common as mc
import mxfp8_block_scaled_mxgemm_amd as pkg
from gpu_common import say, torch_cuda
from test_gpu_block import _backward, _check_quantized, _forward

pytestmark = pytest.mark.gpu


class Layer:
    """r = residual + scale gate norm(x); its norm through a router and gated
    experts; their sum, normed, onto r.  Products by expert, and the router's
    dense, are of FP8 operands with scales of 128."""

    def __init__(self, g, T, H, F, E, k, G, groups=1, top=1, precision="exact"):
        rand = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).cuda()  # noqa: E731
        self.T, self.E, self.k = T, E, k
        self.route = dict(score="sigmoid", bias=rand(E, std=0.1), groups=groups, top_groups=top, scale=2.0)
        self.by = dict(precision=precision)
        both = lambda w: pkg.block_quantize_weight(w, transposed=True)  # noqa: E731
        self.wr, self.wrt = both(rand(E, H, std=H ** -0.5))
        self.w1, self.w1t = both(rand(E, 2 * F, H, std=H ** -0.5).bfloat16())
        self.w2, self.w2t = both(rand(E, H, F, std=F ** -0.5).bfloat16())
        self.norm1 = dict(gate=rand(G, H).bfloat16(), scale=0.5, post_weight=1 + rand(H, std=0.2),
                          pre_weight=1 + rand(H, std=0.2), kind="layer")
        self.norm2 = dict(gate=rand(H), scale=0.7, post_weight=1 + rand(H, std=0.2), kind="rms")

    def forward(self, x, residual):
        k = {}
        k["x"] = x
        k["y"], k["r"] = pkg.add_norm(x, residual, **self.norm1)
        k["yq"], k["yqt"] = pkg.block_quantize(k["y"], cols=True)
        k["logits"] = pkg.block_linear(*k["yq"], *self.wr, out_dtype=torch.float32, **self.by)
        k["ids"], k["weights"] = pkg.route_tokens(k["logits"], self.k, **self.route)
        k["sort"] = s = pkg.sort_tokens(k["ids"], self.E)
        k["rows"] = pkg.dispatch_tokens(k["y"], s)
        k["a"], k["at"] = pkg.block_quantize(k["rows"], sort=s, cols=True)
        k["z"] = pkg.block_linear(*k["a"], *self.w1, s.offsets, **self.by)
        k["b"], k["bt"] = pkg.block_quantize(k["z"], act="silu", gated=True, sort=s, cols=True)
        k["o"] = pkg.block_linear(*k["b"], *self.w2, s.offsets, **self.by)
        k["m"] = pkg.combine_tokens(k["o"], s, k["weights"])
        _, k["r2"] = pkg.add_norm(k["m"], k["r"], **self.norm2)
        return k

    def backward(self, k, d_r2):
        s, d = k["sort"], {}
        d["n2"] = pkg.add_norm_backward(None, d_r2, k["m"], k["r2"], **self.norm2)
        d["o"], d["weights"] = pkg.combine_tokens_backward(d["n2"].d_x, k["o"], s, k["weights"])
        d["b"], d["w2"] = pkg.block_linear_backward(d["o"], None, *k["bt"], *self.w2t, sort=s, **self.by)
        d["rows"], d["w1"] = pkg.block_linear_backward(d["b"], k["z"], *k["at"], *self.w1t, act="silu", gated=True,
                                                       sort=s, fmt="e5m2", out_dtype=torch.bfloat16, **self.by)
        d["logits"] = pkg.route_tokens_backward(d["weights"], k["logits"], k["ids"], score="sigmoid", scale=2.0)
        d["router"], d["wr"] = pkg.block_linear_backward(d["logits"], None, *k["yqt"], *self.wrt, **self.by)
        d["y"] = pkg.dispatch_tokens_backward(d["rows"], s) + d["router"]
        d["n1"] = pkg.add_norm_backward(d["y"], d["n2"].d_residual, k["x"], k["r"], **self.norm1)
        return d

    def step(self, x, residual, d_r2):
        """All tensors of a forward and backward step, flat."""
        k = self.forward(x, residual)
        d = self.backward(k, d_r2)
        return [t for part in (k, d) for v in part.values() for t in _flat(v)]


def _flat(v):
    if isinstance(v, torch.Tensor):
        return [v]
    return [t for p in v for t in _flat(p)] if isinstance(v, tuple) else []


def _by_expert(a, w, ends, T):
    """64-bit product by expert and the sum of its magnitudes."""
    out, size = torch.zeros(T, w.shape[1], dtype=torch.float64), torch.zeros(T, w.shape[1], dtype=torch.float64)
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        out[lo:hi] = a[lo:hi] @ w[e].t()
        size[lo:hi] = a[lo:hi].abs() @ w[e].abs().t()
    return out, size


def _by_inner(a, w, ends):
    pairs = [(a[:, lo:hi], w[:, lo:hi]) for lo, hi in zip(ends, ends[1:])]
    return torch.stack([p @ q.t() for p, q in pairs]), torch.stack([p.abs() @ q.abs().t() for p, q in pairs])


def _near(got, ref, t, what):
    mc.assert_within(got, ref, t + mc.rounding(ref.abs() + t, got.dtype), what)


@pytest.mark.parametrize("T,H,F,E,k,G,groups,top", [(150, 384, 256, 6, 2, 3, 2, 1), (37, 200, 130, 12, 3, 37, 4, 2),
                                                    (1, 136, 128, 4, 2, 1, 1, 1)])
@pytest.mark.parametrize("precision", ["exact", "native"])
def test_layer(T, H, F, E, k, G, groups, top, precision):
    torch_cuda()
    g = torch.Generator().manual_seed(T)
    say(f"layer T={T} H={H} F={F} E={E} {precision}")
    layer = Layer(g, T, H, F, E, k, G, groups, top, precision)
    x, res, d_r2 = (torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(3))
    f = layer.forward(x, res)
    d = layer.backward(f, d_r2)
    wide = lambda t: t.cpu().double()  # noqa: E731
    P = T * k
    s = f["sort"]
    ends, inner = s.offsets.tolist(), s.k_offsets.tolist()

    # the router: its product, its choice, the order and the rows
    val = lambda pair, fmt="e4m3": bc.value(pair[0].cpu(), pair[1].cpu(), fmt)  # noqa: E731
    sq = lambda pair: bc.square_value(pair[0].cpu(), pair[1].cpu(), "e4m3")  # noqa: E731
    y = wide(f["y"])
    _check_quantized(f["yq"], f["yqt"], y, 0 * y, "e4m3")
    a, w = val(f["yq"]), sq(layer.wr)
    _near(f["logits"], a @ w.t(), bc.product_error(a.abs() @ w.abs().t(), a.shape[1], precision), "logits")
    ids, weights = bc.route(f["logits"].cpu(), k, "sigmoid", layer.route["bias"].cpu(), groups, top, True, 2.0)
    assert torch.equal(f["ids"].cpu(), ids)
    mc.assert_within(f["weights"], weights, 64 * bc.U * weights, "weights")
    ref_ends, ref_inner = mc.order(ids, E)[:2]
    assert ends == list(ref_ends) and inner == list(ref_inner)
    rows = wide(f["rows"])
    token = torch.empty(P, dtype=torch.int64)
    token[wide(s.row_of).long().view(-1)] = torch.arange(P) // k
    assert torch.equal(rows, y[token])

    # the experts
    _check_quantized(f["a"], f["at"], rows, 0 * rows, "e4m3", ends, inner, E)
    ref, size = _by_expert(val(f["a"]), sq(layer.w1), ends, P)
    _near(f["z"], ref, bc.product_error(size, bc.up(H), precision), "z")
    h, t = _forward(f["z"].cpu(), "silu", True)
    _check_quantized(f["b"], f["bt"], h, t, "e4m3", ends, inner, E)
    ref, size = _by_expert(val(f["b"]), sq(layer.w2), ends, P)
    _near(f["o"], ref, bc.product_error(size, bc.up(F), precision), "o")
    o, wts, place = wide(f["o"]), wide(f["weights"]), wide(s.row_of).long()
    part = wts.unsqueeze(-1) * o[place]
    _near(f["m"], part.sum(1), (k + 1) * bc.U * part.abs().sum(1), "m")

    # back through the experts, from what arrived
    dm = wide(d["n2"].d_x)
    ref = torch.zeros_like(o)
    ref[place] = wts.unsqueeze(-1) * dm.unsqueeze(1)
    _near(d["o"], ref, 2 * bc.U * ref.abs(), "d_o")
    dot = o[place] * dm.unsqueeze(1)
    mc.assert_within(d["weights"], dot.sum(-1), H * bc.U * dot.abs().sum(-1), "d_weights")
    for name, came, z, wt, at, fmt in (("2", d["o"], None, layer.w2t, f["bt"], "e4m3"),
                                       ("1", d["b"], f["z"], layer.w1t, f["at"], "e5m2")):
        act = dict(act="none" if z is None else "silu", gated=z is not None)
        q, qt = pkg.block_quantize_backward(came, z, sort=s, fmt=fmt, **act)
        dz, t = (wide(came), 0 * wide(came)) if z is None else _backward(came.cpu(), z.cpu(), "silu", True)
        _check_quantized(q, qt, dz, t, fmt, ends, inner, E)
        ref, size = _by_expert(val(q, fmt), sq(wt), ends, P)
        got = d["b"] if name == "2" else d["rows"]
        _near(got, ref, bc.product_error(size, q[0].shape[1], precision), "d_a" + name)
        ref, size = _by_inner(val(qt, fmt), val(at), inner)
        _near(d["w" + name], ref, bc.product_error(size, inner[-1], precision), "d_w" + name)

    # the router's gradient: sigmoid scores over their sum
    l, dw = wide(f["logits"]), wide(d["weights"])
    chosen = ids.long()
    sig = torch.sigmoid(l.gather(1, chosen))
    total = sig.sum(1, keepdim=True)
    ds = 2.0 * (dw / total - (dw * sig).sum(1, keepdim=True) / total ** 2)
    bound = 2.0 * (dw.abs() / total + (dw.abs() * sig).sum(1, keepdim=True) / total ** 2)
    slope = sig * (1 - sig)
    ref = torch.zeros_like(l).scatter_(1, chosen, ds * slope)
    t = torch.zeros_like(l).scatter_(1, chosen, 64 * bc.U * bound * sig)
    mc.assert_within(d["logits"], ref, t, "d_logits")
    q, qt = pkg.block_quantize_backward(d["logits"])
    a, w = val(q), sq(layer.wrt)
    _near(d["router"], a @ w.t(), bc.product_error(a.abs() @ w.abs().t(), a.shape[1], precision), "d_router")
    a, w = val(qt), val(f["yqt"])
    _near(d["wr"], a @ w.t(), bc.product_error(a.abs() @ w.abs().t(), a.shape[1], precision), "d_wr")

    # the residual stream: its gradient passes the second norm as it came
    assert torch.equal(d["n2"].d_residual, d_r2)
    v = wide(f["r"]).requires_grad_()
    n1 = layer.norm1
    out = bc.normed(v, "layer", 1e-6) * wide(n1["pre_weight"])
    ref = torch.autograd.grad(out, v, wide(d["y"]))[0] + wide(d_r2)
    # (64 roundings of the row's sums and of the normed element, each relative
    # to the sizes that enter: |d w| and its mean with the normed row)
    e = (wide(d["y"]) * wide(n1["pre_weight"])).abs()
    hat = bc.normed(v.detach(), "layer", 1e-6).abs() + 1
    rstd = 1 / torch.sqrt(v.detach().var(1, correction=0, keepdim=True) + 1e-6)
    spread = 1 + rstd * v.detach().abs().mean(1, keepdim=True)
    t = 8 * 64 * bc.U * spread * rstd * (e + hat * ((e * hat).mean(1, keepdim=True) + e.mean(1, keepdim=True)))
    _near(d["n1"].d_residual, ref, t + 2 * bc.U * (ref.abs() + wide(d_r2).abs()), "d_residual")


def _sets(g, n, T, H):
    return [[torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(3)] for _ in range(n)]


def _same(a, b):
    """Bit for bit (NaN included)."""
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}
    flat = lambda t: t.contiguous().view(bits[t.element_size()])  # noqa: E731
    return len(a) == len(b) and all(torch.equal(flat(p), flat(q)) for p, q in zip(a, b))


def _capture(f):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    return graph, out


def _split(g):
    """A dense product whose inner axis is split over work-groups."""
    a, w = bc.blocks(torch.randn(40, 7168, generator=g), "e4m3"), bc.blocks(torch.randn(256, 7168, generator=g), "e4m3")
    a, w = tuple(t.cuda() for t in a), tuple(t.cuda() for t in w)
    return lambda: [pkg.block_linear(*a, *w, out_dtype=torch.float32, precision=p) for p in ("exact", "native")]


@pytest.mark.parametrize("T,H,F,E,k,G", [(150, 384, 256, 6, 2, 3), (5000, 256, 128, 16, 2, 5)])
def test_step_in_a_graph(T, H, F, E, k, G):
    """Captured steps replayed on inputs that change (other choices, other
    segments), with eager steps and synchronizations between: the eager bits."""
    torch_cuda()
    g = torch.Generator().manual_seed(H)
    layer = Layer(g, T, H, F, E, k, G)
    split = _split(g)
    sets = _sets(g, 3, T, H)
    held = [t.clone() for t in sets[0]]
    say(f"layer in a graph T={T}")
    whole = lambda x: layer.step(*x) + split()  # noqa: E731
    first, out = _capture(lambda: whole(held))
    second, other = _capture(lambda: whole(held))
    for i in (1, 2, 0, 1):
        ref = whole(sets[i])
        for t, new in zip(held, sets[i]):
            t.copy_(new)
        first.replay()
        if i:
            torch.cuda.synchronize()
        second.replay()
        torch.cuda.synchronize()
        say(f"replay of set {i}")
        assert _same(out, ref) and _same(other, ref)
        assert _same(whole(sets[i]), ref)


def test_steps_on_two_streams_at_once():
    """Steps of two layers in flight together, eager and as graphs."""
    torch_cuda()
    g = torch.Generator().manual_seed(77)
    layers = [Layer(g, 300, 384, 256, 8, 2, 3), Layer(g, 2000, 256, 384, 5, 1, 1, precision="native")]
    splits = [_split(g), _split(g)]
    sets = [_sets(g, 1, 300, 384)[0], _sets(g, 1, 2000, 256)[0]]
    run = lambda i: layers[i].step(*sets[i]) + splits[i]()  # noqa: E731
    refs = [run(0), run(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    say("two streams")
    got = [[], []]
    for _ in range(3):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(run(i))
    torch.cuda.synchronize()
    assert all(_same(one, refs[i]) for i in (0, 1) for one in got[i])
    graphs = [_capture(lambda i=i: run(i)) for i in (0, 1)]
    say("two graphs")
    for _ in range(3):
        for (graph, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(_same(out, refs[i]) for i, (_, out) in enumerate(graphs))


def test_a_layer_without_tokens():
    torch_cuda()
    g = torch.Generator().manual_seed(3)
    layer = Layer(g, 0, 256, 128, 4, 2, 2)
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    say("layer of no tokens")
    f = layer.forward(x, x)
    d = layer.backward(f, x)
    assert f["r2"].shape == (0, 256) and f["ids"].shape == (0, 2)
    for name, shape in (("w1", (4, 256, 256)), ("w2", (4, 256, 128)), ("wr", (4, 256))):
        assert d[name].shape == shape and not d[name].any(), name
    for grad in (d["n1"].d_gate, d["n1"].d_post_weight, d["n1"].d_pre_weight, d["n2"].d_gate, d["n2"].d_post_weight):
        assert not grad.any()


def test_every_token_dropped():
    """No logit can be chosen: ids of -1, empty segments, zeros on the way back."""
    torch_cuda()
    g = torch.Generator().manual_seed(5)
    T, H, F, E = 40, 256, 128, 4
    layer = Layer(g, T, H, F, E, 2, 1)
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    say("layer of dropped tokens")
    ids, weights = pkg.route_tokens(torch.full((T, E), float("-inf"), device="cuda"), 2, **layer.route)
    assert (ids == -1).all() and not weights.any()
    s = pkg.sort_tokens(ids, E)
    rows = pkg.dispatch_tokens(x, s)
    a, at = pkg.block_quantize(rows, sort=s, cols=True)
    z = pkg.block_linear(*a, *layer.w1, s.offsets)
    b, bt = pkg.block_quantize(z, act="silu", gated=True, sort=s, cols=True)
    out = pkg.combine_tokens(pkg.block_linear(*b, *layer.w2, s.offsets), s, weights)
    assert not z.any() and not out.any()
    d_b, d_w2 = pkg.block_linear_backward(rows, None, *bt, *layer.w2t, sort=s)
    d_rows, d_w1 = pkg.block_linear_backward(d_b, z, *at, *layer.w1t, act="silu", gated=True, sort=s)
    assert not d_b.any() and not d_rows.any() and not d_w1.any() and not d_w2.any()
    assert not pkg.route_tokens_backward(weights, torch.zeros(T, E, device="cuda"), ids, score="sigmoid").any()
