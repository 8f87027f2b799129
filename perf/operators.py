"""The expert layer's operators on measured sizes: tokens sorted by expert and
back, and the MXFP8 product with its fused epilogue, dense and by expert,
each with its gradient.

Every case runs either in plain torch (32-bit arithmetic, one rounding at the
end) or, with ``own`` set, through this package's entry points, on the same
inputs.  ``exact`` computes the same outputs from the definitions in 64 bits.

Operators (T tokens, k experts per token, E experts, H columns):
  sort      expert ids [T, k] -> the stable order by expert; an id outside
            [0, E) drops its pair, dropped pairs follow the last expert.
  dispatch  rows[r] = x[token of r], zero for dropped pairs; as the input's
            type with the gradient to x, or quantised to MXFP8.
  combine   out[t] = residual[t] + sum_j w[t, j] rows[row_of[t, j]] over the
            kept pairs, with the gradients to rows and w.
  linear    out = act(a w^T + bias) + residual, a and w in MXFP8.
  mlp       by expert: (silu(g) u) of g, u = a w1^T halves, held in MXFP8,
            times w2^T.
  grad      the gradient of linear to a, w and bias, dense or by expert: dz =
            d_out act'(z) in MXFP8 along N for d_a = dz w and along the
            tokens for d_w = dz^T a.
"""
import math

import torch

own = False

BLOCK = 32          # elements sharing one E8M0 scale
STEP = 128          # granule of a product's inner length
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one decoding step of a small batch: pure latency
        dict(name="sort decode", op="sort", T=4, k=8, E=128, drop=0.0),
        # a long prompt over many experts, a few pairs over capacity dropped
        dict(name="sort prefill", op="sort", T=32768, k=8, E=256, drop=0.02),
        # prompt rows to their experts, quantised once for the MXFP8 product
        dict(name="dispatch mx", op="dispatch", T=8192, k=8, E=64, H=4096, drop=0.02, dtype="bf16", mx=True,
             fmt="e4m3"),
        # a training step's ragged batch in its own type, with the gradient
        dict(name="dispatch grad", op="dispatch", T=5001, k=6, E=40, H=2047, drop=0.1, dtype="fp16", mx=False,
             fmt="e4m3"),
        # one token back from its experts
        dict(name="combine decode", op="combine", T=1, k=8, E=128, H=7168, drop=0.0, dtype="bf16", grad=False,
             residual=True),
        # a training step: forward and both gradients
        dict(name="combine grad", op="combine", T=8192, k=8, E=64, H=4096, drop=0.02, dtype="bf16", grad=True,
             residual=True),
        # a decoding batch through one projection: the weights' bytes count
        dict(name="linear skinny", op="linear", M=64, N=2048, K=7168, act="gelu_tanh", bias=True, residual=False,
             gated=False, dtype="bf16", precision="exact", a_fmt="e4m3", w_fmt="e4m3"),
        # the largest dense projection of the repository's workloads
        dict(name="linear large", op="linear", M=8192, N=8192, K=8192, act="silu", bias=True, residual=True,
             gated=False, dtype="bf16", precision="native", a_fmt="e4m3", w_fmt="e4m3"),
        # eight decoding tokens through their experts
        dict(name="mlp decode", op="mlp", T=8, k=8, E=128, H=2048, F=768, drop=0.0, precision="exact"),
        # a prompt through the experts
        dict(name="mlp prefill", op="mlp", T=4096, k=4, E=32, H=4096, F=2048, drop=0.02, precision="native"),
        # a dense training step's backward
        dict(name="grad dense", op="grad", M=4096, N=4096, K=7168, E=0, k=0, drop=0.0, act="gelu_tanh", gated=False,
             precision="native", fmt="e5m2"),
        # the same by expert, gated, with empty and short experts
        dict(name="grad experts", op="grad", M=4001, N=2048, K=2048, E=24, k=2, drop=0.05, act="silu", gated=True,
             precision="exact", fmt="e4m3"),
    ]


# inner lengths in STEPs, and widths that tiles divide
STEPS = [1, 2, 3, 4, 5, 7, 8, 11, 16, 28, 32, 56, 64]
WIDTHS = [64, 128, 192, 256, 512, 896, 1024, 1536, 2048, 3584, 4096, 7168, 8192]


def _log(rng, lo, hi):
    """Spread over the logarithm; long ones odd, so that no tile divides them."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n | 1 if 2048 < n < hi else n


def _upto(rng, sizes, most):
    return rng.choice([n for n in sizes if n <= most])


def _experts(rng):
    E = rng.choice([4, 8, 24, 40, 64, 128, 200, 256])
    return E, min(E, rng.choice([1, 2, 4, 6, 8]))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "combine", "linear", "mlp", "grad"])
    drop = rng.choice([0.0, 0.0, 0.02, 0.3])
    if op == "sort":
        E, k = _experts(rng)
        return dict(op=op, T=_log(rng, 1, 32768), k=k, E=E, drop=drop)
    if op in ("dispatch", "combine"):
        E, k = _experts(rng)
        H = _log(rng, 64, 8192) if rng.random() < 0.3 else rng.choice(WIDTHS)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        T = min(_log(rng, 1, 16384), max(1, (1 << 29) // (H * k * SIZE[dtype])))
        if op == "combine":
            return dict(op=op, T=T, k=k, E=E, H=H, drop=drop, dtype=dtype, grad=rng.random() < 0.5,
                        residual=rng.random() < 0.5)
        mx = rng.random() < 0.5
        return dict(op=op, T=T, k=k, E=E, H=H // 64 * 64 + (BLOCK if H % 64 else 0) if mx else H, drop=drop,
                    dtype=dtype, mx=mx,
                    fmt=rng.choice(["e4m3", "e5m2"]))
    precision = rng.choice(["exact", "native"])
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    if op == "linear":
        K = STEP * rng.choice(STEPS)
        gated = rng.random() < 0.3
        N = _log(rng, 16, 8192) if rng.random() < 0.3 else rng.choice(WIDTHS)
        M = min(_log(rng, 1, 8192), max(1, (1 << 39) // (2 * N * K)))
        return dict(op=op, M=M, N=N - N % 2 if gated else N, K=K, act=act, bias=rng.random() < 0.7,
                    residual=rng.random() < 0.5, gated=gated, dtype=rng.choice(["bf16", "bf16", "fp16"]),
                    precision=precision, a_fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), w_fmt="e4m3")
    if op == "mlp":
        E, k = _experts(rng)
        H, F = STEP * _upto(rng, STEPS, 32), STEP * _upto(rng, STEPS, 16)
        T = min(_log(rng, 1, 4096), max(1, (1 << 38) // (6 * H * F * k)))
        E = max(k, min(E, 32 * 4096 * 2048 // (H * F)))
        return dict(op=op, T=T, k=k, E=E, H=H, F=F, drop=drop, precision=precision)
    gated = rng.random() < 0.5
    N, K = STEP * _upto(rng, STEPS, 32) + rng.choice([0, 0, 34]), STEP * _upto(rng, STEPS, 32)
    E, k = _experts(rng) if rng.random() < 0.5 else (0, 0)
    E = min(E, 40)
    k = min(E, k)
    M = min(_log(rng, 1, 8192), max(1, (1 << 37) // (N * K * max(1, k))))
    return dict(op=op, M=M, N=N, K=K, E=E, k=k, drop=drop if E else 0.0, act=act, gated=gated, precision=precision,
                fmt=rng.choice(["e4m3", "e5m2"]))


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, scale=1.0, dtype=torch.float32, outliers=False):
    x = torch.randn(*shape, generator=g, device="cuda") * scale
    if outliers:    # a few columns' worth of large activations
        x = torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.002, x * 20, x)
    return x.to(dtype)


def _ids(g, T, k, E, drop):
    """k different experts a token, some experts far more popular than others."""
    logits = torch.rand(T, E, generator=g, device="cuda").log().neg().log().neg()
    logits = logits + 1.2 * torch.randn(E, generator=g, device="cuda")
    ids = logits.topk(k, dim=1).indices.to(torch.int32)
    if drop:
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < drop, -1, ids)
    return ids


def _pack(x, fmt):
    """MXFP8 codes and scale bytes of x along its last axis (a multiple of 32):
    the smallest e with fmax 2^e >= amax, codes round-to-nearest-even."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    m, p = torch.frexp(b.abs().amax(-1))
    top = 9 if fmt == "e4m3" else 16
    e = (p - top + (m > 0.875).int()).clamp(-127, 127)
    e = torch.where(m == 0, -127, e)
    q = torch.ldexp(b, -e.unsqueeze(-1)).flatten(-2).to(F8[fmt])
    return q.view(torch.uint8), (e + 127).to(torch.uint8)


def _value(q, s, fmt):
    """The 32-bit values that codes and scale bytes stand for."""
    v = q.view(F8[fmt]).float().unflatten(-1, (-1, BLOCK))
    return torch.ldexp(v, (s.int() - 127).unsqueeze(-1)).flatten(-2)


def _value64(q, s, fmt):
    v = q.view(F8[fmt]).double().unflatten(-1, (-1, BLOCK))
    return (v * torch.exp2(s.double() - 127).unsqueeze(-1)).flatten(-2)


def _order(ids, E):
    """The sorted layout of ids: offsets, k_offsets, row_of, pair_of."""
    T, k = ids.shape
    key = torch.where((ids >= 0) & (ids < E), ids, E).flatten()
    key, pair = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=key.device, dtype=key.dtype)).to(torch.int32)
    counts = offsets[1:] - offsets[:-1]
    k_offsets = torch.zeros_like(offsets)
    k_offsets[1:] = torch.cumsum((counts + STEP - 1) // STEP * STEP, 0)
    row_of = torch.empty_like(pair)
    row_of[pair] = torch.arange(pair.numel(), device=pair.device)
    return offsets, k_offsets, row_of.view(T, k).to(torch.int32), pair.to(torch.int32)


def _pad_rows(x, n):
    return torch.cat([x, x.new_zeros(n - x.shape[0], x.shape[1])]) if n > x.shape[0] else x


def _up(n, m):
    return -(-n // m) * m


def _layout(case, seed):
    """The inputs of a case, the same for every form of the operator."""
    c, g = case, _generator(seed)
    op = c["op"]
    if op == "sort":
        return dict(ids=_ids(g, c["T"], c["k"], c["E"], c["drop"]))
    if op in ("dispatch", "combine"):
        T, k, H, dt = c["T"], c["k"], c["H"], TYPES[c["dtype"]]
        s = dict(ids=_ids(g, T, k, c["E"], c["drop"]))
        if op == "dispatch":
            s["x"] = _normal(g, T, H, dtype=dt, outliers=True)
            if not c["mx"]:
                s["d_rows"] = _normal(g, T * k, H, dtype=dt)
            return s
        s["rows"] = _normal(g, T * k, H, dtype=dt)
        s["weights"] = torch.softmax(_normal(g, T, k), dim=1)
        s["residual"] = _normal(g, T, H, dtype=dt) if c["residual"] else None
        s["d_out"] = _normal(g, T, H, dtype=dt) if c["grad"] else None
        return s
    if op == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        cols = N // 2 if c["gated"] else N
        a, a_s = _pack(_normal(g, M, K, outliers=True), c["a_fmt"])
        w, w_s = _pack(_normal(g, N, K, scale=K ** -0.5), c["w_fmt"])
        return dict(a=a, a_s=a_s, w=w, w_s=w_s, bias=_normal(g, N, scale=0.5) if c["bias"] else None,
                    residual=_normal(g, M, cols, dtype=TYPES[c["dtype"]]) if c["residual"] else None)
    if op == "mlp":
        T, k, E, H, F = (c[n] for n in ("T", "k", "E", "H", "F"))
        ids = _ids(g, T, k, E, c["drop"])
        a, a_s = _pack(_normal(g, T * k, H, outliers=True), "e4m3")
        w1, w1_s = _pack(_normal(g, E, 2 * F, H, scale=H ** -0.5), "e4m3")
        w2, w2_s = _pack(_normal(g, E, H, F, scale=F ** -0.5), "e4m3")
        return dict(ids=ids, a=a, a_s=a_s, w1=w1, w1_s=w1_s, w2=w2, w2_s=w2_s)
    M, N, K, E = (c[n] for n in ("M", "N", "K", "E"))
    s = {}
    w = _normal(g, max(E, 1), N, K, scale=K ** -0.5)
    if E:
        s["ids"] = _ids(g, M, c["k"], E, c["drop"])
        M = M * c["k"]
        offsets, k_offsets, _, _ = _order(s["ids"], E)
        row = torch.arange(M, device="cuda")
        at = (torch.searchsorted(offsets[1:].contiguous(), row.int(), right=True))
        kept = at < E
        at = at.clamp(max=E - 1)
        column = torch.where(kept, k_offsets[at] + row - offsets[at], 0)
        x = _normal(g, M, K)
        a = x.new_zeros((_up(M, STEP) // STEP + E) * STEP, K)
        a.index_add_(0, column, torch.where(kept.unsqueeze(1), x, 0.0))
    else:
        a = _pad_rows(_normal(g, M, K), _up(M, STEP))
    s["at"], s["at_s"] = _pack(a.t(), "e4m3")
    wt = w.transpose(1, 2)
    if N % STEP:
        wt = torch.cat([wt, wt.new_zeros(*wt.shape[:2], _up(N, STEP) - N)], 2)
    s["wt"], s["wt_s"] = _pack(wt, "e4m3")
    if not E:
        s["wt"], s["wt_s"] = s["wt"][0], s["wt_s"][0]
    s["z"] = _normal(g, M, N, dtype=torch.bfloat16)
    s["d_out"] = _normal(g, M, N // 2 if c["gated"] else N, scale=1e-3, dtype=torch.bfloat16, outliers=True)
    return s


def prepare(case, seed):
    s = _layout(case, seed)
    s["case"] = case
    if "ids" in s and case["op"] != "sort":
        s["sort"] = _order(s["ids"], case["E"])     # such a program has sorted its tokens before
    return s


# ------------------------------------------------------------- plain forms --

def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    return torch.ones_like(z)


def _kept(sort, rows):
    return torch.arange(rows, device="cuda") < sort[0][-1]


def _plain_dispatch(s, c):
    offsets, _, row_of, pair_of = s["sort"]
    rows = torch.where(_kept(s["sort"], pair_of.numel()).unsqueeze(1), s["x"][(pair_of // c["k"]).long()], 0)
    if c["mx"]:
        q, scale = _pack(rows, c["fmt"])
        return q.view(F8[c["fmt"]]), scale
    d = torch.where((row_of < offsets[-1]).unsqueeze(2), s["d_rows"][row_of.long()].float(), 0.0)
    return rows, d.sum(1).to(s["x"].dtype)


def _plain_combine(s, c):
    offsets, _, row_of, pair_of = s["sort"]
    kept = row_of < offsets[-1]
    picked = torch.where(kept.unsqueeze(2), s["rows"][row_of.long()].float(), 0.0)
    w = torch.where(kept, s["weights"], 0.0)
    out = (w.unsqueeze(2) * picked).sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    out = out.to(s["rows"].dtype)
    if not c["grad"]:
        return out
    d_out = s["d_out"].float()
    d_rows = w.flatten()[pair_of.long()].unsqueeze(1) * d_out[(pair_of // c["k"]).long()]
    return out, d_rows.to(s["rows"].dtype), (picked * d_out.unsqueeze(1)).sum(2)


def _plain_linear(s, c):
    z = _value(s["a"], s["a_s"], c["a_fmt"]) @ _value(s["w"], s["w_s"], c["w_fmt"]).t()
    if s["bias"] is not None:
        z = z + s["bias"]
    if c["gated"]:
        gate, up = z.chunk(2, dim=1)
        y = _act(gate, c["act"]) * up
    else:
        y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(TYPES[c["dtype"]])


def _slots(sort, rows, E):
    """Expert and place within it of every row, which rows are kept, and the
    longest expert."""
    offsets = sort[0]
    row = torch.arange(rows, device="cuda")
    expert = torch.searchsorted(offsets[1:].contiguous(), row.int(), right=True)
    kept = expert < E
    expert = expert.clamp(max=E - 1)
    slot = torch.where(kept, row - offsets[expert], 0)
    return expert, slot, kept, _up(max(1, int((offsets[1:] - offsets[:-1]).max())), STEP)


def _spread(x, expert, slot, kept, E, longest):
    """Rows of x as [E, longest, columns], zero where an expert has no row."""
    pad = x.new_zeros(E, longest, x.shape[1])
    return pad.index_put_((expert, slot), torch.where(kept.unsqueeze(1), x, 0), accumulate=True)


def _plain_mlp(s, c):
    E, rows = c["E"], s["a"].shape[0]
    expert, slot, kept, longest = _slots(s["sort"], rows, E)
    a = _spread(_value(s["a"], s["a_s"], "e4m3"), expert, slot, kept, E, longest)
    z = torch.bmm(a, _value(s["w1"], s["w1_s"], "e4m3").transpose(1, 2))
    gate, up = z.chunk(2, dim=2)
    h = _value(*_pack(_act(gate, "silu") * up, "e4m3"), "e4m3")
    y = torch.bmm(h, _value(s["w2"], s["w2_s"], "e4m3").transpose(1, 2))
    return torch.where(kept.unsqueeze(1), y[expert, slot], 0.0).to(torch.bfloat16)


def _plain_grad(s, c):
    E, N = c["E"], c["N"]
    z, d = s["z"].float(), s["d_out"].float()
    if c["gated"]:
        gate, up = z.chunk(2, dim=1)
        dz = torch.cat([d * up * _act_grad(gate, c["act"]), d * _act(gate, c["act"])], 1)
    else:
        dz = d * _act_grad(z, c["act"])
    wide = torch.nn.functional.pad(dz, (0, _up(N, STEP) - N))
    by_row = _value(*_pack(wide, c["fmt"]), c["fmt"])
    at, wt = _value(s["at"], s["at_s"], "e4m3"), _value(s["wt"], s["wt_s"], "e4m3")
    if not E:
        by_col = _value(*_pack(_pad_rows(dz, at.shape[1]).t(), c["fmt"]), c["fmt"])
        return ((by_row @ wt.t()).to(torch.bfloat16), (by_col @ at.t()).to(torch.bfloat16), dz.sum(0))
    expert, slot, kept, longest = _slots(s["sort"], z.shape[0], E)
    d_a = torch.bmm(_spread(by_row, expert, slot, kept, E, longest), wt.transpose(1, 2))[expert, slot]
    spread = _spread(dz, expert, slot, kept, E, longest)
    by_col = _value(*_pack(spread.transpose(1, 2), c["fmt"]), c["fmt"])
    a = at.new_zeros(E, longest, at.shape[0])
    column = (s["sort"][1][expert] + slot).long()
    a = _spread(at.t()[torch.where(kept, column, 0)], expert, slot, kept, E, longest)
    return (torch.where(kept.unsqueeze(1), d_a, 0.0).to(torch.bfloat16), torch.bmm(by_col, a).to(torch.bfloat16),
            spread.sum(1))


# ------------------------------------------------------------ a user's calls --

def _own(s, c):
    import mxfp8_block_scaled_mxgemm_amd as mx
    op = c["op"]
    if op == "sort":
        return tuple(mx.sort_tokens(s["ids"], c["E"]))
    sort = mx.TokenSort(*s["sort"]) if "sort" in s else None
    if op == "dispatch":
        if c["mx"]:
            q, scale = mx.dispatch_tokens_mx(s["x"], sort, fmt=c["fmt"])
            return q.view(F8[c["fmt"]]), scale
        return mx.dispatch_tokens(s["x"], sort), mx.dispatch_tokens_backward(s["d_rows"], sort)
    if op == "combine":
        out = mx.combine_tokens(s["rows"], sort, s["weights"], residual=s["residual"])
        if not c["grad"]:
            return out
        return (out, *mx.combine_tokens_backward(s["d_out"], s["rows"], sort, s["weights"]))
    if op == "linear":
        return mx.linear(s["a"], s["a_s"], s["w"], s["w_s"], bias=s["bias"], act=c["act"], gated=c["gated"],
                         residual=s["residual"], out_dtype=TYPES[c["dtype"]], precision=c["precision"],
                         a_fmt=c["a_fmt"], w_fmt=c["w_fmt"])
    if op == "mlp":
        h, h_s = mx.linear(s["a"], s["a_s"], s["w1"], s["w1_s"], act="silu", gated=True, offsets=sort.offsets,
                           out_dtype="e4m3", precision=c["precision"])
        return mx.linear(h, h_s, s["w2"], s["w2_s"], offsets=sort.offsets, precision=c["precision"])
    return tuple(mx.linear_backward(s["d_out"], s["z"], s["at"], s["at_s"], s["wt"], s["wt_s"], act=c["act"],
                                    gated=c["gated"], sort=sort, fmt=c["fmt"],
                                    precision=c["precision"]))


def run(state):
    s, c = state, state["case"]
    if own:
        return _own(s, c)
    if c["op"] == "sort":
        return _order(s["ids"], c["E"])
    return {"dispatch": _plain_dispatch, "combine": _plain_combine, "linear": _plain_linear, "mlp": _plain_mlp,
            "grad": _plain_grad}[c["op"]](s, c)


def work(case):
    c, op = case, case["op"]
    if op == "sort":
        n = c["T"] * c["k"]
        return {"bytes": 12 * n + 8 * (c["E"] + 1), "flops": n}
    if op == "dispatch":
        one, rows = c["T"] * c["H"], c["T"] * c["k"] * c["H"]
        index = 4 * c["T"] * c["k"]
        if c["mx"]:
            return {"bytes": one * SIZE[c["dtype"]] + rows * 33 / 32 + index, "flops": 2 * one}
        return {"bytes": 2 * (one + rows) * SIZE[c["dtype"]] + 2 * index, "flops": rows}
    if op == "combine":
        one, rows = c["T"] * c["H"], c["T"] * c["k"] * c["H"]
        size = SIZE[c["dtype"]]
        total, flops = (one * (2 if c["residual"] else 1) + rows) * size + 8 * c["T"] * c["k"], 2 * rows
        if c["grad"]:       # the gradient reads rows again and writes as many
            total += (one + rows * 2) * size + 12 * c["T"] * c["k"]
            flops += 3 * rows
        return {"bytes": total, "flops": flops}
    if op == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        out = M * (N // 2 if c["gated"] else N) * SIZE[c["dtype"]]
        return {"bytes": (M + N) * K * 33 / 32 + out * (2 if c["residual"] else 1) + (4 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    if op == "mlp":
        rows, H, F = c["T"] * c["k"], c["H"], c["F"]
        used = min(c["E"], rows)    # experts that can have a row
        return {"bytes": used * 3 * H * F * 33 / 32 + rows * (H * 33 / 32 + 2 * H), "flops": 6 * rows * H * F}
    M, N, K, E = c["M"] * max(1, c["k"]), c["N"], c["K"], max(1, c["E"])
    cols = N // 2 if c["gated"] else N
    return {"bytes": 2 * M * (N + cols) + (M + min(E, M) * N) * K * 33 / 32 + 2 * M * K + E * N * (2 * K + 4),
            "flops": 4 * M * N * K}


# ------------------------------------------------ the definitions in 64 bits --

def _grid64(x, fmt):
    """x (64-bit, last axis in blocks of 32) held in MXFP8, as (codes' values,
    powers of two)."""
    b = x.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / FMAX[fmt]))
    e = torch.where(FMAX[fmt] * torch.exp2(e - 1) >= top, e - 1, e)     # the logarithm's last bit
    e = torch.where(FMAX[fmt] * torch.exp2(e) < top, e + 1, e)
    e = torch.where(top > 0, e.clamp(-127, 127), -127.0)
    y = b / torch.exp2(e)
    bits, low = (3, -6.0) if fmt == "e4m3" else (2, -14.0)
    step = torch.exp2(torch.floor(torch.log2(torch.where(y == 0, 1.0, y.abs()))).clamp(min=low) - bits)
    return torch.round(y / step) * step, torch.exp2(e)


def _held64(x, fmt):
    q, e = _grid64(x, fmt)
    return (q * e).flatten(-2)


def _gelu_like64(z, act):
    """act(z) and its derivative, 64-bit."""
    if act == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0)
    if act == "silu":
        return z * torch.sigmoid(z), torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":      # 0.5 (1 + tanh u) = sigmoid(2 u)
        u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        p = torch.sigmoid(u)
        return z * p, p + z * p * torch.sigmoid(-u) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)
    return z, torch.ones_like(z)


def exact(case, seed):
    c, s = case, _layout(case, seed)
    op = c["op"]
    if op == "sort":
        return None
    if "ids" in s:
        flat = s["ids"].flatten().cpu().tolist()
        lists = [[] for _ in range(c["E"] + 1)]
        for pair, e in enumerate(flat):
            lists[e if 0 <= e < c["E"] else c["E"]].append(pair)
        order = torch.tensor([p for one in lists for p in one], device="cuda")
        ends = [0]
        for one in lists:
            ends.append(ends[-1] + len(one))
        live = ends[c["E"]]
    if op == "dispatch":
        token = order // c["k"]
        rows = s["x"].double()[token]
        rows[live:] = 0
        if c["mx"]:
            q, _ = _grid64(rows, c["fmt"])
            return q.flatten(-2), None
        dx = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
        return rows, dx.index_add_(0, token[:live], s["d_rows"][:live].double())
    if op == "combine":
        token, w = order // c["k"], s["weights"].double().flatten()[order].unsqueeze(1)
        rows = s["rows"].double()
        out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
        out.index_add_(0, token[:live], (w * rows)[:live])
        if s["residual"] is not None:
            out += s["residual"].double()
        if not c["grad"]:
            return out
        d = s["d_out"].double()[token]
        d_w = torch.zeros(c["T"] * c["k"], dtype=torch.float64, device="cuda")
        d_w[order[:live]] = (rows * d).sum(1)[:live]
        d = d * w
        d[live:] = 0
        return out, d, d_w.view(c["T"], c["k"])
    if op == "linear":
        z = torch.mm(_value64(s["a"], s["a_s"], c["a_fmt"]), _value64(s["w"], s["w_s"], c["w_fmt"]).t())
        z = z if s["bias"] is None else z + s["bias"].double()
        half = c["N"] // 2
        y = _gelu_like64(z[:, :half], c["act"])[0] * z[:, half:] if c["gated"] else _gelu_like64(z, c["act"])[0]
        return y if s["residual"] is None else y + s["residual"].double()
    if op == "mlp":
        a, F = _value64(s["a"], s["a_s"], "e4m3"), c["F"]
        out = torch.zeros(a.shape[0], c["H"], dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                z = a[lo:hi] @ _value64(s["w1"][e], s["w1_s"][e], "e4m3").t()
                h = _held64(_gelu_like64(z[:, :F], "silu")[0] * z[:, F:], "e4m3")
                out[lo:hi] = h @ _value64(s["w2"][e], s["w2_s"][e], "e4m3").t()
        return out
    N, E = c["N"], c["E"]
    z, d = s["z"].double(), s["d_out"].double()
    if c["gated"]:
        y, slope = _gelu_like64(z[:, :N // 2], c["act"])
        dz = torch.cat([d * z[:, N // 2:] * slope, d * y], 1)
    else:
        dz = d * _gelu_like64(z, c["act"])[1]
    at, wt = _value64(s["at"], s["at_s"], "e4m3"), _value64(s["wt"], s["wt_s"], "e4m3")
    rows = _held64(torch.nn.functional.pad(dz, (0, wt.shape[-1] - N)), c["fmt"])
    if not E:
        cols = _held64(torch.nn.functional.pad(dz.t(), (0, at.shape[1] - dz.shape[0])), c["fmt"])
        return rows @ wt.t(), cols @ at.t(), dz.sum(0)
    d_a = torch.zeros(z.shape[0], c["K"], dtype=torch.float64, device="cuda")
    d_w = torch.zeros(E, N, c["K"], dtype=torch.float64, device="cuda")
    d_b = torch.zeros(E, N, dtype=torch.float64, device="cuda")
    start = 0
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        n = _up(hi - lo, STEP)
        if n:
            d_a[lo:hi] = rows[lo:hi] @ wt[e].t()
            cols = _held64(torch.nn.functional.pad(dz[lo:hi].t(), (0, n - (hi - lo))), c["fmt"])
            d_w[e] = cols @ at[:, start:start + n].t()
            d_b[e] = dz[lo:hi].sum(0)
        start += n
    return d_a, d_w, d_b
