"""The operators around an expert layer with scales of 128 on measured sizes:
routing of tokens, the FP8 product with a scale for each block of 128 and the
quantisation before it, and the norms before and after a block with its gate
and residual scale, each with its gradient.

Every case runs either in plain torch (32-bit arithmetic, or 64-bit where a
selection hangs on it; one rounding at the end) or, with ``own`` set, through
this package's entry points, on the same inputs.  ``exact`` computes the same
outputs from the definitions in 64 bits.

Operators (T tokens, k experts per token, E experts, H columns):
  route     logits [T, E] -> the k experts of each token and their weights
            (softmax or sigmoid scores; optional selection bias, groups and
            normalisation), with the gradient to the logits.
  quantize  FP8 codes with a float32 scale for each 128 columns of a row, of x
            or of silu(g) u, and, transposed, for each 128 tokens; the same of
            the gradient dz = d act'(z); weights in squares of 128 x 128.
  product   out = a w^T, a with scales of 1 x 128 and w of 128 x 128, dense or
            by expert.
  inner     d_w by expert: products over ranges of the inner axis, both sides
            with scales of 1 x 128.
  norm      r = residual + scale gate post(x), y = pre(r): a block's output
            normalised, gated and added, and the next block's norm of the sum;
            with the gradients to everything.
"""
import math

import torch

own = False

BLOCK = 128
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
TINY = 2.0 ** -126      # smallest scale


def listed():
    return [
        # one decoding step of a small batch: pure latency
        dict(name="route decode", op="route", T=4, k=8, E=128, score="softmax", bias=False, groups=1, top=1,
             normalize=True, scale=1.0, dtype="fp32", grad=False),
        # a training step of a router with a selection bias and groups of experts, and its gradient
        dict(name="route grad", op="route", T=16384, k=8, E=256, score="sigmoid", bias=True, groups=8, top=4,
             normalize=True, scale=2.5, dtype="fp32", grad=True),
        # a prompt's gated hidden rows, between the two products of an expert
        dict(name="quantize gated", op="quantize", M=16384, N=4096, E=32, drop=0.02, act="silu", gated=True,
             back=False, rows=True, cols=False, fmt="e4m3", dtype="bf16"),
        # a training step's gradient of them, both ways, ragged experts
        dict(name="quantize grad", op="quantize", M=8002, N=4096, E=24, drop=0.05, act="silu", gated=True,
             back=True, rows=True, cols=True, fmt="e4m3", dtype="bf16"),
        # all experts' weights after an optimiser's step, both ways
        dict(name="quantize weights", op="weights", N=2048, K=2048, E=24, fmt="e4m3", dtype="bf16"),
        # a decoding batch through one projection: the weights' bytes count
        dict(name="product skinny", op="product", M=64, N=2048, K=7168, E=0, drop=0.0, dtype="bf16",
             precision="exact", a_fmt="e4m3", w_fmt="e4m3"),
        # the largest dense projection of the repository's workloads
        dict(name="product large", op="product", M=8192, N=8192, K=8192, E=0, drop=0.0, dtype="bf16",
             precision="native", a_fmt="e4m3", w_fmt="e4m3"),
        # eight decoding tokens' pairs through their experts
        dict(name="product decode", op="product", M=64, N=1536, K=2048, E=128, drop=0.0, dtype="bf16",
             precision="exact", a_fmt="e4m3", w_fmt="e4m3"),
        # a prompt through the experts
        dict(name="product prefill", op="product", M=16384, N=4096, K=4096, E=32, drop=0.02, dtype="bf16",
             precision="native", a_fmt="e4m3", w_fmt="e4m3"),
        # a training step's weight gradients by expert, kept in 32 bits
        dict(name="inner grad", op="inner", M=2048, N=2048, rows=8002, E=24, drop=0.05, dtype="fp32",
             precision="exact", a_fmt="e5m2", w_fmt="e4m3"),
        # four decoding tokens between two blocks
        dict(name="norm decode", op="norm", T=4, H=7168, G=1, kind="rms", post=True, pre=True, gate=False,
             scale=1.0, dtype="bf16", grad=False),
        # a training step: a gate for each of eight sequences, forward and backward
        dict(name="norm grad", op="norm", T=8192, H=4096, G=8, kind="rms", post=True, pre=True, gate=True,
             scale=0.5, dtype="bf16", grad=True),
    ]


# inner lengths in blocks, and widths that tiles divide
STEPS = [1, 2, 3, 4, 5, 7, 8, 11, 16, 28, 32, 56, 64]
WIDTHS = [64, 128, 192, 256, 512, 896, 1024, 1536, 2048, 3584, 4096, 7168, 8192]


def _log(rng, lo, hi):
    """Spread over the logarithm; long ones odd, so that no tile divides them."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n | 1 if 2048 < n < hi else n


def draw(rng):
    op = rng.choice(["route", "quantize", "weights", "product", "product", "inner", "norm", "norm"])
    drop = rng.choice([0.0, 0.0, 0.02, 0.3])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    precision = rng.choice(["exact", "native"])
    if op == "route":
        E = rng.choice([4, 8, 24, 40, 64, 128, 200, 256, 512, 1000])
        groups = rng.choice([n for n in (1, 1, 2, 4, 8) if E % n == 0 and E // n >= 4])
        top = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, 16384), k=rng.choice([n for n in (1, 2, 4, 6, 8) if n <= E // groups * top]),
                    E=E, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, top=top,
                    normalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), dtype=dtype, grad=rng.random() < 0.5)
    if op == "norm":
        H = _log(rng, 64, 8192) if rng.random() < 0.3 else rng.choice(WIDTHS)
        T, G = _log(rng, 1, 16384), 1
        gate = rng.random() < 0.6
        if gate and rng.random() < 0.6:     # a gate for each of G runs of rows
            G = _log(rng, 1, T)
            T = max(1, T // G) * G
        T = min(T, max(1, (1 << 25) // H) // G * G or G)
        return dict(op=op, T=T, H=H, G=G, kind=rng.choice(["rms", "rms", "layer"]), post=rng.random() < 0.7,
                    pre=rng.random() < 0.8, gate=gate, scale=rng.choice([1.0, 0.5]), dtype=dtype,
                    grad=rng.random() < 0.6)
    E = rng.choice([4, 8, 24, 40, 64, 128])
    if op == "quantize":
        gated = rng.random() < 0.5
        N = _log(rng, 64, 8192) if rng.random() < 0.3 else rng.choice(WIDTHS)
        cols = rng.random() < 0.5
        E = E if rng.random() < 0.6 else 0
        return dict(op=op, M=min(_log(rng, 1, 16384), max(1, (1 << 26) // N)), N=N - N % 2 if gated else N, E=E,
                    drop=drop if E else 0.0, act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                    gated=gated, back=rng.random() < 0.5, rows=rng.random() < 0.7 or not cols, cols=cols, fmt=fmt,
                    dtype=dtype)
    if op == "weights":
        N = _log(rng, 16, 4096) if rng.random() < 0.4 else rng.choice(WIDTHS)
        K = BLOCK * rng.choice(STEPS)
        E = rng.choice([1, 4, 8, 24])
        return dict(op=op, N=N, K=K, E=max(1, min(E, (1 << 26) // (N * K))), fmt=fmt, dtype=dtype)
    if op == "product":
        K = BLOCK * rng.choice(STEPS)
        N = _log(rng, 16, 8192) if rng.random() < 0.3 else rng.choice(WIDTHS)
        if rng.random() < 0.5:
            E = 0
        M = min(_log(rng, 1, 16384), max(1, (1 << 38) // (2 * N * K)))
        return dict(op=op, M=M, N=N, K=K, E=min(E, max(1, (1 << 30) // (N * K))) if E else 0,
                    drop=drop if E else 0.0, dtype=rng.choice(["bf16", "bf16", "fp16"]), precision=precision,
                    a_fmt=fmt, w_fmt="e4m3")
    M, N = (_log(rng, 16, 4096) if rng.random() < 0.3 else BLOCK * rng.choice([n for n in STEPS if n <= 32])
            for _ in range(2))
    E = min(E, 40)
    return dict(op=op, M=M, N=N, rows=min(_log(rng, 1, 16384), max(1, (1 << 37) // (2 * M * N))), E=E, drop=drop,
                dtype=rng.choice(["bf16", "fp32"]) if precision == "exact" else "bf16", precision=precision, a_fmt=fmt,
                w_fmt="e4m3")


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, scale=1.0, dtype=torch.float32, outliers=False):
    x = torch.randn(*shape, generator=g, device="cuda") * scale
    if outliers:    # a few large activations
        x = torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.002, x * 20, x)
    return x.to(dtype)


def _up(n, m):
    return -(-n // m) * m


def _sorted(g, M, E, drop):
    """M rows sorted by expert, some experts far more popular than others, some
    rows dropped: offsets, k_offsets (counts in whole blocks), row_of, pair_of."""
    logits = 1.2 * torch.randn(E, generator=g, device="cuda")
    key = torch.multinomial(torch.softmax(logits, 0), M, replacement=True, generator=g)
    if drop:
        key = torch.where(torch.rand(M, generator=g, device="cuda") < drop, E, key)
    key, pair = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device="cuda")).to(torch.int32)
    k_offsets = torch.zeros_like(offsets)
    k_offsets[1:] = torch.cumsum((offsets[1:] - offsets[:-1] + BLOCK - 1) // BLOCK * BLOCK, 0)
    row_of = torch.empty_like(pair)
    row_of[pair] = torch.arange(M, device="cuda")
    return offsets, k_offsets, row_of.view(M, 1).to(torch.int32), pair.to(torch.int32)


def _pack(x, fmt):
    """FP8 codes of x along its last axis (a multiple of 128) and a float32
    scale for each 128: the largest magnitude over the format's."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    s = (b.abs().amax(-1) / FMAX[fmt]).clamp(min=TINY)
    return (b / s.unsqueeze(-1)).flatten(-2).to(F8[fmt]), s


def _operand(x, fmt):
    """_pack of a product's operand, the scales held block by block (those of
    one block for all rows side by side), as this package's quantiser does."""
    q, s = _pack(x.contiguous(), fmt)
    return q, s.t().contiguous().t()


def _squares(w, fmt):
    """The same with a scale for each 128 x 128; w [.., N, K]."""
    N, K = w.shape[-2:]
    b = torch.nn.functional.pad(w.float(), (0, _up(K, BLOCK) - K, 0, _up(N, BLOCK) - N))
    b = b.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))
    s = (b.abs().amax((-3, -1)) / FMAX[fmt]).clamp(min=TINY)
    q = (b / s[..., :, None, :, None]).flatten(-2).flatten(-3, -2)
    return q[..., :N, :].to(F8[fmt]), s


def _padded(x, sort, E):
    """Rows of x, by expert, each expert's in whole blocks: [all blocks, C]."""
    M = x.shape[0]
    offsets, k_offsets = sort[0], sort[1]
    row = torch.arange(M, device="cuda")
    expert = torch.searchsorted(offsets[1:].contiguous(), row.int(), right=True)
    kept = expert < E
    expert = expert.clamp(max=E - 1)
    column = torch.where(kept, k_offsets[expert] + row - offsets[expert], 0)
    out = x.new_zeros((_up(M, BLOCK) // BLOCK + E) * BLOCK, x.shape[1])
    return out.index_add_(0, column, torch.where(kept.unsqueeze(1), x, 0.0))


def _layout(case, seed):
    """The inputs of a case, the same for every form of the operator."""
    c, g = case, _generator(seed)
    op = c["op"]
    if op == "route":
        T, E = c["T"], c["E"]
        s = dict(logits=(_normal(g, T, E, scale=1.5) + _normal(g, E, scale=0.5)).to(TYPES[c["dtype"]]))
        s["bias"] = _normal(g, E, scale=0.1) if c["bias"] else None
        s["d"] = _normal(g, T, c["k"]) if c["grad"] else None
        return s
    if op == "norm":
        T, H, dt = c["T"], c["H"], TYPES[c["dtype"]]
        s = dict(x=_normal(g, T, H, scale=3.0, dtype=dt, outliers=True), res=_normal(g, T, H, scale=2.0, dtype=dt))
        s["gate"] = _normal(g, c["G"], H, dtype=dt) if c["gate"] else None
        s["post"] = 1 + _normal(g, H, scale=0.2) if c["post"] else None
        s["pre"] = 1 + _normal(g, H, scale=0.2) if c["pre"] else None
        s["d_y"] = _normal(g, T, H, dtype=dt) if c["grad"] and c["pre"] else None
        s["d_r"] = _normal(g, T, H, dtype=dt) if c["grad"] else None
        return s
    if op == "quantize":
        M, N = c["M"], c["N"]
        s = dict(sort=_sorted(g, M, c["E"], c["drop"]) if c["E"] else None)
        if c["back"]:
            s["z"] = _normal(g, M, N, dtype=torch.bfloat16)
            s["x"] = _normal(g, M, N // 2 if c["gated"] else N, scale=1e-3, dtype=TYPES[c["dtype"]], outliers=True)
        else:
            s["x"] = _normal(g, M, N, dtype=TYPES[c["dtype"]], outliers=True)
        return s
    if op == "weights":
        return dict(w=_normal(g, c["E"], c["N"], c["K"], scale=c["K"] ** -0.5, dtype=TYPES[c["dtype"]]))
    if op == "product":
        M, N, K, E = c["M"], c["N"], c["K"], c["E"]
        s = dict(sort=_sorted(g, M, E, c["drop"]) if E else None)
        s["a"], s["a_s"] = _operand(_normal(g, M, K, outliers=True), c["a_fmt"])
        s["w"], s["w_s"] = _squares(_normal(g, *((E,) if E else ()), N, K, scale=K ** -0.5), c["w_fmt"])
        return s
    E = c["E"]
    s = dict(sort=_sorted(g, c["rows"], E, c["drop"]))
    s["a"], s["a_s"] = _operand(_padded(_normal(g, c["rows"], c["M"], scale=1e-3, outliers=True), s["sort"], E).t(),
                                c["a_fmt"])
    s["w"], s["w_s"] = _operand(_padded(_normal(g, c["rows"], c["N"]), s["sort"], E).t(), c["w_fmt"])
    return s


def prepare(case, seed):
    s = _layout(case, seed)
    s["case"] = case
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


def _scores(logits, score):
    """Scores in 64 bits: a selection hangs on them."""
    x = logits.double()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _top(key, k):
    """The k largest of each row, the lower index first where they are equal."""
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]


def _plain_route(s, c):
    score = _scores(s["logits"], c["score"])
    key = score if s["bias"] is None else score + s["bias"].double()
    if s["bias"] is None and c["groups"] == 1:
        key = s["logits"].float()           # the scores' order, exactly
    if c["groups"] > 1:
        by = key.unflatten(1, (c["groups"], -1))
        rank = by.sort(dim=2, descending=True).values[:, :, :2].sum(2)
        open_ = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, _top(rank, c["top"]), True)
        key = torch.where(open_.unsqueeze(2), by, -math.inf).flatten(1)
    ids = _top(key, c["k"])
    picked = score.gather(1, ids)
    total = picked.sum(1, keepdim=True)
    w = c["scale"] * (picked / total if c["normalize"] else picked)
    ids32, w32 = ids.to(torch.int32), w.float()
    if s["d"] is None:
        return ids32, w32
    d = c["scale"] * s["d"].double()
    if c["normalize"]:
        d = (d - (d * picked / total).sum(1, keepdim=True)) / total
    d_score = torch.zeros_like(score).scatter_(1, ids, d)
    if c["score"] == "sigmoid":
        d_logits = d_score * score * (1 - score)
    else:
        d_logits = score * (d_score - (d_score * score).sum(1, keepdim=True))
    return ids32, w32, d_logits.to(s["logits"].dtype)


def _quantized(y, s, c):
    """y's codes and scales along its rows, and by 128 tokens of its transpose."""
    M, C = y.shape
    rows = cols = None
    if s["sort"] is not None:
        kept = torch.arange(M, device="cuda") < s["sort"][0][-1]
    if c["rows"]:
        q, scale = _pack(torch.nn.functional.pad(y, (0, _up(C, BLOCK) - C)), c["fmt"])
        if s["sort"] is not None:
            scale = torch.where(kept.unsqueeze(1), scale, 0.0)
            q = torch.where(kept.unsqueeze(1), q.float(), 0.0).to(F8[c["fmt"]])
        rows = q, scale
    if c["cols"]:
        if s["sort"] is None:
            cols = _pack(torch.nn.functional.pad(y, (0, 0, 0, _up(M, BLOCK) - M)).t(), c["fmt"])
        else:
            q, scale = _pack(_padded(y, s["sort"], c["E"]).t(), c["fmt"])
            used = torch.arange(scale.shape[1], device="cuda") * BLOCK < s["sort"][1][-1]
            cols = q, torch.where(used, scale, 0.0)
    return [x for pair in (rows, cols) if pair is not None for x in pair]


def _plain_quantize(s, c):
    x = s["x"].float()
    half = c["N"] // 2
    if not c["back"]:
        y = _act(x[:, :half], c["act"]) * x[:, half:] if c["gated"] else _act(x, c["act"])
    else:
        z = s["z"].float()
        if c["gated"]:
            y = torch.cat([x * z[:, half:] * _act_grad(z[:, :half], c["act"]), x * _act(z[:, :half], c["act"])], 1)
        else:
            y = x * _act_grad(z, c["act"])
    return _quantized(y, s, c)


def _plain_weights(s, c):
    q, scale = _squares(s["w"], c["fmt"])
    flipped = torch.nn.functional.pad(q.transpose(1, 2).float(), (0, _up(c["N"], BLOCK) - c["N"])).to(F8[c["fmt"]])
    return q, scale, flipped, scale.transpose(1, 2).contiguous()


def _value(q, s):
    """The 32-bit values that codes with scales of 1 x 128 stand for."""
    return (q.float().unflatten(-1, (-1, BLOCK)) * s.unsqueeze(-1)).flatten(-2)


def _square_value(q, s):
    return _value(q, s.repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :])


def _plain_product(s, c):
    a, w = _value(s["a"], s["a_s"]), _square_value(s["w"], s["w_s"])
    dtype = TYPES[c["dtype"]]
    if not c["E"]:
        return (a @ w.t()).to(dtype)
    E, offsets = c["E"], s["sort"][0]
    row = torch.arange(a.shape[0], device="cuda")
    expert = torch.searchsorted(offsets[1:].contiguous(), row.int(), right=True)
    kept = expert < E
    expert = expert.clamp(max=E - 1)
    slot = torch.where(kept, row - offsets[expert], 0)
    longest = max(1, int((offsets[1:] - offsets[:-1]).max()))
    pad = a.new_zeros(E, longest, a.shape[1])
    pad.index_put_((expert, slot), torch.where(kept.unsqueeze(1), a, 0), accumulate=True)
    out = torch.bmm(pad, w.transpose(1, 2))[expert, slot]
    return torch.where(kept.unsqueeze(1), out, 0.0).to(dtype)


def _plain_inner(s, c):
    start, end = s["sort"][1][:-1].long(), s["sort"][1][1:].long()
    longest = max(BLOCK, int((end - start).max()))
    at = start.unsqueeze(1) + torch.arange(longest, device="cuda")
    live = at < end.unsqueeze(1)
    at = torch.where(live, at, 0)
    a = torch.where(live, _value(s["a"], s["a_s"])[:, at], 0.0).transpose(0, 1)
    w = torch.where(live, _value(s["w"], s["w_s"])[:, at], 0.0).permute(1, 2, 0).contiguous()
    return torch.bmm(a, w).to(TYPES[c["dtype"]])


EPS = 1e-6


def _normed(x, kind):
    """x with its mean (layer) taken off and its root mean square one, and 1 / that."""
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    return x * rstd, rstd


def _norm_back(d, hat, rstd, kind):
    d = d - hat * (d * hat).mean(1, keepdim=True)
    if kind == "layer":
        d = d - d.mean(1, keepdim=True)
    return rstd * d


def _norm(x, res, gate, post, pre, d_y, d_r, c, dtype):
    """The norm operator in the arithmetic of its inputs' type; r is rounded to
    ``dtype`` before it is normalised, as it is kept."""
    T, G, work = c["T"], c["G"], x.dtype
    n = x
    if post is not None:
        hat, rstd = _normed(x, c["kind"])
        n = hat * post
    wide = None if gate is None else gate.repeat_interleave(T // G, 0)
    r = (res + c["scale"] * (n if wide is None else n * wide)).to(dtype)
    out = [r]
    if pre is not None:
        r_hat, r_rstd = _normed(r.to(work), c["kind"])
        out.append((r_hat * pre).to(dtype))
    if not c["grad"]:
        return out
    d_res = d_r
    if pre is not None:
        d_res = d_res + _norm_back(d_y * pre, r_hat, r_rstd, c["kind"])
    d_n = c["scale"] * d_res
    if wide is not None:
        out.append((d_n * n).view(G, T // G, -1).sum(1).to(dtype))
        d_n = d_n * wide
    if post is not None:
        out.append((d_n * hat).sum(0))
        d_n = _norm_back(d_n * post, hat, rstd, c["kind"])
    if pre is not None:
        out.append((d_y * r_hat).sum(0))
    return out + [d_n.to(dtype), d_res.to(dtype)]


def _plain_norm(s, c):
    wide = {n: None if s[n] is None else s[n].float() for n in ("x", "res", "gate", "post", "pre", "d_y", "d_r")}
    return _norm(*wide.values(), c, TYPES[c["dtype"]])


# ------------------------------------------------------------ a user's calls --

def _own(s, c):
    import mxfp8_block_scaled_mxgemm_amd as mx
    op = c["op"]
    if op == "route":
        how = dict(score=c["score"], bias=s["bias"], groups=c["groups"], top_groups=c["top"],
                   normalize=c["normalize"], scale=c["scale"])
        ids, w = mx.route_tokens(s["logits"], c["k"], **how)
        if s["d"] is None:
            return ids, w
        del how["bias"], how["groups"], how["top_groups"]
        return ids, w, mx.route_tokens_backward(s["d"], s["logits"], ids, **how)
    if op == "quantize":
        how = dict(act=c["act"], gated=c["gated"], sort=None if s["sort"] is None else mx.TokenSort(*s["sort"]),
                   fmt=c["fmt"], rows=c["rows"], cols=c["cols"])
        if c["back"]:
            rows, cols = mx.block_quantize_backward(s["x"], s["z"], **how)
        else:
            rows, cols = mx.block_quantize(s["x"], **how)
        return [x for q, scale in (rows, cols) if q is not None for x in (q.view(F8[c["fmt"]]), scale)]
    if op == "weights":
        (q, scale), (qt, st) = mx.block_quantize_weight(s["w"], fmt=c["fmt"], transposed=True)
        return q.view(F8[c["fmt"]]), scale, qt.view(F8[c["fmt"]]), st
    if op == "product":
        return mx.block_linear(s["a"].view(torch.uint8), s["a_s"], s["w"].view(torch.uint8), s["w_s"],
                               offsets=s["sort"][0] if c["E"] else None, out_dtype=TYPES[c["dtype"]],
                               precision=c["precision"], a_fmt=c["a_fmt"], w_fmt=c["w_fmt"])
    if op == "inner":
        return mx.block_linear_by_inner(s["a"].view(torch.uint8), s["a_s"], s["w"].view(torch.uint8), s["w_s"],
                                        s["sort"][1], out_dtype=TYPES[c["dtype"]], precision=c["precision"],
                                        a_fmt=c["a_fmt"], w_fmt=c["w_fmt"])
    how = dict(gate=s["gate"], scale=c["scale"], post_weight=s["post"], pre_weight=s["pre"], kind=c["kind"], eps=EPS)
    y, r = mx.add_norm(s["x"], s["res"], **how)
    out = [r] if y is None else [r, y]
    if c["grad"]:
        d = mx.add_norm_backward(s["d_y"], s["d_r"], s["x"], r, **how)
        out += [t for t in (d.d_gate, d.d_post_weight, d.d_pre_weight) if t is not None] + [d.d_x, d.d_residual]
    return out


def run(state):
    s, c = state, state["case"]
    if own:
        return _own(s, c)
    return {"route": _plain_route, "quantize": _plain_quantize, "weights": _plain_weights, "product": _plain_product,
            "inner": _plain_inner, "norm": _plain_norm}[c["op"]](s, c)


def work(case):
    c, op = case, case["op"]
    if op == "route":
        n, size = c["T"] * c["E"], SIZE[c["dtype"]]
        total = n * size + 8 * c["T"] * c["k"] + (4 * c["E"] if c["bias"] else 0)
        if c["grad"]:
            total += 2 * n * size + 8 * c["T"] * c["k"]
        return {"bytes": total, "flops": 4 * n}
    if op == "quantize":
        M, N, size = c["M"], c["N"], SIZE[c["dtype"]]
        held = N // 2 if c["gated"] and not c["back"] else N
        read = M * (N // 2 if c["gated"] else N) * size + 2 * M * N if c["back"] else M * N * size
        ways = int(c["rows"]) + int(c["cols"])
        return {"bytes": read + ways * M * held * (1 + 4 / BLOCK), "flops": 8 * M * N}
    if op == "weights":
        n = c["E"] * c["N"] * c["K"]
        return {"bytes": n * (SIZE[c["dtype"]] + 2), "flops": 2 * n}
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        used = min(c["E"], M) if c["E"] else 1      # experts that can have a row
        return {"bytes": M * K * (1 + 4 / BLOCK) + used * N * K + M * N * SIZE[c["dtype"]], "flops": 2 * M * N * K}
    if op == "inner":
        M, N, rows = c["M"], c["N"], c["rows"]
        return {"bytes": (M + N) * rows * (1 + 4 / BLOCK) + c["E"] * M * N * SIZE[c["dtype"]],
                "flops": 2 * M * N * rows}
    n, size = c["T"] * c["H"], SIZE[c["dtype"]]
    gate = c["G"] * c["H"] * size if c["gate"] else 0
    total = (3 + int(c["pre"])) * n * size + gate
    if c["grad"]:       # reads d_y, d_r, x, r; writes d_x, d_residual
        total += (5 + int(c["pre"])) * n * size + 2 * gate
    return {"bytes": total, "flops": 10 * n}


# ------------------------------------------------ the definitions in 64 bits --

def _codes64(x, s, fmt):
    """x / s on the format's grid, 64-bit (s broadcast)."""
    y = x / torch.where(s > 0, s, 1.0)
    bits, low = (3, -6.0) if fmt == "e4m3" else (2, -14.0)
    step = torch.exp2(torch.floor(torch.log2(torch.where(y == 0, 1.0, y.abs()))).clamp(min=low) - bits)
    return torch.round(y / step) * step


def _blocks64(x, fmt):
    """Codes' values and scales of x, 64-bit, along its last axis."""
    b = x.unflatten(-1, (-1, BLOCK))
    s = torch.clamp(b.abs().amax(-1) / FMAX[fmt], min=TINY)
    return _codes64(b, s.unsqueeze(-1), fmt).flatten(-2), s


def _smooth64(z, act):
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


def _ends(offsets):
    return [int(x) for x in offsets.cpu()]


def _exact_route(s, c):
    x = s["logits"].double()
    score = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
    key = score + (0.0 if s["bias"] is None else s["bias"].double())
    if s["bias"] is None and c["groups"] == 1:
        key = x
    T, E, G = c["T"], c["E"], c["groups"]
    low = torch.full_like(key, -math.inf)
    if G > 1:
        rank = torch.zeros(T, G, dtype=torch.float64, device="cuda")
        for g in range(G):
            part = key[:, g * (E // G):(g + 1) * (E // G)]
            best = part.max(1)
            rest = part.clone().scatter_(1, best.indices.unsqueeze(1), -math.inf)
            rank[:, g] = best.values + rest.max(1).values
        left, shut = rank, torch.ones(T, G, dtype=torch.bool, device="cuda")
        for _ in range(c["top"]):       # the first of the largest, one at a time
            at = (left == left.amax(1, keepdim=True)).int().argmax(1, keepdim=True)
            shut.scatter_(1, at, False)
            left = left.scatter(1, at, -math.inf)
        key = torch.where(shut.repeat_interleave(E // G, 1), low, key)
    ids = []
    for _ in range(c["k"]):
        at = (key == key.amax(1, keepdim=True)).int().argmax(1, keepdim=True)
        ids.append(at)
        key = key.scatter(1, at, -math.inf)
    ids = torch.cat(ids, 1)
    with torch.enable_grad():
        x = x.requires_grad_()
        score = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
        w = score.gather(1, ids)
        if c["normalize"]:
            w = w / w.sum(1, keepdim=True)
        w = w * c["scale"]
    if s["d"] is None:
        return None, w.detach()
    return None, w.detach(), torch.autograd.grad(w, x, s["d"].double())[0]


def exact(case, seed):
    c, s = case, _layout(case, seed)
    op = c["op"]
    if op == "route":
        return _exact_route(s, c)
    if op == "norm":
        # the sums in 64 bits, and for the gradients the rounded r that the path keeps
        wide = {n: None if s[n] is None else s[n].double() for n in ("x", "res", "gate", "post", "pre", "d_y", "d_r")}
        leaf = {n: None if t is None else t.clone().requires_grad_() for n, t in wide.items()}

        def norm(x, weight):
            m = x - x.mean(1, keepdim=True) if c["kind"] == "layer" else x
            return m / torch.sqrt(m.square().mean(1, keepdim=True) + EPS) * weight

        with torch.enable_grad():
            n = leaf["x"] if leaf["post"] is None else norm(leaf["x"], leaf["post"])
            if leaf["gate"] is not None:
                n = (n.view(c["G"], -1, c["H"]) * leaf["gate"].unsqueeze(1)).view(c["T"], c["H"])
            r = leaf["res"] + c["scale"] * n
            kept = r + (r.detach().to(TYPES[c["dtype"]]).double() - r.detach())
            y = None if leaf["pre"] is None else norm(kept, leaf["pre"])
        out = [r.detach()] + ([] if y is None else [y.detach()])
        if not c["grad"]:
            return out
        names = [n for n in ("gate", "post", "pre", "x", "res") if leaf[n] is not None]
        tops = [(kept, wide["d_r"])] + ([] if y is None else [(y, wide["d_y"])])
        grads = torch.autograd.grad([t for t, _ in tops], [leaf[n] for n in names], [d for _, d in tops])
        return out + list(grads)
    if op == "quantize":
        x, half = s["x"].double(), c["N"] // 2
        if not c["back"]:
            y = _smooth64(x[:, :half], c["act"])[0] * x[:, half:] if c["gated"] else _smooth64(x, c["act"])[0]
        else:
            z = s["z"].double()
            if c["gated"]:
                v, slope = _smooth64(z[:, :half], c["act"])
                y = torch.cat([x * z[:, half:] * slope, x * v], 1)
            else:
                y = x * _smooth64(z, c["act"])[1]
        M, C = y.shape
        out = []
        live = M if s["sort"] is None else int(s["sort"][0][-1])
        if c["rows"]:
            q, scale = _blocks64(torch.nn.functional.pad(y, (0, _up(C, BLOCK) - C)), c["fmt"])
            q[live:], scale[live:] = 0, 0
            out += [q, scale]
        if c["cols"]:
            parts, at = [], 0
            ends = [0, M] if s["sort"] is None else _ends(s["sort"][0])
            for lo, hi in zip(ends, ends[1:]):
                parts.append(torch.nn.functional.pad(y[lo:hi], (0, 0, 0, _up(hi - lo, BLOCK) - (hi - lo))))
            used = sum(p.shape[0] for p in parts)
            all_ = _up(M, BLOCK) if s["sort"] is None else (_up(M, BLOCK) // BLOCK + c["E"]) * BLOCK
            q, scale = _blocks64(torch.nn.functional.pad(torch.cat(parts), (0, 0, 0, all_ - used)).t(), c["fmt"])
            scale[:, used // BLOCK:] = 0
            out += [q, scale]
        return out
    if op == "weights":
        N, K, E = c["N"], c["K"], c["E"]
        w, Np = s["w"].double(), _up(N, BLOCK)
        scale = torch.zeros(E, Np // BLOCK, K // BLOCK, dtype=torch.float64, device="cuda")
        for i in range(Np // BLOCK):
            rows = w[:, i * BLOCK:(i + 1) * BLOCK].abs().amax(1)
            scale[:, i] = rows.unflatten(1, (-1, BLOCK)).amax(2) / FMAX[c["fmt"]]
        scale = scale.clamp(min=TINY)
        per = scale.repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)
        q = _codes64(w, per, c["fmt"])
        return q, scale, torch.nn.functional.pad(q.transpose(1, 2), (0, Np - N)), scale.transpose(1, 2)
    wide = lambda q, t: q.double() * t.double().repeat_interleave(BLOCK, 1)  # noqa: E731
    if op == "product":
        N, E = c["N"], c["E"]
        a = wide(s["a"], s["a_s"])
        if not E:
            return a @ wide(s["w"], s["w_s"].repeat_interleave(BLOCK, 0)[:N]).t()
        out = torch.zeros(c["M"], N, dtype=torch.float64, device="cuda")
        ends = _ends(s["sort"][0])
        for e in range(E):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                out[lo:hi] = a[lo:hi] @ wide(s["w"][e], s["w_s"][e].repeat_interleave(BLOCK, 0)[:N]).t()
        return out
    a, w = wide(s["a"], s["a_s"]), wide(s["w"], s["w_s"])
    ends = _ends(s["sort"][1])
    return torch.stack([a[:, lo:hi] @ w[:, lo:hi].t() for lo, hi in zip(ends, ends[1:])])
