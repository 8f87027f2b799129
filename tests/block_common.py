"""References in 64 bits for the operators with scales of 128 and those around
them (imported by test modules, not collected).  Everything runs on the CPU from
the operators' definitions and shares no code with the library."""
import math

import torch

import moe_common as mc

FMAX, F8 = mc.FMAX, mc.F8
LOW = 2.0 ** -126
# largest rounding of a code, relative to its value, and of a subnormal one
REL = {"e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
SUB = {"e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}
U = 2.0 ** -24          # half a step of float32, relative


def up(n, m=128):
    return -(-n // m) * m


# ------------------------------------------------------------------- route --

def route(logits, k, score="softmax", bias=None, groups=1, top_groups=1, normalize=True, scale=1.0):
    """(ids, weights) by definition, one token at a time."""
    T, E = logits.shape
    ids, weights = torch.full((T, k), -1, dtype=torch.int32), torch.zeros(T, k, dtype=torch.float64)
    big = torch.finfo(torch.float32).max
    for t in range(T):
        x = [min(v, big) for v in logits[t].double().tolist()]
        live = [e for e in range(E) if x[e] > -math.inf]        # (NaN is not)
        if not live:
            continue
        top = max(x[e] for e in live)
        if score == "sigmoid":
            s = {e: 1 / (1 + math.exp(-x[e])) if x[e] > -700 else 0.0 for e in live}
        else:
            total = math.fsum(math.exp(x[e] - top) for e in live)
            s = {e: math.exp(x[e] - top) / total for e in live}
        key = {e: s[e] + (0.0 if bias is None else float(bias[e])) for e in live}
        if bias is None and groups == 1:
            key = {e: x[e] for e in live}
        key = {e: v for e, v in key.items() if v > -math.inf}
        if groups > 1:
            size = E // groups
            rank = {}
            for e in key:
                rank.setdefault(e // size, []).append(key[e])
            rank = {g: sum(sorted(v, reverse=True)[:2]) for g, v in rank.items()}
            taken = sorted(rank, key=lambda g: (-rank[g], g))[:top_groups]
            key = {e: v for e, v in key.items() if e // size in taken}
        chosen = sorted(key, key=lambda e: (-key[e], e))[:k]
        if normalize and score == "softmax" and chosen:
            best = max(x[e] for e in chosen)
            w = [math.exp(x[e] - best) for e in chosen]
        else:
            w = [s[e] for e in chosen]
        if normalize:
            total = math.fsum(w)
            w = [v / total if total > 0 else 0.0 for v in w]
        for j, e in enumerate(chosen):
            ids[t, j], weights[t, j] = e, scale * w[j]
    return ids, weights


# ---------------------------------------------------------------- quantise --

def value(q, s, fmt):
    """64-bit values of codes q [.., K] (uint8) with scales s [.., K / 128]."""
    return (q.view(F8[fmt]).double().unflatten(-1, (-1, 128)) * s.double().unsqueeze(-1)).flatten(-2)


def check_blocks(q, s, y, t, fmt, what):
    """Codes q [R, Cp] and scales s [R, Cp / 128] hold y [R, C] (64-bit, known to
    t): each scale the largest magnitude over the format's (one division), each
    value within half a code's step.  The quotient's own roundings, and the one
    of the scale that the value is formed with here, may move it across a tie: 3
    U of the value."""
    q, s = q.cpu(), s.cpu()
    R, C = y.shape
    Cp = up(C)
    assert q.shape == (R, Cp) and s.shape == (R, Cp // 128), (what, q.shape, s.shape)
    assert not q[:, C:].any(), what
    wide = torch.nn.functional.pad(y, (0, Cp - C)).unflatten(-1, (-1, 128))
    tt = torch.nn.functional.pad(torch.broadcast_to(t, y.shape), (0, Cp - C)).unflatten(-1, (-1, 128))
    ref = (wide.abs().amax(-1) / FMAX[fmt]).clamp(min=LOW)
    mc.assert_within(s, ref, tt.amax(-1) / FMAX[fmt] + 2 * U * ref, what + " scales")
    size = wide.abs() + tt
    bound = tt + (REL[fmt] + 3 * U) * size + SUB[fmt] * (1 + 4 * U) * s.double().unsqueeze(-1)
    mc.assert_within(value(q, s, fmt), wide.flatten(-2), bound.flatten(-2), what + " codes")


def blocks(x, fmt):
    """Codes and scales of x (64-bit or float32) along its last axis, for inputs."""
    b = x.float().unflatten(-1, (-1, 128))
    s = (b.abs().amax(-1) / FMAX[fmt]).clamp(min=LOW)
    return (b / s.unsqueeze(-1)).flatten(-2).to(F8[fmt]).view(torch.uint8), s


def squares(w, fmt):
    N, K = w.shape[-2:]
    b = torch.nn.functional.pad(w.float(), (0, 0, 0, up(N) - N)).unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    s = (b.abs().amax((-3, -1)) / FMAX[fmt]).clamp(min=LOW)
    q = (b / s[..., :, None, :, None]).flatten(-2).flatten(-3, -2)[..., :N, :]
    return q.to(F8[fmt]).view(torch.uint8).contiguous(), s


def square_value(q, s, fmt):
    return value(q, s.repeat_interleave(128, -2)[..., :q.shape[-2], :], fmt)


# ----------------------------------------------------------------- product --

def product_error(S, K, precision):
    """Error bound of a product from S = sum |a w|.  Inside a block: FP32 sums of
    groups of eight (16 roundings) on the BF16 unit, or what the FP8 unit drops,
    8 x 2^-13 of a group's largest; the scales' product and its multiplication
    one rounding each; then one addition per block, K group, wave and split (16
    and 16 and 8 at most)."""
    fp32 = (16 + 2 + K / 128 + 40) * U
    return S * (fp32 if precision == "exact" else fp32 + 2.0 ** -10)


# ------------------------------------------------------------------- norm ---

def normed(v, kind, eps):
    m = v - v.mean(1, keepdim=True) if kind == "layer" else v
    return m / torch.sqrt(m.square().mean(1, keepdim=True) + eps)


def norm_r(x, residual, gate, scale, post, kind, eps):
    """r before its rounding, 64-bit; gate [G, H]."""
    n = x if post is None else normed(x, kind, eps) * post
    if gate is not None:
        n = n * gate.repeat_interleave(x.shape[0] // gate.shape[0], 0)
    return scale * n if residual is None else residual + scale * n
