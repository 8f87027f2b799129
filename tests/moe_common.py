"""References in 64 bits for the expert layer's GPU tests (imported by test
modules, not collected).  Everything here runs on the CPU from the operators'
definitions and shares no code with the library."""
import math

import numpy as np
import torch

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
# relative half-step of a rounding to the type: 2^-(stored mantissa bits + 1)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half of the type's smallest step (subnormals)
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def rounding(ref, dtype):
    """Error bound of one rounding of ``ref`` to ``dtype``."""
    return HALF[dtype] * ref.abs() + TINY[dtype]


def order(ids, E):
    """(offsets, k_offsets, row_of, pair_of) as lists, by definition."""
    T, k = ids.shape
    flat = [int(i) for i in ids.flatten().tolist()]
    lists = [[] for _ in range(E + 1)]
    for p, e in enumerate(flat):
        lists[e if 0 <= e < E else E].append(p)
    pair_of = [p for one in lists for p in one]
    row_of = [0] * len(flat)
    for r, p in enumerate(pair_of):
        row_of[p] = r
    offsets, k_offsets = [0], [0]
    for one in lists[:E]:
        offsets.append(offsets[-1] + len(one))
        k_offsets.append(k_offsets[-1] + -(-len(one) // 128) * 128)
    return offsets, k_offsets, np.array(row_of, dtype=np.int64).reshape(T, k), np.array(pair_of, dtype=np.int64)


def ids_of(g, T, k, E, drop=0.0):
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if drop:
        ids[torch.rand(T, k, generator=g) < drop] = -1
    return ids


def value(q, s, fmt):
    """64-bit values of MXFP8 codes q [.., K] and scale bytes [.., K / 32]."""
    v = q.view(F8[fmt]).double().unflatten(-1, (-1, 32))
    e = s.double() - 127
    scale = torch.where(s == 255, math.nan, torch.exp2(e))
    return (v * scale.unsqueeze(-1)).flatten(-2)


def quantize(x, fmt):
    """Codes and scale bytes of finite x (64-bit) along its last axis, by the
    rule: smallest e with fmax 2^e >= amax (clamped), round to nearest even."""
    b = x.double().unflatten(-1, (-1, 32))
    m, p = np.frexp(b.abs().amax(-1).numpy())
    e = p - (9 if fmt == "e4m3" else 16) + (m > 0.875)
    e = np.where(m == 0, -127, np.clip(e, -127, 127)).astype(np.int64)
    e = torch.from_numpy(e)
    # every quotient is exact in float32: the inputs here have at most 24 bits
    q = (b / torch.exp2(e.double()).unsqueeze(-1)).float().flatten(-2).to(F8[fmt])
    return q.view(torch.uint8), (e + 127).to(torch.uint8)


def codes(g, shape, fmt, scale=1.0):
    """Random MXFP8 operand: codes and scale bytes."""
    return quantize((torch.randn(shape, generator=g) * scale).float(), fmt)


def act(z, name):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_grad(z, name):
    """Central differences would do; written out so that it is exact."""
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


# Activations move an error by at most their largest slope (gelu: 1.13), and
# are themselves computed in FP32: hardware exponential, reciprocal and erf
# good to a few units in the last place of |z| (16 of 2^-24 allowed).
SLOPE = 1.13
ACT_ERR = 16 * 2.0 ** -24


def product_error(S, K, precision):
    """Error bound of the product from S = sum |a w|: exact mode sums groups
    of eight products into FP32 (one rounding each, plus one per K-step pair
    and per wave or K group); native mode drops what is 2^13 below the largest
    product of a group of eight, at most 8 * 2^-13 of it."""
    fp32 = (K / 8 + 64) * 2.0 ** -24
    return S * (fp32 if precision == "exact" else fp32 + 2.0 ** -10)


def linear(a, w, bias, name, gated, residual, precision):
    """(out, bound before its rounding, z, bound of z) in 64 bits; a [M, K] and
    w [N, K] are 64-bit values."""
    z = a @ w.t()
    S = a.abs() @ w.abs().t()
    tz = product_error(S, a.shape[1], precision)
    if bias is not None:
        z = z + bias.double()
        tz = tz + 2.0 ** -23 * (z.abs() + S)
    if gated:
        h = z.shape[1] // 2
        y, u = act(z[:, :h], name), z[:, h:]
        ty = SLOPE * tz[:, :h] + ACT_ERR * z[:, :h].abs()
        out = y * u
        t = ty * u.abs() + y.abs() * tz[:, h:] + ty * tz[:, h:] + 2.0 ** -23 * out.abs()
    else:
        out = act(z, name)
        t = SLOPE * tz + ACT_ERR * z.abs()
    if residual is not None:
        out = out + residual.double()
        t = t + 2.0 ** -23 * (out.abs() + residual.double().abs())
    return out, t, z, tz


def mx_bound(ref, t, fmt):
    """Bound of a value held in MXFP8 whose exact value is known to t: half a
    step of the code (relative 2^-4 or 2^-3), the smallest step of a block one
    exponent up, and t itself."""
    b = (ref.abs() + t).unflatten(-1, (-1, 32))
    top = b.amax(-1, keepdim=True).expand_as(b).flatten(-2)
    rel, sub = (2.0 ** -4, 2.0 ** -9) if fmt == "e4m3" else (2.0 ** -3, 2.0 ** -16)
    step = sub * torch.exp2(torch.ceil(torch.log2(torch.clamp(top, min=2.0 ** -100) / FMAX[fmt])))
    return rel * (ref.abs() + t) + step + t


def assert_within(got, ref, bound, what=""):
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound)
    same_nan = torch.isnan(ref) & torch.isnan(got)
    same_inf = torch.isinf(ref) & (got == ref)
    bad &= ~(same_nan | same_inf)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        b = bound[i] if torch.is_tensor(bound) and bound.dim() else bound
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds; first at {i}: got "
                             f"{float(got[i])!r}, reference {float(ref[i])!r}, bound {float(b):.3g}")
