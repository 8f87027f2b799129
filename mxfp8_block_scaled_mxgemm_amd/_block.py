"""Binding of the operators with scales of 128 and of those around them
(declared in ``include/mxgemm_block.h``): the router, quantisation to FP8 with
a float32 scale for each block of 128, the product of such operands, dense and
by expert, and the norms before and after a block; each with its gradient.

As in the expert layer's binding: argument checks and marshalling only, outputs
from torch's caching allocator on the stream the call runs on (the current one
unless ``stream`` is given), inputs recorded on another stream, nothing
synchronises.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional

from . import _moe
from ._moe import (
    _PRECISION, _TYPES, GROUP_INNER, GROUP_NONE, GROUP_ROWS, STEP, TokenSort, _activation, _format,
    _laid_out, _on_stream, _plain, _rows_of, _run, _sort_args, _split_workspace, _up,
)

EXPORTED_BLOCK = [
    "mxgemm_route_tokens", "mxgemm_route_tokens_backward", "mxgemm_block_quantize", "mxgemm_block_quantize_weight",
    "mxgemm_block_linear", "mxgemm_block_linear_workspace", "mxgemm_add_norm", "mxgemm_add_norm_backward",
    "mxgemm_add_norm_workspace",
]

SCORES = {"softmax": 0, "sigmoid": 1}
NORMS = {"rms": 0, "layer": 1}
MAX_NORM_COLS = 8192

# mxgemm_block_linear_t and mxgemm_norm_t, in the header's order
BLOCK_ARGS = struct.Struct("6P13q8iPq")
NORM_ARGS = struct.Struct("15P13q5i2fi")


class NormGrads(NamedTuple):
    d_x: "torch.Tensor"
    d_residual: Optional["torch.Tensor"]
    d_gate: Optional["torch.Tensor"]
    d_post_weight: Optional["torch.Tensor"]
    d_pre_weight: Optional["torch.Tensor"]


_bound = None


def _load():
    """The library with these operators' argument types set."""
    global _bound
    if _bound is None:
        lib = _moe._load()
        i64, i32, vp, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
        lib.mxgemm_route_tokens.argtypes = [vp, i64, i32, i64, i32, i32, i32, vp, i32, i32, i32, f32, vp, vp, vp]
        lib.mxgemm_route_tokens_backward.argtypes = [vp, vp, i64, i32, i64, i32, i32, i32, i32, f32, vp, vp, i64, vp]
        lib.mxgemm_block_quantize.argtypes = [vp, i32, i64, vp, i64, i64, i64, i32, i32, vp, vp, i32, i32, vp, vp, vp,
                                              vp, i64, vp]
        lib.mxgemm_block_quantize_weight.argtypes = [vp, i32, i64, i64, i64, i64, i64, i32, vp, vp, vp, vp, vp]
        lib.mxgemm_block_linear.argtypes = [ctypes.c_char_p, vp]
        lib.mxgemm_add_norm.argtypes = [ctypes.c_char_p, vp]
        lib.mxgemm_add_norm_backward.argtypes = [ctypes.c_char_p, vp]
        for name in EXPORTED_BLOCK:
            getattr(lib, name).restype = ctypes.c_int
        lib.mxgemm_block_linear_workspace.argtypes = lib.mxgemm_add_norm_workspace.argtypes = [i64, i64, i64]
        lib.mxgemm_block_linear_workspace.restype = lib.mxgemm_add_norm_workspace.restype = i64
        _bound = lib
    return _bound


def _pick(table, name, what):
    try:
        return table[name]
    except (KeyError, TypeError):
        raise ValueError(f"unknown {what} {name!r}: one of {', '.join(map(str, table))}") from None


def _new(shape, dtype, device):
    """A contiguous matrix (the quickest of torch's ways to one)."""
    return _moe.torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)


def _new_scales(rows, blocks, device):
    """Scales [rows, blocks], block by block in memory."""
    return _moe.torch.empty_strided((rows, blocks), (1, rows or 1), dtype=_moe.torch.float32, device=device)


def _vector(n, dtype, device):
    return _moe.torch.empty_strided((n,), (1,), dtype=dtype, device=device)


def _matrix(t, name, device=None, dtypes=None, shape=None):
    ld = _rows_of(t, name, device, dtypes, shape)
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a matrix [rows, columns], got {tuple(t.shape)}")
    return ld


# ------------------------------------------------------------------- route --

@_on_stream
def route_tokens(logits, k: int, score="softmax", bias=None, groups: int = 1, top_groups: int = 1, normalize=True,
                 scale: float = 1.0):
    """(ids int32 [T, k], weights float32 [T, k]): the k experts of each token of
    logits [T, E] (bfloat16, float16, float32; at most 1024 experts) and their
    weights, for sort_tokens and combine_tokens.

    Scores are softmax or sigmoid of the logits.  The choice goes by score +
    ``bias`` (float32 [E]) and, with ``groups`` equal runs of experts, among the
    ``top_groups`` runs whose two best sum highest; equal ones to the lowest
    index.  Weights are scale * score, or normalised to the sum ``scale``.
    Experts whose logit (or score + bias) is -inf or NaN are never chosen; where
    they leave fewer than k, the last ids are -1 with weight 0."""
    torch = _moe.torch
    ld = _matrix(logits, "logits", dtypes=_TYPES)
    dev = logits.device
    T, E = logits.shape
    b = None if bias is None else _plain(bias, "bias", dev, torch.float32, (E,))
    k, kind = int(k), _pick(SCORES, score, "score")
    if not 1 <= k <= 64 or not 1 <= E <= 1024 or groups < 1 or E % groups or not 1 <= top_groups <= groups <= 64 or \
            k > E // groups * top_groups:
        raise ValueError(f"cannot choose {k} of {E} experts in {top_groups} of {groups} groups (at most 64 choices, "
                         "1024 experts, 64 groups)")
    ids, weights = _new((T, k), torch.int32, dev), _new((T, k), torch.float32, dev)
    _run(_load().mxgemm_route_tokens, dev, logits.data_ptr(), ld, _TYPES[logits.dtype], T, E, k, kind, b, groups,
         top_groups, 1 if normalize else 0, scale, ids.data_ptr(), weights.data_ptr())
    return ids, weights


@_on_stream
def route_tokens_backward(d_weights, logits, ids, score="softmax", normalize=True, scale: float = 1.0):
    """Gradient of route_tokens' weights to its logits, in their type; the choice
    (and with it bias and groups) has none."""
    torch = _moe.torch
    ld = _matrix(logits, "logits", dtypes=_TYPES)
    dev = logits.device
    T, E = logits.shape
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids: expected [{T}, choices]")
    k = ids.shape[1]
    if not 1 <= k <= min(64, E) or E > 1024:
        raise ValueError(f"{k} choices of {E} experts (at most 64 of 1024)")
    out = _new((T, E), logits.dtype, dev)
    _run(_load().mxgemm_route_tokens_backward, dev, _plain(d_weights, "d_weights", dev, torch.float32, (T, k)),
         logits.data_ptr(), ld, _TYPES[logits.dtype], T, E, k, _pick(SCORES, score, "score"), 1 if normalize else 0,
         scale, _plain(ids, "ids", dev, torch.int32, (T, k)), out.data_ptr(), E)
    return out


# ---------------------------------------------------------------- quantise --

def _quantize(x, z, act, gated, sort, fmt, rows, cols):
    torch = _moe.torch
    ld_x = _matrix(x, "x", dtypes=_TYPES)
    dev = x.device
    M, held = x.shape
    if gated and z is None and held % 2:
        raise ValueError(f"gated columns come in two halves, not {held}")
    C = held if not gated else held // 2 if z is None else 2 * held
    if C < 1:
        raise ValueError("no columns")
    ld_z = 0 if z is None else _matrix(z, "z", dev, (torch.bfloat16,), (M, C))
    E = off = koff = 0
    Mp, Cp = _up(M, STEP), _up(C, STEP)
    ld_qt = Mp
    if sort is not None:
        off, E, _, T, k = _sort_args(sort, dev)
        koff = _plain(sort[1], "sort.k_offsets", dev, torch.int32, (E + 1,))
        if T * k != M:
            raise ValueError(f"x has {M} rows, the sort {T * k}")
        ld_qt = Mp + E * STEP
    fmt, act = _format(fmt), _activation(act)
    q = s = qt = st = None
    if rows:
        q, s = _new((M, Cp), torch.uint8, dev), _new_scales(M, Cp // STEP, dev)
    if cols:
        qt, st = _new((C, ld_qt), torch.uint8, dev), _new_scales(C, ld_qt // STEP, dev)
    if M == 0 and not (cols and sort is not None):      # nothing to write
        return (q, s), (qt, st)
    # (an empty z has no address, and none stands for the forward form: any other does)
    _run(_load().mxgemm_block_quantize, dev, x.data_ptr(), _TYPES[x.dtype], ld_x,
         None if z is None else z.data_ptr() or koff, ld_z, M, C, act, 1 if gated else 0, off or None, koff or None, E, fmt,
         None if q is None else q.data_ptr(), None if s is None else s.data_ptr(),
         None if qt is None else qt.data_ptr(), None if st is None else st.data_ptr(), ld_qt)
    return (q, s), (qt, st)


@_on_stream
def block_quantize(x, act="none", gated=False, sort: Optional[TokenSort] = None, fmt="e4m3", rows=True, cols=False):
    """FP8 of y = act(x), or, gated, act(x[:, :C]) * x[:, C:], with a float32
    scale for each block of 128: ((q, s), (qt, st)); parts not asked for are
    None.

    q [M, Cp] (uint8 codes, zeros past C) and s [M, Cp / 128] are blocked along
    the columns; qt [C, Mp] and st [C, Mp / 128] hold y^T, blocked along the
    rows.  Cp, Mp: rounded up to 128.  A scale is the block's largest magnitude
    over the format's; blocks with a NaN or an infinity are all NaN, past C too.  The
    scales are stored block by block (``s.t()`` is contiguous), as block_linear
    reads them fastest.  With ``sort`` (x in its row order) dropped rows count
    as zero, codes and scales, and every expert's rows are padded to 128 by
    themselves in qt (TokenSort.k_offsets)."""
    return _quantize(x, None, act, gated, sort, fmt, rows, cols)


@_on_stream
def block_quantize_backward(d_out, z=None, act="none", gated=False, sort: Optional[TokenSort] = None, fmt="e4m3",
                            rows=True, cols=True):
    """As block_quantize, of the gradient dz = d_out act'(z), or, gated, [d_out u
    act'(g), d_out act(g)] with [g, u] = z.  d_out [M, cols]; z bfloat16 [M, N],
    None only without activation."""
    if z is None and (gated or _activation(act)):
        raise ValueError("an activation's gradient needs z")
    plain = not gated and not _activation(act)
    return _quantize(d_out, None if plain else z, act, gated, sort, fmt, rows, cols)


@_on_stream
def block_quantize_weight(w, fmt="e4m3", transposed=False):
    """FP8 of weights w [.., N, K] with a float32 scale for each square of 128 x
    128: (q [.., N, Kp], s [.., Np / 128, Kp / 128]); with ``transposed`` the
    pair of these and of w^T, (qt [.., K, Np], st [.., Kp / 128, Np / 128]), the
    same values in the layout that block_linear_backward takes."""
    torch = _moe.torch
    ld = _rows_of(w, "w", dtypes=_TYPES)
    if w.dim() > 3:
        raise ValueError(f"w: expected [N, K] or [experts, N, K], got {tuple(w.shape)}")
    N, K = w.shape[-2:]
    if N < 1 or K < 1:
        raise ValueError(f"w: expected [N, K] or [experts, N, K], got {tuple(w.shape)}")
    lead, dev = w.shape[:-2], w.device
    group = w.stride(0) if lead else 0
    batch = lead[0] if lead else 1
    Np, Kp = _up(N, STEP), _up(K, STEP)
    q = torch.empty((*lead, N, Kp), dtype=torch.uint8, device=dev)
    s = torch.empty((*lead, Np // STEP, Kp // STEP), dtype=torch.float32, device=dev)
    qt = st = None
    if transposed:
        qt = torch.empty((*lead, K, Np), dtype=torch.uint8, device=dev)
        st = torch.empty((*lead, Kp // STEP, Np // STEP), dtype=torch.float32, device=dev)
    _run(_load().mxgemm_block_quantize_weight, dev, w.data_ptr(), _TYPES[w.dtype], ld, group, batch, N, K,
         _format(fmt), q.data_ptr(), s.data_ptr(), None if qt is None else qt.data_ptr(),
         None if st is None else st.data_ptr())
    return ((q, s), (qt, st)) if transposed else (q, s)


# ----------------------------------------------------------------- product --

def _scales(t, name, device, shape):
    """A float32 tensor of scales -> its last two strides."""
    torch = _moe.torch
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise TypeError(f"{name}: expected a tensor on {device}")
    if t.dtype != torch.float32 or t.shape not in shape:
        raise ValueError(f"{name}: expected float32 {' or '.join(str(s) for s in shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    # a stride that no element is reached by may be anything
    return t.stride(-2) if t.shape[-2] > 1 else 0, t.stride(-1) if t.shape[-1] > 1 else 0


def _linear(a, a_scale, w, w_scale, offsets, mode, out_dtype, precision, a_fmt, w_fmt, tile_cfg):
    torch = _moe.torch
    u8 = (torch.uint8,)
    a, w = _laid_out(a), _laid_out(w)
    lda = _matrix(a, "a", dtypes=u8)
    dev = a.device
    M, K = a.shape
    if K % STEP or K == 0:
        raise ValueError(f"K = {K} must be a positive multiple of {STEP}")
    blocks = K // STEP
    as_row, as_k = _scales(a_scale, "a_scale", dev, [(M, blocks)])
    by_row = mode == GROUP_ROWS
    ldw = _rows_of(w, "w", dev, u8)
    if w.dim() != (3 if by_row else 2) or w.shape[-1] != K or w.shape[-2] < 1:
        raise ValueError(f"w: expected {'[experts, N, K]' if by_row else '[N, K]'} with K = {K}, got {tuple(w.shape)}")
    N, lead = w.shape[-2], w.shape[:-2]
    each, square = (*lead, N, blocks), (*lead, _up(N, STEP) // STEP, blocks)
    ws_row, ws_k = _scales(w_scale, "w_scale", dev, [each] if mode == GROUP_INNER else [square, each])
    squares = mode != GROUP_INNER and w_scale.shape == square
    E = off = 0
    if mode != GROUP_NONE:
        if not isinstance(offsets, torch.Tensor):
            raise TypeError(f"offsets: expected a tensor on {dev}")
        if offsets.dim() != 1:
            raise ValueError(f"offsets: expected [experts + 1], got {tuple(offsets.shape)}")
        E = lead[0] if by_row else offsets.shape[0] - 1
        off = _plain(offsets, "offsets", dev, torch.int32, (E + 1,))
        if E < 1:
            raise ValueError("no experts")
    if out_dtype not in _TYPES:
        raise ValueError(f"out_dtype {out_dtype!r} is not a 16- or 32-bit float type")
    out = torch.empty((E, M, N), dtype=out_dtype, device=dev) if mode == GROUP_INNER else _new((M, N), out_dtype, dev)
    work_ptr = work = 0
    # (few rows of squares are not split: block.cpp's choose_tile)
    if mode == GROUP_NONE and not (squares and M <= 64 and -(-M // 32) * -(-N // 16) <= 256 and tile_cfg < 0):
        work = _split_workspace(M, N, K)
    if work:
        work_mem = _vector(work, torch.uint8, dev)
        work_ptr = work_mem.data_ptr()
    # (the only expert's stride may be anything)
    w_group, ws_group = (w.stride(0), w_scale.stride(0)) if by_row and E > 1 else (0, 0)
    _run(_load().mxgemm_block_linear, dev, BLOCK_ARGS.pack(
        a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), out.data_ptr(), off, M, N, K, lda, as_row,
        as_k, ldw, w_group, ws_row, ws_k, ws_group, N, M * N, 1 if squares else 0, mode, E, _format(a_fmt),
        _format(w_fmt), _pick(_PRECISION, precision, "precision mode"), _TYPES[out_dtype], tile_cfg, work_ptr, work))
    return out


@_on_stream
def block_linear(a, a_scale, w, w_scale, offsets=None, out_dtype=None, precision="exact", a_fmt="e4m3", w_fmt="e4m3",
                 tile_cfg=-1):
    """out = a w^T of FP8 operands with a float32 scale for each block of 128.

    a [M, K], w [N, K]: codes (uint8, K a multiple of 128; transposed views are
    first copied into that layout).  a_scale [M, K / 128]; w_scale [N / 128
    (rounded up), K / 128] (block_quantize_weight) or [N, K / 128]
    (block_quantize), any strides.  With ``offsets`` (TokenSort.offsets) w and
    w_scale have a leading axis of experts, and rows offsets[e] .. offsets[e +
    1] of a meet expert e's; rows of no expert give zeros.  out_dtype: bfloat16
    (default), float16 or float32.  precision: "exact" or "native", as for
    SegGemm; every block's sum is formed by itself and added in FP32."""
    return _linear(a, a_scale, w, w_scale, offsets, GROUP_NONE if offsets is None else GROUP_ROWS,
                   _moe.torch.bfloat16 if out_dtype is None else out_dtype, precision, a_fmt, w_fmt, tile_cfg)


@_on_stream
def block_linear_by_inner(a, a_scale, w, w_scale, offsets, out_dtype=None, precision="exact", a_fmt="e4m3",
                          w_fmt="e4m3", tile_cfg=-1):
    """[E, M, N] products a w^T over the inner ranges offsets[e] ..
    offsets[e + 1] (TokenSort.k_offsets): the weights' gradient by expert.
    a_scale [M, K / 128], w_scale [N, K / 128]."""
    return _linear(a, a_scale, w, w_scale, offsets, GROUP_INNER,
                   _moe.torch.bfloat16 if out_dtype is None else out_dtype, precision, a_fmt, w_fmt, tile_cfg)


@_on_stream
def block_linear_backward(d_out, z, at, at_scale, wt, wt_scale, act="none", gated=False,
                          sort: Optional[TokenSort] = None, fmt="e4m3", a_fmt="e4m3", w_fmt="e4m3", out_dtype=None,
                          precision="exact", tile_cfg=-1):
    """Gradients (d_a, d_w) of z = block_linear(a, w) whose act(z) (gated: act(z[:,
    :N/2]) * z[:, N/2:]) went on.

    dz = d_out act'(z) is held in FP8 of ``fmt``: along N for d_a = dz w, along
    the tokens for d_w = dz^T a (block_quantize_backward).  d_out [M, cols]; z
    bfloat16 [M, N], None only without activation; at [K, Mp] with at_scale [K,
    Mp / 128]: a transposed (block_quantize's qt, st); wt [K, Np] with wt_scale
    [K / 128, Np / 128]: w transposed (block_quantize_weight).  By expert, with
    ``sort``: wt [E, K, Np], d_w [E, N, K], dropped rows of d_a are zero.  Both
    of ``out_dtype`` (default bfloat16)."""
    torch = _moe.torch
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if z is None and (gated or _activation(act)):
        raise ValueError("an activation's gradient needs z")
    by, plain = sort is not None, not gated and not _activation(act)
    (q, s), (qt, st) = _quantize(d_out, None if plain else z, act, gated, sort, fmt, True, True)
    d_a = _linear(q, s, wt, wt_scale, sort[0] if by else None, GROUP_ROWS if by else GROUP_NONE, out_dtype, precision,
                  fmt, w_fmt, tile_cfg)
    if qt.shape[1] == 0:        # no tokens: a product of no inner length
        return d_a, torch.zeros((qt.shape[0], at.shape[0]), dtype=out_dtype, device=qt.device)
    d_w = _linear(qt, st, at, at_scale, sort[1] if by else None, GROUP_INNER if by else GROUP_NONE, out_dtype,
                  precision, fmt, a_fmt, tile_cfg)
    return d_a, d_w


# -------------------------------------------------------------------- norm --

def _weight(t, name, device, H):
    torch = _moe.torch
    if t is None:
        return 0, 0
    if not isinstance(t, torch.Tensor) or t.dtype not in _TYPES:
        raise TypeError(f"{name}: expected a 16- or 32-bit float tensor")
    return _plain(t, name, device, t.dtype, (H,)), _TYPES[t.dtype]


def _gate(gate, T, H, device):
    """(pointer, row stride, rows, type) of a gate [H] or [G, H]."""
    if gate is None:
        return 0, 0, 1, 0
    g = gate
    if isinstance(g, _moe.torch.Tensor) and g.dim() == 1:
        g = g[None]
    ld = _matrix(g, "gate", device, _TYPES)
    G = g.shape[0]
    if g.shape[1] != H or G < 1 or T % G:
        raise ValueError(f"gate: expected [{H}] or [G, {H}] with G a divisor of {T} rows, got {tuple(gate.shape)}")
    return g.data_ptr(), ld, G, _TYPES[g.dtype]


@_on_stream
def add_norm(x, residual=None, gate=None, scale: float = 1.0, post_weight=None, pre_weight=None, kind="rms",
             eps: float = 1e-6):
    """(y, r): the end of one block and the start of the next.

    r = residual + scale * gate * norm(x) post_weight; y = norm(r) pre_weight, of
    r as rounded to its type.  Without post_weight x enters as it is; without
    pre_weight y is None.  x, residual [T, H] of one type (bfloat16, float16,
    float32; H at most 8192); gate [H], or [G, H] with row i for the i-th run of
    T / G rows (each sequence its own; G = T: each token); weights [H]; gate and
    weights may be of any of the types.  kind: "rms" or "layer" (mean taken
    off)."""
    ld_x = _matrix(x, "x", dtypes=_TYPES)
    dev = x.device
    T, H = x.shape
    if not 1 <= H <= MAX_NORM_COLS:
        raise ValueError(f"{H} columns: 1 to {MAX_NORM_COLS} are possible")
    res_ptr = ld_res = 0
    if residual is not None:
        ld_res = _matrix(residual, "residual", dev, (x.dtype,), (T, H))
        res_ptr = residual.data_ptr()
    g_ptr, ld_g, G, g_type = _gate(gate, T, H, dev)
    post, post_type = _weight(post_weight, "post_weight", dev, H)
    pre, pre_type = _weight(pre_weight, "pre_weight", dev, H)
    r = _new((T, H), x.dtype, dev)
    y = None if pre_weight is None else _new((T, H), x.dtype, dev)
    _run(_load().mxgemm_add_norm, dev, NORM_ARGS.pack(
        x.data_ptr(), res_ptr, g_ptr, post, pre, r.data_ptr(), 0 if y is None else y.data_ptr(), 0, 0, 0, 0, 0, 0, 0,
        0, 0, T, H, G, ld_x, ld_res, ld_g, H, H, 0, 0, 0, 0, _TYPES[x.dtype], g_type, post_type, pre_type,
        _pick(NORMS, kind, "norm"), scale, eps, 0))
    return y, r


@_on_stream
def add_norm_backward(d_y, d_r, x, r, gate=None, scale: float = 1.0, post_weight=None, pre_weight=None, kind="rms",
                      eps: float = 1e-6, residual=True) -> NormGrads:
    """Gradients of add_norm from d_y (None without pre_weight, or for zero) and
    d_r (what arrives at r by other ways; None: zero), with x and the r that
    add_norm returned: d_x and d_residual (None unless ``residual``) of x's
    type, d_gate of the gate's type and shape, d_post_weight and d_pre_weight in
    float32."""
    torch = _moe.torch
    ld_x = _matrix(x, "x", dtypes=_TYPES)
    dev = x.device
    T, H = x.shape
    if not 1 <= H <= MAX_NORM_COLS:
        raise ValueError(f"{H} columns: 1 to {MAX_NORM_COLS} are possible")
    one = (x.dtype,)
    ld_r = _matrix(r, "r", dev, one, (T, H))
    if d_y is not None and pre_weight is None:
        raise ValueError("d_y comes with pre_weight")
    ld_dy = 0 if d_y is None else _matrix(d_y, "d_y", dev, one, (T, H))
    ld_dr = 0 if d_r is None else _matrix(d_r, "d_r", dev, one, (T, H))
    g_ptr, ld_g, G, g_type = _gate(gate, T, H, dev)
    post, post_type = _weight(post_weight, "post_weight", dev, H)
    pre, pre_type = _weight(pre_weight, "pre_weight", dev, H)
    d_x = _new((T, H), x.dtype, dev)
    d_res = _new((T, H), x.dtype, dev) if residual else None
    d_gate = None
    if gate is not None:
        d_gate = _vector(H, gate.dtype, dev) if gate.dim() == 1 else _new((G, H), gate.dtype, dev)
    d_post = _vector(H, torch.float32, dev) if post else None
    d_pre = _vector(H, torch.float32, dev) if pre else None
    lib = _load()
    size = lib.mxgemm_add_norm_workspace(T, H, G)
    work = _vector(size, torch.uint8, dev)
    ptr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    _run(lib.mxgemm_add_norm_backward, dev, NORM_ARGS.pack(
        x.data_ptr(), 0, g_ptr, post, pre, r.data_ptr(), 0, ptr(d_y), ptr(d_r), d_x.data_ptr(), ptr(d_res),
        ptr(d_gate), ptr(d_post), ptr(d_pre), work.data_ptr(), size, T, H, G, ld_x, 0, ld_g, ld_r, 0,
        ld_dy, ld_dr, H, H, _TYPES[x.dtype], g_type, post_type, pre_type, _pick(NORMS, kind, "norm"), scale, eps, 0))
    return NormGrads(d_x, d_res, d_gate, d_post, d_pre)
