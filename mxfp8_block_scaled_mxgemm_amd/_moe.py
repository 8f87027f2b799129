"""Binding of the expert layer (declared in ``include/mxgemm_moe.h``): tokens
sorted by expert and back, and the MXFP8 product with its fused epilogue,
dense and by expert, each with its gradient.

Argument checks and marshalling only; every computation runs in the HIP
library.  Outputs are allocated from torch's caching allocator on the stream
the call runs on (the current one unless ``stream`` is given); with another
stream, the inputs are recorded on it.  Nothing synchronises.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional

from . import _lib
from ._lib import FMT_E4M3, FMT_E5M2, PRECISION_EXACT, PRECISION_NATIVE, check

EXPORTED_MOE = [
    "mxgemm_sort_tokens", "mxgemm_sort_tokens_workspace", "mxgemm_dispatch_tokens",
    "mxgemm_dispatch_tokens_mx", "mxgemm_combine_tokens", "mxgemm_combine_tokens_backward",
    "mxgemm_linear", "mxgemm_linear_workspace", "mxgemm_epilogue_backward", "mxgemm_transpose_bytes",
]

GROUP_NONE, GROUP_ROWS, GROUP_INNER = 0, 1, 2
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
TYPE_MXE4M3, TYPE_MXE5M2 = 3, 4
_MX_OUT = {"e4m3": TYPE_MXE4M3, "e5m2": TYPE_MXE5M2}
_FMT = {"e4m3": FMT_E4M3, "e5m2": FMT_E5M2, FMT_E4M3: FMT_E4M3, FMT_E5M2: FMT_E5M2}
_PRECISION = {"exact": PRECISION_EXACT, "native": PRECISION_NATIVE, PRECISION_EXACT: PRECISION_EXACT,
              PRECISION_NATIVE: PRECISION_NATIVE}
STEP = 128          # granule of a product's inner length and of k_offsets


# mxgemm_linear_t: ten pointers, fourteen int64, ten int32, the workspace, in
# the header's order
LINEAR_ARGS = struct.Struct("10P14q10iPq")


class TokenSort(NamedTuple):
    """The (token, choice) pairs of ids [T, k] in stable order by expert.

    offsets [E + 1]: expert e holds rows offsets[e] .. offsets[e + 1]; rows
    from offsets[E] on are dropped pairs.  k_offsets [E + 1]: the same with
    every expert's count rounded up to 128.  row_of [T, k]: row of each pair.
    pair_of [T k]: pair (t k + j) of each row.  All int32."""
    offsets: "torch.Tensor"
    k_offsets: "torch.Tensor"
    row_of: "torch.Tensor"
    pair_of: "torch.Tensor"


class LinearGrads(NamedTuple):
    d_a: "torch.Tensor"
    d_w: "torch.Tensor"
    d_bias: Optional["torch.Tensor"]


_bound = None


def _load():
    """The library with the expert layer's argument types set."""
    global _bound
    if _bound is None:
        lib = _lib.load()
        i64, i32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
        lib.mxgemm_sort_tokens.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp, vp, vp, i64, vp]
        lib.mxgemm_sort_tokens_workspace.argtypes = [i64, i32, i32]
        lib.mxgemm_dispatch_tokens.argtypes = [vp, i64, i32, i64, i32, i64, vp, i32, vp, vp, i64, vp]
        lib.mxgemm_dispatch_tokens_mx.argtypes = [vp, i64, i32, i64, i32, i64, vp, i32, vp, vp, vp, i32, vp]
        lib.mxgemm_combine_tokens.argtypes = [vp, i64, i32, i64, i32, i64, vp, i32, vp, vp, vp, i64, vp, i64, vp]
        lib.mxgemm_combine_tokens_backward.argtypes = [vp, i64, vp, i64, i32, i64, i32, i64, vp, i32, vp, vp, vp,
                                                       i64, vp, vp]
        lib.mxgemm_linear.argtypes = [ctypes.c_char_p, vp]
        lib.mxgemm_epilogue_backward.argtypes = [vp, i32, i64, vp, i64, i64, i64, i32, i32, vp, vp, i32, i32, vp,
                                                 vp, vp, vp, i64, vp, vp, i64, vp]
        lib.mxgemm_transpose_bytes.argtypes = [vp, i64, i64, i64, i64, i64, vp, vp]
        for name in EXPORTED_MOE:
            getattr(lib, name).restype = ctypes.c_int
        lib.mxgemm_linear_workspace.argtypes = [i64, i64, i64]
        lib.mxgemm_sort_tokens_workspace.restype = lib.mxgemm_linear_workspace.restype = i64
        _bound = lib
    return _bound


torch = None        # bound by the first call: the package loads without it
_TYPES = {}


def _bind():
    """Fills the table of types, then binds torch: a thread that finds it bound
    finds the table filled."""
    global torch
    import torch as module
    _TYPES.update({module.bfloat16: 0, module.float16: 1, module.float32: 2})
    torch = module


def _on_stream(fn):
    """Runs ``fn`` with its ``stream`` as torch's current one, so that what it
    allocates belongs to that stream, and records its inputs there."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if torch is None:
            _bind()
        if stream is None:
            return fn(*args, **kw)
        if stream == torch.cuda.current_stream(stream.device):
            with torch.cuda.device(stream.device):
                return fn(*args, **kw)
        with torch.cuda.stream(stream):
            out = fn(*args, **kw)
        for x in (*args, *kw.values()):
            for t in x if isinstance(x, tuple) else (x,):
                if isinstance(t, torch.Tensor) and t.is_cuda:
                    t.record_stream(stream)
        return out
    return call


def _run(fn, device, *args):
    """fn(*args, stream) on ``device`` and its current stream."""
    i = device.index
    if i == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(i):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    if rc:
        check(rc)


def _rows_of(t, name, device=None, dtypes=None, shape=None):
    """A device matrix with contiguous rows -> its row stride."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name}: {t.dtype} is not one of {', '.join(map(str, dtypes))}")
    have = t.shape
    if len(have) < 2 or (shape is not None and have != shape):
        raise ValueError(f"{name}: expected shape {shape if shape is not None else '[rows, columns]'}, "
                         f"got {tuple(have)}")
    stride = t.stride()
    if stride[-1] != 1 and have[-1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    # a stride that no element is reached by may be anything
    return stride[-2] if have[-2] > 1 else have[-1]


def _plain(t, name, device, dtype, shape):
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise TypeError(f"{name}: expected a tensor on {device}")
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _format(fmt):
    try:
        return _FMT[fmt.lower() if isinstance(fmt, str) else fmt]
    except (KeyError, TypeError):
        raise ValueError(f"unknown FP8 format {fmt!r}") from None


def _activation(act):
    try:
        return ACTIVATIONS[act or "none"]
    except (KeyError, TypeError):
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTIVATIONS)}") from None


def _up(n, m):
    return -(-n // m) * m


# ------------------------------------------------------------------ tokens --

@_on_stream
def sort_tokens(expert_ids, num_experts: int) -> TokenSort:
    """Stable order by expert of the pairs of ``expert_ids`` [T, k] (int32 or
    int64); an id outside [0, num_experts) drops its pair."""
    ids = expert_ids
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda:
        raise TypeError("expert_ids: expected a device tensor")
    if ids.dtype not in (torch.int32, torch.int64) or ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("expert_ids must be a contiguous int32 or int64 [tokens, choices] tensor")
    T, k = ids.shape
    lib = _load()
    E1 = int(num_experts) + 1
    if not 1 <= E1 - 1 <= 1024 or k < 1:
        raise ValueError(f"1 to 1024 experts and at least one choice are needed, not {num_experts} and {k}")
    if T * k >= (1 << 31) - (1 << 20):
        raise ValueError(f"{T} x {k} pairs exceed 2^31 - 2^20")
    n = T * k
    work = lib.mxgemm_sort_tokens_workspace(T, k, E1 - 1)
    # one allocation: the four arrays, each from a 16-byte boundary, and the workspace
    e4, n4 = _up(E1, 4), _up(n, 4)
    mem = torch.empty(2 * e4 + 2 * n4 + work // 4, dtype=torch.int32, device=ids.device)
    offsets, _, k_offsets, _, row_of, _, pair_of, _ = mem.split_with_sizes(
        (E1, e4 - E1, E1, e4 - E1, n, n4 - n, n, n4 - n + work // 4))
    p = mem.data_ptr()
    _run(lib.mxgemm_sort_tokens, ids.device, ids.data_ptr(), ids.element_size(), T, k, E1 - 1, p, p + 4 * e4,
         p + 8 * e4, p + 8 * e4 + 4 * n4, p + 8 * e4 + 8 * n4, work)
    return TokenSort(offsets, k_offsets, row_of.view(T, k), pair_of)


def _sort_args(sort, device, T=None):
    """(offsets pointer, experts, row_of pointer, T, k) of a TokenSort."""
    offsets, _, row_of, _ = sort
    if row_of.dim() != 2 or offsets.dim() != 1 or (T is not None and row_of.shape[0] != T):
        raise ValueError(f"sort: row_of {tuple(row_of.shape)} is not [tokens{'' if T is None else f' = {T}'}, choices]")
    T, k = row_of.shape
    E = offsets.shape[0] - 1
    return (_plain(offsets, "sort.offsets", device, torch.int32, (E + 1,)), E,
            _plain(row_of, "sort.row_of", device, torch.int32, (T, k)), T, k)


@_on_stream
def dispatch_tokens(x, sort: TokenSort):
    """Rows [T k, H] of the sorted order from tokens x [T, H] (bfloat16,
    float16 or float32); rows of dropped pairs are zero."""
    ld = _rows_of(x, "x", dtypes=_TYPES)
    T, H = x.shape
    off, E, row_of, T, k = _sort_args(sort, x.device, T)
    rows = torch.empty((T * k, H), dtype=x.dtype, device=x.device)
    _run(_load().mxgemm_dispatch_tokens, x.device, x.data_ptr(), ld, _TYPES[x.dtype], T, k, H, off, E, row_of,
         rows.data_ptr(), H)
    return rows


@_on_stream
def dispatch_tokens_mx(x, sort: TokenSort, fmt="e4m3"):
    """As dispatch_tokens, quantised to MXFP8: (codes [T k, H], scales [T k,
    H / 32]), both uint8; H a multiple of 32."""
    ld = _rows_of(x, "x", dtypes=_TYPES)
    T, H = x.shape
    if H % 32:
        raise ValueError(f"{H} columns are not a multiple of the MX block 32")
    off, E, row_of, T, k = _sort_args(sort, x.device, T)
    q = torch.empty((T * k, H), dtype=torch.uint8, device=x.device)
    s = torch.empty((T * k, H // 32), dtype=torch.uint8, device=x.device)
    _run(_load().mxgemm_dispatch_tokens_mx, x.device, x.data_ptr(), ld, _TYPES[x.dtype], T, k, H, off, E, row_of,
         q.data_ptr(), s.data_ptr(), _format(fmt))
    return q, s


@_on_stream
def combine_tokens(rows, sort: TokenSort, weights=None, residual=None):
    """Tokens back from their rows: residual[t] + sum_j weights[t, j]
    rows[row_of[t, j]] over the kept pairs, in FP32, rounded once.  rows [T k,
    H]; weights float32 [T, k] (default ones); residual [T, H] of rows' type."""
    ld = _rows_of(rows, "rows", dtypes=_TYPES)
    off, E, row_of, T, k = _sort_args(sort, rows.device)
    n, H = rows.shape
    if n != T * k:
        raise ValueError(f"rows has {n} rows, the sort {T * k}")
    w = None if weights is None else _plain(weights, "weights", rows.device, torch.float32, (T, k))
    ld_res = 0 if residual is None else _rows_of(residual, "residual", rows.device, (rows.dtype,), (T, H))
    out = torch.empty((T, H), dtype=rows.dtype, device=rows.device)
    _run(_load().mxgemm_combine_tokens, rows.device, rows.data_ptr(), ld, _TYPES[rows.dtype], T, k, H, off, E,
         row_of, w, None if residual is None else residual.data_ptr(), ld_res, out.data_ptr(), H)
    return out


def dispatch_tokens_backward(d_rows, sort: TokenSort, stream=None):
    """Gradient of dispatch_tokens: the sum of each token's kept rows."""
    return combine_tokens(d_rows, sort, stream=stream)


@_on_stream
def combine_tokens_backward(d_out, rows, sort: TokenSort, weights=None):
    """Gradients of combine_tokens to its rows ([T k, H] of rows' type) and
    weights (float32 [T, k]); the residual's is d_out itself."""
    ld = _rows_of(rows, "rows", dtypes=_TYPES)
    off, E, row_of, T, k = _sort_args(sort, rows.device)
    n, H = rows.shape
    if n != T * k:
        raise ValueError(f"rows has {n} rows, the sort {T * k}")
    ld_d = _rows_of(d_out, "d_out", rows.device, (rows.dtype,), (T, H))
    w = None if weights is None else _plain(weights, "weights", rows.device, torch.float32, (T, k))
    d_rows = torch.empty((n, H), dtype=rows.dtype, device=rows.device)
    d_w = torch.empty((T, k), dtype=torch.float32, device=rows.device)
    _run(_load().mxgemm_combine_tokens_backward, rows.device, d_out.data_ptr(), ld_d, rows.data_ptr(), ld,
         _TYPES[rows.dtype], T, k, H, off, E, row_of, w, d_rows.data_ptr(), H, d_w.data_ptr())
    return d_rows, d_w


# ----------------------------------------------------------------- product --

def _laid_out(t):
    """``t``, or where its other axis is the contiguous one (a transposed view)
    a copy with contiguous rows; [.., N, K] bytes."""
    if torch is None:
        _bind()
    stride = t.stride() if isinstance(t, torch.Tensor) else ()
    if not 2 <= len(stride) <= 3 or stride[-1] == 1 or t.dtype != torch.uint8 or not t.is_cuda:
        return t            # as it should be, or refused by the checks that follow
    shape = t.shape
    if shape[-1] <= 1 or stride[-2] != 1 or stride[-1] < shape[-2]:
        return t
    out = torch.empty(shape, dtype=torch.uint8, device=t.device)
    _run(_load().mxgemm_transpose_bytes, t.device, t.data_ptr(), stride[-1], stride[0] if len(shape) == 3 else 0,
         shape[-1], shape[-2], shape[0] if len(shape) == 3 else 1, out.data_ptr())
    return out


def _split_workspace(M, N, K):
    """mxgemm_linear_workspace's rule, without a call into the library."""
    return 4 << 20 if M > 32 and K >= 2048 and -(-M // 64) * -(-N // 64) <= 128 else 0


def _linear(a, a_scale, w, w_scale, bias, act, gated, residual, offsets, mode, out_dtype, preact, precision, a_fmt,
            w_fmt, tile_cfg):
    u8 = (torch.uint8,)
    a, a_scale, w, w_scale = _laid_out(a), _laid_out(a_scale), _laid_out(w), _laid_out(w_scale)
    lda = _rows_of(a, "a", dtypes=u8)
    dev = a.device
    if a.dim() != 2:
        raise ValueError(f"a: expected [rows, K], got {tuple(a.shape)}")
    M, K = a.shape
    if K % STEP:
        raise ValueError(f"K = {K} must be a multiple of {STEP}")
    lda_s = _rows_of(a_scale, "a_scale", dev, u8, (M, K // 32))
    by_row = mode == GROUP_ROWS
    ldw = _rows_of(w, "w", dev, u8)
    if w.dim() != (3 if by_row else 2) or w.shape[-1] != K:
        raise ValueError(f"w: expected {'[experts, N, K]' if by_row else '[N, K]'} with K = {K}, got {tuple(w.shape)}")
    N = w.shape[-2]
    ldw_s = _rows_of(w_scale, "w_scale", dev, u8, (*w.shape[:-1], K // 32))
    E = off = 0
    if mode != GROUP_NONE:
        E = w.shape[0] if by_row else offsets.shape[0] - 1
        off = _plain(offsets, "offsets", dev, torch.int32, (E + 1,))
    if gated and N % 2:
        raise ValueError(f"a gated product needs an even N, not {N}")
    cols = N // 2 if gated else N
    mx = isinstance(out_dtype, str)
    if mx and out_dtype not in _MX_OUT or not mx and out_dtype not in _TYPES:
        raise ValueError(f"out_dtype {out_dtype!r} is not a 16- or 32-bit float type, 'e4m3' or 'e5m2'")
    if mx and cols % 32:
        raise ValueError(f"MXFP8 output needs columns in blocks of 32, not {cols}")
    if precision not in _PRECISION:
        raise ValueError(f"unknown precision mode {precision!r}")
    bias_ptr = res_ptr = scale_ptr = z_ptr = ld_res = bias_type = 0
    if bias is not None:
        if bias.dtype not in _TYPES:
            raise TypeError(f"bias: {bias.dtype} is not a 16- or 32-bit float type")
        bias_ptr = _plain(bias, "bias", dev, bias.dtype, (E, N) if by_row else (N,))
        bias_type = _TYPES[bias.dtype]
    if residual is not None:
        ld_res = _rows_of(residual, "residual", dev, (torch.bfloat16 if mx else out_dtype,), (M, cols))
        res_ptr = residual.data_ptr()
    out = torch.empty((E, M, cols) if mode == GROUP_INNER else (M, cols), dtype=torch.uint8 if mx else out_dtype,
                      device=dev)
    result = [out]
    if mx:
        scale = torch.empty((M, cols // 32), dtype=torch.uint8, device=dev)
        scale_ptr = scale.data_ptr()
        result.append(scale)
    if preact:
        z = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        z_ptr = z.data_ptr()
        result.append(z)
    work_ptr = 0
    work = _split_workspace(M, N, K) if mode == GROUP_NONE else 0
    if work:
        work_mem = torch.empty(work, dtype=torch.uint8, device=dev)
        work_ptr = work_mem.data_ptr()
    # (the only expert's stride may be anything)
    w_group, w_scale_group = (w.stride(0), w_scale.stride(0)) if by_row and E > 1 else (0, 0)
    _run(_load().mxgemm_linear, dev, LINEAR_ARGS.pack(
        a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), bias_ptr, res_ptr, out.data_ptr(),
        scale_ptr, z_ptr, off, M, N, K, lda, lda_s, ldw, ldw_s, w_group, w_scale_group, ld_res, cols, M * cols,
        cols // 32, N, mode, E, _format(a_fmt), _format(w_fmt), _PRECISION[precision], bias_type, _activation(act),
        1 if gated else 0, _MX_OUT[out_dtype] if mx else _TYPES[out_dtype], tile_cfg, work_ptr, work))
    return result[0] if len(result) == 1 else tuple(result)


@_on_stream
def linear(a, a_scale, w, w_scale, bias=None, act="none", gated=False, residual=None, offsets=None, out_dtype=None,
           preact=False, precision="exact", a_fmt="e4m3", w_fmt="e4m3", tile_cfg=-1):
    """out = act(z) + residual with z = a w^T + bias; gated: act(z[:, :N/2]) *
    z[:, N/2:] + residual.

    a [M, K], w [N, K]: MXFP8 codes (uint8, K a multiple of 128) with scales
    [.., K / 32]; transposed views (K strided, the other axis contiguous) are
    first copied into that layout.  With ``offsets`` (TokenSort.offsets) w is [E, N, K], bias
    [E, N], and rows offsets[e] .. offsets[e + 1] of a meet expert e's; rows
    of no expert give zeros.  act: none, relu, gelu, gelu_tanh, silu.
    out_dtype: bfloat16 (default), float16, float32, or "e4m3" / "e5m2" for
    MXFP8 codes and scales, ready for the next product.  precision: "exact" or
    "native", as for SegGemm.  Returns out, or a tuple of out, its scales
    (MXFP8) and z in bfloat16 (``preact``, for linear_backward)."""
    return _linear(a, a_scale, w, w_scale, bias, act, gated, residual, offsets,
                   GROUP_NONE if offsets is None else GROUP_ROWS, torch.bfloat16 if out_dtype is None else out_dtype,
                   preact, precision, a_fmt, w_fmt, tile_cfg)


@_on_stream
def linear_by_inner(a, a_scale, w, w_scale, offsets, out_dtype=None, precision="exact", a_fmt="e4m3", w_fmt="e4m3",
                    tile_cfg=-1):
    """[E, M, N] products a w^T over the inner ranges offsets[e] ..
    offsets[e + 1] (TokenSort.k_offsets): the weights' gradient by expert."""
    return _linear(a, a_scale, w, w_scale, None, "none", False, None, offsets, GROUP_INNER,
                   torch.bfloat16 if out_dtype is None else out_dtype, False, precision, a_fmt, w_fmt, tile_cfg)


def _epilogue_backward(d_out, z, act, gated, sort, fmt, rows, cols, bias):
    """(q, s), (qt, st), d_bias of mxgemm_epilogue_backward; None where not
    asked for."""
    dev = d_out.device
    ld_d = _rows_of(d_out, "d_out", dtypes=_TYPES)
    if d_out.dim() != 2:
        raise ValueError(f"expected a matrix [rows, columns], got {tuple(d_out.shape)}")
    M = d_out.shape[0]
    N = d_out.shape[1] * (2 if gated else 1)
    if z is None and (gated or _activation(act)):
        raise ValueError("an activation's gradient needs z")
    ld_z = 0 if z is None else _rows_of(z, "z", dev, (torch.bfloat16,), (M, N))
    E = off = koff = 0
    ld_qt = _up(M, STEP)
    if sort is not None:
        off, E, _, T, k = _sort_args(sort, dev)
        koff = _plain(sort[1], "sort.k_offsets", dev, torch.int32, (E + 1,))
        if T * k != M:
            raise ValueError(f"d_out has {M} rows, the sort {T * k}")
        ld_qt = (ld_qt // STEP + E) * STEP
    u8 = dict(dtype=torch.uint8, device=dev)
    Np = _up(N, STEP)
    q = s = qt = st = db = work = None
    if rows:
        q, s = torch.empty((M, Np), **u8), torch.empty((M, Np // 32), **u8)
    if cols:
        qt, st = torch.empty((N, ld_qt), **u8), torch.empty((N, ld_qt // 32), **u8)
    if bias:
        db = torch.empty((E, N) if E else (N,), dtype=torch.float32, device=dev)
        work = torch.empty((ld_qt // STEP, N), dtype=torch.float32, device=dev)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _run(_load().mxgemm_epilogue_backward, dev, d_out.data_ptr(), _TYPES[d_out.dtype], ld_d, ptr(z), ld_z, M, N,
         _activation(act), 1 if gated else 0, off or None, koff or None, E, _format(fmt), ptr(q), ptr(s), ptr(qt),
         ptr(st), ld_qt, ptr(db), ptr(work), 0 if work is None else work.numel() * 4)
    return (q, s), (qt, st), db


@_on_stream
def epilogue_backward(d_out, z=None, act="none", gated=False, sort=None, fmt="e4m3", rows=True, cols=True, bias=True):
    """dz = d_out act'(z) (gated: both halves) in MXFP8 both ways: ((q, s)
    along the columns [M, Np], (qt, st) transposed along the tokens [N, ..],
    d_bias float32); parts not asked for are None.  Np is N rounded up to 128.
    With ``sort`` the tokens of expert e take columns k_offsets[e] ..
    k_offsets[e + 1] of qt, and d_bias is [E, N]; rows of dropped pairs and
    columns past the last segment are zero."""
    return _epilogue_backward(d_out, z, act, gated, sort, fmt, rows, cols, bias)


@_on_stream
def quantize_transposed(x, sort=None, fmt="e4m3"):
    """MXFP8 codes and scales of x^T along x's rows: x [M, C] (bfloat16,
    float16, float32) -> [C, M rounded up to 128] and [C, ../32], zeros past
    M.  This is the layout of at and wt in linear_backward; with ``sort`` (x
    in its row order) every expert's rows are padded to 128 by themselves."""
    _, (qt, st), _ = _epilogue_backward(x, None, "none", False, sort, fmt, False, True, False)
    return qt, st


@_on_stream
def linear_backward(d_out, z, at, at_scale, wt, wt_scale, act="none", gated=False, sort=None, bias=True, fmt="e4m3",
                    a_fmt="e4m3", w_fmt="e4m3", out_dtype=None, precision="exact", tile_cfg=-1) -> LinearGrads:
    """Gradient of linear to a, w and bias (the residual's is d_out itself).

    dz = d_out act'(z) is held in MXFP8 of ``fmt``: along N for d_a = dz w,
    along the tokens for d_w = dz^T a.  d_out [M, cols]; z: linear's preact
    output (None only without activation); at [K, Mp], wt [K, Np]: a and w
    transposed (quantize_transposed), Mp and Np rounded up to 128.  By expert,
    with ``sort``: wt [E, K, Np], at in the padded layout of
    quantize_transposed(.., sort); d_w is [E, N, K], d_bias [E, N], and
    dropped rows of d_a are zero.  d_a and d_w are of ``out_dtype`` (default
    bfloat16), d_bias float32."""
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if isinstance(out_dtype, str):
        raise ValueError("gradients are not written in MXFP8")
    by = sort is not None
    (q, s), (qt, st), db = _epilogue_backward(d_out, z, act, gated, sort, fmt, True, True, bias)
    d_a = _linear(q, s, wt, wt_scale, None, "none", False, None, sort[0] if by else None,
                  GROUP_ROWS if by else GROUP_NONE, out_dtype, False, precision, fmt, w_fmt, tile_cfg)
    if not by and d_out.shape[0] == 0:      # no tokens: a product of no inner length
        return LinearGrads(d_a, torch.zeros((qt.shape[0], at.shape[0]), dtype=out_dtype, device=qt.device), db)
    d_w = _linear(qt, st, at, at_scale, None, "none", False, None, sort[1] if by else None,
                  GROUP_INNER if by else GROUP_NONE, out_dtype, False, precision, fmt, a_fmt, tile_cfg)
    return LinearGrads(d_a, d_w, db)
