"""CPU-only checks of the expert layer's C ABI: exports, the layout of the
argument struct, argument rules that need no GPU."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

import mxfp8_block_scaled_mxgemm_amd as pkg
from mxfp8_block_scaled_mxgemm_amd import _lib, _moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxgemm_moe.h")


def _declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(mxgemm_\w+)\s*\(", text)))


def test_library_exports_every_declared_symbol():
    lib = _moe._load()
    assert sorted(pkg.EXPORTED_MOE) == _declared()
    assert all(hasattr(lib, name) for name in _declared())


def test_header_is_c_and_the_struct_is_the_bindings(tmp_path):
    """The header compiles as C, and the packed argument block has the
    struct's size and field order."""
    src = tmp_path / "layout.c"
    text = open(HEADER).read()
    body = text[text.index("typedef struct mxgemm_linear {"):text.index("} mxgemm_linear_t;")]
    fields = re.findall(r"[\w*]+\s+\*?\s*([\w, ]+);", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
    names = [n.strip() for group in fields for n in group.split(",")]
    lines = "".join(f'printf("{n} %zu\\n", offsetof(mxgemm_linear_t, {n}));' for n in names)
    src.write_text('#include "mxgemm_moe.h"\n#include <stddef.h>\n#include <stdio.h>\n'
                   f'int main(void) {{ printf("size %zu\\n", sizeof(mxgemm_linear_t)); {lines} return 0; }}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], check=True, capture_output=True,
                                                       text=True).stdout.splitlines())
    assert int(got.pop("size")) == _moe.LINEAR_ARGS.size
    sizes = [8] * 24 + [4] * 10 + [8] * 2
    at = 0
    for name, size in zip(names, sizes):
        assert int(got[name]) == at, name
        at += size
    assert len(names) == len(sizes)


def test_sort_workspace():
    ws = _moe._load().mxgemm_sort_tokens_workspace
    assert ws(0, 1, 1) == 0 and ws(512, 8, 256) == 0            # one work-group
    assert ws(513, 8, 256) > 0 and ws(1 << 20, 8, 256) <= 128 * 257 * 4
    assert ws(1, 1, 1025) == 0 and ws(1 << 31, 1, 4) == 0 and ws(-1, 1, 4) == 0


def test_linear_workspace():
    ws = _moe._load().mxgemm_linear_workspace
    assert ws(64, 2048, 7168) == 256 * 64 * 64 * 4
    assert ws(32, 2048, 7168) == 0 and ws(64, 2048, 1024) == 0 and ws(8192, 8192, 8192) == 0 and ws(0, 64, 4096) == 0


def _args(**kw):
    names = ("a a_scale w w_scale bias residual out out_scale z offsets rows N K lda ld_a_scale ldw ld_w_scale w_group "
             "w_scale_group ld_residual ld_out out_group ld_out_scale ld_z mode experts a_format w_format precision "
             "bias_type act gated out_type tile_cfg workspace workspace_bytes").split()
    v = dict.fromkeys(names, 0)
    v.update(rows=4, N=64, K=256, lda=256, ld_a_scale=8, ldw=256, ld_w_scale=8, ld_out=64, tile_cfg=-1)
    v.update(kw)
    return _moe.LINEAR_ARGS.pack(*(v[n] for n in names))


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), _lib.MXGEMM_EINVAL), (dict(N=0), _lib.MXGEMM_EINVAL), (dict(K=48), _lib.MXGEMM_EINVAL),
    (dict(K=96, lda=96, ldw=96), _lib.MXGEMM_EUNSUPPORTED), (dict(mode=3), _lib.MXGEMM_EINVAL),
    (dict(mode=1), _lib.MXGEMM_EINVAL), (dict(act=5), _lib.MXGEMM_EINVAL), (dict(out_type=5), _lib.MXGEMM_EINVAL),
    (dict(bias=16, bias_type=3), _lib.MXGEMM_EINVAL), (dict(a_format=2), _lib.MXGEMM_EINVAL),
    (dict(precision=2), _lib.MXGEMM_EINVAL), (dict(gated=1, N=63), _lib.MXGEMM_EINVAL),
    (dict(out_type=3, N=40, ld_out=40), _lib.MXGEMM_EINVAL), (dict(out_type=3, ld_out_scale=1), _lib.MXGEMM_EINVAL),
    (dict(lda=128), _lib.MXGEMM_EINVAL), (dict(lda=264), _lib.MXGEMM_EINVAL), (dict(ld_a_scale=10), _lib.MXGEMM_EINVAL),
    (dict(ld_out=63), _lib.MXGEMM_EINVAL), (dict(residual=16, ld_residual=1), _lib.MXGEMM_EINVAL),
    (dict(z=16, ld_z=1), _lib.MXGEMM_EINVAL), (dict(tile_cfg=5), _lib.MXGEMM_EINVAL),
    (dict(tile_cfg=0, precision=0), _lib.MXGEMM_EINVAL), (dict(rows=1 << 31), _lib.MXGEMM_EUNSUPPORTED),
    (dict(lda=1 << 24), _lib.MXGEMM_EUNSUPPORTED),
    (dict(mode=2, experts=2, offsets=16, act=1), _lib.MXGEMM_EINVAL),
    (dict(gated=1, N=1 << 25, ldw=256, ld_out=1 << 24), _lib.MXGEMM_EUNSUPPORTED),
    (dict(gated=1, N=1 << 21, ld_w_scale=1 << 22, ld_out=1 << 20), _lib.MXGEMM_EUNSUPPORTED),
])
def test_linear_refuses_before_touching_a_gpu(kw, code):
    lib = _moe._load()
    assert lib.mxgemm_linear(_args(**kw), None) == code
    assert pkg.last_error()


def test_linear_without_rows_is_nothing():
    assert _moe._load().mxgemm_linear(_args(rows=0), None) == 0
    assert _moe._load().mxgemm_linear(None, None) == _lib.MXGEMM_EINVAL


@pytest.mark.parametrize("args,code", [
    ((-1, 1, 4), _lib.MXGEMM_EINVAL), ((4, 0, 4), _lib.MXGEMM_EINVAL), ((4, 1, 0), _lib.MXGEMM_EINVAL),
    ((4, 1, 1025), _lib.MXGEMM_EUNSUPPORTED), ((1 << 31, 1, 4), _lib.MXGEMM_EUNSUPPORTED),
])
def test_token_rules(args, code):
    lib = _moe._load()
    T, k, E = args
    p = ctypes.c_void_p(16)
    assert lib.mxgemm_sort_tokens(p, 4, T, k, E, p, p, p, p, None, 0, None) == code
    assert lib.mxgemm_dispatch_tokens(p, 8, 0, T, k, 8, p, E, p, p, 8, None) == code
    assert lib.mxgemm_combine_tokens(p, 8, 0, T, k, 8, p, E, p, None, None, 0, p, 8, None) == code
    assert lib.mxgemm_combine_tokens_backward(p, 8, p, 8, 0, T, k, 8, p, E, p, None, p, 8, p, None) == code


def test_more_token_rules():
    lib = _moe._load()
    p = ctypes.c_void_p(16)
    E = _lib.MXGEMM_EINVAL
    assert lib.mxgemm_sort_tokens(p, 2, 4, 1, 4, p, p, p, p, None, 0, None) == E        # id_bytes
    assert lib.mxgemm_dispatch_tokens(p, 8, 3, 4, 1, 8, p, 4, p, p, 8, None) == E       # type
    assert lib.mxgemm_dispatch_tokens(p, 7, 0, 4, 1, 8, p, 4, p, p, 8, None) == E       # stride
    assert lib.mxgemm_dispatch_tokens(p, 8, 0, 4, 1, 0, p, 4, p, p, 8, None) == E       # no columns
    assert lib.mxgemm_dispatch_tokens_mx(p, 48, 0, 4, 1, 48, p, 4, p, p, p, 0, None) == E
    assert lib.mxgemm_dispatch_tokens_mx(p, 64, 0, 4, 1, 64, p, 4, p, p, p, 2, None) == E
    assert lib.mxgemm_dispatch_tokens(p, 8, 0, 0, 1, 8, p, 4, p, p, 8, None) == 0       # no tokens
    # epilogue_backward: z needed, codes with scales, ld_qt, workspace
    eb = lib.mxgemm_epilogue_backward
    assert eb(p, 0, 64, None, 0, 4, 64, 4, 0, None, None, 0, 0, p, p, p, p, 128, None, None, 0, None) == E
    assert eb(p, 0, 64, None, 0, 4, 64, 0, 0, None, None, 0, 0, p, None, p, p, 128, None, None, 0, None) == E
    assert eb(p, 0, 64, None, 0, 4, 64, 0, 0, None, None, 0, 0, p, p, p, p, 256, None, None, 0, None) == E
    assert eb(p, 0, 64, None, 0, 4, 64, 0, 0, None, None, 2, 0, p, p, p, p, 128, None, None, 0, None) == E
    assert eb(p, 0, 64, None, 0, 4, 64, 0, 0, None, None, 0, 0, p, p, p, p, 128, p, p, 8, None) == E
    assert lib.mxgemm_transpose_bytes(p, 3, 0, 4, 4, 1, p, None) == E
    assert lib.mxgemm_transpose_bytes(p, 4, 0, 0, 4, 1, p, None) == 0


def test_binding_refuses_host_tensors_without_a_gpu():
    torch = pytest.importorskip("torch")
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        pkg.sort_tokens(ids, 4)
    with pytest.raises(TypeError):
        pkg.dispatch_tokens(torch.zeros(4, 8), (ids, ids, ids, ids))
    u8 = torch.zeros(4, 128, dtype=torch.uint8)
    with pytest.raises(TypeError):
        pkg.linear(u8, u8[:, :4], u8, u8[:, :4])
    with pytest.raises(ValueError):
        pkg.linear_backward(torch.zeros(4, 8), None, u8, u8, u8, u8, out_dtype="e4m3")
    assert sys.modules["mxfp8_block_scaled_mxgemm_amd"].TokenSort._fields == ("offsets", "k_offsets", "row_of",
                                                                              "pair_of")
