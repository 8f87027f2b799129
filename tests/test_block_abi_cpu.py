"""CPU-only checks of the C ABI of the operators with scales of 128 and those
around them: exports, the layout of the argument structs, argument rules that
need no GPU."""
import ctypes
import os
import re
import subprocess

import pytest

import mxfp8_block_scaled_mxgemm_amd as pkg
from mxfp8_block_scaled_mxgemm_amd import _block, _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxgemm_block.h")
P = ctypes.c_void_p(16)
EINVAL, EUNSUPPORTED = _lib.MXGEMM_EINVAL, _lib.MXGEMM_EUNSUPPORTED


def _text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_library_exports_every_declared_symbol():
    declared = sorted(set(re.findall(r"\b(mxgemm_\w+)\s*\(", _text())))
    lib = _block._load()
    assert sorted(pkg.EXPORTED_BLOCK) == declared
    assert all(hasattr(lib, name) for name in declared)


@pytest.mark.parametrize("tag,packed", [("mxgemm_block_linear", _block.BLOCK_ARGS), ("mxgemm_norm", _block.NORM_ARGS)])
def test_header_is_c_and_the_structs_are_the_bindings(tag, packed, tmp_path):
    """The header compiles as C, and the packed argument blocks have the structs'
    sizes and field offsets."""
    text = _text()
    body = text[text.index(f"typedef struct {tag} {{"):text.index(f"}} {tag}_t;")]
    fields = []
    for kind, names in re.findall(r"(?:const )?(\w+)\s*(\*?\s*[\w, ]+);", body):
        for n in names.split(","):
            fields.append((n.replace("*", "").strip(), 8 if "*" in names or kind in ("int64_t",) else 4))
    lines = "".join(f'printf("{n} %zu\\n", offsetof({tag}_t, {n}));' for n, _ in fields)
    src = tmp_path / "layout.c"
    src.write_text('#include "mxgemm_block.h"\n#include <stddef.h>\n#include <stdio.h>\n'
                   f'int main(void) {{ printf("size %zu\\n", sizeof({tag}_t)); {lines} return 0; }}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], check=True, capture_output=True,
                                                       text=True).stdout.splitlines())
    assert int(got.pop("size")) == packed.size
    kinds = [c for n, c in re.findall(r"(\d*)([Pqif])", packed.format if isinstance(packed.format, str) else
                                      packed.format.decode()) for _ in range(int(n or 1))]
    assert [8 if c in "Pq" else 4 for c in kinds] == [size for _, size in fields]
    at = 0
    for name, size in fields:
        assert int(got[name]) == at, name
        at += size


# ------------------------------------------------------------------- route --

def _route(tokens=4, experts=8, k=2, ld=8, type=2, score=0, groups=1, top=1):
    return _block._load().mxgemm_route_tokens(P, ld, type, tokens, experts, k, score, None, groups, top, 1, 1.0, P, P,
                                              None)


def _route_backward(tokens=4, experts=8, k=2, ld=8, type=2, score=0, ld_d=8):
    return _block._load().mxgemm_route_tokens_backward(P, P, ld, type, tokens, experts, k, score, 1, 1.0, P, P, ld_d,
                                                       None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), EINVAL), (dict(experts=0), EINVAL), (dict(k=0), EINVAL), (dict(k=9), EINVAL),
    (dict(ld=7), EINVAL), (dict(type=3), EINVAL), (dict(type=-1), EINVAL), (dict(score=2), EINVAL),
    (dict(experts=1025, ld=1025), EUNSUPPORTED), (dict(experts=100, ld=100, k=65), EUNSUPPORTED),
    (dict(tokens=1 << 41), EUNSUPPORTED),
])
def test_route_rules(kw, code):
    assert _route(**kw) == code and pkg.last_error()
    if "ld" not in kw or "experts" in kw:
        kw = dict(kw, ld_d=1025)
    assert _route_backward(**kw) == code


def test_more_route_rules():
    assert _route(groups=3) == _route(groups=0) == _route(groups=2, top=3) == _route(top=0) == EINVAL
    assert _route(groups=8, top=1, k=2) == EINVAL                      # one expert a group
    assert _route(experts=130, ld=130, groups=65, top=2) == EUNSUPPORTED
    assert _route_backward(ld_d=7) == EINVAL
    assert _route(tokens=0) == 0 and _route_backward(tokens=0) == 0


# ---------------------------------------------------------------- quantise --

def _quantize(rows=4, C=128, ld_x=128, z=None, ld_z=0, type=0, act=0, gated=0, off=None, koff=None, E=0, fmt=0, q=P,
              s=P, qt=P, st=P, ld_qt=128):
    return _block._load().mxgemm_block_quantize(P, type, ld_x, z, ld_z, rows, C, act, gated, off, koff, E, fmt, q, s,
                                                qt, st, ld_qt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), EINVAL), (dict(C=0), EINVAL), (dict(E=-1), EINVAL), (dict(type=3), EINVAL), (dict(act=5), EINVAL),
    (dict(fmt=2), EINVAL), (dict(z=P, ld_z=127, C=127, gated=1), EINVAL), (dict(s=None), EINVAL), (dict(qt=None), EINVAL),
    (dict(E=2), EINVAL), (dict(ld_qt=256), EINVAL), (dict(ld_qt=130, E=1, off=P, koff=P), EINVAL),
    (dict(ld_x=127), EINVAL), (dict(gated=1), EINVAL), (dict(z=P, ld_z=127), EINVAL),
    (dict(rows=65534 * 128 + 1), EUNSUPPORTED), (dict(C=(1 << 30) + 1), EUNSUPPORTED),
    (dict(E=65536, off=P, koff=P), EUNSUPPORTED), (dict(E=1, off=P, koff=P, ld_qt=65535 * 128), EUNSUPPORTED),
])
def test_quantize_rules(kw, code):
    assert _quantize(**kw) == code and pkg.last_error()


def _weight(type=0, ld=128, group=0, batch=1, N=4, K=128, fmt=0, qt=P, st=P):
    return _block._load().mxgemm_block_quantize_weight(P, type, ld, group, batch, N, K, fmt, P, P, qt, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), EINVAL), (dict(ld=127), EINVAL), (dict(batch=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL),
    (dict(fmt=-1), EINVAL), (dict(qt=None), EINVAL), (dict(group=-1), EINVAL), (dict(batch=65536), EUNSUPPORTED),
    (dict(N=65535 * 128 + 1), EUNSUPPORTED), (dict(batch=0), 0),
])
def test_quantize_weight_rules(kw, code):
    assert _weight(**kw) == code


# ----------------------------------------------------------------- product --

def _args(**kw):
    names = ("a a_scale w w_scale out offsets rows N K lda a_scale_row a_scale_k ldw w_group w_scale_row w_scale_k "
             "w_scale_group ld_out out_group squares mode experts a_format w_format precision out_type tile_cfg "
             "workspace workspace_bytes").split()
    v = dict.fromkeys(names, 0)
    v.update(rows=4, N=64, K=256, lda=256, a_scale_row=1, a_scale_k=4, ldw=256, w_scale_row=2, w_scale_k=1, ld_out=64,
             squares=1, tile_cfg=-1)
    v.update(kw)
    return _block.BLOCK_ARGS.pack(*(v[n] for n in names))


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(K=192, lda=192, ldw=192), EINVAL),
    (dict(mode=3), EINVAL), (dict(mode=1), EINVAL), (dict(mode=1, experts=2), EINVAL),
    (dict(mode=2, experts=2, offsets=16), EINVAL), (dict(out_type=3), EINVAL), (dict(a_format=2), EINVAL),
    (dict(w_format=-1), EINVAL), (dict(precision=2), EINVAL), (dict(lda=128), EINVAL), (dict(lda=264), EINVAL),
    (dict(ldw=255), EINVAL), (dict(w_group=8, mode=1, experts=2, offsets=16), EINVAL), (dict(ld_out=63), EINVAL),
    (dict(a_scale_row=-1), EINVAL), (dict(w_scale_k=-1), EINVAL), (dict(tile_cfg=5), EINVAL),
    (dict(tile_cfg=0), EINVAL), (dict(tile_cfg=0, precision=1, squares=0), EINVAL), (dict(tile_cfg=3, squares=0), EINVAL),
    (dict(rows=1 << 31), EUNSUPPORTED), (dict(N=1 << 31, ld_out=1 << 31), EUNSUPPORTED),
    (dict(lda=1 << 24), EUNSUPPORTED), (dict(a_scale_row=(1 << 21) + 1), EUNSUPPORTED),
    (dict(w_scale_row=(1 << 21) + 1), EUNSUPPORTED), (dict(mode=1, experts=(1 << 20) + 1, offsets=16), EUNSUPPORTED),
])
def test_block_linear_refuses_before_touching_a_gpu(kw, code):
    assert _block._load().mxgemm_block_linear(_args(**kw), None) == code
    assert pkg.last_error()


def test_block_linear_without_rows_is_nothing():
    assert _block._load().mxgemm_block_linear(_args(rows=0), None) == 0
    assert _block._load().mxgemm_block_linear(None, None) == EINVAL


def test_workspaces():
    lib = _block._load()
    assert lib.mxgemm_block_linear_workspace(64, 2048, 7168) == 256 * 64 * 64 * 4
    assert lib.mxgemm_block_linear_workspace(32, 2048, 7168) == 0
    ws = lib.mxgemm_add_norm_workspace
    assert ws(0, 64, 1) == ws(4, 0, 1) == ws(4, 64, 3) == ws(4, 64, 0) == ws(4, 8193, 1) == 0
    for rows, cols, gates in ((1, 1, 1), (8192, 4096, 8), (5000, 100, 5000), (100000, 8192, 1)):
        n = ws(rows, cols, gates)
        assert 0 < n <= 3 * 4 * cols * min(rows, 4096)


# ------------------------------------------------------------------- norm ---

def _norm(**kw):
    names = ("x residual gate post_weight pre_weight r y d_y d_r d_x d_residual d_gate d_post_weight d_pre_weight "
             "workspace workspace_bytes rows cols gate_rows ld_x ld_residual ld_gate ld_r ld_y ld_d_y ld_d_r ld_d_x "
             "ld_d_residual type gate_type post_type pre_type kind scale eps reserved").split()
    v = dict.fromkeys(names, 0)
    v.update(rows=4, cols=64, gate_rows=1, x=16, r=16, y=16, scale=1.0, eps=1e-6, workspace=16,
             workspace_bytes=1 << 30, **{n: 64 for n in names if n.startswith("ld_")})
    v.update(kw)
    return _block.NORM_ARGS.pack(*(v[n] for n in names))


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), EINVAL), (dict(cols=0), EINVAL), (dict(cols=8193), EUNSUPPORTED), (dict(type=3), EINVAL),
    (dict(kind=2), EINVAL), (dict(gate=16, gate_type=3), EINVAL), (dict(post_weight=16, post_type=-1), EINVAL),
    (dict(pre_weight=16, pre_type=7), EINVAL), (dict(gate=16, gate_rows=3), EINVAL), (dict(gate=16, gate_rows=0), EINVAL),
    (dict(gate=16, ld_gate=-1), EINVAL), (dict(ld_x=63), EINVAL), (dict(ld_r=63), EINVAL),
    (dict(rows=0, gate=16, gate_rows=70000), EUNSUPPORTED),
])
def test_norm_rules(kw, code):
    lib = _block._load()
    assert lib.mxgemm_add_norm(_norm(**kw), None) == code and pkg.last_error()
    assert lib.mxgemm_add_norm_backward(_norm(**kw), None) == code


def test_more_norm_rules():
    lib = _block._load()
    assert lib.mxgemm_add_norm(_norm(residual=16, ld_residual=63), None) == EINVAL
    assert lib.mxgemm_add_norm(_norm(pre_weight=16, ld_y=63), None) == EINVAL
    assert lib.mxgemm_add_norm_backward(_norm(d_y=16), None) == EINVAL              # without pre_weight
    assert lib.mxgemm_add_norm_backward(_norm(d_r=16, ld_d_r=63), None) == EINVAL
    assert lib.mxgemm_add_norm_backward(_norm(ld_d_x=63), None) == EINVAL
    assert lib.mxgemm_add_norm_backward(_norm(d_residual=16, ld_d_residual=63), None) == EINVAL
    assert lib.mxgemm_add_norm_backward(_norm(workspace_bytes=0), None) == EINVAL
    assert lib.mxgemm_add_norm(_norm(rows=0), None) == 0
    assert lib.mxgemm_add_norm(None, None) == lib.mxgemm_add_norm_backward(None, None) == EINVAL


def test_binding_refuses_without_a_gpu():
    torch = pytest.importorskip("torch")
    u8, f = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 128)
    for call in (lambda: pkg.route_tokens(f, 2), lambda: pkg.route_tokens_backward(f[:, :2], f, f[:, :2].int()),
                 lambda: pkg.block_quantize(f), lambda: pkg.block_quantize_weight(f),
                 lambda: pkg.block_linear(u8, f[:, :1], u8, f[:, :1]), lambda: pkg.add_norm(f),
                 lambda: pkg.add_norm_backward(None, f, f, f)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: pkg.block_quantize_backward(f, None, act="silu"),
                 lambda: pkg.block_quantize_backward(f, None, gated=True),
                 lambda: pkg.block_linear_backward(f, None, u8, f, u8, f, act="gelu")):
        with pytest.raises(ValueError):
            call()
