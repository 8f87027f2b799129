"""CPU-only checks of edges of the expert layer's host side."""
import ctypes

import pytest

import mxfp8_block_scaled_mxgemm_amd as pkg
from mxfp8_block_scaled_mxgemm_amd import _lib, _moe


def test_grids_of_2_to_32_threads_are_refused():
    """What one launch cannot hold is EUNSUPPORTED before anything else is
    looked at."""
    lib = _moe._load()
    p = ctypes.c_void_p(16)
    eb = lib.mxgemm_epilogue_backward
    N = 1 << 30
    assert eb(p, 0, N, None, 0, 4, N, 0, 0, None, None, 0, 0, p, p, p, p, 128, None, None, 0,
              None) == _lib.MXGEMM_EUNSUPPORTED
    rows = 65535 * 128
    assert eb(p, 0, 64, None, 0, rows, 64, 0, 0, p, p, 2, 0, p, p, p, p, 128, None, None, 0,
              None) == _lib.MXGEMM_EUNSUPPORTED
    assert lib.mxgemm_transpose_bytes(p, 1 << 31, 0, 4, 1 << 31, 1, p, None) == _lib.MXGEMM_EUNSUPPORTED


def test_no_rows_need_no_preactivation():
    """A NULL z is refused for real rows only."""
    eb = _moe._load().mxgemm_epilogue_backward
    args = lambda rows, ld: (None, 0, 64, None, 64, rows, 64, 4, 0, None, None, 0, 0, None, None, None, None,  # noqa: E731
                             ld, None, None, 0, None)
    assert eb(*args(4, 128)) == _lib.MXGEMM_EINVAL and "needs z" in pkg.last_error()
    assert eb(*args(0, 0)) != _lib.MXGEMM_EINVAL        # without a GPU the call ends at the device


def test_first_call_from_two_threads():
    """torch counts as bound only once the table of types is filled."""
    torch = pytest.importorskip("torch")

    class Watched(dict):
        def update(self, *a, **kw):
            seen.append(_moe.torch)
            super().update(*a, **kw)

    seen, before = [], (_moe.torch, _moe._TYPES)
    _moe.torch, _moe._TYPES = None, Watched()
    try:
        _moe._bind()
        assert seen and all(t is None for t in seen)
        assert _moe.torch is torch and len(_moe._TYPES) == 3
    finally:
        _moe.torch, _moe._TYPES = before


def test_the_bindings_workspace_rule_is_the_librarys():
    ws = _moe._load().mxgemm_linear_workspace
    edges = [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 512, 1000, 2047, 2048, 2049, 4096, 8191, 8192, 8193]
    for M in edges:
        for N in edges:
            for K in (128, 1920, 2048, 2176, 7168):
                assert _moe._split_workspace(M, N, K) == ws(M, N, K), (M, N, K)
