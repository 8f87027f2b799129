"""Registers, scratch and occupancy of every kernel of the operators with scales
of 128 and those around them, as the compiler reports them: nothing is spilled to
memory, and as many waves fit on a SIMD as the launch code and the tiles count on;
and vector writes only, in every format pair.  This file is CPU-only."""
import os
import re
import shutil
import subprocess

import pytest

from test_block_isa_cpu import WRITERS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mxfp8_block_scaled_mxgemm_amd", "csrc")
PRODUCTS = ["block_e4m3_e4m3.hip", "block_e4m3_e5m2.hip", "block_e5m2_e4m3.hip", "block_e5m2_e5m2.hip"]
SOURCES = ["route.hip", "norm.hip", "block_quant.hip", *PRODUCTS]
LDS = 160 * 1024        # of a compute unit


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    """{source: (assembly, {kernel: {what: number}})}"""
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    from mxfp8_block_scaled_mxgemm_amd import build
    d = tmp_path_factory.mktemp("occupancy")
    procs = {src: subprocess.Popen([hipcc, "-x", "hip", *build.HIP_FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                                    "--cuda-device-only", "-S", os.path.join(CSRC, src), "-o", str(d / (src + ".s")),
                                    "-Rpass-analysis=kernel-resource-usage"], stdout=subprocess.PIPE,
                                   stderr=subprocess.PIPE, text=True) for src in SOURCES}
    out = {}
    for src, p in procs.items():
        _, err = p.communicate(timeout=900)
        assert p.returncode == 0, err[-2000:]
        kernels, name = {}, None
        for line in err.splitlines():
            m = re.search(r"Function Name: (\S+)", line)
            if m:
                name = m.group(1)
                kernels[name] = {}
                continue
            m = re.search(r"remark:\s+([A-Za-z ]+?)(?:\s*\[[^\]]*\])?: (\d+)", line)
            if m and name:
                kernels[name][m.group(1).strip()] = int(m.group(2))
        assert kernels, src
        out[src] = (d / (src + ".s")).read_text(), kernels
    return out


@pytest.mark.parametrize("src", SOURCES)
def test_nothing_spills_to_memory(compiled, src):
    for kernel, v in compiled[src][1].items():
        assert v["VGPRs Spill"] == v["ScratchSize"] == 0, (kernel, v)


@pytest.mark.parametrize("src", PRODUCTS)
def test_products_write_by_vector_writes_without_packed_fp32(compiled, src):
    asm = compiled[src][0]
    assert {w.split("_")[0].strip() for w in WRITERS.findall(asm)} == {"global", "ds"}
    assert not re.search(r"v_pk_(?:add|mul|fma)_f32", asm)


@pytest.mark.parametrize("src", PRODUCTS)
def test_products_share_compute_units_as_planned(compiled, src):
    """Waves of a SIMD, work-groups of a compute unit: 256 x 256 tiles one of
    eight waves, 128 x 128 two of four, 64 x 64 one of four."""
    tiles = {"ILi256ELi256ELi2ELi4ELi1ELi1E": (2, 1), "ILi128ELi128ELi2ELi2ELi1ELi2E": (2, 2),
             "ILi64ELi64ELi1ELi1ELi4ELi1E": (1, 1)}
    seen = dict.fromkeys(tiles, 0)
    for kernel, v in compiled[src][1].items():
        for tile, (waves, groups) in tiles.items():
            if "block_linear_kernel" + tile in kernel:
                seen[tile] += 1
                assert v["Occupancy"] >= waves and v["LDS Size"] * groups <= LDS, (kernel, v)
    assert list(seen.values()) == [1, 4, 4]         # the largest: native, squares; the others both of both
    skinny = [v for k, v in compiled[src][1].items() if "block_skinny_kernel" in k]
    assert len(skinny) == 16 and all(v["Occupancy"] >= 3 for v in skinny)


def test_rows_of_norms_routers_and_quantisers(compiled):
    """The norms' gradient is launched for sixteen waves of a compute unit, four of
    a SIMD, and has three where a wave takes a row; the others' grids are larger
    than what is resident anyway."""
    kernels = compiled["norm.hip"][1]
    back = {k: v["Occupancy"] for k, v in kernels.items() if "norm_backward_kernel" in k}
    assert len(back) == 30
    for k, waves in back.items():
        assert waves >= (3 if re.search(r"ILi\dELi64E", k) else 4), (k, waves)
    assert all(v["Occupancy"] >= 5 for k, v in kernels.items() if "11norm_kernel" in k)
    for k, v in compiled["route.hip"][1].items():
        if "route_rows_kernel" in k:
            assert v["Occupancy"] >= 4, (k, v)
    for k, v in compiled["block_quant.hip"][1].items():
        assert v["Occupancy"] >= (3 if re.search(r"pair_kernelILi\dELi2E", k) else 4), (k, v)
