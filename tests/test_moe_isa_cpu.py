"""Build-time properties of the expert layer's gfx950 code: vector-only memory
writes, nothing spilled to scratch, and the occupancy its tiles are made for.
This file is CPU-only."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mxfp8_block_scaled_mxgemm_amd", "csrc")
SOURCES = ["tokens.hip", "grad.hip", "layout.hip", "linear_finish.hip", "linear_e4m3_e4m3.hip", "linear_e5m2_e4m3.hip"]
WRITERS = re.compile(r"^\s+(?:global|flat|ds|buffer|s)_(?:store|atomic|write)\w*", re.MULTILINE)


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    from mxfp8_block_scaled_mxgemm_amd import build
    d = tmp_path_factory.mktemp("isa")
    procs = {}
    for src in SOURCES:
        cmd = [hipcc, "-x", "hip", *build.HIP_FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
               "--cuda-device-only", "-S", os.path.join(CSRC, src), "-o", str(d / (src + ".s")),
               "-Rpass-analysis=kernel-resource-usage"]
        procs[src] = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
    out = {}
    for src, p in procs.items():
        _, err = p.communicate(timeout=900)
        assert p.returncode == 0, err[-2000:]
        usage, name = {}, None
        for line in err.splitlines():
            m = re.search(r"Function Name: (\S+)", line)
            if m:
                name = m.group(1)
                usage[name] = {}
                continue
            m = re.search(r"remark:\s+([A-Za-z ]+?)(?:\s*\[[^\]]*\])?: (\d+)", line)
            if m and name:
                usage[name][m.group(1).strip()] = int(m.group(2))
        out[src] = ((d / (src + ".s")).read_text(), usage)
    return out


@pytest.mark.parametrize("src", SOURCES)
def test_writes_are_vector_writes_and_nothing_spills(compiled, src):
    asm, usage = compiled[src]
    assert usage
    assert {w.split("_")[0].strip() for w in WRITERS.findall(asm)} <= {"global", "ds"}
    for kernel, v in usage.items():
        assert v.get("VGPRs Spill", 0) == 0 and v.get("ScratchSize", 0) == 0, (kernel, v)


def test_packed_fp32_is_off(compiled):
    for src, (asm, _) in compiled.items():
        assert not re.search(r"v_pk_(?:add|mul|fma)_f32", asm), src


def test_tiles_share_compute_units_as_planned(compiled):
    _, usage = compiled["linear_e4m3_e4m3.hip"]
    for tile, per_simd, lds in (("ILi256ELi256ELi2ELi2ELi1ELi1ELb0E", 1, 160), ("ILi128ELi128ELi2ELi2ELi1ELi2ELb0E", 2, 80),
                                ("ILi128ELi128ELi2ELi2ELi1ELi2ELb1E", 2, 80), ("ILi64ELi64ELi1ELi1ELi4ELi1ELb1E", 1, 160)):
        v = [u for k, u in usage.items() if "linear_kernel" + tile in k]
        assert len(v) == 1 and v[0]["Occupancy"] == per_simd and v[0]["LDS Size"] <= lds * 1024, (tile, v)
