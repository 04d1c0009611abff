"""bench.py's key of a measured HBM traffic: the sources that the workload's kernel is built from, and no others (CPU)."""
import os
import shutil

import pytest

import bench


@pytest.fixture
def csrc(tmp_path):
    to = tmp_path / "csrc"
    shutil.copytree(bench.CSRC, to)
    return to


def keys(csrc):
    return {w: bench.kernel_hash(w, str(csrc)) for w in bench.ORDER}


def append(path):
    with open(path, "a") as f:
        f.write("\n// one more line\n")


def test_every_workload_has_its_unit():
    assert set(bench.KERNEL_UNIT) == set(bench.ORDER)
    assert all(os.path.exists(os.path.join(bench.CSRC, f)) for f in bench.KERNEL_UNIT.values())


def test_a_copy_has_the_same_keys(csrc):
    assert keys(csrc) == {w: bench.kernel_hash(w) for w in bench.ORDER}


def test_sources_of_other_operators_leave_the_keys(csrc):
    before = keys(csrc)
    for f in os.listdir(csrc):
        if not f.startswith(("gemm", "tcm")) or f == "gemm_w4.hip":
            append(csrc / f)
    (csrc / "another_operator.hip").write_text("// new\n")
    assert keys(csrc) == before


@pytest.mark.parametrize("file,changed", [
    ("tcm_device.h", bench.ORDER), ("tcm_internal.h", bench.ORDER), ("tcm_api.cpp", bench.ORDER),
    ("gemm16_mx.h", ["mxfp8_8192", "mxfp6_8192", "mxfp4_8192"]), ("gemm16_nv4.h", ["nvfp4_8192"]),
    ("gemm_tn.hip", ["bf16_8192", "bf16_4096", "batched", "tile_f16"]), ("gemm_mn_b.hip", ["bf16_8192_nn"]),
    ("gemm_mx_mn_ab.hip", ["mxfp8_8192_mn"]), ("gemm_mx_mn.h", ["mxfp8_8192_mn"])])
def test_sources_of_a_kernel_change_its_key(csrc, file, changed):
    before = keys(csrc)
    append(csrc / file)
    after = keys(csrc)
    assert sorted(w for w in bench.ORDER if before[w] != after[w]) == sorted(changed)


def test_flags_change_the_keys(monkeypatch):
    from tensor_core_matrix_amd import build

    before = bench.kernel_hash("bf16_8192")
    monkeypatch.setattr(build, "DEVICE", build.DEVICE + ["-DONE_MORE"])
    assert bench.kernel_hash("bf16_8192") != before
