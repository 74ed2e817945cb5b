"""The fingerprint by which the bench knows that its DRAM captures are of the present decode kernel (CPU
only): it covers what that kernel is compiled from, and no other kernel's code."""
import os
import shutil

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "paged_kv_attention_pa_gb300", "csrc")


@pytest.mark.parametrize("name,part", [
    ("pa_decode_kernel.cuh", True), ("pa_device.cuh", True), ("pa_params.h", True), ("pa_inst_bf16_d128.cu", True),
    ("pa_inst_fp8_bf16_d128.cu", True), ("pa_attend.cuh", False), ("pa_tcgen05.cuh", False), ("pa_decode_int4.cuh", False),
    ("pa_inst_attend_bf16_d128.cu", False), ("pa_rows.cu", False), ("pa_api.cu", False)])
def test_what_the_fingerprint_covers(tmp_path, name, part):
    csrc = tmp_path / "csrc"
    shutil.copytree(CSRC, csrc)
    before = bench.kernel_sources_sha256(str(csrc))
    assert before == bench.kernel_sources_sha256()
    with open(csrc / name, "a") as f:
        f.write("\n// a comment\n")
    assert bench.kernel_sources_sha256(str(csrc)) == before
    with open(csrc / name, "a") as f:
        f.write("\nnamespace pa { constexpr int one_more = 1; }\n")
    assert (bench.kernel_sources_sha256(str(csrc)) != before) == part


def test_a_file_beside_the_kernel_changes_nothing(tmp_path):
    csrc = tmp_path / "csrc"
    shutil.copytree(CSRC, csrc)
    (csrc / "pa_other.cuh").write_text("namespace pa { constexpr int other = 1; }\n")
    (csrc / "pa_inst_other_d128.cu").write_text('#include "pa_other.cuh"\n')
    assert bench.kernel_sources_sha256(str(csrc)) == bench.kernel_sources_sha256()
