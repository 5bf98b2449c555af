"""The recorded counters of the scan belong to its kernels' code: edits of host code and of comments
keep them, an edit of a kernel voids them."""

import os
import shutil

import bench
from selective_state_space_13_b200 import build


def copies(tmp_path, monkeypatch):
    paths = []
    for f in build.KERNEL_FILES:
        paths.append(str(tmp_path / os.path.basename(f)))
        shutil.copy(f, paths[-1])
    monkeypatch.setattr(build, "KERNEL_FILES", paths)
    return paths


def test_the_record_applies():
    for workload in ("m130", "long", "vim", "ss2d", "cromb"):
        assert bench.recorded_counters(workload)["dram_bytes_per_launch"] > 0


def test_host_code_is_not_in_it():
    names = {os.path.basename(f) for f in build.KERNEL_FILES}
    assert {"ss_scan_kernels.cuh", "ss_device.cuh", "ss_scan_bf16.cu"} <= names
    assert not names & {"ss_api.cu", "ss_host.cu", "ss_noalloc.cu", "selective_scan.h"}


def test_comments_keep_it_and_code_voids_it(tmp_path, monkeypatch):
    before = bench.kernel_source_digest()
    paths = copies(tmp_path, monkeypatch)
    for p in paths:
        assert bench.kernel_source_digest() == before
        with open(p, "a") as fh:
            fh.write("// a remark\n")
        assert bench.kernel_source_digest() == before
    with open(paths[0], "a") as fh:
        fh.write("constexpr int kOneMore = 1;\n")
    assert bench.kernel_source_digest() != before and not bench.recorded_counters("m130")
