"""bench.py reports recorded DRAM bytes only while every source that decides
them is the one they were taken on."""
import os
import shutil

import pytest

import bench

CSRC = os.path.join("mtp_speculative_decoding_gb300", "csrc")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    shutil.copytree(os.path.join(bench.ROOT, "include"), tmp_path / "include")
    (tmp_path / "profiles").mkdir()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    (tmp_path / "profiles" / "dram_traffic.txt").write_text(
        f"workload=w kernel=k source_hash={bench.kernel_source_hash()} dram_bytes_per_launch=3 read=2 write=1\n")
    assert bench.recorded_traffic("w") == 3
    return tmp_path


@pytest.mark.parametrize("name", ["api.cu", "host.cuh", "common.cuh", "draft_kernel.cuh", "draft_dispatch.cu", "verify.cu", "sample.cuh",
                                  "a_new_one.cuh", "../../include/mtp.h"])
def test_a_changed_source_drops_the_recorded_bytes(tree, name):
    with open(tree / CSRC / name, "a") as f:
        f.write("\n// changed\n")
    assert bench.recorded_traffic("w") is None


@pytest.mark.parametrize("name", ["kv_append.cu", "logprobs.cuh", "paged.cuh", "paged_api.cu", "paged_attn.cu", "paged_attn_tc.cu"])
def test_operators_that_no_workload_launches_do_not(tree, name):
    with open(tree / CSRC / name, "a") as f:
        f.write("\n// changed\n")
    assert bench.recorded_traffic("w") == 3
