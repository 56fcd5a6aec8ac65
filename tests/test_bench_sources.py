"""The hash that ties committed profiler counters to the code they were taken
on: changed by the timed calls' own code and by nothing else."""

import os
import shutil
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.fixture()
def sources(tmp_path, monkeypatch):
    import bench

    csrc = tmp_path / "cross_entropy_gb300" / "csrc"
    shutil.copytree(os.path.join(bench.ROOT, "cross_entropy_gb300", "csrc"), csrc)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return bench, csrc


def test_other_calls_and_comments_do_not_change_it(sources):
    bench, csrc = sources
    was = bench.kernel_source_hash()
    for name in ("gbce_linear.cu", "gbce_linear_mma.cu", "gbce_embedding.cu", "gbce_another.cu"):
        with open(csrc / name, "a") as f:
            f.write("\nint another;\n")
    with open(csrc / "gbce_persistent.cuh", "a") as f:
        f.write("\n// a comment /* in one */\n\n")
    assert bench.kernel_source_hash() == was


@pytest.mark.parametrize("name", ["gbce_api.cu", "gbce_kernels_bf16.cu", "gbce_reduce.cu", "gbce_dispatch.cuh",
                                  "gbce_persistent.cuh", "gbce_kernels.cuh", "gbce_device.cuh", "gbce_internal.h"])
def test_the_timed_calls_own_code_does(sources, name):
    bench, csrc = sources
    was = bench.kernel_source_hash()
    with open(csrc / name, "a") as f:
        f.write("\nint another;\n")
    assert bench.kernel_source_hash() != was
