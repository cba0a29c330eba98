"""``bench.py``'s stored DRAM traffic figures: which sources they are keyed to,
and that they are of the present kernels."""

import os
import shutil

import pytest

import bench


@pytest.fixture
def csrc(tmp_path, monkeypatch):
    """A copy of the kernels' folder that a test may change."""
    at = str(tmp_path / "csrc")
    shutil.copytree(bench.CSRC, at)
    monkeypatch.setattr(bench, "CSRC", at)
    return at


def _append(csrc, name):
    with open(os.path.join(csrc, name), "a") as f:
        f.write("// one more line\n")


def test_traffic_figures_are_of_the_present_kernels():
    """A figure whose sources changed is null in the bench line: take it again,
    or take it out."""
    for (workload, kernel), t in bench.NCU_TRAFFIC.items():
        assert t["src"] == bench._src_sha(bench.KERNEL_SRC[kernel]), (workload, kernel)
    assert ("million_decode", "index_score") in bench.NCU_TRAFFIC  # the default line's


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SRC))
def test_key_covers_what_a_kernel_includes(csrc, kernel):
    src = bench.KERNEL_SRC[kernel]
    used = [os.path.basename(p) for p in bench._sources(src)]
    assert src in used and {"csa_internal.cuh", "tc.cuh"} <= set(used)
    key = bench._src_sha(src)
    for name in used:
        _append(csrc, name)
        assert bench._src_sha(src) != key, name
        key = bench._src_sha(src)


def test_key_leaves_out_what_no_kernel_of_its_includes(csrc):
    keys = {s: bench._src_sha(s) for s in bench.KERNEL_SRC.values()}
    for name in ("headvec.cuh", "paged_common.cuh", "k_paged_chunk.cu"):
        _append(csrc, name)
    with open(os.path.join(csrc, "unrelated.cuh"), "w") as f:
        f.write("#pragma once\n")
    assert {s: bench._src_sha(s) for s in keys} == keys
