"""The bench's recorded DRAM bytes hold while the kernels' code does, the code that they include too."""

import os
import shutil

import pytest

import bench


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the sources, and the records as if they had been captured on it."""
    dirs = tuple(str(tmp_path / str(i)) for i in range(len(bench.SOURCE_DIRS)))
    for src, dst in zip(bench.SOURCE_DIRS, dirs):
        shutil.copytree(src, dst)
    monkeypatch.setattr(bench, "SOURCE_DIRS", dirs)
    monkeypatch.setattr(bench, "NCU_TRAFFIC", {
        key: {"sources": {s: bench._code_digest(s) for s in rec["sources"]}, "bytes": rec["bytes"]}
        for key, rec in bench.NCU_TRAFFIC.items()})
    return lambda name: next(p for p in (os.path.join(d, name) for d in dirs) if os.path.exists(p))


def _current():
    return {kernel for kernel, workload in bench.NCU_TRAFFIC if bench._traffic(kernel, workload) is not None}


ALL = {kernel for kernel, _ in bench.NCU_TRAFFIC}


def test_unchanged_sources_keep_their_records(tree):
    assert _current() == ALL and bench._traffic("fwd_kernel", "no such workload") is None


@pytest.mark.parametrize("name,stale", [
    ("softmax.cuh", {"fwd_kernel", "fwd_kernel_fp8", "fwd_persist_kernel", "causal_sharded4"}),
    ("bwd_common.cuh", {"bwd_dkdv_kernel"}),
    ("stage_io.cuh", {"fwd_kernel", "fwd_kernel_fp8", "fwd_persist_kernel", "causal_sharded4", "bwd_dkdv_kernel"}),
    ("fa_decode.cu", {"decode_split_kernel", "decode_split_kernel_paged", "causal_sharded4"}),
    ("fa_fwd.cu", {"fwd_kernel", "fwd_kernel_fp8", "fwd_persist_kernel", "causal_sharded4"}),
    ("ptx.cuh", ALL), ("internal.h", ALL), ("fattn.h", ALL), ("fa_rope.cu", set())])
def test_a_change_of_code_ends_the_records_it_reaches(tree, name, stale):
    path = tree(name)
    with open(path) as f:
        text = f.read()
    with open(path, "w") as f:
        f.write(text + "\n// a remark\n\n/* and\n another */\n")
    assert _current() == ALL
    with open(path, "w") as f:
        f.write(text + "\nconstexpr int kAnother = 1;\n")
    assert _current() == ALL - stale
    os.remove(path)
    assert _current() <= ALL - stale
