"""The DRAM traffic that bench.py reports is a recorded capture's, valid while the dense forward's
sources are as they were."""

import os
import shutil

import pytest

import bench


@pytest.fixture
def sources(monkeypatch, tmp_path):
    at = tmp_path / "csrc"
    shutil.copytree(bench.CSRC, at)
    monkeypatch.setattr(bench, "CSRC", str(at))
    return at


def touch(path):
    path.write_text(path.read_text() + "\n")


def test_other_operators_leave_the_record_valid(sources):
    want = bench.kernel_source_hash()
    names = os.listdir(sources)
    for name in sorted(n for n in names if n.startswith(("fa_rope", "fa_kv_append", "fa_paged", "fa_bwd", "fa_combine"))):
        touch(sources / name)
        assert bench.kernel_source_hash() == want, name
    touch(sources / "fa_fwd_window.cu")
    assert bench.kernel_source_hash() == want


@pytest.mark.parametrize("name", ["fa_fwd_tm.cuh", "fa_fwd_common.cuh", "fa_fwd_win.cuh", "fa_fwd_d128.cu", "fa_api.cu",
                                  "fa_internal.h", "sm103_ptx.cuh"])
def test_the_forward_sources_do_not(sources, name):
    want = bench.kernel_source_hash()
    touch(sources / name)
    assert bench.kernel_source_hash() != want


def test_names_that_do_not_count_are_files():
    assert set(bench.NOT_FORWARD) <= set(os.listdir(bench.CSRC))
