"""The compiled calls are an addition: the binding and the build do without them where they are
missing, do not load or do not compile. CPU only."""

import os
import subprocess
import sys
import types
import warnings

import pytest

import exact_attention_80_gb300 as fa
from exact_attention_80_gb300 import build as fa_build

torch = pytest.importorskip("torch")
NAME = fa.__name__ + "._calls"
needs_cuda_torch = pytest.mark.skipif(torch.version.cuda is None, reason="a PyTorch without CUDA has no compiled calls")


@pytest.fixture
def unloaded(monkeypatch):
    """The binding as before its first call."""
    fa.load_library()
    monkeypatch.setattr(fa, "_lib", None)
    monkeypatch.setattr(fa, "_compiled", None)
    monkeypatch.delattr(fa, "_calls", raising=False)


def works_without():
    with pytest.warns(RuntimeWarning, match="compiled calls"):
        assert fa.fa_splitkv_workspace_bytes(1, 1, 1, 64, 2) == 528
    assert fa._compiled is None
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # said once
        assert fa.fa_splitkv_workspace_bytes(1, 1, 1, 64, 2) == 528
        assert fa.fa_paged_num_splits(1, 8, 8, 1, 4096, 64) >= 1
    with pytest.raises((TypeError, ValueError)):  # the Python form's own checks
        fa.rope(torch.zeros(4, 2, 64), None, torch.zeros(9, 64), torch.zeros(4, dtype=torch.int32))


@needs_cuda_torch
def test_missing_module(unloaded, monkeypatch):
    monkeypatch.setitem(sys.modules, NAME, None)
    works_without()


@needs_cuda_torch
@pytest.mark.parametrize("fake", [{"torch_version": "0.1"}, {}])
def test_module_of_another_pytorch(unloaded, monkeypatch, fake):
    module = types.ModuleType(NAME)
    module.__dict__.update(fake, init=lambda *a: pytest.fail("taken all the same"))
    monkeypatch.setitem(sys.modules, NAME, module)
    monkeypatch.setattr(fa, "_calls", module, raising=False)
    works_without()


@needs_cuda_torch
def test_module_that_was_built_here(unloaded):
    """What the build leaves beside the library is loaded, with no warning."""
    if not os.path.exists(fa_build.CALLS):
        pytest.skip("not built")
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        fa.load_library()
    assert fa._compiled is not None and fa._compiled.torch_version == str(torch.__version__)


def test_a_load_that_failed_is_not_kept(unloaded, monkeypatch):
    def fails(lib):
        raise OSError("no such thing")

    monkeypatch.setattr(fa, "_load_calls", fails)
    for _ in range(2):
        with pytest.raises(OSError):
            fa.fa_splitkv_workspace_bytes(1, 1, 1, 64, 2)


@needs_cuda_torch
@pytest.mark.parametrize("failure", ["status", "no compiler"])
def test_build_goes_on_without_the_module(monkeypatch, tmp_path, capsys, failure):
    """A module that does not compile is reported and leaves no older one behind."""
    calls = tmp_path / "_calls.so"
    calls.write_bytes(b"older")
    monkeypatch.setattr(fa_build, "CALLS", str(calls))

    def run(cmd, **kw):
        if failure == "status":
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        raise FileNotFoundError("g++")

    monkeypatch.setattr(fa_build.subprocess, "run", run)
    assert fa_build.build_calls() is None and not calls.exists()
    assert "_calls was not built" in capsys.readouterr().err


def test_build_with_a_pytorch_without_cuda(monkeypatch, tmp_path):
    (tmp_path / "lib").mkdir()
    monkeypatch.setattr(fa_build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(fa_build.importlib.util, "find_spec",
                        lambda name: types.SimpleNamespace(submodule_search_locations=[str(tmp_path)]))
    monkeypatch.setattr(fa_build.subprocess, "run", lambda *a, **k: pytest.fail("nothing to compile against"))
    assert fa_build.build_calls() is None
