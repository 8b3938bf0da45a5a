"""The codec's build without torch or Python's headers, which only the paged
cache's binding is built against (the binding's compiler runs are recorded in
place of being made)."""
import subprocess
import sys
import sysconfig

import pytest

from lossless_entropy_coded_dfc_amd.csrc import build as b


@pytest.fixture
def runs(monkeypatch):
    made = []
    monkeypatch.setattr(b, "_run", lambda cmd, verbose: made.append(cmd))
    monkeypatch.setattr(b.os, "replace", lambda a, c: made.append((a, c)))
    return made


def test_the_build_goes_on_without_torch(runs, monkeypatch, capsys):
    monkeypatch.setattr(b, "_hipcc", lambda: "hipcc")
    monkeypatch.setitem(sys.modules, "torch", None)
    assert b.build() == b.OUT
    assert any(r[-1] == b.OUT for r in runs) and any(r[-1] == b.PROBE_OUT for r in runs)
    assert not any(b.BIND_OUT in str(r) for r in runs)
    assert "torch cannot be imported" in capsys.readouterr().err


def test_the_build_goes_on_without_pythons_headers(runs, monkeypatch, tmp_path, capsys):
    pytest.importorskip("torch")
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(sysconfig, "get_paths", lambda: paths)
    b._build_bind(False)
    assert not runs and "Python.h" in capsys.readouterr().err


def test_an_error_of_the_compiler_is_still_one(monkeypatch):
    pytest.importorskip("torch")

    def fails(cmd, verbose):
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(b, "_run", fails)
    with pytest.raises(subprocess.CalledProcessError):
        b._build_bind(False)


def test_a_binding_of_another_torch_is_refused(monkeypatch):
    # it reads tensors by that torch's structures
    torch = pytest.importorskip("torch")
    import lossless_entropy_coded_dfc_amd as dfc
    from lossless_entropy_coded_dfc_amd import paged
    monkeypatch.setattr(paged, "_BIND", None)
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    x = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(dfc.DfcLibraryMissing, match="1.0.0"):
        dfc.paged_plan(x, x, x, x, x, 16, 1)
    monkeypatch.undo()
    with pytest.raises(TypeError):  # (this torch's: as far as the arguments)
        dfc.paged_plan(x, x, x[None], x, x, 16, 1)
