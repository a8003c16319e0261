"""The binding's hot path is optional: the library is built first and without it, and a module built for another
torch is neither kept nor used."""
import ctypes
import subprocess
import types

import pytest
import torch

import paged_kv_cache_462_b200 as pkv
from paged_kv_cache_462_b200 import build


@pytest.fixture
def at(tmp_path, monkeypatch):
    """The extension's files in a folder of their own, g++ a stand-in that counts."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "FASTCALL", str(tmp_path / "_fastcall.so"))
    monkeypatch.setattr(build.subprocess, "run", run)
    return ran


@pytest.mark.parametrize("fault", ["no compiler", "no torch", "compile error"])
def test_the_library_does_without_it(tmp_path, monkeypatch, capfd, fault):
    built = []
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "FASTCALL", str(tmp_path / "_fastcall.so"))
    monkeypatch.setattr(build, "build_library", lambda force=False, verbose=False: built.append("library"))
    if fault == "no compiler":
        monkeypatch.setenv("CXX", str(tmp_path / "missing"))
    elif fault == "no torch":
        real = build.importlib.util.find_spec
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda n, *a: None if n == "torch" else real(n, *a))
    else:
        monkeypatch.setattr(build.subprocess, "run", lambda *a, **k: subprocess.CompletedProcess(a, 1, "", "no"))
    assert build.build() == build.LIB and built == ["library"]
    assert "warning" in capfd.readouterr().err
    with pytest.raises((OSError, RuntimeError)):
        build.build(strict=True)
    assert built == ["library"] * 2


def test_built_anew_for_another_torch(at, monkeypatch):
    build.build_fastcall()
    build.build_fastcall()
    assert len(at) == 1
    monkeypatch.setattr(build, "torch_version", lambda: "0.1")
    build.build_fastcall()
    build.build_fastcall()
    assert len(at) == 2 and '-DPKV_TORCH_VERSION="0.1"' in at[1]


def test_a_module_for_another_torch_is_left_alone(monkeypatch):
    build.build(strict=True)
    lib = ctypes.CDLL(pkv.LIB_PATH)
    monkeypatch.setattr(pkv, "_fast", None)
    pkv._bind_fast(lib)
    assert pkv._fast is not None and pkv._fast.torch_version == torch.__version__
    monkeypatch.setattr(pkv, "_fast", None)
    monkeypatch.setattr(torch, "__version__", "0.1")
    pkv._bind_fast(lib)
    assert pkv._fast is None
