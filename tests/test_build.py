"""The build of the marshalling module: where its headers are found and when it is built again (no GPU needed)."""
import importlib.util
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _build_module(monkeypatch, nvcc):
    monkeypatch.setenv("NVCC", nvcc)
    spec = importlib.util.spec_from_file_location("build_under_test", os.path.join(ROOT, "block_sparse_cluster_b200", "build.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _toolkit(path):
    (path / "bin").mkdir(parents=True)
    (path / "include").mkdir()
    (path / "include" / "cuda_runtime.h").write_text("")
    nvcc = path / "bin" / "nvcc"
    nvcc.write_text("#!/bin/sh\n")
    nvcc.chmod(0o755)
    return nvcc


def _includes(module, monkeypatch):
    """The include directories of the compiler call that build_call makes."""
    calls = []
    monkeypatch.setattr(module.subprocess, "run", lambda cmd, **kw: calls.append(cmd) or subprocess.CompletedProcess(cmd, 0, "", ""))
    module.build_call()
    return [a[2:] for a in calls[0] if a.startswith("-I")]


@pytest.mark.parametrize("how", ["path", "name", "link", "wrapper"])
def test_headers_are_found_however_nvcc_is_named(how, tmp_path, monkeypatch):
    """By its path, by a name on PATH, by a link elsewhere; and by a program elsewhere, with the toolkit in CUDA_HOME."""
    nvcc = _toolkit(tmp_path / "toolkit")
    elsewhere = tmp_path / "bin"
    elsewhere.mkdir()
    monkeypatch.delenv("CUDA_HOME", raising=False)
    name = str(nvcc)
    if how == "name":
        monkeypatch.setenv("PATH", str(nvcc.parent) + os.pathsep + os.environ["PATH"])
        name = "nvcc"
    elif how == "link":
        (elsewhere / "nvcc").symlink_to(nvcc)
        name = str(elsewhere / "nvcc")
    elif how == "wrapper":
        (elsewhere / "nvcc").write_text("#!/bin/sh\n")
        (elsewhere / "nvcc").chmod(0o755)
        name = str(elsewhere / "nvcc")
        monkeypatch.setenv("CUDA_HOME", str(tmp_path / "toolkit"))
    found = _includes(_build_module(monkeypatch, name), monkeypatch)
    assert str(tmp_path / "toolkit" / "include") in [os.path.realpath(d) for d in found]


def test_marshalling_module_is_built_again_for_another_torch(tmp_path, monkeypatch):
    """Sources untouched: built for the first time, kept, and built again once torch or Python is another."""
    module = _build_module(monkeypatch, "nvcc")
    for name in ("LIB", "FAULT_LIB", "CALL_LIB"):
        path = tmp_path / name
        path.write_text("")
        monkeypatch.setattr(module, name, str(path))
    monkeypatch.setattr(module, "BUILD", str(tmp_path / "_build"))
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "__init__.py").write_text("")
    (torch / "version.py").write_text("__version__ = '1'\n")
    monkeypatch.setattr(module.importlib.util, "find_spec", lambda name: importlib.util.spec_from_file_location(name, torch / "__init__.py"))
    built = []
    monkeypatch.setattr(module, "build_call", lambda: built.append(1))
    module.build()
    assert built == [1]                      # a module that is not known to be this torch's
    module.build()
    assert built == [1]
    (torch / "version.py").write_text("__version__ = '2'\n")
    module.build()
    module.build()
    assert built == [1, 1]
    monkeypatch.setattr(module.sysconfig, "get_config_var", lambda name: "another")
    module.build()
    assert built == [1, 1, 1]
