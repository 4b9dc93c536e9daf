"""The compiled argument checks as a file: which torch and interpreter they
belong to (no GPU needed; the compiler is a stand-in)."""

import os
import sysconfig
import types

import pytest
import torch


@pytest.fixture()
def built(monkeypatch, tmp_path):
    """(build module, package, list of compiler calls), the package's file being
    one in tmp_path; the stand-in compiler writes an empty output."""
    import paged_kv_cache_50_gb300 as pa
    from paged_kv_cache_50_gb300 import build
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=run))
    monkeypatch.setattr(pa, "BINDING_PATH", str(tmp_path / os.path.basename(pa.BINDING_PATH)))
    return build, pa, calls


def test_the_file_names_its_torch_and_interpreter():
    import paged_kv_cache_50_gb300 as pa
    name = os.path.basename(pa.BINDING_PATH)
    assert f"torch-{torch.__version__}" in name
    assert name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def test_checks_of_another_torch_are_not_current(built, monkeypatch):
    build, pa, calls = built
    assert build.build_binding() == pa.BINDING_PATH and len(calls) == 1
    assert build.build_binding() == pa.BINDING_PATH and len(calls) == 1     # current
    there = pa.BINDING_PATH
    other = there.replace(torch.__version__, "9.9.9+cu999")
    assert other != there
    monkeypatch.setattr(pa, "BINDING_PATH", other)
    assert build.build_binding() == other and len(calls) == 2
    assert os.path.exists(there) and os.path.exists(other)


def test_checks_of_another_torch_are_not_loaded(built, monkeypatch):
    build, pa, calls = built
    build.build_binding()
    monkeypatch.setattr(pa, "_steps", None)
    monkeypatch.setattr(pa, "BINDING_PATH",
                        pa.BINDING_PATH.replace(torch.__version__, "9.9.9+cu999"))
    with pytest.raises(RuntimeError, match="is missing: build it"):
        pa._binding()


def test_library_alone_builds_without_python_headers(built, monkeypatch, tmp_path):
    """libpa.so, and a warning instead of an error for the checks."""
    build, pa, calls = built
    made = []
    monkeypatch.setattr(build, "_build_lib", lambda lib, *rest: made.append(lib))
    assert build.binding_headers_missing() == ""
    build.build()
    assert made == [build.LIB] and len(calls) == 1
    monkeypatch.setattr(build, "sysconfig", types.SimpleNamespace(
        get_paths=lambda: {"include": str(tmp_path)}))
    os.remove(pa.BINDING_PATH)
    with pytest.warns(RuntimeWarning, match="Python.h is missing"):
        assert build.build() == build.LIB
    assert made == [build.LIB] * 2 and len(calls) == 1


def test_first_callers_load_the_checks_once(monkeypatch):
    """Two threads that both find them not loaded yet."""
    import importlib.machinery
    import threading

    import paged_kv_cache_50_gb300 as pa
    from paged_kv_cache_50_gb300 import build
    build.build()
    real, loads, both = importlib.machinery.ExtensionFileLoader.exec_module, [], []
    lib, meet = pa.lib(), threading.Barrier(2)

    def exec_module(self, module):
        loads.append(1)
        return real(self, module)

    def first(*args):      # both are past the unlocked test when they come here
        meet.wait(timeout=60)
        return lib

    monkeypatch.setattr(importlib.machinery.ExtensionFileLoader, "exec_module", exec_module)
    monkeypatch.setattr(pa, "_steps", None)
    monkeypatch.setattr(pa, "lib", first)
    threads = [threading.Thread(target=lambda: both.append(pa._binding())) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(loads) == 1 and both[0] is both[1] and pa._steps is both[0]
