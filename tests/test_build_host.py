"""When the build is due, and what it builds against, on stand-ins for the
compiled files and for torch; CPU only, nothing is compiled."""

import importlib.util
import os
import time

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(ROOT, "newton_schulz_shape_gb300", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for name in ("csrc", "include", "_build"):
        (tmp_path / name).mkdir()
    (tmp_path / "csrc" / "a.cu").write_text("")
    (tmp_path / "include" / "nsgb300.h").write_text("")
    for name, path in (("CSRC", "csrc"), ("INCLUDE", "include"), ("BUILD", "_build"), ("LIB", "lib.so"), ("BINDING", "_training.so")):
        monkeypatch.setattr(mod, name, str(tmp_path / path))
    return mod


def fake_torch(tmp_path, monkeypatch, build, cuda=True, version="1.0"):
    d = tmp_path / "torch"
    (d / "lib").mkdir(parents=True, exist_ok=True)
    (d / "__init__.py").write_text("")
    (d / "version.py").write_text(f"__version__ = {version!r}\n")
    if cuda:
        (d / "lib" / "libc10_cuda.so").write_text("")
    spec = importlib.util.spec_from_file_location("torch", str(d / "__init__.py"))
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: spec if name == "torch" else None)


def pretend_to_build(build, monkeypatch):
    """build(), with every compiler command replaced by writing its output."""
    def run(cmd, what):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(what)
        return ""
    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "_nvcc", lambda: "/nowhere/bin/nvcc")
    build.build()
    later = time.time() + 100                      # newer than this file and the sources
    for f in (build.LIB, build.BINDING):
        if os.path.exists(f):
            os.utime(f, (later, later))


def test_a_torch_without_cuda_builds_the_library_alone(build, tmp_path, monkeypatch):
    fake_torch(tmp_path, monkeypatch, build, cuda=False)
    pretend_to_build(build, monkeypatch)
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert not build._stale()


def test_without_torch_too(build, monkeypatch):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    pretend_to_build(build, monkeypatch)
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert not build._stale()


def test_a_torch_with_cuda_builds_the_binding(build, tmp_path, monkeypatch):
    fake_torch(tmp_path, monkeypatch, build)
    pretend_to_build(build, monkeypatch)
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING)
    assert not build._stale()
    os.remove(build.BINDING)
    assert build._stale()


def test_entry_point_imports_what_was_built(monkeypatch):
    # the package alone where there is no binding
    import builtins

    import __graft_entry__ as entry
    seen = []
    real = builtins.__import__

    def record(name, *args, **kwargs):
        if name.startswith("newton_schulz_shape_gb300"):
            seen.append(name)
        return real(name, *args, **kwargs)

    class Stub:
        BINDING = "/nowhere/_training.so"

        @staticmethod
        def build():
            pass
    monkeypatch.setattr(importlib.util, "module_from_spec", lambda spec: Stub)
    monkeypatch.setattr(importlib.util, "spec_from_file_location", lambda *a: type("S", (), {"loader": type("L", (), {"exec_module": staticmethod(lambda m: None)})}))
    monkeypatch.setattr(builtins, "__import__", record)
    entry.build()
    monkeypatch.undo()
    assert seen and "newton_schulz_shape_gb300.training" not in seen


def test_another_torch_or_python_makes_the_binding_stale(build, tmp_path, monkeypatch):
    fake_torch(tmp_path, monkeypatch, build)
    pretend_to_build(build, monkeypatch)
    assert not build._stale()
    fake_torch(tmp_path, monkeypatch, build, version="1.1")
    assert build._stale()
    pretend_to_build(build, monkeypatch)
    assert not build._stale()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399-nowhere" if name == "SOABI" else None)
    assert build._stale()
    pretend_to_build(build, monkeypatch)
    assert not build._stale()


def test_a_binding_of_unknown_origin_is_stale(build, tmp_path, monkeypatch):
    fake_torch(tmp_path, monkeypatch, build)
    pretend_to_build(build, monkeypatch)
    for f in os.listdir(build.BUILD):
        os.remove(os.path.join(build.BUILD, f))
    assert build._stale()
