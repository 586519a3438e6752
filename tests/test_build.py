"""When build() compiles what: the C library from its sources alone, the torch binding for the torch and Python in use.

The compilers are stand-ins that only leave the file they were asked for; a folder of the test's own takes the results.
"""
import importlib.util
import os
import subprocess
import sys
import sysconfig
import types

import pytest

from chunked_gated_delta_prepare_gb300 import build


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """The outputs of the compiler runs since the last look at it."""
    made = []

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        made.append(os.path.basename(out).split(".tmp")[0])
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=run))
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libgdr.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_gdr_layer.so"))

    def look():
        now = sorted(made)
        made.clear()
        return now
    return look


def test_a_second_build_compiles_nothing(compiled):
    build.build()
    first = compiled()
    assert "libgdr.so" in first and "_gdr_layer.so" in first and len(first) == len(build._sources()) + 3
    build.build()
    assert compiled() == []


def test_the_library_builds_without_torch(compiled, tmp_path):
    """In an interpreter that has the standard library alone, on the results of a build that lack the binding."""
    build.build()
    (tmp_path / "_gdr_layer.so").unlink()
    script = f"""
import importlib.util, sys
spec = importlib.util.spec_from_file_location("build", {build.__file__!r})
build = importlib.util.module_from_spec(spec)
spec.loader.exec_module(build)
build.BUILD, build.LIB, build.BINDING = {build.BUILD!r}, {build.LIB!r}, {build.BINDING!r}
build._nvcc = lambda: "/usr/local/cuda/bin/nvcc"
assert build.build() == build.LIB
"""
    ran = subprocess.run([sys.executable, "-I", "-S", "-c", script], capture_output=True, text=True)
    assert ran.returncode == 0, ran.stderr
    assert not os.path.exists(build.BINDING)


def test_the_binding_is_compiled_again_for_another_torch(compiled, monkeypatch, tmp_path):
    build.build()
    compiled()
    other = tmp_path / "elsewhere" / "torch"
    other.mkdir(parents=True)
    (other / "__init__.py").touch()
    (other / "version.py").write_text("__version__ = '0.0.1'\n")
    found = importlib.util.find_spec("torch")
    spec = types.SimpleNamespace(origin=str(other / "__init__.py"))
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else None)
    build.build()
    assert compiled() == ["_gdr_layer.so", "layer_binding.o"]
    build.build()
    assert compiled() == []
    (other / "version.py").write_text("__version__ = '0.0.2'\n")            # the same place, another version
    build.build()
    assert compiled() == ["_gdr_layer.so", "layer_binding.o"]
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: found)
    build.build()
    assert compiled() == ["_gdr_layer.so", "layer_binding.o"]


def test_the_binding_is_compiled_again_for_another_python(compiled, monkeypatch):
    build.build()
    compiled()
    here = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399" if name == "SOABI" else here(name))
    build.build()
    assert compiled() == ["_gdr_layer.so", "layer_binding.o"]
    build.build()
    assert compiled() == []
