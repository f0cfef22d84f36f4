"""What a build leaves behind when the module of the calls with rotation cannot be built: the library all the same,
and an error that names the module and the tool.  No GPU; one small CUDA source stands for the library's."""
import os
import shutil

import pytest

from decode_attention_append_gb300 import build


@pytest.fixture
def own(tmp_path, monkeypatch):
    if not os.path.exists(build._nvcc()):
        pytest.skip("nvcc unavailable")
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "_build" / "libdaa.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_build" / "_binding.so"))
    monkeypatch.setattr(build, "SOURCES", ["noalloc.cu"])
    return tmp_path


def _tool(path, script):
    path.write_text("#!/bin/sh\n" + script + "\n")
    path.chmod(0o755)
    return str(path)


def _error(own):
    return (own / "_build" / "_binding.error").read_text()


def test_library_without_module(own, monkeypatch, capsys):
    """A compiler that finds no Python.h, then none at all: the library stands, a module of before is taken away, and the
    package's error has the reason."""
    import decode_attention_append_gb300 as daa
    daa.load_library()
    monkeypatch.setattr(build.shutil, "which", _which(_tool(own / "g++", "echo 'fatal error: Python.h: No such file' >&2; exit 1")))
    (own / "_build").mkdir()
    (own / "_build" / "_binding.so").write_text("of another torch")
    lib = build.build()
    assert lib == build.LIB and os.path.getsize(lib) > 0
    assert not os.path.exists(build.BINDING)
    assert "g++ failed" in _error(own) and "Python.h" in _error(own)
    assert "_binding.so is not built" in capsys.readouterr().err
    monkeypatch.setattr(daa, "_native", None)
    monkeypatch.setattr(daa, "_HERE", str(own))
    with pytest.raises(ImportError, match="_binding.so.*g\\+\\+ failed.*Python.h"):
        daa._load_native()
    monkeypatch.setattr(build.shutil, "which", _which(str(own / "none")))
    before = os.path.getmtime(lib)
    assert build.build() == lib and os.path.getmtime(lib) == before
    assert "could not be run" in _error(own)


def test_a_later_build_brings_the_module(own, monkeypatch):
    flags = []
    script = 'while [ $# -gt 0 ]; do if [ "$1" = -o ]; then echo x > "$2"; fi; shift; done'
    monkeypatch.setattr(build.shutil, "which", _which(_tool(own / "g++", script)))
    monkeypatch.setattr(build, "_torch_flags", lambda torch: flags)
    build.build()
    assert os.path.exists(build.BINDING) and not (own / "_build" / "_binding.error").exists()
    os.remove(build.BINDING)
    (own / "_build" / "_binding.error").write_text("of before")
    build.build()
    assert os.path.exists(build.BINDING) and not (own / "_build" / "_binding.error").exists()


def test_a_failing_nvcc_is_named(own, monkeypatch):
    nvcc = _tool(own / "nvcc", "echo no >&2; exit 3")
    monkeypatch.setattr(build, "_nvcc", lambda: nvcc)
    with pytest.raises(RuntimeError, match="nvcc failed.*no"):
        build.build()


_shutil_which = shutil.which


def _which(gxx):
    return lambda name, *a, **k: gxx if name == "g++" else _shutil_which(name, *a, **k)
