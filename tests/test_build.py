"""The build on the CPU: the library and the Python extension beside it do not depend on each other."""
import os
import sysconfig

import pytest

from exact_attention_staged_gb300 import api, build


@pytest.fixture()
def elsewhere(monkeypatch, tmp_path):
    """Build targets in a folder of their own, with one small translation unit."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfa.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / os.path.basename(build.BINDING)))
    monkeypatch.setattr(build, "SOURCES", ["fa_rope.cu"])
    return tmp_path


def test_the_library_is_linked_where_the_extension_does_not_compile(elsewhere, monkeypatch, capfd):
    (elsewhere / "headers").mkdir()
    real = sysconfig.get_path
    monkeypatch.setattr(sysconfig, "get_path", lambda name, *a, **k: str(elsewhere / "headers")
                        if name == "include" else real(name, *a, **k))
    with open(build.BINDING, "w") as f:
        f.write("of older sources")
    os.utime(build.BINDING, (1, 1))
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert "Python.h" in capfd.readouterr().err
    assert not os.path.exists(build.BINDING)
    # once the headers are there, the extension alone is made
    monkeypatch.setattr(sysconfig, "get_path", real)
    made = os.path.getmtime(build.LIB)
    build.build()
    assert os.path.exists(build.BINDING) and os.path.getmtime(build.LIB) == made


def test_the_library_is_linked_without_a_host_compiler_for_the_extension(elsewhere, monkeypatch, capfd):
    which = build.shutil.which
    monkeypatch.setattr(build.shutil, "which", lambda name, *a, **k: str(elsewhere / "no-such-compiler")
                        if name == "gcc" else which(name, *a, **k))
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert "binding.c" in capfd.readouterr().err


def test_calls_that_need_the_extension_raise_without_it(monkeypatch):
    build.build()
    api.load()
    monkeypatch.setattr(api, "_binding", None)
    exists = os.path.exists
    monkeypatch.setattr(os.path, "exists", lambda p: "_binding" not in str(p) and exists(p))
    with pytest.raises(RuntimeError, match="missing"):
        api._calls()


def test_the_extension_carries_this_interpreters_suffix():
    build.build()
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert suffix != ".so" and build.BINDING == api.BINDING_PATH
    assert build.BINDING.endswith(f"{os.sep}_binding{suffix}")
    api.load()
    assert os.path.samefile(api._calls().__file__, build.BINDING)
