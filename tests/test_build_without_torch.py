"""The library builds without PyTorch (a C program's case), and is not built again when it is there.
Host only; nvcc is stood in for."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def module(tmp_path, monkeypatch):
    """rmsnorm_row_b200/build.py on targets of its own, with its compiler and linker counted."""
    spec = importlib.util.spec_from_file_location("build_alone", os.path.join(ROOT, "rmsnorm_row_b200", "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.ran = []
    monkeypatch.setattr(m, "LIB", str(tmp_path / "libfused_norm.so"))
    monkeypatch.setattr(m, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(m, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(m, "_compile", lambda src, verbose: m.ran.append("compile") or src)

    def link(cmd, **kw):
        m.ran.append("link")
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(m.subprocess, "run", link)
    monkeypatch.setattr(m, "nvcc", lambda: "nvcc")
    return m


def test_without_torch(module, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setitem(__import__("sys").modules, "torch", None)  # importing it raises ImportError
    assert module.build() == module.LIB and os.path.exists(module.LIB) and not os.path.exists(module.BINDING)
    assert module.ran.count("link") == 1
    del module.ran[:]
    assert module.build() == module.LIB and module.ran == []


def test_only_the_binding_is_missing(module, monkeypatch):
    made = []
    monkeypatch.setattr(module, "_build_binding", lambda: made.append(1) or open(module.BINDING, "w").close())
    module.build()
    assert made == [1] and "link" in module.ran
    del module.ran[:], made[:]
    module.build()
    assert made == [] and module.ran == []
    os.remove(module.BINDING)
    module.build()
    assert made == [1] and module.ran == []
