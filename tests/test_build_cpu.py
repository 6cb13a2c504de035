"""What build() compiles and in which order, with the compilers replaced by a fake."""
import os
import subprocess
import sys

import pytest

from exact_attention_40_gb300 import build


class Compilers:
    """Stands in for subprocess.run: notes what is made, and fails for `broken`."""

    def __init__(self):
        self.made, self.broken = [], None

    def __call__(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).split(".tmp")[0]
        if name == self.broken:
            return subprocess.CompletedProcess(cmd, 1, "", "no such thing")
        with open(out, "w") as f:
            f.write(name)
        self.made.append(name)
        return subprocess.CompletedProcess(cmd, 0, "", "")


@pytest.fixture
def box(tmp_path, monkeypatch):
    """An empty place to build into, on a machine with torch and Python's headers."""
    torch = tmp_path / "torch"
    (torch / "include" / "ATen").mkdir(parents=True)
    (torch / "include" / "ATen" / "ATen.h").write_text("")
    (torch / "version.py").write_text("__version__ = '1'")
    python = tmp_path / "python"
    python.mkdir()
    (python / "Python.h").write_text("")
    fake = Compilers()
    fake.torch, fake.python, fake.lib = torch, python, tmp_path / "libexattn.so"
    fake.binding = tmp_path / "_binding.so"
    monkeypatch.setattr(build, "LIB", str(fake.lib))
    monkeypatch.setattr(build, "BINDING", str(fake.binding))
    monkeypatch.setattr(build, "BINDING_KEY", str(tmp_path / "_build" / "binding.key"))
    monkeypatch.setattr(build, "_torch_dir", lambda: str(torch))
    monkeypatch.setattr(build, "_python_include", lambda: str(python))
    monkeypatch.setattr(build.subprocess, "run", fake)
    return fake


OBJECTS = {src.replace(".cu", ".o") for src in build.SOURCES}


def test_all_is_built_once(box):
    assert build.build() == str(box.lib)
    assert set(box.made) == OBJECTS | {"libexattn.so", "binding.o", "_binding.so"}
    assert box.made.index("libexattn.so") < box.made.index("_binding.so")
    box.made.clear()
    build.build()
    assert box.made == []
    build.build(force=True)
    assert len(box.made) == len(OBJECTS) + 3


@pytest.mark.parametrize("missing", ["Python.h", "ATen.h", "torch"])
def test_without_the_bindings_headers_the_library_is_built_alone(box, monkeypatch, missing):
    if missing == "torch":
        monkeypatch.setattr(build, "_torch_dir", lambda: None)
    else:
        (box.python / missing if missing == "Python.h" else box.torch / "include" / "ATen" / missing).unlink()
    for force in (False, True):
        box.made.clear()
        assert build.build(force) == str(box.lib)
        assert set(box.made) == OBJECTS | {"libexattn.so"}
    box.made.clear()
    build.build()
    assert box.made == [] and not box.binding.exists()


@pytest.mark.parametrize("broken", ["binding.o", "_binding.so"])
def test_a_binding_that_does_not_build_is_reported_once_the_library_is_there(box, broken):
    box.broken = broken
    for _ in range(2):
        with pytest.raises(RuntimeError, match="no such thing"):
            build.build()
        assert box.lib.exists() and not box.binding.exists()
    assert box.made.count("libexattn.so") == 1  # the second time only the binding is tried
    box.broken = None
    build.build()
    assert box.binding.exists()


def test_another_torch_rebuilds_the_binding(box):
    build.build()
    box.made.clear()
    (box.torch / "version.py").write_text("__version__ = '2'")
    build.build()
    assert set(box.made) == {"binding.o", "_binding.so"}
    box.made.clear()
    build.build()
    assert box.made == []


def test_a_library_that_does_not_build_is_reported(box):
    box.broken = "rope.o"
    with pytest.raises(RuntimeError, match="rope.cu"):
        build.build()
    assert not box.lib.exists()


def test_calls_say_what_they_lack_without_the_binding(monkeypatch):
    pytest.importorskip("torch")
    build.build()
    import exact_attention_40_gb300 as package
    from exact_attention_40_gb300 import exattn
    monkeypatch.setattr(exattn, "_native", None)
    monkeypatch.delattr(package, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, "exact_attention_40_gb300._binding", None)
    with pytest.raises(ImportError, match="python -m exact_attention_40_gb300.build"):
        exattn.attn_rope_axes(None, None, None, (32,))
