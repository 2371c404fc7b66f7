"""What build() makes, and when it makes it again (compilers are stand-ins that
write down what they are asked for)."""
import os
import subprocess
import types

import pytest


@pytest.fixture()
def b(tmp_path, monkeypatch):
    """The build module over a source tree of its own, with `made` telling what was linked."""
    from draft_vocab_lm_gb300 import build as real
    m = types.ModuleType("build_copy")
    m.__file__ = str(tmp_path / "pkg" / "build.py")
    (tmp_path / "pkg" / "csrc").mkdir(parents=True)
    (tmp_path / "include").mkdir()
    (tmp_path / "torch" / "lib").mkdir(parents=True)
    (tmp_path / "torch" / "lib" / "libc10_cuda.so").write_text("")
    (tmp_path / "torch" / "version.py").write_text("__version__ = '1'\n")
    (tmp_path / "torch" / "__init__.py").write_text("")
    for name in ("csrc/a.cu", "csrc/ranks.cpp", "csrc/step_binding.cc", "csrc/x.cuh", "build.py"):
        (tmp_path / "pkg" / name).write_text("")
    (tmp_path / "include" / "dvl.h").write_text("")
    exec(compile(open(real.__file__).read(), real.__file__, "exec"), m.__dict__)
    m.made, m.torch = [], tmp_path / "torch"

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        if "-c" not in cmd:
            m.made.append(os.path.basename(out).split(".tmp")[0])
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(m, "subprocess", types.SimpleNamespace(run=run))
    monkeypatch.setattr(m, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    spec = types.SimpleNamespace(origin=str(m.torch / "__init__.py"))
    monkeypatch.setattr(m.importlib.util, "find_spec", lambda name: spec if m.torch.exists() else None)
    return m


def touch(b, *path):
    """A file changed after everything that was built."""
    p = os.path.join(os.path.dirname(b.__file__), *path)
    t = max(os.path.getmtime(x) for x in (b.LIB, b.STEP) if os.path.exists(x)) + 10
    os.utime(p, (t, t))


def again(b):
    b.made.clear()
    b.build()
    return b.made


def test_both_are_built_once(b):
    assert b.build() == b.LIB and b.made == ["libdvl.so", "_step.so"]
    assert b.up_to_date() and again(b) == []
    b.made.clear()
    b.build(force=True)
    assert b.made == ["libdvl.so", "_step.so"]


@pytest.mark.parametrize("path,made", [
    (("csrc", "a.cu"), ["libdvl.so"]), (("csrc", "x.cuh"), ["libdvl.so"]), (("csrc", "ranks.cpp"), ["libdvl.so"]),
    (("csrc", "step_binding.cc"), ["_step.so"]), (("..", "include", "dvl.h"), ["libdvl.so", "_step.so"]),
])
def test_a_changed_source_makes_what_it_is_part_of(b, path, made):
    b.build()
    touch(b, *path)
    assert not b.up_to_date() and again(b) == made


@pytest.mark.parametrize("missing", ["torch", "cuda"])
def test_the_library_needs_no_pytorch(b, missing):
    if missing == "torch":
        b.torch.rename(b.torch.with_name("gone"))
    else:
        (b.torch / "lib" / "libc10_cuda.so").unlink()
    assert b.build() == b.LIB and b.made == ["libdvl.so"]
    assert b.up_to_date() and again(b) == []
    # installed later: the module follows, the library stays
    if missing == "torch":
        b.torch.with_name("gone").rename(b.torch)
    else:
        (b.torch / "lib" / "libc10_cuda.so").write_text("")
    assert not b.up_to_date() and again(b) == ["_step.so"]


@pytest.mark.parametrize("what", ["version", "place", "python"])
def test_the_module_is_remade_for_another_pytorch(b, monkeypatch, what):
    b.build()
    if what == "version":
        old = os.path.getmtime(b.torch / "version.py")
        (b.torch / "version.py").write_text("__version__ = '2'\n")
        os.utime(b.torch / "version.py", (old, old))  # an older file than what was built
    elif what == "place":
        other = b.torch.with_name("elsewhere")
        b.torch.rename(other)
        b.torch.mkdir()
        spec = types.SimpleNamespace(origin=str(other / "__init__.py"))
        monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: spec)
    else:
        monkeypatch.setattr(b.sysconfig, "get_config_var", lambda name: "cpython-999")
    assert not b.up_to_date() and again(b) == ["_step.so"]
    assert b.up_to_date() and again(b) == []
