"""Builds the Python module of the drafting step's operators against
step_host.cc, so that what it does around the library's calls can be watched
without a GPU."""
import importlib.machinery
import importlib.util
import os
import subprocess

from conftest import ROOT


_loaded = []


def load(folder):
    """(the module of the operators, the module that drives it), built in `folder` by the first call."""
    if not _loaded:
        _loaded.append(_load(folder))
    return _loaded[0]


def _load(folder):
    from draft_vocab_lm_gb300 import build
    so = os.path.join(folder, "_step.so")
    objs = []
    for src in (os.path.join(build.CSRC, "step_binding.cc"), os.path.join(ROOT, "tests", "step_host.cc")):
        obj = os.path.join(folder, os.path.basename(src) + ".o")
        cmd = build._step_compile(obj)
        cmd[cmd.index("-c") + 1] = src
        objs.append((subprocess.Popen(["-O0" if x == "-O2" else x for x in cmd], stdout=subprocess.PIPE,
                                      stderr=subprocess.STDOUT, text=True), obj))
    for p, _ in objs:
        out, _ = p.communicate()
        assert p.returncode == 0, out
    link = [x for x in build._step_link(objs[0][1], so) if not x.startswith("-l:")]
    link[link.index(objs[0][1]):link.index(objs[0][1]) + 1] = [o for _, o in objs]
    r = subprocess.run(link + ["-Wl,-Bsymbolic"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def module(name):
        loader = importlib.machinery.ExtensionFileLoader(name, so)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader(name, loader))
        loader.exec_module(m)
        return m

    return module("_step"), module("step_host")
