"""The package's names can be imported where the library is not built or
PyTorch is missing; calling what needs them says so."""
import os
import shutil
import subprocess
import sys

import pytest

from conftest import ROOT

NAMES = """
import sys
{before}
from draft_vocab_lm_gb300 import *
import draft_vocab_lm_gb300 as d
assert all(n in globals() for n in d.__all__)
write_ranks_txt("ranks.txt", [3, 1])
assert read_ranks_txt("ranks.txt").tolist() == [3, 1]
for call in (add_rmsnorm, paged_attention, beam_select, beam_reorder, d.add_rmsnorm, d.step.beam_select):
    try:
        call(None, None)
    except {error} as e:
        assert "{says}" in str(e), e
    else:
        raise AssertionError("no error")
for module in (d, d.step):
    try:
        module.no_such_name
    except AttributeError:
        pass
    else:
        raise AssertionError("no error")
"""


def run(folder, code, **kw):
    path = os.pathsep.join([str(folder)] + [p for p in os.environ.get("PYTHONPATH", "").split(os.pathsep) if p])
    r = subprocess.run([sys.executable, "-c", code], cwd=folder, env=dict(os.environ, PYTHONPATH=path),
                       capture_output=True, text=True, **kw)
    assert r.returncode == 0, r.stderr


@pytest.fixture()
def unbuilt(tmp_path):
    shutil.copytree(os.path.join(ROOT, "draft_vocab_lm_gb300"), tmp_path / "draft_vocab_lm_gb300",
                    ignore=shutil.ignore_patterns("*.so", "_build", "csrc", "__pycache__"))
    return tmp_path


def test_names_without_the_library(unbuilt):
    run(unbuilt, NAMES.format(before="", error="RuntimeError", says="is missing"))


def test_names_without_pytorch(unbuilt):
    run(unbuilt, NAMES.format(before="sys.modules['torch'] = None", error="ImportError", says="torch"))


def test_names_with_the_library():
    from draft_vocab_lm_gb300 import build
    build.build()
    import draft_vocab_lm_gb300 as d
    import draft_vocab_lm_gb300.step as step
    try:
        op = step._load("add_rmsnorm")
    except ImportError:  # a PyTorch without CUDA
        pytest.skip("the compiled module does not load here")
    assert d.add_rmsnorm is op and vars(d)["add_rmsnorm"] is op and vars(step)["beam_select"] is d.beam_select
    with pytest.raises(ValueError):
        d.add_rmsnorm(None, None)
