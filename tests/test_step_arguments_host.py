"""Arguments of the drafting step's operators that are no numbers, truth values
or streams (no GPU here: step_host)."""
import pytest

import step_host
from test_step_device_host import arguments

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return step_host.load(str(tmp_path_factory.mktemp("step")))


class NoTruth:
    def __bool__(self):
        raise LookupError("no truth value")


@pytest.mark.parametrize("op,kw,error", [
    ("add_rmsnorm", dict(bf16=NoTruth()), LookupError), ("add_rmsnorm", dict(eps="x"), TypeError),
    ("add_rmsnorm", dict(fp8_group=1.5), TypeError), ("add_rmsnorm", dict(stream="x"), TypeError),
    ("add_rmsnorm", dict(no_such=1), TypeError), ("paged_attention", dict(want_lse=NoTruth()), LookupError),
    ("paged_attention", dict(scale="x"), TypeError), ("beam_select", dict(k=4), TypeError),
    ("beam_reorder", dict(states=[]), TypeError),
])
def test_the_arguments_own_error_comes_out(host, op, kw, error):
    step, drive = host
    args, outs = arguments(drive.tensor, 0)[op]
    outs.pop("lse", None)
    drive.state(0, 0)
    with pytest.raises(error):
        getattr(step, op)(*args, **outs, **kw)
    assert not any(e.startswith(op) for e in drive.events()[0])


@pytest.mark.parametrize("bf16,wanted", [(True, True), (1, True), (None, True), (False, False), ([], False)])
def test_truth_values(host, bf16, wanted):
    step, drive = host
    (x, w), _ = arguments(drive.tensor, 0)["add_rmsnorm"]
    drive.state(0, 0)
    assert (step.add_rmsnorm(x, w, bf16=bf16, fp8_group=0)[0] is not None) == wanted
