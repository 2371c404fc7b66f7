"""What the drafting step's operators allocate for themselves belongs to the
stream they run on (no GPU here: step_host)."""
import pytest

import step_host
from test_step_device_host import OPERATORS, FakeCache, arguments

torch = pytest.importorskip("torch")

# outputs and, where there is one, the workspace that a bare call makes
MADE = {"add_rmsnorm": 1, "paged_attention": 2, "beam_select": 3, "beam_reorder": 1}


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return step_host.load(str(tmp_path_factory.mktemp("step")))


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def bare(drive, op, dev):
    """A call of the operator that brings no outputs, but its workspace."""
    args, kw = arguments(drive.tensor, dev)[op]
    return args, {k: v for k, v in kw.items() if k == "ws"}


@pytest.mark.parametrize("op", OPERATORS)
@pytest.mark.parametrize("dev", [0, 1])
@pytest.mark.parametrize("stream", [None, 64, Stream(64)])
def test_on_the_current_stream_outputs_are_its_own(host, op, stream, dev):
    step, drive = host
    args, kw = bare(drive, op, dev)
    drive.state(0, 64)
    getattr(step, op)(*args, **kw, stream=stream)
    assert drive.events() == ([f"empty device {dev} stream 64"] * MADE[op] + [f"{op} device {dev} stream 64"], 0, 64)


@pytest.mark.parametrize("op", OPERATORS)
@pytest.mark.parametrize("current,other", [(64, 128), (0, 128), (64, 0)])
@pytest.mark.parametrize("wrap", [int, Stream])
def test_on_another_stream_outputs_are_that_streams(host, op, current, other, wrap):
    step, drive = host
    args, kw = bare(drive, op, 1)
    drive.state(0, current)
    getattr(step, op)(*args, **kw, stream=wrap(other))
    made = [f"empty device 1 stream {other}", f"record device 1 stream {current}"] * MADE[op]
    assert drive.events() == (made + [f"{op} device 1 stream {other}"], 0, current)


@pytest.mark.parametrize("op", OPERATORS)
def test_a_failed_call_leaves_the_current_stream(host, op):
    step, drive = host
    args, kw = bare(drive, op, 0)
    drive.state(0, 64)
    # an output of the wrong type, found after others were made
    name = {"add_rmsnorm": "codes", "paged_attention": "lse", "beam_select": "tokens", "beam_reorder": "states_out"}[op]
    wrong = drive.tensor(0x30000, (2, 3, 8), torch.int64, 0)
    bad = {name: [wrong] if op == "beam_reorder" else wrong}
    if op == "add_rmsnorm":
        bad["fp8_group"] = 0
    with pytest.raises(ValueError):
        getattr(step, op)(*args, **kw, **bad, stream=128)
    assert drive.events()[1:] == (0, 64)


@pytest.mark.parametrize("op", ["paged_attention", "beam_select"])
def test_a_workspace_of_the_calls_own_is_made_for_its_stream(host, op, monkeypatch):
    import draft_vocab_lm_gb300.step as made_by
    step, drive = host
    asked = []

    def workspace(*_, stream=None):
        asked.append(stream)
        return drive.tensor(0x20000, (4096,), torch.uint8, 0)

    monkeypatch.setattr(made_by, "attention_workspace", workspace)
    monkeypatch.setattr(made_by, "_beam_workspace_on", workspace)
    args, _ = bare(drive, op, 0)
    for stream in (None, 128):
        drive.state(0, 64)
        getattr(step, op)(*args, stream=stream)
    assert asked == [None, 128]


class Torch:
    """The parts of torch that memory for a stream is taken through."""

    uint8 = torch.uint8

    def __init__(self):
        self.log = log = []
        self.now = "current"
        t = self

        class Stream:
            def __init__(self, name, handle):
                self.name, self.cuda_stream, self.device = name, handle, torch.device("cuda:0")

        class Block:
            def record_stream(self, s):
                log.append(("record", s.name))

        class use:
            def __init__(self, s):
                self.s = s

            def __enter__(self):
                self.was, t.now = t.now, self.s.name

            def __exit__(self, *_):
                t.now = self.was

        class cuda:
            pass

        cuda.Stream, cuda.stream = Stream, use
        cuda.current_stream = staticmethod(lambda _: Stream("current", 64))
        cuda.default_stream = staticmethod(lambda _: Stream("default", 0))
        cuda.ExternalStream = staticmethod(lambda handle, device: Stream(f"external {handle}", handle))
        self.cuda, self.device = cuda, torch.device

        def empty(*_, **__):
            log.append(("empty", t.now))
            return Block()

        self.empty = empty


@pytest.mark.parametrize("given,where", [(None, "current"), (64, "current"), (128, "external 128"), (0, "default")])
def test_memory_for_a_stream(monkeypatch, given, where):
    import draft_vocab_lm_gb300 as dvl
    t = Torch()
    monkeypatch.setattr(dvl, "_torch", lambda: t)
    dvl._empty(16, t.uint8, "cuda:0", given)
    assert t.log == [("empty", where)] + ([("record", "current")] if where != "current" else [])
    if given is not None:  # as a stream object
        t = Torch()
        monkeypatch.setattr(dvl, "_torch", lambda: t)
        dvl._empty(16, t.uint8, "cuda:0", t.cuda.Stream("mine" if where != "current" else "current", given))
        assert t.log[0] == ("empty", "mine" if where != "current" else "current")
