"""The drafting step's operators run on their tensors' device, whichever is
current, and leave the current one as it was (no GPU here: step_host)."""
import ctypes

import pytest

import step_host

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return step_host.load(str(tmp_path_factory.mktemp("step")))


class FakeCache:
    """What the module reads of a KVCache."""

    def __init__(self, device):
        from draft_vocab_lm_gb300._native import DvlKVCache
        self._struct = DvlKVCache(0, 8, 16, 2, 64, 0, 0x1000, 0x2000, 2048, 128, 64, 2048, 128, 64, 1.0, 1.0)
        self._address, self._dev = ctypes.addressof(self._struct), device


def arguments(t, dev):
    """Positional and keyword arguments of a complete call of each operator on device `dev`."""
    def x(shape, dtype):
        return t(0x10000, shape, dtype, dev)

    bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    return {
        "add_rmsnorm": ((x((4, 64), bf), x((64,), bf)), dict(out=x((4, 64), bf))),
        "paged_attention": ((FakeCache(dev), x((2, 1, 4, 64), bf), x((2, 3), i32), x((2,), i32)),
                            dict(out=x((2, 1, 4, 64), bf), lse=x((2, 1, 4), f32), ws=x((4096,), u8))),
        "beam_select": ((x((2, 3, 100), f32), x((2, 3), f32), 4),
                        dict(out_scores=x((2, 4), f32), parents=x((2, 4), i32), tokens=x((2, 4), i32),
                             ws=x((4096,), u8))),
        "beam_reorder": ((x((2, 3), i32), [x((2, 3, 8), f32)]), dict(states_out=[x((2, 3, 8), f32)])),
    }


OPERATORS = ("add_rmsnorm", "paged_attention", "beam_select", "beam_reorder")


@pytest.mark.parametrize("op", OPERATORS)
@pytest.mark.parametrize("current,dev", [(0, 0), (0, 1), (1, 0), (3, 2)])
def test_calls_run_on_the_tensors_device(host, op, current, dev):
    step, drive = host
    args, kw = arguments(drive.tensor, dev)[op]
    drive.state(current, 0)
    getattr(step, op)(*args, **kw)
    assert drive.events() == ([f"{op} device {dev} stream 0"], current, 0)


@pytest.mark.parametrize("op", OPERATORS)
def test_a_refusal_leaves_the_current_device(host, op):
    step, drive = host
    args, kw = arguments(drive.tensor, 1)[op]
    name = {"add_rmsnorm": "out", "paged_attention": "out", "beam_select": "tokens", "beam_reorder": "states_out"}[op]
    other = arguments(drive.tensor, 0)[op][1][name]  # an output on another device
    drive.state(0, 0)
    with pytest.raises(ValueError):
        getattr(step, op)(*args, **dict(kw, **{name: other}))
    assert drive.events() == ([], 0, 0)


def test_workspaces_are_made_on_their_device(monkeypatch):
    from draft_vocab_lm_gb300 import step
    seen = []

    class On:
        def __init__(self, device):
            self.device = torch.device(device)

        def __enter__(self):
            seen.append(self.device.index)

        def __exit__(self, *_):
            seen.pop()

    class Lib:
        def dvl_attention_workspace_bytes(self, *_):
            assert seen == [1]  # its grid is the current device's
            return 4096

        def dvl_beam_workspace_bytes(self, *_):
            return 4096

    class Bytes:
        def __init__(self, n, dtype, device):
            self.n, self.device = n, torch.device(device)

        def record_stream(self, _):
            pass

    zeroed = []
    monkeypatch.setattr(step, "lib", Lib)
    monkeypatch.setattr(step, "workspace_init", lambda ws, stream: zeroed.append((seen[-1], ws.device.index)))
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(torch, "empty", Bytes)
    cache = type("Cache", (), {"_struct": None, "device": torch.device("cuda:1")})()
    assert step.attention_workspace(cache, 1, 1, 4).device.index == 1
    assert step._beam_workspace_on(1, 4, 100, 2).device.index == 2
    assert zeroed == [(1, 1), (2, 2)] and seen == []
