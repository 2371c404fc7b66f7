"""What qk_norm_rope and cache_keep do around the library's calls: device,
stream, the tensors they make and the arguments they refuse (no GPU here)."""
import importlib.machinery
import importlib.util
import os
import subprocess

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    """(the module of the operators, the module that drives its stand-in library)"""
    from draft_vocab_lm_gb300 import build
    folder = str(tmp_path_factory.mktemp("cache"))
    objs = []
    for src in (os.path.join(build.CSRC, "step_binding.cc"), os.path.join(ROOT, "tests", "cache_host.cc")):
        obj = os.path.join(folder, os.path.basename(src) + ".o")
        cmd = ["-O0" if x == "-O2" else x for x in build._step_compile(obj)]
        cmd[cmd.index("-c") + 1] = src
        objs.append((subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True), obj))
    for p, _ in objs:
        out, _ = p.communicate()
        assert p.returncode == 0, out
    so = os.path.join(folder, "_step.so")
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


class FakeCache:
    def __init__(self, dev):
        from draft_vocab_lm_gb300._native import DvlKVCache
        import ctypes
        self._struct = DvlKVCache(0, 8, 16, 2, 64, 0, 0x1000, 0x2000, 2048, 128, 64, 2048, 128, 64, 1.0, 1.0)
        self._address, self._dev = ctypes.addressof(self._struct), dev


class FakeRope:
    def __init__(self, drive, dev, dim=64):
        self.freq, self.dim, self.interleaved = drive.tensor(0x9000, (dim // 2,), torch.int64, dev), dim, False


def arguments(drive, dev, op):
    def t(shape, dtype=torch.int32, at=0x30000):
        return drive.tensor(at, shape, dtype, dev)
    if op == "qk_norm_rope":
        q, kv = t((6, 4, 64), torch.bfloat16), t((6, 2, 64), torch.bfloat16)
        return [q, kv, kv], dict(rope=FakeRope(drive, dev), cache=FakeCache(dev), table=t((3, 4)), lengths=t((3,)))
    return [FakeCache(dev), t((3, 4)), t((3,)), t((3,)), t((3, 7)), t((3,))], {}


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


OPS = ["qk_norm_rope", "cache_keep"]


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("current,other", [(64, None), (64, 128), (0, 128), (64, 0)])
@pytest.mark.parametrize("wrap", [int, Stream])
def test_device_stream_and_what_is_made(host, op, current, other, wrap):
    step, drive = host
    args, kw = arguments(drive, 1, op)
    drive.state(0, current)
    getattr(step, op)(*args, **kw, stream=None if other is None else wrap(other))
    on = current if other is None else other
    made = [f"empty device 1 stream {on}"] + ([] if on == current else [f"record device 1 stream {current}"])
    assert drive.events() == (made + [f"{op} device 1 stream {on}"], 0, current)


def refuse(host, op, change, says):
    step, drive = host
    args, kw = arguments(drive, 0, op)
    kw.update(change(drive, args) or {})
    drive.state(0, 64)
    with pytest.raises(ValueError, match=says):
        getattr(step, op)(*args, **kw)
    events, device, stream = drive.events()
    assert device == 0 and stream == 64 and not any(op in e for e in events)


@pytest.mark.parametrize("name,shape,dtype,dev", [
    ("q_weight", (63,), torch.bfloat16, 0), ("k_weight", (64,), torch.float32, 0), ("positions", (5,), torch.int32, 0),
    ("positions", (6,), torch.int64, 0), ("table", (3, 4), torch.int64, 0), ("table", (4, 4), torch.int32, 0),
    ("lengths", (2,), torch.int32, 0), ("lengths", (3,), torch.int32, 1), ("starts", (3,), torch.int32, 0),
    ("q_out", (6, 4, 32), torch.bfloat16, 0), ("q_out", (6, 4, 64), torch.float32, 0),
    ("k_out", (6, 4, 64), torch.bfloat16, 0), ("k_out", (6, 2, 64), torch.bfloat16, 1),
])
def test_rope_tensors_of_another_kind(host, name, shape, dtype, dev):
    refuse(host, "qk_norm_rope", lambda d, a: {name: d.tensor(0x50000, shape, dtype, dev)}, "must be")


@pytest.mark.parametrize("i,shape,dtype,dev", [
    (0, (6, 4), torch.bfloat16, 0), (1, (6, 2, 32), torch.bfloat16, 0), (1, (5, 2, 64), torch.bfloat16, 0),
    (2, (6, 3, 64), torch.bfloat16, 0), (2, (6, 2, 64), torch.float16, 0), (1, (6, 2, 64), torch.bfloat16, 1),
])
def test_rope_inputs_of_another_kind(host, i, shape, dtype, dev):
    def change(d, args):
        args[i] = d.tensor(0x50000, shape, dtype, dev)
    refuse(host, "qk_norm_rope", change, "must be")


def test_rope_arguments_that_go_together(host):
    for name in ("table", "lengths"):
        refuse(host, "qk_norm_rope", lambda d, a: {name: None}, "goes with")
    refuse(host, "qk_norm_rope", lambda d, a: {"cache": None}, "go with a cache")
    refuse(host, "qk_norm_rope", lambda d, a: a.__setitem__(2, None), "goes with v")
    refuse(host, "qk_norm_rope", lambda d, a: {"cache": FakeCache(1)}, "on q's device")
    refuse(host, "qk_norm_rope", lambda d, a: {"rope": FakeRope(d, 1)}, "on q's device")
    refuse(host, "qk_norm_rope", lambda d, a: {"rope": FakeRope(d, 0, 80)}, "more values than a head")
    refuse(host, "qk_norm_rope", lambda d, a: {"rope": 3}, "must be a Rope")
    refuse(host, "qk_norm_rope", lambda d, a: {"cache": 3}, "must be a KVCache")

    def alone(d, a):
        a[2] = None
        return dict(cache=None, table=None, lengths=None)
    refuse(host, "qk_norm_rope", alone, "goes with positions")

    def batched(d, a):
        a[0], a[1], a[2] = (d.tensor(0x30000, (3, 2, h, 64), torch.bfloat16, 0) for h in (4, 2, 2))
        return dict(starts=d.tensor(0x50000, (4,), torch.int32, 0))
    refuse(host, "qk_norm_rope", batched, "goes with q as")


def test_rope_with_the_rows_as_sequences_and_tokens(host):
    step, drive = host
    _, kw = arguments(drive, 0, "qk_norm_rope")
    q, k = (drive.tensor(0x30000, (3, 2, h, 64), torch.bfloat16, 0) for h in (4, 2))
    out, k_out = step.qk_norm_rope(q, k, k, **kw)
    assert out.shape == q.shape and k_out is None
    out, k_out = step.qk_norm_rope(q, k, positions=drive.tensor(0x40000, (3, 2), torch.int32, 0), rope=kw["rope"])
    assert out.shape == q.shape and k_out.shape == k.shape


@pytest.mark.parametrize("i,shape,dtype", [
    (1, (3,), torch.int32), (1, (3, 4), torch.int64), (2, (4,), torch.int32), (3, (3,), torch.int64),
    (4, (2, 7), torch.int32), (4, (3, 7), torch.int64), (5, (3, 1), torch.int32),
])
def test_keep_tensors_of_another_kind(host, i, shape, dtype):
    def change(d, args):
        args[i] = d.tensor(0x50000, shape, dtype, 0)
    refuse(host, "cache_keep", change, "must be")
    refuse(host, "cache_keep", lambda d, a: {"lengths_out": d.tensor(0x50000, shape + (2,), dtype, 0)}, "must be")


@pytest.mark.parametrize("op", OPS)
def test_wrong_argument_lists(host, op):
    step, drive = host
    args, kw = arguments(drive, 0, op)
    with pytest.raises(TypeError):
        getattr(step, op)(*args, *args)
    with pytest.raises(TypeError):
        getattr(step, op)(*args, **kw, no_such=1)
    with pytest.raises(ValueError):
        getattr(step, op)(*args[:1])
