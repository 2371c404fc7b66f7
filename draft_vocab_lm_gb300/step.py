"""The drafting step around the head: attention of the new tokens over a paged
key-value cache, residual addition with norm, beam selection, and the
reordering of what belongs to a beam (include/dvl.h has the definitions).

    cache = KVCache(k, v)                          # CUDA [pages][page][heads][D]
    ws = attention_workspace(cache, B, T, Hq)
    o, lse = paged_attention(cache, q, table, lengths, ws=ws)
    h, residual, _, _ = add_rmsnorm(x, weight, residual)
    scores, parents, tokens = beam_select(logits, scores, k, d2t=d2t)
    states, table, lengths = beam_reorder(parents, states, cache=cache, table=table,
                                          lengths=lengths, spare=spare)

The four operators live in the compiled module _step (csrc/step_binding.cc),
which checks and marshals their arguments in a few hundred nanoseconds; what
is made once -- the cache's handle, the workspaces -- is here.  Output tensors
can be passed in; the ones that are not are allocated.  With `stream`, a call
runs on that stream, after what that stream holds; the caller orders it behind
whatever else makes its inputs.  What the call allocates is that stream's own.
None of the four has a backward pass: their results are detached, also from
inputs that require gradients."""
from __future__ import annotations

import ctypes
import os

from . import _empty, _torch, workspace_init
from ._native import DVL_BF16, DVL_FP8, DvlKVCache, lib

_OPERATORS = ("add_rmsnorm", "paged_attention", "beam_select", "beam_reorder")
__all__ = [*_OPERATORS, "KVCache", "attention_workspace", "beam_workspace"]


def _load(name):
    # The compiled module needs PyTorch; it is loaded with the first use of an
    # operator.  There is no fallback: a missing module raises.
    _torch()
    lib()
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_step.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    from . import _step
    for op in _OPERATORS:
        globals()[op] = getattr(_step, op)
    return globals()[name]


def __getattr__(name):
    if name not in _OPERATORS:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    try:
        return _load(name)
    except (ImportError, OSError, RuntimeError):
        # Naming an operator, as `from .. import *` does, is no use of it: what
        # is missing raises when it is called.
        def later(*args, **kw):
            return _load(name)(*args, **kw)
        later.__name__ = later.__qualname__ = name
        return later


def _t():
    return _torch()


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


class KVCache:
    """A paged key-value cache on one CUDA device.

    k, v: bf16, or E4M3 (float8_e4m3fn, or uint8 codes), each
          [pages][page_size][heads][D]; the D values of a head are
          contiguous, the other strides are free (so a [pages][heads][page]
          [D] pool goes in transposed), rows on 16-byte boundaries.
    k_scale, v_scale: the value of code 1 of an E4M3 cache.
    """

    def __init__(self, k, v, *, k_scale: float = 1.0, v_scale: float = 1.0):
        torch = _t()
        _need(k.is_cuda and k.dim() == 4 and v.shape == k.shape and v.dtype == k.dtype
              and v.device == k.device, "k and v must be CUDA [pages][page_size][heads][D] tensors alike")
        _need(k.dtype in (torch.bfloat16, torch.float8_e4m3fn, torch.uint8),
              "a cache holds bf16 or E4M3 (float8_e4m3fn or uint8) values")
        _need(k.stride(3) == 1 and v.stride(3) == 1, "the values of a head must be contiguous")
        self.k, self.v = k, v
        self.fp8 = k.dtype != torch.bfloat16
        _need(self.fp8 or (k_scale == 1.0 and v_scale == 1.0), "scales go with an E4M3 cache")
        self.pages, self.page_size, self.heads, self.D = k.shape
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.device = k.device
        self._struct = DvlKVCache(DVL_FP8 if self.fp8 else DVL_BF16, self.pages, self.page_size,
                                  self.heads, self.D, 0, k.data_ptr(), v.data_ptr(), *k.stride()[:3],
                                  *v.stride()[:3], self.k_scale, self.v_scale)
        # what the compiled module reads
        self._address = ctypes.addressof(self._struct)
        self._dev = k.get_device()


def _workspace(n: int, device, stream):
    """n zeroed bytes on the device."""
    torch = _t()
    ws = _empty(n, torch.uint8, device, stream)
    with torch.cuda.device(ws.device):
        workspace_init(ws, stream)
    return ws


def attention_workspace(cache: KVCache, B: int, T: int, Hq: int, *, stream=None):
    """A zeroed workspace for paged_attention calls with this cache, T new
    tokens per sequence and Hq query heads (any batch: B is not used)."""
    with _t().cuda.device(cache.device):
        n = int(lib().dvl_attention_workspace_bytes(cache._struct, T, Hq))
        _need(n > 0, "T or Hq outside the library's limits")
        return _workspace(n, cache.device, stream)


def beam_workspace(batch: int, beams: int, N: int, k: int = 1, *, device=None, stream=None):
    """A zeroed workspace for beam_select calls of this size (any k)."""
    n = int(lib().dvl_beam_workspace_bytes(batch, beams, N))
    _need(n > 0, "batch, beams or N outside the library's limits")
    return _workspace(n, device or "cuda", stream)


def _beam_workspace_on(batch: int, beams: int, N: int, device: int, *, stream=None):
    return beam_workspace(batch, beams, N, device=f"cuda:{device}", stream=stream)
