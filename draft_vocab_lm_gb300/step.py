"""The drafting step around the head: norm and rotation of the new queries and
keys and their way into a paged key-value cache, attention of the new tokens
over it, residual addition with norm, beam selection, the reordering of what
belongs to a beam, and the cached tokens that a verification keeps
(include/dvl.h has the definitions).

    cache = KVCache(k, v)                          # CUDA [pages][page][heads][D]
    rope = Rope(D, theta=1e6)
    q, _ = qk_norm_rope(q, k_new, v_new, rope=rope, q_weight=wq, k_weight=wk,
                        cache=cache, table=table, lengths=lengths)
    ws = attention_workspace(cache, B, T, Hq)
    o, lse = paged_attention(cache, q, table, lengths, ws=ws)
    h, residual, _, _ = add_rmsnorm(x, weight, residual)
    scores, parents, tokens = beam_select(logits, scores, k, d2t=d2t)
    states, table, lengths = beam_reorder(parents, states, cache=cache, table=table,
                                          lengths=lengths, spare=spare)
    lengths = cache_keep(cache, table, lengths, first, keep, counts)

The operators live in the compiled module _step (csrc/step_binding.cc),
which checks and marshals their arguments in a few hundred nanoseconds; what
is made once -- the cache's handle, the workspaces -- is here.  Output tensors
can be passed in; the ones that are not are allocated.  With `stream`, a call
runs on that stream, after what that stream holds; the caller orders it behind
whatever else makes its inputs.  What the call allocates is that stream's own.
None has a backward pass: their results are detached, also from inputs that
require gradients."""
from __future__ import annotations

import ctypes
import math
import os

from . import _empty, _torch, workspace_init
from ._native import DVL_BF16, DVL_FP8, DVL_NVFP4, DvlKVCache, lib

_OPERATORS = ("add_rmsnorm", "paged_attention", "beam_select", "beam_reorder", "qk_norm_rope", "cache_keep")
__all__ = [*_OPERATORS, "KVCache", "Rope", "attention_workspace", "beam_workspace"]


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
          [D] pool goes in transposed), rows on 16-byte boundaries.  With
          k_blocks and v_blocks an NVFP4 cache: uint8 [pages][page_size]
          [heads][D / 2], two E2M1 codes to a byte (low nibble = even d), D a
          multiple of 64, strides multiples of D / 2.
    k_scale, v_scale: the value of code 1 of an E4M3 cache, the scale of all of
          an NVFP4 one.
    k_blocks, v_blocks: E4M3 (float8_e4m3fn or uint8) [pages][page_size][heads]
          [D / 16], one scale per 16 values; strides an eighth of k's and v's.
    """

    def __init__(self, k, v, *, k_scale: float = 1.0, v_scale: float = 1.0, k_blocks=None, v_blocks=None):
        torch = _t()
        if k_blocks is not None or v_blocks is not None:
            self._nvfp4(k, v, float(k_scale), float(v_scale), k_blocks, v_blocks)
            return
        _need(k.is_cuda and k.dim() == 4 and v.shape == k.shape and v.dtype == k.dtype
              and v.device == k.device, "k and v must be CUDA [pages][page_size][heads][D] tensors alike")
        _need(k.dtype in (torch.bfloat16, torch.float8_e4m3fn, torch.uint8),
              "a cache holds bf16 or E4M3 (float8_e4m3fn or uint8) values")
        _need(k.stride(3) == 1 and v.stride(3) == 1, "the values of a head must be contiguous")
        self.k, self.v = k, v
        self.nvfp4, self.k_blocks, self.v_blocks = False, None, None
        self.fp8 = k.dtype != torch.bfloat16
        _need(self.fp8 or (k_scale == 1.0 and v_scale == 1.0), "scales go with an E4M3 cache")
        self.pages, self.page_size, self.heads, self.D = k.shape
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.device = k.device
        self._struct = DvlKVCache(DVL_FP8 if self.fp8 else DVL_BF16, self.pages, self.page_size,
                                  self.heads, self.D, 0, k.data_ptr(), v.data_ptr(), *k.stride()[:3],
                                  *v.stride()[:3], self.k_scale, self.v_scale, None, None)
        # what the compiled module reads
        self._address = ctypes.addressof(self._struct)
        self._dev = k.get_device()

    def _nvfp4(self, k, v, k_scale, v_scale, k_blocks, v_blocks):
        torch = _t()
        _need(k_blocks is not None and v_blocks is not None, "k_blocks and v_blocks go together")
        _need(k.is_cuda and k.dim() == 4 and v.shape == k.shape and v.device == k.device and
              k.dtype == v.dtype == torch.uint8 and k.shape[3] % 32 == 0,
              "k and v of an NVFP4 cache must be CUDA uint8 [pages][page_size][heads][D / 2] tensors alike, "
              "D a multiple of 64")
        for codes, blocks in ((k, k_blocks), (v, v_blocks)):
            _need(blocks.device == k.device and blocks.dtype in (torch.float8_e4m3fn, torch.uint8) and
                  blocks.shape == (*k.shape[:3], k.shape[3] // 8),
                  "k_blocks and v_blocks must be E4M3 [pages][page_size][heads][D / 16] tensors on k's device")
            # (the stride of an axis of one is nobody's)
            _need(codes.stride(3) == 1 and (blocks.stride(3) == 1 or blocks.shape[3] == 1) and
                  all(n == 1 or s == 8 * t for n, s, t in zip(k.shape[:3], codes.stride(), blocks.stride())),
                  "the values of a head must be contiguous, and the scales' strides an eighth of the codes'")
        self.k, self.v, self.k_blocks, self.v_blocks = k, v, k_blocks, v_blocks
        self.fp8, self.nvfp4 = False, True
        self.pages, self.page_size, self.heads = k.shape[:3]
        self.D = 2 * k.shape[3]
        self.k_scale, self.v_scale = k_scale, v_scale
        self.device = k.device
        strides = [2 * s if n > 1 else 0 for x in (k, v) for n, s in zip(x.shape, x.stride()[:3])]  # in values
        self._struct = DvlKVCache(DVL_NVFP4, self.pages, self.page_size, self.heads, self.D, 0, k.data_ptr(),
                                  v.data_ptr(), *strides, k_scale, v_scale, k_blocks.data_ptr(),
                                  v_blocks.data_ptr())
        self._address = ctypes.addressof(self._struct)
        self._dev = k.get_device()


_inverse = {}  # by its bits


def _inverse_turn(bits: int) -> int:
    """2^bits / (2 pi), within 1, from pi = 16 atan(1/5) - 4 atan(1/239) in integers."""
    if bits not in _inverse:
        one = 1 << (2 * bits + 64)

        def atan(n):  # of 1 / n
            power, total, k = one // n, 0, 0
            while power:
                total += (-1) ** k * (power // (2 * k + 1))
                power //= n * n
                k += 1
            return total

        _inverse[bits] = (one << bits) // (2 * (16 * atan(5) - 4 * atan(239)))
    return _inverse[bits]


def _turns(f: float) -> int:
    """f radians in turns, modulo one, as a signed 64-bit fraction: position x turns,
    modulo one turn, is then an integer product that wraps.  Exact but for its last
    bit, which the quotient of two 64-bit floating-point numbers is not."""
    m, d = f.as_integer_ratio()
    # 64 bits of the fraction, as many as f has above one, and some to round with
    bits = 96 + max(0, math.frexp(f)[1])
    down = d << (bits - 64)
    turns = (2 * m * _inverse_turn(bits) + down) // (2 * down)
    return (turns + (1 << 63)) % (1 << 64) - (1 << 63)


class Rope:
    """The rotation frequencies of a model, for qk_norm_rope.

    dim:   rotated values of a head (its first ones), a multiple of 16.
    theta: pair i turns by theta^(-2 i / dim) radians per position, unless
    freqs: the dim / 2 frequencies themselves, in radians per position.
    interleaved: the pairs are (2i, 2i + 1) instead of (i, i + dim / 2).
    """

    def __init__(self, dim: int, *, theta: float = 10000.0, freqs=None, interleaved: bool = False, device="cuda"):
        torch = _t()
        _need(dim >= 16 and dim % 16 == 0, "dim must be a positive multiple of 16")
        if freqs is None:
            _need(theta > 0 and math.isfinite(theta), "theta must be positive")
            freqs = [theta ** (-2 * i / dim) for i in range(dim // 2)]
        freqs = [float(f) for f in freqs]
        _need(len(freqs) == dim // 2 and all(math.isfinite(f) for f in freqs), "freqs must be dim / 2 finite numbers")
        self.dim, self.interleaved = dim, bool(interleaved)
        # (the copy has ended when this returns: any stream may use it)
        self.freq = torch.tensor([_turns(f) for f in freqs], dtype=torch.int64).to(device)


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
