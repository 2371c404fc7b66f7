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

Like the rest of the binding these only check and marshal arguments.  Output
tensors can be passed in; the ones that are not are allocated.  A step of a
few rows takes about as long on the GPU as its checks take here, so they read
each tensor's properties once."""
from __future__ import annotations

import ctypes

from . import _call_stream, _torch, workspace_init
from ._native import (DVL_BF16, DVL_F32, DVL_FP8, DVL_MAX_STATES, DvlBeamPages, DvlKVCache, DvlNorm,
                      DvlState, check, lib)

__all__ = ["add_rmsnorm", "KVCache", "attention_workspace", "paged_attention", "beam_workspace",
           "beam_select", "beam_reorder"]

_cached = None  # the torch module


def _t():
    global _cached
    if _cached is None:
        _cached = _torch()
    return _cached


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _rows(t, shape, dtypes, dev: int, name: str):
    """Data pointer and row stride of a 2-D tensor whose rows are contiguous."""
    s = t.stride()
    if (t.get_device() != dev or t.dtype not in dtypes or t.shape != shape
            or (s[1] != 1 and shape[1] != 1)):
        raise ValueError(f"{name} must be a CUDA {'/'.join(str(d)[6:] for d in dtypes)} tensor of "
                         f"shape {tuple(shape)} with contiguous rows, on x's device")
    return t.data_ptr(), s[0]


def _flat(t, shape, dtype, dev: int, name: str) -> int:
    """Data pointer of a contiguous tensor."""
    if (t.get_device() != dev or t.dtype != dtype or t.shape != shape
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA {str(dtype)[6:]} tensor of shape "
                         f"{tuple(shape)} on the inputs' device")
    return t.data_ptr()


def add_rmsnorm(x, weight, residual=None, *, eps: float = 1e-6, bf16: bool = True, fp8_group=None,
                out=None, residual_out=None, codes=None, scales=None, stream=None):
    """u = x + residual; y = u * weight / sqrt(mean(u^2) + eps), per row.

    x:         CUDA bf16 [rows][K] (rows may be strided).
    residual:  bf16 or fp32 [rows][K], or None (u = x).
    bf16:      whether y is wanted in bf16.
    fp8_group: None, or the number of values per scale of E4M3 codes of y
               (16, 32, 64, 128, 256; 0: one scale per row).
    Returns (out, residual_out, codes, scales) with None for what was not asked
    for; y ~ codes * scales.  residual_out (u in the residual's type) may be
    the residual itself; codes is float8_e4m3fn (a given one may be uint8)."""
    torch = _t()
    dev = x.get_device()
    _need(dev >= 0 and x.dim() == 2 and weight.dim() == 1, "x must be a CUDA [rows][K] tensor, weight [K]")
    shape = x.shape
    rows, K = shape
    half = (torch.bfloat16,)
    px, sx = _rows(x, shape, half, dev, "x")
    pw = _flat(weight, (K,), torch.bfloat16, dev, "weight")
    pr = sr = pro = sro = 0
    rtype = DVL_BF16
    if residual is not None:
        if residual.dtype == torch.float32:
            rtype = DVL_F32
        pr, sr = _rows(residual, shape, (torch.bfloat16, torch.float32), dev, "residual")
        if residual_out is None:
            residual_out = torch.empty((rows, K), dtype=residual.dtype, device=x.device)
        pro, sro = _rows(residual_out, shape, (residual.dtype,), dev, "residual_out")
    else:
        _need(residual_out is None, "residual_out goes with a residual")
    po = so = pc = sc = ps = 0
    if bf16:
        if out is None:
            out = torch.empty((rows, K), dtype=torch.bfloat16, device=x.device)
        po, so = _rows(out, shape, half, dev, "out")
    else:
        _need(out is None, "out goes with bf16=True")
    if fp8_group is not None:
        _need(fp8_group in (0, 16, 32, 64, 128, 256), "fp8_group must be 0, 16, 32, 64, 128 or 256")
        groups = -(-K // fp8_group) if fp8_group else 1
        if codes is None:
            codes = torch.empty((rows, K), dtype=torch.float8_e4m3fn, device=x.device)
        if scales is None:
            scales = torch.empty((rows, groups), dtype=torch.float32, device=x.device)
        pc, sc = _rows(codes, shape, (torch.float8_e4m3fn, torch.uint8), dev, "codes")
        ps = _flat(scales, (rows, groups), torch.float32, dev, "scales")
    else:
        _need(codes is None and scales is None, "codes and scales go with fp8_group")
    _need(bf16 or fp8_group is not None, "no output asked for")
    if rows:
        st = lib().dvl_add_rmsnorm(
            DvlNorm(rows, K, rtype, fp8_group or 0, eps, px, sx, pw, pr, sr, pro, sro, po, so, pc, sc, ps),
            _call_stream(stream, x))
        if st:
            check("dvl_add_rmsnorm", st)
    return out, residual_out, codes, scales


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
        self._dev = k.get_device()


def attention_workspace(cache: KVCache, B: int, T: int, Hq: int, *, stream=None):
    """A zeroed workspace for paged_attention calls with this cache, T new
    tokens per sequence and Hq query heads (any batch: B is not used)."""
    n = int(lib().dvl_attention_workspace_bytes(cache._struct, T, Hq))
    _need(n > 0, "T or Hq outside the library's limits")
    ws = _t().empty(n, dtype=_t().uint8, device=cache.device)
    workspace_init(ws, stream)
    return ws


def paged_attention(cache: KVCache, q, table, lengths, *, scale=None, out=None, lse=None,
                    want_lse: bool = True, ws=None, stream=None):
    """Attention of the T newest tokens of each sequence over its cached keys
    and values (its own included: lengths counts them).

    q:       bf16 [B][T][Hq][D], or [B][Hq][D] for one token.
    table:   int32 [B][width]: the page of each page_size tokens.
    lengths: int32 [B].
    scale:   of the scores; 1 / sqrt(D) by default.
    Returns (out, lse): bf16 of q's shape and fp32 without the D axis (None
    without want_lse).  An empty sequence, and a token that sees no position,
    give 0 and -inf."""
    torch = _t()
    dev = q.get_device()
    shape = q.shape
    st = q.stride()
    if len(shape) == 4:
        B, T, Hq, D = shape
        sb, stt, sh, sd = st
    elif len(shape) == 3:
        B, Hq, D = shape
        T, stt = 1, 0
        sb, sh, sd = st
    else:
        raise ValueError("q must be [B][T][Hq][D] or [B][Hq][D]")
    if dev != cache._dev or q.dtype != torch.bfloat16 or D != cache.D or sd != 1:
        raise ValueError("q must be bf16 on the cache's device, its last axis the cache's D, contiguous")
    ts = table.shape
    if (table.get_device() != dev or table.dtype != torch.int32 or len(ts) != 2 or ts[0] != B
            or (table.stride(1) != 1 and ts[1] != 1)):
        raise ValueError("table must be a CUDA int32 [B][width] tensor with contiguous rows")
    pl = _flat(lengths, (B,), torch.int32, dev, "lengths")
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(shape[:-1], dtype=torch.float32, device=q.device)
    po = _flat(out, shape, torch.bfloat16, dev, "out")
    pe = _flat(lse, shape[:-1], torch.float32, dev, "lse") if lse is not None else 0
    if ws is None:
        ws = attention_workspace(cache, B, T, Hq, stream=stream)
    _need(ws.get_device() == dev, "ws must be on the cache's device")
    rc = lib().dvl_paged_attention(
        cache._struct, q.data_ptr(), sb if B > 1 else 0, stt if T > 1 else 0, sh if Hq > 1 else 0, B, T, Hq,
        table.data_ptr(), table.stride(0) if B > 1 else 0, ts[1], pl,
        D ** -0.5 if scale is None else scale, po, pe, ws.data_ptr(), ws.numel(),
        _call_stream(stream, q))
    if rc:
        check("dvl_paged_attention", rc)
    return out, lse


def beam_workspace(batch: int, beams: int, N: int, k: int = 1, *, device=None, stream=None):
    """A zeroed workspace for beam_select calls of this size (any k)."""
    n = int(lib().dvl_beam_workspace_bytes(batch, beams, N))
    _need(n > 0, "batch, beams or N outside the library's limits")
    ws = _t().empty(n, dtype=_t().uint8, device=device or "cuda")
    workspace_init(ws, stream)
    return ws


def beam_select(logits, scores, k: int, *, d2t=None, out_scores=None, parents=None, tokens=None,
                ws=None, stream=None):
    """The k best next beams of each request, best first: score(j, n) =
    scores[j] + log_softmax(logits[j])[n].

    logits: CUDA bf16 or fp32 [batch][beams][N], rows contiguous.
    scores: fp32 [batch][beams]; -inf marks a dead beam.
    d2t:    int32 [N] full-vocabulary id of each row, or None (the row).
    Returns (scores fp32, parents int32, tokens int32), each [batch][k]; places
    without a candidate hold (-inf, -1, -1)."""
    torch = _t()
    dev = logits.get_device()
    shape = logits.shape
    st = logits.stride()
    if dev < 0 or len(shape) != 3 or (st[2] != 1 and shape[2] != 1):
        raise ValueError("logits must be a CUDA [batch][beams][N] tensor with contiguous rows")
    batch, beams, N = shape
    if logits.dtype == torch.float32:
        dtype = DVL_F32
    elif logits.dtype == torch.bfloat16:
        dtype = DVL_BF16
    else:
        raise ValueError("logits must be bf16 or fp32")
    p_in = _flat(scores, (batch, beams), torch.float32, dev, "scores")
    pd = _flat(d2t, (N,), torch.int32, dev, "d2t") if d2t is not None else 0
    k = int(k)
    got = (batch, k)
    if out_scores is None:
        out_scores = torch.empty(got, dtype=torch.float32, device=logits.device)
    if parents is None:
        parents = torch.empty(got, dtype=torch.int32, device=logits.device)
    if tokens is None:
        tokens = torch.empty(got, dtype=torch.int32, device=logits.device)
    po = _flat(out_scores, got, torch.float32, dev, "out_scores")
    pp = _flat(parents, got, torch.int32, dev, "parents")
    pt = _flat(tokens, got, torch.int32, dev, "tokens")
    if ws is None:
        ws = beam_workspace(batch, beams, N, k, device=logits.device, stream=stream)
    _need(ws.get_device() == dev, "ws must be on the logits' device")
    if batch:
        rc = lib().dvl_beam_select(logits.data_ptr(), dtype, st[0], st[1], p_in, batch, beams, N, k, pd, po,
                                   pp, pt, ws.data_ptr(), ws.numel(), _call_stream(stream, logits))
        if rc:
            check("dvl_beam_select", rc)
    return out_scores, parents, tokens


def beam_reorder(parents, states=(), *, states_out=None, cache: KVCache | None = None, table=None,
                 table_out=None, lengths=None, lengths_out=None, spare=None, stream=None):
    """Give each new beam its parent's rows: state[b][parents[b][i]] for every
    state, zeros for a parent outside [0, beams).

    parents: int32 [batch][k].
    states:  CUDA tensors [batch][beams][...], contiguous, any dtype.
    With cache, table [batch][beams][width], lengths [batch][beams] and spare
    [batch][k] (int32): the page tables and lengths move the same way, and the
    new beam gets its spare page in place of the parent's partly filled last
    page, with that page's tokens copied (in the cache, in place).
    Returns (states, table, lengths) as new tensors [batch][k][...]; the last
    two None without a cache."""
    torch = _t()
    dev = parents.get_device()
    _need(dev >= 0 and parents.dim() == 2, "parents must be a CUDA int32 [batch][k] tensor")
    batch, k = parents.shape
    p_par = _flat(parents, (batch, k), torch.int32, dev, "parents")
    n = len(states)
    _need(n <= DVL_MAX_STATES, f"at most {DVL_MAX_STATES} states")
    _need(n > 0 or cache is not None, "nothing to reorder")
    beams = states[0].shape[1] if n else table.shape[1]
    if states_out is None:
        states_out = [torch.empty((batch, k) + tuple(s.shape[2:]), dtype=s.dtype, device=s.device)
                      for s in states]
    _need(len(states_out) == n, "states_out must match states")
    items = []
    for s, d in zip(states, states_out):
        tail = s.shape[2:]
        size = s.element_size() * tail.numel()
        _need(size > 0, "a state's rows must not be empty")
        items.append((_flat(s, (batch, beams, *tail), s.dtype, dev, "a state"),
                      _flat(d, (batch, k, *tail), s.dtype, dev, "a state's output"), size, size, size))
    items = (DvlState * n)(*items) if n else None
    pages = None
    if cache is not None:
        _need(table is not None and lengths is not None and spare is not None,
              "a cache goes with table, lengths and spare")
        width = table.shape[-1]
        if table_out is None:
            table_out = torch.empty((batch, k, width), dtype=torch.int32, device=table.device)
        if lengths_out is None:
            lengths_out = torch.empty((batch, k), dtype=torch.int32, device=table.device)
        _need(cache._dev == dev, "the cache must be on the parents' device")
        pages = DvlBeamPages(_flat(table, (batch, beams, width), torch.int32, dev, "table"),
                             _flat(table_out, (batch, k, width), torch.int32, dev, "table_out"),
                             _flat(lengths, (batch, beams), torch.int32, dev, "lengths"),
                             _flat(lengths_out, (batch, k), torch.int32, dev, "lengths_out"),
                             _flat(spare, (batch, k), torch.int32, dev, "spare"), width, 0)
    else:
        _need(table is None and lengths is None and spare is None, "table, lengths and spare go with a cache")
    if batch:
        rc = lib().dvl_beam_reorder(items, n, pages, cache._struct if cache is not None else None, p_par,
                                    batch, beams, k, _call_stream(stream, parents))
        if rc:
            check("dvl_beam_reorder", rc)
    return list(states_out), table_out, lengths_out
