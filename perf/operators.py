"""The operators of one drafting step, in their plain form and through the library.

A drafter's step around its LM head: the new tokens' attention over the paged
key-value cache (paged_attention), the residual addition and norm before a
projection or the head (add_rmsnorm), the choice of the next beams from the
head's logits (beam_select) and the reordering of what belongs to a beam
(beam_reorder).  The widths are this library's own (2,560 and 5,120), as are
the vocabulary (248,320) and the shortlists (16,000 and 52,755 rows); head
counts, lengths, pages and beams are generic serving sizes.

`run` computes an operator from elementary torch operations in 32 bits, or,
with `own` true, calls the library's entry points.
"""
import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
E4M3_MAX = 448.0
INF = float("inf")


def listed():
    return [
        # the norm before the head at one draft step: pure latency
        {"name": "norm_draft_step", "op": "norm", "rows": 1, "K": 2560, "residual": "bf16", "bf16": True, "group": -1},
        # a batched verify step that feeds an 8-bit projection: one scale per 128 values
        {"name": "norm_verify_fp8", "op": "norm", "rows": 96, "K": 5120, "residual": "bf16", "bf16": True, "group": 128},
        # prefill: a long ragged batch with the residual stream kept in 32 bits, one scale per row
        {"name": "norm_prefill_fp8", "op": "norm", "rows": 20011, "K": 2560, "residual": "fp32", "bf16": False, "group": 0},
        # one request, one new token, a chat-sized cache: latency
        {"name": "attn_draft_step", "op": "attn", "B": 1, "T": 1, "hq": 20, "hkv": 4, "D": 128, "longest": 731,
         "page": 16, "fp8": False},
        # a verify step of three tokens for a few requests of unequal length
        {"name": "attn_verify3", "op": "attn", "B": 8, "T": 3, "hq": 40, "hkv": 8, "D": 128, "longest": 4101,
         "page": 64, "fp8": False},
        # one request with a very long context, few wide heads: the split over the length carries it
        {"name": "attn_long_context", "op": "attn", "B": 1, "T": 1, "hq": 16, "hkv": 2, "D": 256, "longest": 262139,
         "page": 64, "fp8": False},
        # a full serving batch on an 8-bit cache
        {"name": "attn_batch_fp8", "op": "attn", "B": 64, "T": 1, "hq": 40, "hkv": 8, "D": 128, "longest": 16381,
         "page": 32, "fp8": True},
        # the first step of a beam search on the 16k shortlist: one live beam of four
        {"name": "beam_first_16k", "op": "beam", "batch": 1, "beams": 4, "live": 1, "N": 16000, "k": 4,
         "bf16": False, "d2t": True, "banned": 0.0},
        # a batch on the merged 52,755-row list, bf16 logits as a bf16 projection leaves them (odd row length)
        {"name": "beam_union_bf16", "op": "beam", "batch": 8, "beams": 4, "live": 4, "N": 52755, "k": 8,
         "bf16": True, "d2t": True, "banned": 0.0},
        # the full vocabulary, wide beams, part of the vocabulary banned by a grammar
        {"name": "beam_full_vocab", "op": "beam", "batch": 8, "beams": 8, "live": 8, "N": 248320, "k": 16,
         "bf16": False, "d2t": False, "banned": 0.02},
        # four beams of one request: hidden rows, page tables, the partly filled pages
        {"name": "reorder_one_request", "op": "reorder", "batch": 1, "beams": 4, "state": 0, "K": 2560, "len": 731,
         "hkv": 4, "D": 128, "page": 16, "fp8": False},
        # a batch of wide beams with a recurrent state of 512 KB each
        {"name": "reorder_batch_state", "op": "reorder", "batch": 16, "beams": 8, "state": 8, "K": 2560, "len": 1901,
         "hkv": 8, "D": 128, "page": 64, "fp8": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "attn", "attn", "beam", "reorder"])
    if op == "norm":
        # the library's widths, other multiples of eight, and widths no vector load fits
        K = rng.choice([2560, 5120, 8 * rng.randrange(9, 300), 2 * rng.randrange(40, 1000) + 1])
        rows = 2 * _log_int(rng, 1, 25_000_000 // K if K > 2500 else 10_000) - 1
        bf16, group = rng.choice([(True, -1), (True, 0), (False, 0), (True, 128), (False, 64)])
        return {"op": op, "rows": rows, "K": K, "residual": rng.choice(["none", "bf16", "fp32"]), "bf16": bf16, "group": group}
    if op == "attn":
        D = rng.choice([64, 80, 128, 128, 256])
        hkv, G, T = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 1, 1, 2, 3, 5])
        fp8 = rng.random() < 0.4
        longest, B = _log_int(rng, 1, 60_000), _log_int(rng, 1, 96)
        row = hkv * D * (1 if fp8 else 2)  # one cached token's keys
        B = max(1, min(B, 200_000_000 // (row * longest)))
        return {"op": op, "B": B, "T": T, "hq": hkv * G, "hkv": hkv, "D": D, "longest": longest,
                "page": rng.choice([16, 32, 48, 64, 128]), "fp8": fp8}
    if op == "beam":
        N = rng.choice([16000, 52755, 248320, 2 * _log_int(rng, 200, 60_000) + 1])
        beams = rng.choice([1, 2, 4, 5, 8])
        batch = _log_int(rng, 1, 8)
        return {"op": op, "batch": batch, "beams": beams, "live": rng.randrange(1, beams + 1), "N": N,
                "k": rng.choice([beams, 2 * beams]), "bf16": rng.random() < 0.4, "d2t": rng.random() < 0.5,
                "banned": rng.choice([0.0, 0.0, 0.3])}
    return {"op": op, "batch": _log_int(rng, 1, 16), "beams": rng.choice([2, 3, 4, 8]), "state": rng.choice([0, 0, 1, 4]),
            "K": rng.choice([2560, 5120]), "len": _log_int(rng, 1, 2600), "hkv": rng.choice([1, 2, 4, 8]),
            "D": rng.choice([64, 128, 256]), "page": rng.choice([16, 32, 64]), "fp8": rng.random() < 0.4}


def _plan(case):
    """A generator that depends on the case's sizes alone, for what its work depends on."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """The batch's lengths, the longest among them; prepare() puts them in another order for each seed."""
    r, n = _plan(case), case["longest"]
    return [n] + [r.randint(max(1, n // 8), n) if r.random() > 0.02 else 0 for _ in range(case["B"] - 1)]


def _parents(case):
    """[batch][beams]: parents as a selection leaves them -- the better beams more often, some never, rarely an empty slot."""
    r, n = _plan(case), case["beams"]
    return [[-1 if r.random() < 0.02 else min(r.randrange(n), r.randrange(n)) for _ in range(n)] for _ in range(case["batch"])]


# ---------------------------------------------------------------------------
# What a user's program has in hand
# ---------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _pool(g, pages, page, hkv, D, fp8):
    """One page pool (keys or values) and the value of its code 1."""
    out = torch.empty((pages, page, hkv, D), dtype=FP8 if fp8 else torch.bfloat16, device="cuda")
    step = max(1, (1 << 26) // (page * hkv * D))
    for i in range(0, pages, step):
        part = out[i:i + step]
        part.copy_(_normal(g, *part.shape, std=40.0 if fp8 else 1.0).clamp_(-E4M3_MAX, E4M3_MAX))
    return out, 0.025 if fp8 else 1.0


def _prepare_norm(case, g):
    rows, K, kind = case["rows"], case["K"], case["residual"]
    s = {"x": _normal(g, rows, K).bfloat16(), "weight": (1 + _normal(g, K, std=0.1)).bfloat16(), "eps": 1e-6}
    s["residual"] = None
    if kind != "none":
        s["residual"] = _normal(g, rows, K, std=3.0).to(torch.float32 if kind == "fp32" else torch.bfloat16)
    return s


def _prepare_attn(case, g):
    B, T, page = case["B"], case["T"], case["page"]
    lens = _lengths(case)
    order = torch.randperm(B, generator=g, device="cuda").tolist()
    lens = [lens[i] for i in order]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=g, device="cuda").int()
    width = max(max(need), 1)
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    k, k_scale = _pool(g, pages, page, case["hkv"], case["D"], case["fp8"])
    v, v_scale = _pool(g, pages, page, case["hkv"], case["D"], case["fp8"])
    return {"q": _normal(g, B, T, case["hq"], case["D"], std=2.0).bfloat16(), "k": k, "v": v, "k_scale": k_scale,
            "v_scale": v_scale, "table": table, "lengths": torch.tensor(lens, dtype=torch.int32, device="cuda"),
            "scale": case["D"] ** -0.5}


def _prepare_beam(case, g):
    batch, beams, N = case["batch"], case["beams"], case["N"]
    logits = _normal(g, batch, beams, N, std=1.5)
    # a model's logits: a broad floor and some hundreds of favoured tokens
    likely = torch.rand(logits.shape, generator=g, device="cuda") < 400 / N
    lift = 12.0 * torch.rand(logits.shape, generator=g, device="cuda").square_()
    logits = torch.where(likely, 0.5 * logits + lift, logits)
    if case["banned"]:
        logits.masked_fill_((torch.rand(N, generator=g, device="cuda") < case["banned"]), -INF)
    scores = -8.0 * torch.rand((batch, beams), generator=g, device="cuda").sort(dim=1).values
    scores[:, case["live"]:] = -INF
    d2t = None
    if case["d2t"]:
        V = max(248320, N)
        d2t = torch.randperm(V, generator=g, device="cuda")[:N].sort().values.int()
    return {"logits": logits.bfloat16() if case["bf16"] else logits, "scores": scores, "d2t": d2t, "k": case["k"]}


def _prepare_reorder(case, g):
    batch, beams, page = case["batch"], case["beams"], case["page"]
    n = case["len"]
    full, width = n // page, (n + 31) // page + 1
    # beams of one request share their full pages; each has its own last page, and a spare one
    shared = batch * full
    pages = shared + 2 * batch * beams
    ids = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.zeros((batch, beams, width), dtype=torch.int32, device="cuda")
    table[:, :, :full] = ids[:shared].view(batch, 1, full)
    table[:, :, full] = ids[shared:shared + batch * beams].view(batch, beams)
    k, k_scale = _pool(g, pages, page, case["hkv"], case["D"], case["fp8"])
    v, v_scale = _pool(g, pages, page, case["hkv"], case["D"], case["fp8"])
    states = [_normal(g, batch, beams, case["K"]).bfloat16()]
    if case["state"]:
        states.append(_normal(g, batch, beams, case["state"], 128, 128))
    parents = _parents(case)
    order = torch.randperm(batch, generator=g, device="cuda").tolist()
    return {"states": states, "parents": torch.tensor([parents[i] for i in order], dtype=torch.int32, device="cuda"),
            "k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale, "table": table,
            "lengths": torch.full((batch, beams), n, dtype=torch.int32, device="cuda"),
            "spare": ids[shared + batch * beams:].view(batch, beams).contiguous()}


def prepare(case, seed):
    make = {"norm": _prepare_norm, "attn": _prepare_attn, "beam": _prepare_beam, "reorder": _prepare_reorder}
    return {"case": case, **make[case["op"]](case, _generator(seed))}


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _plain_norm(s):
    case = s["case"]
    u, out = s["x"].float(), {}
    if s["residual"] is not None:
        u = u + s["residual"].float()
        out["residual"] = u.to(s["residual"].dtype)
    y = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    if case["bf16"]:
        out["out"] = y.bfloat16()
    if case["group"] >= 0:
        rows, K = y.shape
        size = case["group"] or K
        groups = -(-K // size)
        y = torch.nn.functional.pad(y, (0, groups * size - K)).view(rows, groups, size)
        amax = y.abs().amax(-1, keepdim=True)
        codes = torch.where(amax > 0, y * (E4M3_MAX / amax), torch.zeros_like(y))
        out["codes"] = codes.view(rows, groups * size)[:, :K].to(FP8)
        out["scales"] = (amax / E4M3_MAX).view(rows, groups)
    return out


def _plain_attn(s):
    case, table = s["case"], s["table"].long()
    B, T, hq, D = s["q"].shape
    hkv, n = case["hkv"], table.shape[1] * case["page"]
    q = s["q"].float().view(B, T, hkv, hq // hkv, D)
    k = s["k"][table].view(B, n, hkv, D).float()
    x = torch.einsum("bthgd,bnhd->bthgn", q, k) * (s["scale"] * s["k_scale"])
    del k
    sees = s["lengths"].view(B, 1) - (T - 1 - torch.arange(T, device="cuda"))  # [B][T]
    seen = torch.arange(n, device="cuda") < sees.view(B, T, 1, 1, 1)
    x = x.masked_fill(~seen, -INF)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -INF, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    v = s["v"][table].view(B, n, hkv, D).float()
    o = torch.einsum("bthgn,bnhd->bthgd", p, v) * s["v_scale"]
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return {"out": o.reshape(B, T, hq, D).bfloat16(), "lse": (m + torch.log(total)).reshape(B, T, hq)}


def _plain_beam(s):
    x, k = s["logits"].float(), s["k"]
    batch, beams, N = x.shape
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    score = (s["scores"].view(batch, beams, 1) + (x - lse)).view(batch, beams * N)
    score = torch.where(torch.isnan(score), torch.full_like(score, -INF), score) + 0.0
    # one whole number per candidate: the score's order first, then the lower index
    bits = score.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    best = torch.topk(order * (1 << 32) + ((1 << 32) - 1 - torch.arange(beams * N, device="cuda")), k).values
    at = (1 << 32) - 1 - (best & ((1 << 32) - 1))
    score = score.gather(1, at)
    none = score == -INF
    token = at % N
    token = s["d2t"][token].long() if s["d2t"] is not None else token
    return {"scores": score, "parents": torch.where(none, -1, at // N).int(), "tokens": torch.where(none, -1, token).int()}


def _plain_reorder(s):
    parents = s["parents"].long()
    batch, beams = parents.shape
    page = s["case"]["page"]
    live = parents >= 0
    rows = (parents.clamp(min=0) + beams * torch.arange(batch, device="cuda").view(-1, 1)).view(-1)

    def moved(x):
        y = x.reshape(batch * beams, -1)[rows]
        return torch.where(live.view(-1, 1), y, torch.zeros_like(y)).view(x.shape)

    lengths = moved(s["lengths"].view(batch, beams, 1)).view(batch, beams)
    table = moved(s["table"])
    slot = (lengths // page).long().clamp(max=table.shape[2] - 1)
    source = table.gather(2, slot.unsqueeze(2)).view(-1).long()
    filled = torch.where(live, lengths % page, torch.zeros_like(lengths)).view(-1, 1, 1, 1)
    spare = s["spare"].view(-1).long()
    copies = torch.arange(page, device="cuda").view(1, page, 1, 1) < filled
    for pool in (s["k"], s["v"]):
        raw = pool.view(torch.uint8)
        raw[spare] = torch.where(copies, raw[source], raw[spare])
    table.scatter_(2, slot.unsqueeze(2), torch.where(live, s["spare"], table.gather(2, slot.unsqueeze(2)).squeeze(2)).unsqueeze(2))
    return {"states": [moved(x) for x in s["states"]], "table": table, "lengths": lengths, "k": s["k"], "v": s["v"]}


# ---------------------------------------------------------------------------
# The library
# ---------------------------------------------------------------------------

def _own(s):
    import draft_vocab_lm_gb300 as dvl

    case = s["case"]
    was = s.setdefault("outputs", {})  # a serving loop's output buffers: made by its first pass, written by every later one
    if case["op"] == "norm":
        group = case["group"] if case["group"] >= 0 else None
        r = dvl.add_rmsnorm(s["x"], s["weight"], s["residual"], eps=s["eps"], bf16=case["bf16"], fp8_group=group,
                            out=was.get("out"), residual_out=was.get("residual"), codes=was.get("codes"),
                            scales=was.get("scales"))
        s["outputs"] = {n: v for n, v in zip(("out", "residual", "codes", "scales"), r) if v is not None}
        return s["outputs"]
    if case["op"] == "beam":
        if "ws" not in s:  # the loop's workspace
            s["ws"] = dvl.beam_workspace(*s["logits"].shape, s["k"])
        r = dvl.beam_select(s["logits"], s["scores"], s["k"], d2t=s["d2t"], out_scores=was.get("scores"),
                            parents=was.get("parents"), tokens=was.get("tokens"), ws=s["ws"])
        s["outputs"] = dict(zip(("scores", "parents", "tokens"), r))
        return s["outputs"]
    if "cache" not in s:  # the loop's handle of its page pool
        s["cache"] = dvl.KVCache(s["k"], s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if case["op"] == "attn":
        if "ws" not in s:
            s["ws"] = dvl.attention_workspace(s["cache"], *s["q"].shape[:3])
        r = dvl.paged_attention(s["cache"], s["q"], s["table"], s["lengths"], scale=s["scale"], out=was.get("out"),
                                lse=was.get("lse"), ws=s["ws"])
        s["outputs"] = dict(zip(("out", "lse"), r))
        return s["outputs"]
    r = dvl.beam_reorder(s["parents"], s["states"], states_out=was.get("states"), cache=s["cache"], table=s["table"],
                         table_out=was.get("table"), lengths=s["lengths"], lengths_out=was.get("lengths"),
                         spare=s["spare"])
    s["outputs"] = dict(zip(("states", "table", "lengths"), r))
    return {**s["outputs"], "k": s["k"], "v": s["v"]}


def run(state):
    if own:
        return _own(state)
    plain = {"norm": _plain_norm, "attn": _plain_attn, "beam": _plain_beam, "reorder": _plain_reorder}
    return plain[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        n, rows, K = case["rows"] * case["K"], case["rows"], case["K"]
        moved = 2 * n + 2 * K + {"none": 0, "bf16": 4, "fp32": 8}[case["residual"]] * n + 2 * n * case["bf16"]
        if case["group"] >= 0:
            moved += n + 4 * rows * (-(-K // (case["group"] or K)))
        return {"bytes": moved, "flops": 6 * n}
    if op == "attn":
        lens, T, hq, D = _lengths(case), case["T"], case["hq"], case["D"]
        size = 1 if case["fp8"] else 2
        pages = sum(-(-n // case["page"]) for n in lens)
        moved = 2 * sum(lens) * case["hkv"] * D * size + case["B"] * T * hq * (4 * D + 4) + 4 * pages + 4 * case["B"]
        return {"bytes": moved, "flops": 4 * hq * D * sum(max(0, n - t) for n in lens for t in range(T))}
    if op == "beam":
        rows, N = case["batch"] * case["beams"], case["N"]
        moved = rows * (N * (2 if case["bf16"] else 4) + 4) + case["batch"] * case["k"] * (12 + 4 * case["d2t"])
        return {"bytes": moved, "flops": 5 * rows * N}
    rows, page = case["batch"] * case["beams"], case["page"]
    read = sum(len({p for p in row if p >= 0}) for row in _parents(case))  # a parent of several beams is read once
    kept = sum(p >= 0 for row in _parents(case) for p in row)
    state = 2 * case["K"] + case["state"] * 128 * 128 * 4
    table = 4 * ((case["len"] + 31) // page + 1) + 4
    tail = 2 * (case["len"] % page) * case["hkv"] * case["D"] * (1 if case["fp8"] else 2)
    return {"bytes": (state + table) * (read + rows) + tail * (read + kept) + 8 * rows, "flops": 0}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_norm(s):
    case, K = s["case"], s["case"]["K"]
    out = {}
    u = s["x"].double()
    if s["residual"] is not None:
        u += s["residual"].double()
        out["residual"] = u.clone()
    u /= ((u * u).sum(1) / K + s["eps"]).sqrt()[:, None]
    u *= s["weight"].double()
    if case["bf16"]:
        out["out"] = u
    if case["group"] >= 0:
        parts = u.split(case["group"] or K, dim=1)
        largest = [p.abs().max(dim=1).values / E4M3_MAX for p in parts]
        out["scales"] = torch.stack(largest, dim=1)
        out["codes"] = torch.cat([p / a.clamp(min=1e-300)[:, None] for p, a in zip(parts, largest)], dim=1)
    return out


def _exact_attn(s):
    case = s["case"]
    B, T, hq, D = s["q"].shape
    hkv, page = case["hkv"], case["page"]
    out = torch.zeros((B, T, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, hq), -INF, dtype=torch.float64, device="cuda")
    q = s["q"].double()
    for b, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            continue
        used = s["table"][b, :-(-n // page)].long()
        k = s["k"][used].flatten(0, 1)[:n].double() * s["k_scale"]  # [n][hkv][D]
        v = s["v"][used].flatten(0, 1)[:n].double() * s["v_scale"]
        for t in range(T):
            last = n - (T - 1 - t)
            if last <= 0:
                continue
            for h in range(hkv):
                heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                x = s["scale"] * (q[b, t, heads] @ k[:last, h].T)
                z = torch.logsumexp(x, dim=1)
                lse[b, t, heads] = z
                out[b, t, heads] = torch.exp(x - z[:, None]) @ v[:last, h]
    return {"out": out, "lse": lse}


def _exact_beam(s):
    logp = torch.log_softmax(s["logits"].double(), dim=2) + s["scores"].double()[:, :, None]
    batch, beams, N = logp.shape
    flat = logp.nan_to_num(nan=-INF, neginf=-INF).reshape(batch, -1)
    best, at = torch.sort(flat, dim=1, descending=True, stable=True)
    best, at = best[:, :s["k"]], at[:, :s["k"]]
    return {"scores": best, "parents": None, "tokens": None}


def exact(case, seed):
    if case["op"] == "reorder":  # nothing is computed: rows move
        return None
    with torch.no_grad():
        return {"norm": _exact_norm, "attn": _exact_attn, "beam": _exact_beam}[case["op"]](prepare(case, seed))
