"""The cache's side of a drafting step, in plain form and through the library.

What a drafter's layer does with its paged key-value cache around the attention
itself: the norm of the new queries and keys for each head with the position
rotation, the new keys and values going to their places of the cache in the same
pass (qk_norm_rope); attention over a cache held in 4 bits (paged_attention with
an NVFP4 cache: E2M1 codes, one E4M3 scale per 16 values); and, after a
verification, the tokens that were accepted moving together where the rejected
ones lay between them (cache_keep).  Head counts, lengths and pages are generic
serving sizes, those of this library's other operators' cases among them.

`run` computes an operator from elementary torch operations in 32 bits (the
rotation's angles in 64: a far position times a frequency), or, with `own` true,
calls the library's entry points.
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
        # one new token of one request in front of its attention: pure latency
        {"name": "rope_draft_step", "op": "rope", "B": 1, "T": 1, "rows": 1, "past": 731, "hq": 20, "hkv": 4, "D": 128,
         "rot": 128, "interleaved": False, "norm": True, "page": 16, "fp8": False},
        # a verify step of three tokens for a full batch, on an 8-bit cache
        {"name": "rope_verify3_fp8", "op": "rope", "B": 64, "T": 3, "rows": 192, "past": 4101, "hq": 40, "hkv": 8, "D": 128,
         "rot": 128, "interleaved": False, "norm": True, "page": 64, "fp8": True},
        # ragged prompts of a few requests in one pass, padded rows behind them
        {"name": "rope_prefill", "op": "rope", "B": 5, "T": 0, "rows": 16381, "past": 1021, "hq": 40, "hkv": 8, "D": 128,
         "rot": 128, "interleaved": False, "norm": True, "page": 16, "fp8": False},
        # the same with wide heads of which a quarter is rotated, in neighbouring pairs
        {"name": "rope_prefill_partial_fp8", "op": "rope", "B": 3, "T": 0, "rows": 8191, "past": 40001, "hq": 16, "hkv": 2,
         "D": 256, "rot": 64, "interleaved": True, "norm": False, "page": 48, "fp8": True},
        # one request, one new token, a chat-sized cache: latency
        {"name": "attn4_draft_step", "op": "attn4", "B": 1, "T": 1, "hq": 20, "hkv": 4, "D": 128, "longest": 731, "page": 16},
        # a verify step of three tokens for a few requests of unequal length
        {"name": "attn4_verify3", "op": "attn4", "B": 8, "T": 3, "hq": 40, "hkv": 8, "D": 128, "longest": 4101, "page": 64},
        # one request with a very long context, few wide heads
        {"name": "attn4_long_context", "op": "attn4", "B": 1, "T": 1, "hq": 16, "hkv": 2, "D": 256, "longest": 262139,
         "page": 64},
        # a full serving batch
        {"name": "attn4_batch", "op": "attn4", "B": 64, "T": 1, "hq": 40, "hkv": 8, "D": 128, "longest": 16381, "page": 32},
        # one request's tree of drafts after its verification: a path of a few nodes stays
        {"name": "keep_tree", "op": "keep", "B": 1, "nodes": 63, "kept": 7, "past": 731, "hkv": 4, "D": 128, "page": 16,
         "kind": "bf16"},
        # the same for a full batch on an 8-bit cache
        {"name": "keep_tree_batch_fp8", "op": "keep", "B": 64, "nodes": 31, "kept": 9, "past": 4101, "hkv": 8, "D": 128,
         "page": 64, "kind": "fp8"},
        # long 4-bit caches of which half of the tokens are dropped
        {"name": "keep_half_4bit", "op": "keep", "B": 16, "nodes": 16381, "kept": 8191, "past": 3, "hkv": 8, "D": 128,
         "page": 32, "kind": "nvfp4"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "attn4", "attn4", "keep"])
    if op == "rope":
        D = rng.choice([64, 80, 128, 128, 256])
        hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
        case = {"op": op, "hq": hkv * G, "hkv": hkv, "D": D, "rot": rng.choice([D, D, 16 * rng.randrange(1, D // 16 + 1)]),
                "interleaved": rng.random() < 0.3, "norm": rng.random() < 0.7, "page": rng.choice([16, 32, 48, 64, 128]),
                "fp8": rng.random() < 0.4}
        most = max(64, min(16000, 700_000_000 // ((G + 2) * hkv * D * 8)))
        if rng.random() < 0.5:
            B, T = _log_int(rng, 1, 64), rng.choice([1, 1, 2, 3, 5, 8])
            return {**case, "B": B, "T": T, "rows": B * T, "past": _log_int(rng, 1, 4000)}
        return {**case, "B": _log_int(rng, 1, 16), "T": 0, "rows": 2 * _log_int(rng, 8, most // 2) + 1,
                "past": _log_int(rng, 1, 8000)}
    if op == "attn4":
        D = rng.choice([64, 128, 128, 192, 256])
        hkv, G, T = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 1, 1, 2, 3, 5])
        longest, B = _log_int(rng, 1, 60_000), _log_int(rng, 1, 96)
        B = max(1, min(B, 400_000_000 // (hkv * D * longest)))
        return {"op": op, "B": B, "T": T, "hq": hkv * G, "hkv": hkv, "D": D, "longest": longest,
                "page": rng.choice([16, 32, 48, 64, 128])}
    nodes = _log_int(rng, 1, 8000)
    return {"op": op, "B": _log_int(rng, 1, 32), "nodes": nodes, "kept": _log_int(rng, 1, nodes), "past": _log_int(rng, 1, 2000),
            "hkv": rng.choice([1, 2, 4, 8]), "D": rng.choice([64, 128, 256]), "page": rng.choice([16, 32, 48, 64]),
            "kind": rng.choice(["bf16", "fp8", "nvfp4"])}


def _plan(case):
    """A generator that depends on the case's sizes alone, for what its work depends on."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """The batch's lengths, the longest among them; prepare() puts them in another order for each seed."""
    r, n = _plan(case), case["longest"]
    return [n] + [r.randint(max(1, n // 8), n) if r.random() > 0.02 else 0 for _ in range(case["B"] - 1)]


def _news(case):
    """[(tokens cached before, new tokens)] of the batch's sequences."""
    r, B, past = _plan(case), case["B"], case["past"]
    pasts = [past] + [r.randint(0, past) for _ in range(B - 1)]
    if case["T"]:
        return [(p, case["T"]) for p in pasts]
    used = case["rows"] - case["rows"] // 50  # the rest of the rows is padding
    cuts = sorted(r.randint(0, used) for _ in range(B - 1))
    return [(p, b - a) for p, a, b in zip(pasts, [0] + cuts, cuts + [used])]


def _kept(case):
    """[(tokens before the nodes, nodes, the nodes that stay)] of the batch's sequences."""
    r, out = _plan(case), []
    for _ in range(case["B"]):
        nodes = r.randint((case["nodes"] + 1) // 2, case["nodes"])
        n = min(nodes, r.randint((case["kept"] + 1) // 2, case["kept"]))
        out.append((r.randint(0, case["past"]), nodes, [0] + sorted(r.sample(range(1, nodes), n - 1))))
    return out


# ---------------------------------------------------------------------------
# What a user's program has in hand
# ---------------------------------------------------------------------------

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


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


def _pool4(g, pages, page, hkv, D):
    """One page pool in 4 bits: codes (two to a byte), scales of 16 values, and the scale of all."""
    codes = torch.empty((pages, page, hkv, D // 2), dtype=torch.uint8, device="cuda")
    blocks = torch.empty((pages, page, hkv, D // 16), dtype=FP8, device="cuda")
    scale = 6.0 / (6 * E4M3_MAX)  # the largest value is near 6
    middles = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])], device="cuda")
    step = max(1, (1 << 25) // (page * hkv * D))
    for i in range(0, pages, step):
        x = _normal(g, *codes[i:i + step].shape[:3], D // 16, 16)
        s = (x.abs().amax(-1) / (6 * scale)).clamp_(max=E4M3_MAX).to(FP8)
        x /= (s.float() * scale).clamp(min=1e-30).unsqueeze(-1)
        c = torch.bucketize(x.abs(), middles, out_int32=True) + 8 * (x < 0)
        c = c.to(torch.uint8).view(*codes[i:i + step].shape, 2)
        codes[i:i + step] = c[..., 0] + 16 * c[..., 1]
        blocks[i:i + step] = s
    return codes, blocks, scale


def _tables(g, lens, page):
    """Page tables [B][width] of these lengths over a pool of shuffled pages; the pool's pages, a page of no table."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.zeros((len(lens), max(max(need), 1)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pages, ids[-1:]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_rope(case, g):
    hq, hkv, D, rows = case["hq"], case["hkv"], case["D"], case["rows"]
    news = _news(case)
    news = [news[i] for i in torch.randperm(len(news), generator=g, device="cuda").tolist()]
    table, pages, _ = _tables(g, [p + n for p, n in news], case["page"])
    # the projection's rows: queries, keys and values next to each other
    qkv = _normal(g, rows, hq + 2 * hkv, D, std=2.0).bfloat16()
    starts = None
    if case["T"] == 0:
        starts = [0]
        for _, n in news:
            starts.append(starts[-1] + n)
    k, k_scale = _pool(g, pages, case["page"], hkv, D, case["fp8"])
    v, v_scale = _pool(g, pages, case["page"], hkv, D, case["fp8"])
    weights = [(1 + _normal(g, D, std=0.1)).bfloat16() if case["norm"] else None for _ in range(2)]
    return {"q": qkv[:, :hq], "k_new": qkv[:, hq:hq + hkv], "v_new": qkv[:, hq + hkv:], "q_weight": weights[0],
            "k_weight": weights[1], "eps": 1e-6, "theta": 1e6, "table": table, "lengths": _ints([p + n for p, n in news]),
            "starts": None if starts is None else _ints(starts), "k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale,
            "q_out": torch.zeros((rows, hq, D), dtype=torch.bfloat16, device="cuda")}


def _prepare_attn4(case, g):
    B, T = case["B"], case["T"]
    lens = _lengths(case)
    lens = [lens[i] for i in torch.randperm(B, generator=g, device="cuda").tolist()]
    table, pages, _ = _tables(g, lens, case["page"])
    k, k_blocks, k_scale = _pool4(g, pages, case["page"], case["hkv"], case["D"])
    v, v_blocks, v_scale = _pool4(g, pages, case["page"], case["hkv"], case["D"])
    return {"q": _normal(g, B, T, case["hq"], case["D"], std=2.0).bfloat16(), "k": k, "v": v, "k_blocks": k_blocks,
            "v_blocks": v_blocks, "k_scale": k_scale, "v_scale": v_scale, "table": table, "lengths": _ints(lens),
            "scale": case["D"] ** -0.5}


def _prepare_keep(case, g):
    B, hkv, D, page = case["B"], case["hkv"], case["D"], case["page"]
    kept = _kept(case)
    kept = [kept[i] for i in torch.randperm(B, generator=g, device="cuda").tolist()]
    lens = [first + nodes for first, nodes, _ in kept]
    table, pages, spare = _tables(g, lens, page)
    width = case["kept"]
    s = {"table": table, "lengths": _ints(lens), "first": _ints([first for first, _, _ in kept]),
         "keep": _ints([nodes + [-1] * (width - len(nodes)) for _, _, nodes in kept]),
         "counts": _ints([len(nodes) for _, _, nodes in kept]), "spare": spare}
    if case["kind"] == "nvfp4":
        # what the codes stand for plays no part: any bytes, any scales but NaN
        for n in ("k", "v"):
            s[n] = torch.randint(256, (pages, page, hkv, D // 2), generator=g, device="cuda", dtype=torch.uint8)
            s[n + "_blocks"] = torch.randint(127, (pages, page, hkv, D // 16), generator=g, device="cuda",
                                             dtype=torch.uint8).view(FP8)
            s[n + "_scale"] = 1.0
    else:
        s["k"], s["k_scale"] = _pool(g, pages, page, hkv, D, case["kind"] == "fp8")
        s["v"], s["v_scale"] = _pool(g, pages, page, hkv, D, case["kind"] == "fp8")
    return s


def prepare(case, seed):
    make = {"rope": _prepare_rope, "attn4": _prepare_attn4, "keep": _prepare_keep}
    return {"case": case, **make[case["op"]](case, _generator(seed))}


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _rows_of_sequences(s):
    """(sequence, place in the cache, row it stands for, whether it is a row of a sequence) of every row."""
    rows, lengths = s["q"].shape[0], s["lengths"].long()
    r = torch.arange(rows, device="cuda")
    if s["starts"] is None:
        T = s["case"]["T"]
        b, end = r // T, (r // T + 1) * T
        used = r >= 0
    else:
        starts = s["starts"].long()
        b = (torch.searchsorted(starts, r, right=True) - 1).clamp(max=len(starts) - 2)
        end, used = starts[b + 1], r < starts[-1]
    # the rows behind the last sequence stand for its last row
    row = torch.where(used, r, used.sum() - 1)
    return b[row], (lengths[b] - (end - r))[row], row, used


def _plain_rope(s):
    case = s["case"]
    D, rot, page = case["D"], case["rot"], case["page"]
    b, pos, row, used = _rows_of_sequences(s)
    half = rot // 2
    freq = s["theta"] ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = pos.double().view(-1, 1) * freq
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)

    def normed(x, weight):
        x = x.float()
        if weight is None:
            return x
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()

    def rotated(x):
        if case["interleaved"]:
            x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1).flatten(-2)
        else:
            x1, x2 = x[..., :half], x[..., half:rot]
            turned = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)
        return torch.cat((turned, x[..., rot:]), -1)

    q = rotated(normed(s["q"], s["q_weight"])).bfloat16()
    s["q_out"].copy_(torch.where(used.view(-1, 1, 1), q, s["q_out"]))
    slot = s["table"][b, pos // page].long() * page + pos % page
    for pool, x, scale in ((s["k"], rotated(normed(s["k_new"], s["k_weight"])), s["k_scale"]),
                           (s["v"], s["v_new"].float(), s["v_scale"])):
        if case["fp8"]:
            x = (x / scale).clamp(-E4M3_MAX, E4M3_MAX)
        x = x.to(pool.dtype)
        bits = torch.uint8 if case["fp8"] else torch.int16
        pool.view(bits).flatten(0, 1).index_copy_(0, slot, x.view(bits)[row])
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _decoded(codes, blocks, scale):
    """The values [..][D] that 4-bit codes [..][D/2] and their scales stand for."""
    one = torch.tensor(E2M1 + [-x for x in E2M1], device=codes.device)
    pairs = torch.stack((one.repeat(16), one.repeat_interleave(16)), -1)  # of each byte: low, high
    x = pairs.index_select(0, codes.reshape(-1).int()).view(*blocks.shape, 16)
    return (x * (blocks.float() * scale).unsqueeze(-1)).flatten(-2)


def _plain_attn4(s):
    case, table = s["case"], s["table"].long()
    B, T, hq, D = s["q"].shape
    hkv, n = case["hkv"], table.shape[1] * case["page"]
    q = s["q"].float().view(B, T, hkv, hq // hkv, D)
    k = _decoded(s["k"][table], s["k_blocks"].view(torch.uint8)[table].view(FP8), s["k_scale"]).view(B, n, hkv, D)
    x = torch.einsum("bthgd,bnhd->bthgn", q, k) * s["scale"]
    del k
    sees = s["lengths"].view(B, 1) - (T - 1 - torch.arange(T, device="cuda"))  # [B][T]
    seen = torch.arange(n, device="cuda") < sees.view(B, T, 1, 1, 1)
    x = x.masked_fill(~seen, -INF)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -INF, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    v = _decoded(s["v"][table], s["v_blocks"].view(torch.uint8)[table].view(FP8), s["v_scale"]).view(B, n, hkv, D)
    o = torch.einsum("bthgn,bnhd->bthgd", p, v)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return {"out": o.reshape(B, T, hq, D).bfloat16(), "lse": (m + torch.log(total)).reshape(B, T, hq)}


def _pools(s):
    return {n: s[n] for n in ("k", "v", "k_blocks", "v_blocks") if n in s}


def _plain_keep(s):
    page, keep = s["case"]["page"], s["keep"].long()
    B, M = keep.shape
    i = torch.arange(M, device="cuda").view(1, M)
    valid = i < s["counts"].view(B, 1)
    first = s["first"].long().view(B, 1)

    def slots(pos):
        at = s["table"].gather(1, (pos // page).clamp(max=s["table"].shape[1] - 1)).long() * page + pos % page
        # a place of no sequence keeps what it holds
        return torch.where(valid, at, s["spare"].long() * page).view(-1)

    src, dst = slots(first + keep.clamp(min=0)), slots(first + i)
    for pool in _pools(s).values():
        raw = pool.view(torch.uint8).flatten(0, 1)
        raw[dst] = raw[src]
    return {**_pools(s), "lengths": s["first"] + s["counts"]}


# ---------------------------------------------------------------------------
# The library
# ---------------------------------------------------------------------------

def _own(s):
    import draft_vocab_lm_gb300 as dvl

    case = s["case"]
    was = s.setdefault("outputs", {})  # a serving loop's output buffers: made by its first pass, written by every later one
    if "cache" not in s:  # the loop's handle of its page pool
        four = {n: s[n] for n in ("k_blocks", "v_blocks") if n in s}
        s["cache"] = dvl.KVCache(s["k"], s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"], **four)
    if case["op"] == "rope":
        if "rope" not in s:  # a model's frequencies
            s["rope"] = dvl.Rope(case["rot"], theta=s["theta"], interleaved=case["interleaved"])
        dvl.qk_norm_rope(s["q"], s["k_new"], s["v_new"], rope=s["rope"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                         eps=s["eps"], cache=s["cache"], table=s["table"], lengths=s["lengths"], starts=s["starts"],
                         q_out=s["q_out"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if case["op"] == "attn4":
        if "ws" not in s:
            s["ws"] = dvl.attention_workspace(s["cache"], *s["q"].shape[:3])
        r = dvl.paged_attention(s["cache"], s["q"], s["table"], s["lengths"], scale=s["scale"], out=was.get("out"),
                                lse=was.get("lse"), ws=s["ws"])
        s["outputs"] = dict(zip(("out", "lse"), r))
        return s["outputs"]
    lengths = dvl.cache_keep(s["cache"], s["table"], s["lengths"], s["first"], s["keep"], s["counts"],
                             lengths_out=was.get("lengths"))
    s["outputs"] = {"lengths": lengths}
    return {**_pools(s), "lengths": lengths}


def run(state):
    if own:
        return _own(state)
    plain = {"rope": _plain_rope, "attn4": _plain_attn4, "keep": _plain_keep}
    return plain[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, D, hkv = case["op"], case["D"], case["hkv"]
    if op == "rope":
        rows = sum(n for _, n in _news(case))
        moved = rows * D * (4 * case["hq"] + 2 * hkv * (2 + (1 if case["fp8"] else 2))) + 4 * rows + 12 * case["B"]
        return {"bytes": moved + 4 * D * case["norm"], "flops": rows * D * (case["hq"] + hkv) * (3 + 4 * case["norm"])}
    if op == "attn4":
        lens, T, hq = _lengths(case), case["T"], case["hq"]
        pages = sum(-(-n // case["page"]) for n in lens)
        moved = 2 * sum(lens) * hkv * (D // 2 + D // 16) + case["B"] * T * hq * (4 * D + 4) + 4 * pages + 4 * case["B"]
        return {"bytes": moved, "flops": 4 * hq * D * sum(max(0, n - t) for n in lens for t in range(T))}
    kept = _kept(case)
    row = 2 * hkv * {"bf16": 2 * D, "fp8": D, "nvfp4": D // 2 + D // 16}[case["kind"]]
    moved = sum(n != i for _, _, nodes in kept for i, n in enumerate(nodes))  # a node in its place already stays
    return {"bytes": 2 * row * moved + 8 * sum(len(nodes) for _, _, nodes in kept) + 16 * case["B"], "flops": 0}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rope(s):
    case = s["case"]
    D, rot, page, rows = case["D"], case["rot"], case["page"], s["q"].shape[0]
    lengths = s["lengths"].tolist()
    starts = s["starts"].tolist() if s["starts"] is not None else [b * case["T"] for b in range(case["B"] + 1)]
    out = s["q_out"].double()
    pools = {"k": s["k"].double(), "v": s["v"].double()}

    def turn(x, weight, angle):
        x = x.double()
        if weight is not None:
            x = x / ((x * x).sum(-1, keepdim=True) / D + s["eps"]).sqrt() * weight.double()
        pairs = list(range(0, rot, 2)) if case["interleaved"] else list(range(rot // 2))
        first = torch.tensor(pairs, device="cuda")
        second = first + (1 if case["interleaved"] else rot // 2)
        z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None, :]
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    freq = torch.tensor([s["theta"] ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device="cuda")
    for b, n in enumerate(lengths):
        lo, hi = starts[b], starts[b + 1]
        pos = torch.arange(n - (hi - lo), n, device="cuda")
        angle = pos.double()[:, None] * freq[None, :]
        out[lo:hi] = turn(s["q"][lo:hi], s["q_weight"], angle)
        page_of = s["table"][b].long()[pos // page]
        pools["k"][page_of, pos % page] = turn(s["k_new"][lo:hi], s["k_weight"], angle) / s["k_scale"]
        pools["v"][page_of, pos % page] = s["v_new"][lo:hi].double() / s["v_scale"]
    return {"q": out, **pools}


def _exact_attn4(s):
    case = s["case"]
    B, T, hq, D = s["q"].shape
    hkv = case["hkv"]
    out = torch.zeros((B, T, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, hq), -INF, dtype=torch.float64, device="cuda")
    q = s["q"].double()

    def values(name, pages, n):
        c = s[name][pages].flatten(0, 1)[:n]  # [n][hkv][D/2]
        c = torch.stack((c & 15, c >> 4), -1).flatten(-2).int()
        exponent, odd = (c >> 1) & 3, (c & 1).double()
        x = torch.where(exponent == 0, odd / 2, (1 + odd / 2) * 2.0 ** (exponent - 1).double())
        x = torch.where(c >= 8, -x, x).view(n, hkv, D // 16, 16)
        block = s[name + "_blocks"][pages].flatten(0, 1)[:n].double()
        return (x * block.unsqueeze(-1) * s[name + "_scale"]).view(n, hkv, D)

    for b, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // case["page"])].long()
        k, v = values("k", pages, n), values("v", pages, n)
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


def exact(case, seed):
    if case["op"] == "keep":  # nothing is computed: rows move
        return None
    with torch.no_grad():
        return {"rope": _exact_rope, "attn4": _exact_attn4}[case["op"]](prepare(case, seed))
