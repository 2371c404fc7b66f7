"""Beam drafting with one attention layer and a trimmed head, on random weights.

One step, for batch x beams rows:

    x = embed[token]
    h = add_rmsnorm(x)                          -> queries, keys, values (matmul)
    qk_norm_rope(queries, keys, values)         keys, values -> the beam's next cache slot
                                                (this layer neither norms nor rotates them)
    o = paged_attention(h's queries over the cache)
    h, _ = add_rmsnorm(o wo, residual=x)        residual addition and norm
    logits = h . W_trim^T                       (matmul; W_trim from trim_head)
    scores, parents, tokens = beam_select(logits, scores, d2t)
    states, table, lengths = beam_reorder(parents, ..)

Every beam keeps its own page tables over one page pool: full pages are
shared by the beams that came from the same parent, the page a beam writes to
is its own (beam_reorder hands it a spare one).

    python examples/beam_draft.py [--steps 8] [--batch 4] [--beams 4]
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import draft_vocab_lm_gb300 as dvl  # noqa: E402


class Drafter:
    """Weights of the layer and the trimmed head (random, fixed seed)."""

    def __init__(self, V=20_000, K=2560, heads=20, kv_heads=4, D=128, shortlist=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()

        self.V, self.K, self.heads, self.kv_heads, self.D = V, K, heads, kv_heads, D
        self.embed = normal(V, K, std=1.0)
        self.wqkv = normal((heads + 2 * kv_heads) * D, K, std=K ** -0.5)
        self.wo = normal(K, heads * D, std=(heads * D) ** -0.5)
        self.norm1 = (1 + normal(K, std=0.1).float()).bfloat16()
        self.norm2 = (1 + normal(K, std=0.1).float()).bfloat16()
        ranks = torch.randperm(V, generator=torch.Generator().manual_seed(seed))[:shortlist].sort().values
        self.w_trim, _, self.d2t, _ = dvl.trim_head(normal(V, K, std=2.0 * K ** -0.5), ranks.numpy())


class Beams:
    """The beams of a batch of requests: page pool, tables, scores, tokens."""

    def __init__(self, model: Drafter, batch: int, beams: int, steps: int, page: int = 16, fp8: bool = False):
        self.model, self.batch, self.beams, self.page = model, batch, beams, page
        rows = batch * beams
        # one spare page per row and step: an engine would take freed pages instead
        pages = rows * (steps + 2)
        shape = (pages, page, model.kv_heads, model.D)
        kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
        self.scale = 0.05 if fp8 else 1.0
        self.k, self.v = (torch.zeros(shape, dtype=kind, device="cuda") for _ in range(2))
        self.cache = dvl.KVCache(self.k, self.v, k_scale=self.scale, v_scale=self.scale)
        self.ws = dvl.attention_workspace(self.cache, rows, 1, model.heads)
        self.select_ws = dvl.beam_workspace(batch, beams, model.w_trim.shape[0])
        self.free = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.used = 0
        width = (steps + 2 * page) // page
        self.table = torch.zeros((batch, beams, width), dtype=torch.int32, device="cuda")
        self.table[:, :, 0] = self.take()
        self.lengths = torch.zeros((batch, beams), dtype=torch.int32, device="cuda")
        # one live beam per request at first
        self.scores = torch.full((batch, beams), -float("inf"), device="cuda")
        self.scores[:, 0] = 0
        self.history = torch.zeros((batch, beams, steps + 1), dtype=torch.int32, device="cuda")
        self.done = 0

    def take(self):
        """A page for every row."""
        n = self.batch * self.beams
        self.used += n
        return self.free[self.used - n:self.used].view(self.batch, self.beams)

    def start(self, tokens):
        """tokens [batch]: the last token of each request's prompt."""
        self.history[:, :, 0] = tokens.view(-1, 1)

    def append(self, q, k, v):
        """Write one token's keys and values [rows][kv_heads][D] to each row's next slot."""
        self.lengths += 1
        dvl.qk_norm_rope(q, k, v, cache=self.cache, table=self.table.view(-1, self.table.shape[2]),
                         lengths=self.lengths.view(-1), q_out=q)

    def step(self):
        m, rows = self.model, self.batch * self.beams
        x = m.embed[self.history[:, :, self.done].view(-1).long()]
        h, _, _, _ = dvl.add_rmsnorm(x, m.norm1)
        qkv = torch.matmul(h, m.wqkv.t()).view(rows, m.heads + 2 * m.kv_heads, m.D)
        q, k, v = qkv.split([m.heads, m.kv_heads, m.kv_heads], dim=1)
        self.append(q, k, v)
        o, _ = dvl.paged_attention(self.cache, q, self.table.view(rows, -1), self.lengths.view(-1),
                                   want_lse=False, ws=self.ws)
        h, _, _, _ = dvl.add_rmsnorm(torch.matmul(o.view(rows, -1), m.wo.t()), m.norm2, x)
        logits = torch.matmul(h, m.w_trim.t()).view(self.batch, self.beams, -1)
        self.scores, parents, tokens = dvl.beam_select(logits, self.scores, self.beams, d2t=m.d2t,
                                                       ws=self.select_ws)
        spare = self.take()
        (self.history,), self.table, self.lengths = dvl.beam_reorder(
            parents, [self.history], cache=self.cache, table=self.table, lengths=self.lengths, spare=spare)
        # an unused slot's table is all page 0, another beam's: what it appends goes to its own page
        self.table[:, :, 0] = torch.where(parents < 0, spare, self.table[:, :, 0])
        self.done += 1
        self.history[:, :, self.done] = tokens
        return tokens


def draft(model: Drafter, tokens, beams: int, steps: int, **kw) -> Beams:
    """Draft `steps` tokens after each request's last token; returns the beams."""
    b = Beams(model, tokens.shape[0], beams, steps, **kw)
    b.start(tokens)
    for _ in range(steps):
        b.step()
    return b


def main() -> None:
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--beams", type=int, default=4)
    p.add_argument("--fp8", action="store_true", help="an E4M3 cache")
    a = p.parse_args()
    model = Drafter()
    b = draft(model, torch.arange(a.batch, dtype=torch.int32, device="cuda"), a.beams, a.steps, fp8=a.fp8)
    for r in range(a.batch):
        for j in range(a.beams):
            print(f"request {r} beam {j} score {b.scores[r, j].item():8.3f}  tokens "
                  + " ".join(str(t) for t in b.history[r, j].tolist()))


if __name__ == "__main__":
    main()
