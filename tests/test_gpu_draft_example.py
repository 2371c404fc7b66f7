"""The beam drafting example end to end: what each final beam's page table
holds is its own path's keys, and its score is the path's log probability.

Bounds: a key depends on its token alone; the example and the check round it
to bf16 (2^-8) or E4M3 (2^-4 of it, 2^-10 of the scale) from sums of 2,560
products in another order.  A path's score: each of its steps rounds the
attention output, the projected row, the normed row (2^-8 relative each, with
logits of standard deviation 2 about 0.03 in a logit) and the logits (bf16,
below 16: 2^-5), so about 0.1 a step; an E4M3 cache adds about as much."""
import importlib.util
import os

import numpy as np
import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from draft_vocab_lm_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("beam_draft", os.path.join(ROOT, "examples", "beam_draft.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Plain:
    """The model's weights in 64 bits on the CPU."""

    def __init__(self, m):
        for name in ("embed", "wqkv", "wo", "norm1", "norm2", "w_trim"):
            setattr(self, name, getattr(m, name).double().cpu())
        self.heads, self.kv_heads, self.D = m.heads, m.kv_heads, m.D


def plain_step(m, tokens):
    """64-bit forward of the last of `tokens` (a path): (keys of all, log
    probabilities).  The first norm's output is rounded to bf16 as the example
    rounds it, so that both sides sum the same products for a key."""
    x = m.embed[tokens.long().cpu()]

    def norm(u, w):
        return u / (u.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w

    qkv = (norm(x, m.norm1).bfloat16().double() @ m.wqkv.t()).view(len(tokens), -1, m.D)
    q, k, v = qkv[-1, :m.heads], qkv[:, m.heads:m.heads + m.kv_heads], qkv[:, m.heads + m.kv_heads:]
    g = m.heads // m.kv_heads
    s = torch.einsum("hd,nhd->hn", q, k.repeat_interleave(g, 1)) * m.D ** -0.5
    o = torch.einsum("hn,nhd->hd", s.softmax(-1), v.repeat_interleave(g, 1)).reshape(1, -1)
    h = norm(x[-1:] + o @ m.wo.t(), m.norm2)
    return k, torch.log_softmax(h @ m.w_trim.t(), -1)[0]


@pytest.mark.parametrize("fp8,page,steps", [(False, 4, 9), (True, 16, 6)])
def test_beam_draft_example(example, fp8, page, steps):
    model = example.Drafter(V=3000, K=512, heads=8, kv_heads=2, D=64, shortlist=700, seed=3)
    start = torch.tensor([5, 17, 1000], dtype=torch.int32, device="cuda")
    b = example.draft(model, start, 4, steps, page=page, fp8=fp8)
    assert torch.equal(b.lengths, torch.full((3, 4), steps, dtype=torch.int32, device="cuda"))
    plain = Plain(model)
    row_of = {int(t): i for i, t in enumerate(model.d2t.tolist())}
    seen = set()
    for r in range(3):
        assert torch.all(b.scores[r][:-1] >= b.scores[r][1:])
        for j in range(4):
            path = b.history[r, j]
            assert int(path[0]) == int(start[r])
            assert (r, *path.tolist()) not in seen
            seen.add((r, *path.tolist()))
            total = 0.0
            for t in range(steps):
                keys, logp = plain_step(plain, path[:t + 1])
                total += float(logp[row_of[int(path[t + 1])]])
            ids = b.table[r, j, :-(-steps // page)].long()
            held = b.k[ids].flatten(0, 1)[:steps].double().cpu() * b.scale
            tol = keys.abs() * (2.0 ** -4 if fp8 else 2.0 ** -7) + (b.scale * 2.0 ** -9 if fp8 else 0) + 1e-3
            assert torch.all((held - keys).abs() <= tol)
            assert abs(float(b.scores[r, j]) - total) <= (0.2 if fp8 else 0.1) * steps


def test_one_beam_is_greedy(example):
    import draft_vocab_lm_gb300 as dvl
    model = example.Drafter(V=3000, K=512, heads=8, kv_heads=2, D=64, shortlist=700, seed=4)
    b = example.draft(model, torch.tensor([9], dtype=torch.int32, device="cuda"), 1, 5)
    # the head's own argmax picks the token of the largest logit too
    head = dvl.Head(model.w_trim, V=model.V, d2t=model.d2t)
    for t in range(5):
        _, logp = plain_step(Plain(model), b.history[0, 0, :t + 1])
        best = logp.max()
        mine = logp[model.d2t.tolist().index(int(b.history[0, 0, t + 1]))]
        assert float(best - mine) <= 0.1
    h = torch.randn(4, 512, device="cuda").bfloat16()
    ids, vals = dvl.draft_argmax(head, h)
    logits = torch.matmul(h.float(), model.w_trim.float().t())
    _, parents, tokens = dvl.beam_select(logits.view(4, 1, -1), torch.zeros(4, 1, device="cuda"), 1, d2t=model.d2t)
    gap = logits.topk(2, dim=1).values
    clear = (gap[:, 0] - gap[:, 1]) > 1e-3 * logits.abs().amax(1)
    assert torch.equal(ids[clear], tokens[clear, 0]) and torch.all(parents == 0)
    assert np.allclose(vals.cpu(), gap[:, 0].cpu(), rtol=2e-3)
