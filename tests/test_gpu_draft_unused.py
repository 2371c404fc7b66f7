"""The beam drafting example where a shortlist has fewer rows than there are
beams: unused slots write into no other beam's pages."""
import importlib.util
import os

import pytest

from conftest import ROOT
from test_gpu_draft_example import Plain, plain_step

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


@pytest.mark.parametrize("page", [1, 4])
@pytest.mark.parametrize("steps", [1, 2, 3])
def test_unused_beams_leave_the_others_pages_alone(example, steps, page):
    # two rows in the head, five beams: 2, 4, then 5 live ones
    model = example.Drafter(V=300, K=512, heads=8, kv_heads=2, D=64, shortlist=2, seed=5)
    b = example.draft(model, torch.tensor([5, 17], dtype=torch.int32, device="cuda"), 5, steps, page=page)
    plain = Plain(model)
    live = min(5, 2 ** steps)
    for r in range(2):
        assert torch.isfinite(b.scores[r, :live]).all() and torch.all(b.scores[r, live:] == -float("inf"))
        for j in range(live):
            path = b.history[r, j]
            keys, _ = plain_step(plain, path[:steps])
            ids = b.table[r, j, :-(-steps // page)].long()
            held = b.k[ids].flatten(0, 1)[:steps].double().cpu()
            assert torch.all((held - keys).abs() <= keys.abs() * 2.0 ** -7 + 1e-3)
    # every row, used or not, writes its next token to a page of its own
    at = (b.lengths // page).long().unsqueeze(2)
    pages = b.table.gather(2, at).flatten().tolist()
    assert len(set(pages)) == len(pages)
