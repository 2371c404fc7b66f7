"""The cache's operators as a drafter runs them, one after the other: new tokens
into the cache, attention over it, and the accepted ones kept; eagerly, as a
replayed graph, and on another stream."""
import numpy as np
import pytest

import cache_reference as C
import step_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dvl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from draft_vocab_lm_gb300 import build
    build.build()
    import draft_vocab_lm_gb300 as d
    return d


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Loop:
    """A cache of B sequences and the calls of one verify step of T tokens."""

    def __init__(self, dvl, kind, B=3, T=4, Hq=8, H=2, D=64, page=16, width=8, seed=0):
        self.dvl, self.kind, self.B, self.T, self.Hq, self.H, self.D, self.page = dvl, kind, B, T, Hq, H, D, page
        g = torch.Generator().manual_seed(seed)
        self.g = g
        pages = B * width
        shape = (pages, page, H)
        if kind == "nvfp4":
            self.pools = [torch.zeros(*shape, n, dtype=torch.uint8, device="cuda") for n in (D // 2, D // 2, D // 16, D // 16)]
            self.scales = (0.005, 0.005)
            self.cache = dvl.KVCache(*self.pools[:2], k_scale=0.005, v_scale=0.005, k_blocks=self.pools[2], v_blocks=self.pools[3])
        else:
            t = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
            self.pools = [torch.zeros(*shape, D, dtype=t, device="cuda") for _ in range(2)]
            self.scales = (1.0, 1.0) if kind == "bf16" else (0.02, 0.02)
            self.cache = dvl.KVCache(*self.pools, k_scale=self.scales[0], v_scale=self.scales[1])
        self.table = torch.randperm(pages, generator=g).int().view(B, width).cuda()
        self.rope = dvl.Rope(D, theta=10000.0)
        self.wq, self.wk = ((1 + 0.2 * torch.randn(D, generator=g)).bfloat16().cuda() for _ in range(2))
        self.ws = dvl.attention_workspace(self.cache, B, T, Hq)
        self.qkv = torch.empty(B, T, Hq + 2 * H, D, dtype=torch.bfloat16, device="cuda")
        self.before = ints([0, 17, 40])[:B].clone()
        self.keep, self.counts = ints(np.zeros((B, T))), ints(np.zeros(B))
        self.new()

    def new(self):
        """Another step's inputs, in the same memory."""
        self.qkv.copy_((torch.randn(self.qkv.shape, generator=self.g) * 2).bfloat16())
        self.keep.copy_(torch.tensor([[0, 2, 3, -1], [0, 1, 2, 3], [0, 3, -1, -1]], dtype=torch.int32)[:self.B])
        self.counts.copy_(torch.tensor([3, 4, 2], dtype=torch.int32)[:self.B])

    def step(self, stream=None):
        q, k, v = (x for x in self.qkv.split([self.Hq, self.H, self.H], dim=2))
        lengths = self.before + self.T
        qo, _ = self.dvl.qk_norm_rope(q, k, v, rope=self.rope, q_weight=self.wq, k_weight=self.wk, cache=self.cache,
                                      table=self.table, lengths=lengths, stream=stream)
        out, lse = self.dvl.paged_attention(self.cache, qo, self.table, lengths, ws=self.ws, stream=stream)
        after = self.dvl.cache_keep(self.cache, self.table, lengths, self.before, self.keep, self.counts, stream=stream)
        return qo, out, lse, after

    def values(self):
        if self.kind == "nvfp4":
            c = [x.cpu().numpy() for x in self.pools]
            return [C.decode(c[i], c[i + 2], self.scales[i]) for i in range(2)]
        return [x.float().cpu().numpy().astype(np.float64) * s for x, s in zip(self.pools, self.scales)]

    def check(self):
        """A step against the 64-bit forms, each from what the one before left."""
        was = [x.contiguous().view(torch.uint8).cpu().numpy() for x in self.pools]
        q, k, v = (x.float().cpu().numpy().astype(np.float64).reshape(self.B * self.T, -1, self.D)
                   for x in self.qkv.split([self.Hq, self.H, self.H], dim=2))
        before, table = self.before.cpu().numpy(), self.table.cpu().numpy()
        where = C.places(self.B * self.T, before + self.T)
        got = [x.clone() for x in self.step()]
        freqs = [10000.0 ** (-2 * i / self.D) for i in range(self.D // 2)]
        w = [x.float().cpu().numpy().astype(np.float64) for x in (self.wq, self.wk)]
        pos = [p for _, p in where]
        z, err = C.turned(q, w[0], 1e-6, pos, freqs, False)
        qo = got[0].float().cpu().numpy().astype(np.float64)
        assert np.all(np.abs(qo.reshape(z.shape) - z) <= C.bf16_bound(z, err))
        # the cache as it is now holds the kept tokens; the dropped ones' slots
        # still hold what was there before they moved, so the full state before
        # the move is made again by another call
        for x, y in zip(self.pools, was):
            x.view(torch.uint8).copy_(torch.from_numpy(y))
        lengths = self.before + self.T
        a, b, c = self.qkv.split([self.Hq, self.H, self.H], dim=2)
        self.dvl.qk_norm_rope(a, b, c, rope=self.rope, q_weight=self.wq, k_weight=self.wk, cache=self.cache,
                              table=self.table, lengths=lengths)
        kk, vv = self.values()
        zk, ek = C.turned(k, w[1], 1e-6, pos, freqs, False)
        held = np.stack([kk[table[s, p // self.page], p % self.page] for s, p in where])
        loose = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -4, "nvfp4": 2.0 ** -2}[self.kind]
        assert np.all(np.abs(held - zk) <= loose * np.abs(zk).max(axis=-1, keepdims=True) + ek)
        ref = R.attention(qo, kk, vv, table, lengths.cpu().numpy(), self.D ** -0.5)
        tol, tol_lse = R.attention_bounds(*ref, n_max=int(lengths.max()), fp8=self.kind != "bf16")
        assert np.all(np.abs(got[1].float().cpu().numpy() - ref[0]) <= tol)
        assert np.all(np.abs(got[2].cpu().numpy() - ref[1]) <= tol_lse)
        full = [x.contiguous().view(torch.uint8).cpu().numpy() for x in self.pools]
        self.dvl.cache_keep(self.cache, self.table, lengths, self.before, self.keep, self.counts)
        for x, y in zip(self.pools, full):
            moved = C.kept(y, table, lengths.cpu().numpy(), before, self.keep.cpu().numpy(), self.counts.cpu().numpy())
            assert np.array_equal(x.contiguous().view(torch.uint8).cpu().numpy(), moved)
        assert got[3].tolist() == (before + self.counts.cpu().numpy()).tolist()
        self.before.copy_(got[3])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "nvfp4"])
def test_steps_follow_each_other(dvl, kind):
    loop = Loop(dvl, kind)
    for _ in range(4):
        loop.check()
        loop.new()


def snapshot(loop):
    return [x.clone().view(torch.uint8) for x in loop.pools]


@pytest.mark.parametrize("kind", ["bf16", "nvfp4"])
def test_a_replayed_step_is_the_eager_one(dvl, kind):
    eager, replayed = Loop(dvl, kind, seed=3), Loop(dvl, kind, seed=3)
    replayed.step()  # everything loaded before the capture; the cache's change is the first step's own
    eager.step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = replayed.step()
    for _ in range(3):
        eager.new(), replayed.new()
        want = eager.step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        for a, b in zip(snapshot(eager), snapshot(replayed)):
            assert torch.equal(a, b)
        eager.before.copy_(want[3]), replayed.before.copy_(out[3])


@pytest.mark.parametrize("handle", [False, True])
def test_a_step_on_another_stream(dvl, handle):
    here, there = Loop(dvl, "nvfp4", seed=4), Loop(dvl, "nvfp4", seed=4)
    want = [x.clone() for x in here.step()]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
    lengths = there.before + there.T  # (made on the current stream, in time)
    torch.cuda.current_stream().synchronize()
    on = st.cuda_stream if handle else st
    q, k, v = there.qkv.split([there.Hq, there.H, there.H], dim=2)
    qo, _ = dvl.qk_norm_rope(q, k, v, rope=there.rope, q_weight=there.wq, k_weight=there.wk, cache=there.cache,
                             table=there.table, lengths=lengths, stream=on)
    out, lse = dvl.paged_attention(there.cache, qo, there.table, lengths, ws=there.ws, stream=on)
    after = dvl.cache_keep(there.cache, there.table, lengths, there.before, there.keep, there.counts, stream=on)
    held = [torch.full((x.numel() * x.element_size(),), 0x55, dtype=torch.uint8, device="cuda") for x in want for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    st.synchronize()
    for a, b in zip((qo, out, lse, after), want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for a, b in zip(snapshot(here), snapshot(there)):
        assert torch.equal(a, b)
    del held


def test_two_steps_at_once(dvl):
    # two loops with workspaces of their own on two streams
    loops = [Loop(dvl, "nvfp4", seed=s, T=4) for s in (5, 6)]
    twins = [Loop(dvl, "nvfp4", seed=s, T=4) for s in (5, 6)]
    want = [[x.clone() for x in t.step()] for t in twins]
    streams = [torch.cuda.Stream() for _ in loops]
    torch.cuda.synchronize()
    got = []
    for loop, st in zip(loops, streams):
        with torch.cuda.stream(st):
            got.append(loop.step())
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    for a, b in zip(twins, loops):
        for x, y in zip(snapshot(a), snapshot(b)):
            assert torch.equal(x, y)
