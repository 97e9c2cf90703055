"""The operators around shared pages as a server of several samples a prompt uses them
together: rows forked from prompts, draft blocks through norm, projections and attention,
rows that grow, end and begin again from others, and the pools moved together.

Tables, lengths and copied rows are compared exactly; the attention with the definition in
64 bits, within 2^-8 (sum_k p_k |v_k| + |out|) for the roundings of the weights and of
the result to bf16 and 1e-4 of that for the rest."""
import numpy as np
import pytest
import torch

from block_diffusion_speculative_fusion_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32
B, LAYERS, PAGE, MAX_PAGES, NUM = 7, 2, 16, 24, 120
D_MODEL, HQ, HKV, D, N_Q = 512, 4, 2, 128, 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_fusion_gb300 import build
    build.build()
    api.lib()


def _i32(x):
    return torch.tensor(x, dtype=I32, device=DEV)


class Model:
    """Norm, fused projection and attention of two layers, the attention's output the next
    layer's input and the sum its residual."""

    def __init__(self, seed):
        t = torch.Generator().manual_seed(seed)
        self.norm = [(1 + 0.1 * torch.randn(D_MODEL, generator=t)).bfloat16().to(DEV) for _ in range(LAYERS)]
        self.w = [api.fp8_quant((torch.randn(((HQ + 2 * HKV) * D, D_MODEL), generator=t) * 0.1).bfloat16().to(DEV), 128)
                  for _ in range(LAYERS)]

    def round(self, x, pools, table, ctx, group, prefix, ws=None, check=None):
        """[(K, V) of the block by layer], and the last layer's attention."""
        res, blocks = torch.zeros_like(x), []
        for l in range(LAYERS):
            n = api.rms_norm(x, self.norm[l], 1e-6, residual=res, fp8=True)
            res = n["sum"]
            qkv = api.fp8_gemm(n["q"], n["scale"], *self.w[l], ws=None if ws is None else ws[0])
            q, k, v = (p.reshape(B, N_Q, -1, D).contiguous() for p in qkv.split([HQ * D, HKV * D, HKV * D], 1))
            kp, vp = pools[2 * l], pools[2 * l + 1]
            a = api.prefix_attn(q, k, v, kp, vp, table, ctx, group, prefix, causal=l == 1,
                                ws=None if ws is None else ws[1])
            if check is not None:
                check(l, q, k, v, a)
            blocks.append((k, v))
            x = a.view(B * N_Q, HQ * D)
        return blocks, x


def _attention(q, k, v, causal):
    z = torch.einsum("ihd,khd->hik", q.double(), k.double().repeat_interleave(HQ // HKV, 1)) * D ** -0.5
    v = v.double().repeat_interleave(HQ // HKV, 1)
    if causal:
        i, j = torch.arange(len(q), device=DEV)[:, None], torch.arange(len(k), device=DEV)[None]
        z = z.masked_fill(j > len(k) - len(q) + i, -torch.inf)
    p = torch.softmax(z, -1)
    return torch.einsum("hik,khd->ihd", p, v), torch.einsum("hik,khd->ihd", p, v.abs())


class Server:
    """The device's tables and pools beside a plain copy of every row's K/V."""

    def __init__(self, seed):
        self.t, self.g = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        self.pools = [torch.full((NUM, PAGE, HKV, D), float("nan"), dtype=torch.bfloat16, device=DEV)
                      for _ in range(2 * LAYERS)]
        self.table = torch.full((B, MAX_PAGES), -1, dtype=I32, device=DEV)
        self.n_pages, self.shares = _i32([0] * B), _i32([0] * NUM)
        self.free, self.n_free = torch.randperm(NUM, generator=self.t).to(I32).to(DEV), _i32([NUM])
        self.len = [0] * B
        self.rows = [[torch.empty((0, HKV, D), dtype=torch.bfloat16, device=DEV)] * B for _ in range(2 * LAYERS)]
        self.group, self.prefix = [-1] * B, [0, 0]

    def grow(self, new):
        """new[b]: per pool the rows that sequence b gets."""
        want = [n + len(new[b][0]) for b, n in enumerate(self.len)]
        o = api.pages_resize(_i32(want), self.table, self.n_pages, self.free, self.n_free, PAGE)
        assert not o["short"].any()
        self.n_pages, self.n_free = o["n_pages"], o["n_free"]
        for b in range(B):
            pos = torch.arange(self.len[b], want[b], device=DEV)
            page = self.table[b].long()[pos // PAGE]
            for i, pool in enumerate(self.pools):
                pool[page, pos % PAGE] = new[b][i]
                self.rows[i][b] = torch.cat([self.rows[i][b], new[b][i]])
        self.len = want

    def fork(self, parent):
        o = api.pages_fork(_i32(parent), _i32(self.len), self.table, self.n_pages, self.shares, self.free, self.n_free,
                           PAGE, self.pools)
        assert not o["short"].any()
        self.n_pages, self.n_free, self.shares = o["n_pages"], o["n_free"], o["shares"]
        for b, p in enumerate(parent):
            if p >= 0:
                self.len[b], self.group[b] = self.len[p], self.group[p]
                for r in self.rows:
                    r[b] = r[p]

    def end(self, gone):
        for b in gone:
            self.len[b], self.group[b] = 0, -1
            for r in self.rows:
                r[b] = r[b][:0]
        o = api.pages_release(_i32(self.len), self.table, self.n_pages, self.shares, self.free, self.n_free, PAGE)
        self.n_pages, self.n_free, self.shares = o["n_pages"], o["n_free"], o["shares"]

    def compact(self):
        o = api.pages_compact(self.table, self.n_pages, self.shares, PAGE, self.pools)
        self.table, self.shares, self.free, self.n_free = o["page_table"], o["shares"], o["free_pages"], o["n_free"]

    def check(self):
        held = set()
        for b, n in enumerate(self.len):
            pages = self.table[b, :-(-n // PAGE)].tolist()
            assert int(self.n_pages[b]) == len(pages)
            held.update(pages)
            pos = torch.arange(n, device=DEV)
            for r, pool in zip(self.rows, self.pools):
                assert torch.equal(pool[self.table[b].long()[pos // PAGE], pos % PAGE], r[b])
        free = self.free[:int(self.n_free)].tolist()
        assert sorted(free) == sorted(set(range(NUM)) - held)
        return held

    def args(self):
        return self.pools, self.table, _i32(self.len), _i32(self.group), _i32(self.prefix)

    def rand(self, n):
        return [torch.randn((n, HKV, D), generator=self.t).bfloat16().to(DEV) for _ in range(2 * LAYERS)]

    def hidden(self):
        return torch.randn((B * N_Q, D_MODEL), generator=self.t).bfloat16().to(DEV)


def _prompts(s):
    """Rows 0 and 1 hold prompts of 150 and 64 tokens; 2, 3 and 5 begin as row 0, 4 as row 1."""
    s.grow([s.rand(150), s.rand(64)] + [s.rand(0) for _ in range(B - 2)])
    s.group[:2], s.prefix = [0, 1], [150 // PAGE * PAGE, 64]
    s.fork([-1, -1, 0, 0, 1, 0, -1])


@pytest.mark.parametrize("seed", [0, 1])
def test_samples_of_two_prompts(seed):
    s, m = Server(seed), Model(seed)
    _prompts(s)
    for turn in range(5):
        s.check()

        def check(l, q, k, v, a):
            for b, n in enumerate(s.len):
                want, size = _attention(q[b], torch.cat([s.rows[2 * l][b], k[b]]), torch.cat([s.rows[2 * l + 1][b], v[b]]),
                                        l == 1)
                assert torch.all((a[b].double() - want).abs() <= 2.0 ** -8 * (size + want.abs()) * (1 + 1e-4) + 1e-4 * size)

        x = s.hidden()
        blocks, last = m.round(x, *s.args(), check=check)
        if turn in (1, 3):
            # the pools moved together: the same rows, and the same results bit for bit
            before = s.check()
            s.compact()
            assert s.check() == set(range(len(before)))
            assert torch.equal(m.round(x, *s.args())[1], last)
        # what each living row keeps of its block
        take = [int(s.g.integers(0, N_Q + 1)) if s.len[b] else 0 for b in range(B)]
        s.grow([[t[b, :take[b]] for kv in blocks for t in kv] for b in range(B)])
        if turn == 2:
            s.end([0, 4])                        # row 0's pages live on in its samples
            s.check()
            s.fork([2, -1, -1, -1, -1, -1, 1])   # rows ended or never begun: samples of rows as they are now
            assert s.len[0] == s.len[2] and s.len[6] == s.len[1]
    s.end(range(B))
    assert s.check() == set() and int(s.n_free) == NUM and not s.shares.any()


def test_round_captured_and_replayed():
    s, m = Server(5), Model(5)
    _prompts(s)
    x = s.hidden()
    m.round(x, *s.args())                         # workspaces
    ctx, group, prefix, table = _i32(s.len), _i32(s.group), _i32(s.prefix), s.table.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        blocks, last = m.round(x, s.pools, table, ctx, group, prefix)
    for turn in range(3):
        graph.replay()
        want_blocks, want = m.round(x, *s.args())
        assert torch.equal(last, want)
        for (k, v), (wk, wv) in zip(blocks, want_blocks):
            assert torch.equal(k, wk) and torch.equal(v, wv)
        # other lengths and rows, in the buffers that the graph reads
        s.grow([[t[b, :(b + turn) % N_Q if s.len[b] else 0].clone() for kv in blocks for t in kv] for b in range(B)])
        if turn == 1:
            s.end([3])
            s.fork([-1, -1, -1, 1, -1, -1, -1])
        ctx.copy_(_i32(s.len))
        group.copy_(_i32(s.group))
        table.copy_(s.table)
        x.copy_(s.hidden())


def test_two_streams_at_once():
    s, m = Server(6), Model(6)
    _prompts(s)
    xs = [s.hidden(), s.hidden()]
    args = s.args()
    want = [m.round(x, *args)[1].clone() for x in xs]
    size = [max(w.numel() for (_, of), w in api.cached_workspaces() if of == slot) for slot in (3, 6)]
    own = [[torch.zeros(n, dtype=torch.uint8, device=DEV) for n in size] for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = m.round(xs[i], *args, ws=own[i])[1]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
