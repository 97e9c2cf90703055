"""GPU parity of the attention over shared prefixes (dflash_prefix_attn) with the
definition in 64 bits.

Tolerance of an output element, from the roundings: the weights p (exact sum 1) meet
the values in bf16, each off by at most half a step (2^-8 of itself), and the result
is rounded once more: 2^-8 (sum_k p_k |v_k| + |out|). Scores (fp32 sums of bf16
products), exponentials and fp32 sums add less than 1e-4 of the same."""
import numpy as np
import pytest
import torch

from block_diffusion_speculative_fusion_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_fusion_gb300 import build
    build.build()
    api.lib()


class Case:
    """Tables whose groups share the pages of their prefixes; the pages' rows past a
    context, the pages in no context and the table past the context hold junk."""

    def __init__(self, ctx, group, prefix, n_q=4, n_kv=None, Hq=4, Hkv=2, D=128, page=16, dtype=torch.bfloat16, seed=0,
                 junk=float("nan")):
        g = self.g = np.random.default_rng(seed)
        t = torch.Generator().manual_seed(seed)
        B = len(ctx)
        n_kv = n_q if n_kv is None else n_kv
        self.ctx, self.group, self.prefix = list(ctx), list(group), list(prefix)
        max_pages = max(1, max(-(-c // page) for c in ctx) + 1)
        shared = {}
        table, nxt = np.full((B, max_pages), 1 << 20, dtype=np.int64), 0
        for b, c in enumerate(ctx):
            gr = group[b]
            low = min((ctx[i] for i in range(B) if group[i] == gr), default=0)
            n = -(-c // page)
            for i in range(n):
                # a page is shared if all its positions lie in the part in common
                if 0 <= gr < len(prefix) and (i + 1) * page <= min(prefix[gr], low):
                    if (gr, i) not in shared:
                        shared[gr, i] = nxt
                        nxt += 1
                    table[b, i] = shared[gr, i]
                else:
                    table[b, i] = nxt
                    nxt += 1
        num = nxt + 3
        perm = g.permutation(num)
        ok = table < num
        table[ok] = perm[table[ok]]
        # a prefix that ends inside a page: that page's rows must be the same ones too
        self.page = page
        shape = (num, page, Hkv, D)
        k, v = torch.randn(shape, generator=t), torch.randn(shape, generator=t)
        for gr, n in enumerate(prefix):
            rows = [b for b in range(B) if group[b] == gr]
            if not rows:
                continue
            n = max(0, min(n, min(ctx[b] for b in rows)))
            for b in rows[1:]:
                if n % page:
                    src, dst = table[rows[0], n // page], table[b, n // page]
                    k[dst, :n % page], v[dst, :n % page] = k[src, :n % page], v[src, :n % page]
        used = np.zeros((num, page), dtype=bool)
        for b, c in enumerate(ctx):
            for i in range(c):
                used[table[b, i // page], i % page] = True
        k[torch.from_numpy(~used)] = junk
        v[torch.from_numpy(~used)] = junk
        self.k, self.v = k.to(dtype).to(DEV), v.to(dtype).to(DEV)
        self.q = torch.randn((B, n_q, Hq, D), generator=t).to(dtype).to(DEV)
        self.kb = torch.randn((B, n_kv, Hkv, D), generator=t).to(dtype).to(DEV)
        self.vb = torch.randn((B, n_kv, Hkv, D), generator=t).to(dtype).to(DEV)
        table[~ok] = -5
        self.table = torch.from_numpy(table.astype(np.int32)).to(DEV)

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def run(self, causal=False, **kw):
        return api.prefix_attn(self.q, self.kb, self.vb, self.k, self.v, self.table, self.i32(self.ctx),
                               self.i32(self.group), self.i32(self.prefix), causal=causal, **kw)

    def reference(self, causal=False, scale=None):
        """(out, size of a tolerance's terms) in 64 bits."""
        B, n_q, Hq, D = self.q.shape
        n_kv, Hkv = self.kb.shape[1:3]
        scale = D ** -0.5 if scale is None else scale
        out = torch.zeros((B, n_q, Hq, D), dtype=torch.float64, device=DEV)
        size = torch.zeros_like(out)
        for b, c in enumerate(self.ctx):
            slot = torch.arange(c, device=DEV)
            slot = self.table[b].long()[slot // self.page] * self.page + slot % self.page
            k = torch.cat([self.k.view(-1, Hkv, D)[slot], self.kb[b]]).double().repeat_interleave(Hq // Hkv, 1)
            v = torch.cat([self.v.view(-1, Hkv, D)[slot], self.vb[b]]).double().repeat_interleave(Hq // Hkv, 1)
            if c + n_kv == 0:
                continue
            z = torch.einsum("ihd,khd->hik", self.q[b].double(), k) * scale
            if causal:
                i, j = torch.arange(n_q, device=DEV)[:, None], torch.arange(c + n_kv, device=DEV)[None]
                z = z.masked_fill(j > c + i + n_kv - n_q, -torch.inf)
            p = torch.softmax(z, -1)
            out[b] = torch.einsum("hik,khd->ihd", p, v)
            size[b] = torch.einsum("hik,khd->ihd", p, v.abs())
        return out, size

    def check(self, causal=False, **kw):
        got = self.run(causal, **kw)
        ref, size = self.reference(causal, kw.get("scale"))
        half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -22
        tol = (size + ref.abs()) * (half + 1e-4) if got.dtype == torch.bfloat16 else (size + ref.abs()) * 2e-5
        err = (got.double() - ref).abs()
        assert bool(torch.isfinite(got.float()).all())
        assert bool((err <= tol + 1e-30).all()), float((err / (tol + 1e-30)).max())
        assert torch.equal(got, self.run(causal, **kw))          # the same bits each time
        assert set(api.error_words().values()) == {0}
        return got


@pytest.mark.parametrize("prefix", [0, 1, 100, 127, 128, 129, 255, 256, 300, 640, 1000, 2048])
@pytest.mark.parametrize("causal", [False, True])
def test_one_group(prefix, causal):
    own = [0, 5, 1, 130, 17, 64, 0, 300]
    Case([prefix + n for n in own], [0] * 8, [prefix], n_q=16, Hq=8, seed=prefix).check(causal)


@pytest.mark.parametrize("n_q,Hq,Hkv", [(1, 4, 4), (1, 8, 1), (1, 32, 8), (3, 5, 5), (7, 6, 2), (16, 32, 8), (10, 32, 8),
                                        (33, 8, 2), (40, 8, 2), (64, 16, 4), (70, 4, 1), (128, 2, 2)])
def test_heads_and_blocks(n_q, Hq, Hkv):
    # packed rows of 1 to 280 a sequence, 7 to 1960 a group
    Case([700, 650, 641, 640, 1030, 900, 777], [0] * 7, [640], n_q=n_q, Hq=Hq, Hkv=Hkv, seed=n_q).check()


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_page_sizes(page, causal):
    ctx = [512, 513, 517, 640, 1100, 385, 384, 2]
    Case(ctx, [0, 1, 0, 1, 0, 1, 1, -1], [512, 390], n_q=8, Hq=8, page=page, seed=page).check(causal)


@pytest.mark.parametrize("n_kv", [0, 1, 2, 15, 17, 33, 64, 100, 128])
def test_block_rows(n_kv):
    c = Case([300, 256, 1000, 0, 257], [0, 0, 0, 1, 0], [256, 0], n_q=2, n_kv=n_kv, seed=n_kv)
    c.check()
    if n_kv >= 2:
        c.check(True)


@pytest.mark.parametrize("seed", range(6))
def test_many_groups(seed):
    g = np.random.default_rng(seed)
    B, n = int(g.integers(2, 80)), int(g.integers(1, 12))
    prefix = [int(x) for x in g.integers(0, 900, n)]
    group = [int(x) for x in g.integers(-2, n + 2, B)]           # some belong to none
    ctx = [(prefix[x] if 0 <= x < n else 0) + int(g.integers(0, 200)) for x in group]
    ctx[0] = 0                                                    # and its group's prefix counts for nothing
    prefix += [-4] * (n < 3 <= B - n)                             # a group without sequences
    Case(ctx, group, prefix[:B], n_q=int(g.integers(1, 17)), Hq=8, page=[16, 32][seed % 2], seed=seed).check(seed % 2 == 0)


def test_no_groups_and_lone_sequences():
    for group, prefix in (([0, 0, 0], []), ([0, 1, 2], [500, 700, 2]), ([-1, 7, -9], [300])):
        c = Case([500, 700, 3], group, prefix, n_q=8, Hq=8)
        got = c.check()
        want = api.block_attn(c.q, c.kb, c.vb, c.k, c.v, c.table, c.i32(c.ctx))
        assert float((got.float() - want.float()).abs().max()) < 2e-2


def test_long_prefix_of_many_sequences():
    # 20 sequences of 16 x 4 rows on 8 heads: five blocks of 256 rows, cut into pieces
    g = np.random.default_rng(3)
    own = [int(x) for x in g.integers(0, 400, 20)]
    Case([4000 + n for n in own], [0] * 20, [4000], n_q=16, Hq=32, Hkv=8, seed=9).check()


def test_long_context_of_one_sequence():
    Case([9000, 100, 128, 140], [0] * 4, [100], n_q=16, Hq=32, Hkv=8, seed=10).check()


@pytest.mark.parametrize("Hkv", [1, 2, 3, 8])
@pytest.mark.parametrize("own", [0, 300])
def test_groups_of_all_sizes(Hkv, own):
    # groups of 2 to 41 sequences of 16 packed rows: Q tiles alone, two on the same keys, of two
    # heads, several of each to a CTA, prefixes of an odd number of tiles and of one
    g = np.random.default_rng(Hkv)
    sizes, prefix = [2, 3, 8, 9, 16, 17, 41, 2, 3], [1000, 64, 3000, 64, 1500, 832, 3500, 2200, 130]
    group = [i for i, n in enumerate(sizes) for _ in range(n)]
    g.shuffle(group)
    ctx = [prefix[i] + (int(g.integers(0, own)) if own else 0) for i in group]
    Case(ctx, group, prefix, n_q=4, Hq=4 * Hkv, Hkv=Hkv, seed=Hkv).check()


def test_many_query_rows():
    Case([700, 650, 3], [0, 0, 1], [640, 0], n_q=260, n_kv=60, Hq=8, Hkv=2, seed=20).check()


def test_a_thousand_sequences():
    g = np.random.default_rng(4)
    n = [int(x) for x in g.integers(0, 40, 1024)]
    group = [b % 3 for b in range(1024)]
    Case([[256, 128, 140][b % 3] + n[b] for b in range(1024)], group, [256, 128, 140], n_q=1, Hq=4, Hkv=1, seed=11).check()


def test_scores_that_grow_along_the_keys():
    # each tile's largest score far above the one before: O is rescaled again and again
    c = Case([1500, 1400, 1300], [0] * 3, [1280], n_q=16, Hq=8, seed=12)
    pos = torch.arange(1500, device=DEV)
    for b in range(3):
        slot = c.table[b].long()[pos[:c.ctx[b]] // 16] * 16 + pos[:c.ctx[b]] % 16
        k = c.k.view(-1, 2, 128)
        k[slot] = (torch.sign(c.q[0, 0, 0].float()) * (pos[:c.ctx[b], None, None] / 100.0)).to(torch.bfloat16).expand(-1, 2, -1)
    c.check()
    c.check(scale=1.0)


@pytest.mark.parametrize("kw", [dict(dtype=torch.float32, D=16), dict(dtype=torch.float32, D=128), dict(D=64),
                                dict(n_kv=130, n_q=2), dict(page=4)])
def test_calls_outside_the_shared_kernel(kw):
    Case([130, 128, 200, 3], [0, 0, 0, -1], [128], n_q=kw.pop("n_q", 3), seed=13, junk=0.0, **kw).check()


def test_query_off_a_vector():
    c = Case([300, 290], [0, 0], [256], n_q=4, seed=14, junk=0.0)
    buf = torch.empty(c.q.numel() + 4, dtype=torch.bfloat16, device=DEV)
    q = buf[4:].view(c.q.shape)
    q.copy_(c.q)
    c.q = q
    c.check()


def test_output_rows_of_the_batch_alone_are_written():
    c = Case([300, 290, 5], [0, 0, 0], [256], n_q=4, seed=15)
    buf = torch.full((5, *c.q.shape[1:]), 7.0, dtype=torch.bfloat16, device=DEV)
    c.run(out=buf[1:4])
    assert bool((buf[0] == 7).all()) and bool((buf[4] == 7).all())


def test_a_bad_page_is_recorded():
    c = Case([300, 290], [0, 0], [256], n_q=4, seed=16, junk=0.0)
    need = 64 << 20
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    c.run(ws=ws)
    assert api.device_error_word(ws) == 0
    c.table[0, 1] = 1 << 30
    c.run(ws=ws)
    assert api.device_error_word(ws) == api.DEVERR_BAD_PAGE


def test_captured_and_replayed_with_other_lengths():
    c = Case([700, 650, 641, 640], [0] * 4, [640], n_q=16, Hq=8, seed=17)
    ctx, group, prefix = c.i32(c.ctx), c.i32(c.group), c.i32(c.prefix)
    out = torch.empty_like(c.q)
    args = (c.q, c.kb, c.vb, c.k, c.v, c.table, ctx, group, prefix)
    api.prefix_attn(*args, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.prefix_attn(*args, out=out)
    for lens, gr, pre in (([700, 650, 641, 640], [0] * 4, [640]), ([640, 640, 2, 640], [0, 0, 1, 0], [500]),
                          ([0, 0, 0, 0], [0] * 4, [640]), ([700, 650, 641, 640], [-1] * 4, [0])):
        ctx.copy_(c.i32(lens))
        group.copy_(c.i32(gr))
        prefix.copy_(c.i32(pre))
        out.zero_()
        graph.replay()
        want = api.prefix_attn(*args)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        c.ctx = lens
        ref, size = c.reference()
        assert bool(((out.double() - ref).abs() <= (size + ref.abs()) * (2.0 ** -8 + 1e-4)).all())


def test_a_wait_that_runs_out_ends_the_call():
    # a limit below the first copy's time: the launch returns, the word holds a wait's
    # code, and with the limit restored the same workspace gives the same bits
    c = Case([2100, 2050, 2048], [0] * 3, [2048], n_q=16, Hq=32, Hkv=8, seed=18)
    ws = torch.zeros(256 << 20, dtype=torch.uint8, device=DEV)
    want = c.run(ws=ws)
    torch.cuda.synchronize()
    api.set_wait_limit_ns(200)
    try:
        c.run(ws=ws)
        torch.cuda.synchronize()
    finally:
        api.set_wait_limit_ns(0)
    assert 1 <= api.device_error_word(ws) <= 99
    api.clear_counters(ws)
    assert torch.equal(c.run(ws=ws), want) and api.device_error_word(ws) == 0


def test_pages_past_four_gigabytes():
    # the same rows in pages at the end of pools of 140,000 (4.6 GB each)
    c = Case([700, 650, 641], [0] * 3, [640], n_q=16, Hq=32, Hkv=8, seed=21)
    want = c.check()
    num = 140000
    first = num - c.k.shape[0]
    big = [torch.empty((num, *c.k.shape[1:]), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for pool, old in zip(big, (c.k, c.v)):
        pool[first:] = old
    table = torch.where(c.table >= 0, c.table + first, c.table)
    got = api.prefix_attn(c.q, c.kb, c.vb, *big, table, c.i32(c.ctx), c.i32(c.group), c.i32(c.prefix))
    assert torch.equal(got, want)


@pytest.mark.parametrize("debug", [False, True], ids=["release", "debug"])
def test_lengths_out_of_range_are_clamped(debug):
    # above max_ctx: max_ctx; below zero: none; only the debug library records them
    from block_diffusion_speculative_fusion_gb300 import build
    build.build(debug=True)
    c = Case([700, 650, 648, 0], [0, 0, 0, 0], [640], n_q=4, Hq=8, seed=22)
    top = 640
    api.select_library(debug=debug)
    try:
        ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
        args = (c.q, c.kb, c.vb, c.k, c.v, c.table)
        rest = (c.i32(c.group), c.i32(c.prefix))
        for lens, bad in (([top] * 3 + [0], [700, 650, 1 << 30, 0]), ([top] * 3 + [0], [top] * 3 + [-9])):
            want = api.prefix_attn(*args, c.i32(lens), *rest, max_ctx=top, ws=ws)
            ws.zero_()
            got = api.prefix_attn(*args, c.i32(bad), *rest, max_ctx=top, ws=ws)
            assert torch.equal(got, want)
            assert api.device_error_word(ws) == (api.DEVERR_BAD_CTX_LEN if debug else 0)
            ws.zero_()
    finally:
        api.select_library(debug=False)
