"""A decode round of a serving program, all of it on the device and in the order a
server runs it: headroom reserved in the block tables, the block's slots mapped,
block attention, the requests' rules on the target logits, the greedy verify, the
commit materialised with 8-bit weights, the rest of the headroom given back.

Every number is chosen so that fp32 holds it exactly (logits in steps of 1/16,
penalties and biases in powers of two), so the rounds' integers are compared with
the oracle's exactly."""
import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_speculative_fusion_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, K, PAGE, MAX_PAGES, V = 5, 6, 16, 8, 1003
L, HQ, HKV, D, DM, M = 2, 4, 2, 128, 256, 2
HIST = 96


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_fusion_gb300 import build
    build.build()
    api.lib()


def _bf(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).to(DEV)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    """The persistent state of the sequences, and one round."""

    def __init__(self, num_pages, seed):
        g = self.g = np.random.default_rng(seed)
        self.num_pages = num_pages
        self.ctx = [_i32([30, 0, 15, 47, 1]), torch.empty(B, dtype=torch.int32, device=DEV)]
        self.table = torch.full((B, MAX_PAGES), -1, dtype=torch.int32, device=DEV)
        self.free = torch.from_numpy(g.permutation(num_pages).astype(np.int32)).to(DEV)
        self.held = [torch.zeros(B, dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)]
        self.n_free = [_i32([num_pages]), torch.empty(1, dtype=torch.int32, device=DEV)]
        self.short = torch.empty(B, dtype=torch.uint8, device=DEV)
        shape = (num_pages, PAGE, HKV, D)
        self.kp = [_bf(g.normal(0, 1, shape)) for _ in range(L)]
        self.vp = [_bf(g.normal(0, 1, shape)) for _ in range(L)]
        self.hist = torch.from_numpy(g.integers(0, V, (B, HIST))).to(DEV)
        self.hist_len, self.prompt_len = _i32([30, 0, 15, 40, 1]), _i32([20, 0, 15, 0, 1])
        self.W_f = api.fp8_quant(_bf(g.normal(0, 0.05, (DM, M * DM))), block_rows=128)
        w, s = api.fp8_quant(_bf(g.normal(0, 0.05, (L * 2 * HKV * D, DM))), block_rows=128)
        self.W_kv = (w.view(L, 2, HKV * D, DM), s)
        self.k_norm = _bf(np.ones((L, D)))
        self.rules = dict(repetition=torch.full((B,), 2.0, device=DEV), presence=torch.full((B,), 0.5, device=DEV),
                          frequency=torch.full((B,), 0.25, device=DEV),
                          bias_tok=torch.from_numpy(g.integers(0, V, (B, 7))).to(DEV),
                          bias_val=torch.from_numpy(g.choice([-8.0, 4.0, 2.0], (B, 7)).astype(np.float32)).to(DEV))
        self.z = torch.zeros((B, K, V), dtype=torch.bfloat16, device=DEV)
        self.attn = [torch.zeros((B, K, HQ, D), dtype=torch.bfloat16, device=DEV) for _ in range(L)]
        self.verified = {}

    def inputs(self):
        g = self.g
        x = {f"{n}{layer}": _bf(g.normal(0, 1, (B, K, h, D))) for layer in range(L)
             for n, h in (("q", HQ), ("k", HKV), ("v", HKV))}
        x["logits"] = _bf(g.integers(-128, 129, (B, K, V)) / 16)
        x["cand"] = torch.from_numpy(g.integers(0, V, (B, K))).to(DEV)
        x["hidden"] = _bf(g.normal(0, 1, (B, K, M * DM)))
        keep = g.random((B, K, 32 * 32)) < 0.6
        bits = (keep.reshape(B, K, 32, 32) * (1 << np.arange(32, dtype=np.int64))).sum(-1)
        x["mask"] = torch.from_numpy(bits.astype(np.uint32).view(np.int32)).to(DEV)
        x["mask_on"] = torch.from_numpy((np.arange(B) % 2 == 0).astype(np.uint8)).to(DEV)
        x["n_draft"] = _i32(g.integers(0, K, B).tolist())
        return x

    def round(self, x):
        ctx, new = self.ctx
        held, n_free = self.held, self.n_free
        api.pages_resize(ctx + 2 * K, self.table, held[0], self.free, n_free[0], PAGE,
                         out={"n_pages": held[1], "n_free": n_free[1], "short": self.short})
        self.slots = api.slot_map(ctx, torch.full_like(ctx, K), self.table, PAGE, self.num_pages, B * K)
        for layer in range(L):
            api.block_attn(x[f"q{layer}"], x[f"k{layer}"], x[f"v{layer}"], self.kp[layer], self.vp[layer], self.table,
                           ctx, out=self.attn[layer])
        api.logits_rules(x["logits"], cand=x["cand"], n_draft=x["n_draft"], hist=self.hist, hist_len=self.hist_len,
                         prompt_len=self.prompt_len, mask=x["mask"], mask_on=x["mask_on"], out=self.z, **self.rules)
        v = api.verify_greedy(self.z, x["cand"], x["n_draft"], out=self.verified)
        api.materialize_ctx_kv_fp8(x["hidden"], v["commit_len"], ctx, *self.W_f, None, *self.W_kv, self.k_norm, 1e-6,
                                   1e4, self.kp, self.vp, self.table, new_len=new)
        api.pages_resize(new, self.table, held[1], self.free, n_free[1], PAGE,
                         out={"n_pages": held[0], "n_free": n_free[0], "short": self.short})
        # the committed tokens join the history
        at = self.hist_len[:, None] + torch.arange(K, device=DEV)[None]
        put = torch.arange(K, device=DEV)[None] < v["commit_len"][:, None]
        old = self.hist.gather(1, at.long())
        self.hist.scatter_(1, at.long(), torch.where(put, v["out_tokens"], old))
        self.hist_len.add_(v["commit_len"])
        ctx.copy_(new)


def _check_round(s, before, x):
    """One round's integers against the oracle, from the state before it."""
    ctx, table, held, free, n_free, hist, hist_len = before
    t1, h1, f1, n1, short = O.pages_resize(ctx + 2 * K, table, held, free, n_free, PAGE)
    assert not short.any()
    r = O.slot_map(ctx, [K] * B, t1, PAGE, s.num_pages, B * K)
    for name, want in zip(("cu_rows", "row_seq", "positions", "slots"), r):
        assert np.array_equal(s.slots[name].cpu().numpy(), want), name
    host = {k: x[k].cpu().float().numpy() if x[k].is_floating_point() else x[k].cpu().numpy()
            for k in ("logits", "cand", "n_draft", "mask", "mask_on")}
    z, _ = O.logits_rules(host["logits"], cand=host["cand"], n_draft=host["n_draft"], hist=hist, hist_len=hist_len,
                          prompt_len=s.prompt_len.cpu().numpy(), mask=host["mask"], mask_on=host["mask_on"],
                          **{k: v.cpu().numpy() for k, v in s.rules.items()})
    z = torch.from_numpy(z).to(torch.bfloat16).float().numpy()
    got = s.z.float().cpu().numpy()
    for b in range(B):
        n = int(host["n_draft"][b]) + 1
        assert np.array_equal(got[b, :n], z[b, :n])
    v = O.verify_greedy(z.astype(np.float64), host["cand"], host["n_draft"])
    for k in ("accept_len", "bonus", "commit_len", "out_tokens"):
        assert np.array_equal(s.verified[k].cpu().numpy(), v[k]), k
    new = ctx + v["commit_len"]
    assert np.array_equal(s.ctx[0].cpu().numpy(), new)
    t2, h2, f2, n2, _ = O.pages_resize(new, t1, h1, f1, n1, PAGE)
    assert np.array_equal(s.table.cpu().numpy(), t2) and np.array_equal(s.held[0].cpu().numpy(), h2)
    assert np.array_equal(s.free.cpu().numpy(), f2) and int(s.n_free[0]) == n2
    return v


def _snapshot(s):
    return (s.ctx[0].cpu().numpy(), s.table.cpu().numpy(), s.held[0].cpu().numpy(), s.free.cpu().numpy(),
            int(s.n_free[0]), s.hist.cpu().numpy(), s.hist_len.cpu().numpy())


def test_rounds_against_the_oracle():
    s = Server(40, seed=1)
    for _ in range(4):
        x = s.inputs()
        # a candidate that the rules let through, so that some drafts are accepted
        z0 = api.logits_rules(x["logits"], hist=s.hist, hist_len=s.hist_len, prompt_len=s.prompt_len, mask=x["mask"],
                              mask_on=x["mask_on"], **s.rules)
        x["cand"][::2, 1] = z0[::2, 0].float().argmax(-1)
        before = _snapshot(s)
        pools = [p.clone() for p in s.kp + s.vp]
        s.round(x)
        v = _check_round(s, before, x)
        # the pools change at the committed rows' slots and nowhere else
        rows = [int(s.slots["cu_rows"][b]) + j for b in range(B) for j in range(int(v["commit_len"][b]))]
        slots = s.slots["slots"][rows]
        for new, old in zip(s.kp + s.vp, pools):
            changed = (new != old).view(-1, HKV * D).any(1).nonzero().flatten()
            assert set(changed.tolist()) == set(slots.tolist())
            assert torch.isfinite(new.float()).all()
        assert all(torch.isfinite(a.float()).all() for a in s.attn)
    assert set(api.error_words().values()) == {0}


def test_captured_round_replays():
    s, t = Server(40, seed=2), Server(40, seed=2)
    first = s.inputs()
    t.inputs()
    s.round(first)                             # workspaces exist and kernels are loaded before the capture
    t.round(first)
    x = s.inputs()
    fixed = {k: v.clone() for k, v in x.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.round(fixed)
    for _ in range(3):
        for k in fixed:
            fixed[k].copy_(x[k])
        graph.replay()
        s.round(x)
        for a, b in zip([s.z, s.hist, s.hist_len, s.table, s.free, s.ctx[0], s.n_free[0], *s.kp, *s.vp, *s.attn],
                        [t.z, t.hist, t.hist_len, t.table, t.free, t.ctx[0], t.n_free[0], *t.kp, *t.vp, *t.attn]):
            assert torch.equal(a, b)
        x = s.inputs()


def test_rounds_until_the_pool_is_dry():
    # a pool that holds the sequences but not everyone's headroom: those left short keep
    # what they have, and get theirs once another sequence ends
    s = Server(12, seed=3)
    s.round(s.inputs())
    assert int(s.held[0].sum()) + int(s.n_free[0]) == 12
    ctx = s.ctx[0]
    r = api.pages_resize(ctx + 100, s.table, s.held[0], s.free, s.n_free[0], PAGE)
    assert int(r["short"].sum()) > 0
    ended = torch.where(torch.arange(B, device=DEV) == 3, 0, ctx + 16).int()
    r2 = api.pages_resize(ended, s.table, r["n_pages"], s.free, r["n_free"], PAGE)
    assert int(r2["n_pages"][3]) == 0
    live = torch.cat([s.table[b, :int(r2["n_pages"][b])] for b in range(B)] + [s.free[:int(r2["n_free"])]])
    assert sorted(live.tolist()) == list(range(12))


@pytest.mark.parametrize("captured", [False, True])
def test_launches_that_overlap_see_each_others_results(captured):
    """Every operator's launch may begin while the kernel before it ends: calls
    in a row that read what the one before wrote, over the same buffers, give
    what the same calls give one at a time."""
    B, R, V, T, K, N, page, max_pages = 4, 3, 5000, 40, 1024, 640, 16, 64
    g = torch.Generator().manual_seed(12)
    n = 6
    logits = torch.randn((n, B, R, V), generator=g).to(torch.bfloat16).to(DEV)
    hist = torch.randint(0, V, (n, B, 300), generator=g).to(DEV)
    x = torch.randn((n, T, K), generator=g).to(torch.bfloat16).to(DEV)
    w, ws = api.fp8_quant(torch.randn((N, K), generator=g).to(torch.bfloat16).to(DEV), block_rows=128)
    length = torch.randint(0, page * max_pages, (n, B), generator=g).to(torch.int32).to(DEV)
    length[-1] = 0
    hl = torch.full((B,), 300, dtype=torch.int32, device=DEV)
    rep = torch.full((B,), 1.5, device=DEV)
    zero = torch.zeros(B, dtype=torch.int32, device=DEV)
    buf = dict(z=torch.empty_like(logits[0]), hist=torch.empty_like(hist[0]), x=torch.empty_like(x[0]),
               q=torch.empty((T, K), dtype=torch.float8_e4m3fn, device=DEV),
               s=torch.empty((T, K // 128), dtype=torch.float32, device=DEV),
               y=torch.empty((T, N), dtype=torch.bfloat16, device=DEV),
               len=torch.empty(B, dtype=torch.int32, device=DEV),
               table=torch.empty((B, max_pages), dtype=torch.int32, device=DEV),
               free=torch.empty(B * max_pages, dtype=torch.int32, device=DEV))
    pages = [{k: torch.zeros(m, dtype=t, device=DEV) for k, m, t in
              (("n_pages", B, torch.int32), ("n_free", 1, torch.int32), ("short", B, torch.uint8))} for _ in range(2)]
    y = torch.empty((n, T, N), dtype=torch.bfloat16, device=DEV)
    z = torch.empty_like(logits)
    slots = torch.empty((n, B * 8), dtype=torch.int64, device=DEV)

    def run(one_at_a_time):
        def call(fn, *args, **kw):
            fn(*args, **kw)
            if one_at_a_time:
                torch.cuda.synchronize()
        call(buf["table"].fill_, -1)
        call(buf["free"].copy_, torch.arange(B * max_pages, dtype=torch.int32, device=DEV))
        call(pages[0]["n_pages"].zero_)
        call(pages[0]["n_free"].fill_, B * max_pages)
        yq, ys = buf["q"].view(-1)[:T * N].view(T, N), buf["s"].view(-1)[:T * 5].view(T, 5)
        for i in range(n):
            call(buf["x"].copy_, x[i])
            call(api.fp8_quant, buf["x"], q=buf["q"], scale=buf["s"])
            call(api.fp8_gemm, buf["q"], buf["s"], w, ws, out=buf["y"])
            call(api.fp8_gemm, buf["q"], buf["s"], w, ws, out=y[i])
            call(api.fp8_quant, buf["y"], q=yq, scale=ys)
            old, new = pages[i % 2], pages[1 - i % 2]
            call(api.pages_resize, length[i], buf["table"], old["n_pages"], buf["free"], old["n_free"], page, out=new)
            call(api.slot_map, zero, new["n_pages"], buf["table"], page, B * max_pages, B * 8, out=dict(slots=slots[i]))
            call(buf["hist"].copy_, hist[i])
            call(buf["z"].copy_, logits[i])
            call(api.logits_rules, buf["z"], hist=buf["hist"], hist_len=hl, repetition=rep, out=buf["z"])
            call(api.logits_rules, buf["z"], hist=buf["hist"], hist_len=hl, repetition=rep, out=z[i])

    def result():
        torch.cuda.synchronize()
        return [t.clone() for t in (y, z, slots, buf["table"], buf["free"], pages[n % 2]["n_free"])]

    run(True)
    want = result()
    assert int(want[-1]) == B * max_pages and bool((want[2][:-1] >= 0).any())
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(False)
    for _ in range(5):
        for t in (y, z, slots):
            t.zero_()
        graph.replay() if captured else run(False)
        for a, b in zip(result(), want):
            assert torch.equal(a, b)
