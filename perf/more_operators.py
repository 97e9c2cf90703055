"""Sequences that share a prefix, and the norm in front of an 8-bit product, as cases to measure.

Five operators, each in its plain form (elementary torch operations) and through
the library's binding (``own``):

  attn      the draft block's attention for a batch whose sequences share long
            prefixes in groups: a prefix's K/V stand once in the paged cache
  fork      new sequences that begin as copies of others: their whole pages are
            held together (counted), the rows of a page begun are copied
  release   pages that sequences let go, freed where no other one holds them
  compact   the pages in use moved to the pools' low end, tables rewritten
  norm      root-mean-square norm of a sum with the residual, in e4m3 with one
            scale per 128 values

Sizes are those of the workloads (Llama-3.1-8B and Qwen3-4B draft shapes: d =
4096 / 2560, 32 query and 8 K/V heads of 128, five draft layers, blocks of 8 to 16
rows, 16-token pages, contexts up to 8192) or generic odd ones.
"""
import math

import torch

own = False

GROUP = 128           # values per scale
E4M3_MAX = 448.0
NORMAL_MIN = 2.0 ** -126
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attn(**kw):
    base = dict(op="attn", dtype="bf16", Hq=32, Hkv=8, D=128, page=16, causal=False)
    return dict(base, **kw)


def listed():
    return [
        # four samples of one short prompt, a token at a time: the latency of a call
        _attn(name="attn_b4_q1_p500", B=4, n_q=1, groups=1, p_lo=500, p_hi=500, s_hi=64),
        # eight samples of one prompt, the Qwen3-4B draft's block
        _attn(name="attn_b8_q16_p1024", B=8, n_q=16, groups=1, p_lo=1024, p_hi=1024, s_hi=200),
        # the DLoop batch under several prompts of odd lengths, the causal variant
        _attn(name="attn_b32_q8_groups", B=32, n_q=8, groups=7, p_lo=33, p_hi=4096, s_hi=1000, causal=True),
        # the throughput workload's batch behind one long system prompt
        _attn(name="attn_b64_q16_p8192", B=64, n_q=16, groups=1, p_lo=8192, p_hi=8192, s_hi=512),
        # eight samples begun from one prompt
        dict(name="fork_b8", op="fork", B=8, family=8, max_len=2048, layers=5, page=16, row=1024),
        # a thousand rows, 128 prompts of which each is sampled eight times
        dict(name="fork_b1024", op="fork", B=1024, family=8, max_len=2048, layers=5, page=16, row=1024),
        # samples of eight prompts, a quarter of them at their end
        dict(name="release_b64", op="release", B=64, family=8, max_len=8192, ended=0.25, page=16),
        # a thousand sequences, most of them at their end
        dict(name="release_b1024", op="release", B=1024, family=5, max_len=4096, ended=0.75, page=16),
        # one layer's cache of a few sequences
        dict(name="compact_b8", op="compact", B=8, family=2, max_len=1024, ended=0.25, layers=1, page=16, row=1024),
        # the five layers of the throughput workload after half of it has ended
        dict(name="compact_b64", op="compact", B=64, family=4, max_len=8192, ended=0.5, layers=5, page=16, row=1024),
        # the rows of one block
        dict(name="norm_t10_d4096", op="norm", dtype="bf16", T=10, d=4096, residual=True, fp8=True),
        # the rows of a prefill
        dict(name="norm_t8190_d4096", op="norm", dtype="bf16", T=8190, d=4096, residual=True, fp8=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "fork", "release", "compact", "norm", "norm"])
    if op == "attn":
        if rng.random() < 0.1:
            # the tiny fp32 configuration's heads
            return _attn(dtype="f32", Hq=4, Hkv=2, D=16, B=rng.randint(1, 4), n_q=rng.randint(1, 4), groups=1,
                         p_lo=1, p_hi=_log(rng, 16, 256), s_hi=_log(rng, 1, 32), causal=rng.random() < 0.5)
        Hkv, g = rng.choice([(8, 4), (8, 4), (4, 4), (8, 2), (2, 8), (4, 1)])
        B, n_q, hi = _log(rng, 1, 64), rng.choice([1, 1, rng.randint(2, 16), 16]), _log(rng, 16, 8192)
        return _attn(B=B, n_q=n_q, Hq=Hkv * g, Hkv=Hkv, groups=rng.choice([1, 1, _log(rng, 1, max(1, B // 2))]),
                     p_lo=rng.choice([hi, rng.randint(1, hi)]), p_hi=hi, s_hi=_log(rng, 1, 512),
                     page=rng.choice([16, 16, 32, 64]), causal=rng.random() < 0.3)
    if op == "norm":
        wide = rng.random() < 0.5
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), T=_log(rng, 1, 4095),
                    d=rng.choice([2560, 4096]) if wide else 16 * _log(rng, 1, 256), residual=rng.random() < 0.7,
                    fp8=rng.random() < 0.7)
    B = _log(rng, 2, 64 if op == "compact" else 1024)
    c = dict(op=op, B=B, family=rng.randint(2 if op == "fork" else 1, min(B, 9)), page=rng.choice([16, 16, 32]),
             max_len=_log(rng, 20, 8192 if op == "compact" else 2048))
    if op != "fork":
        c["ended"] = rng.choice([0.0, 0.1, 0.5, 0.9])
    if op != "release":
        c["layers"], c["row"] = rng.randint(1, 5), rng.choice([1024, 512, 256])
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randint(lo, hi, shape, g, dtype=torch.int32):
    """Uniform whole numbers lo .. hi, both included."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(dtype)


def _normal(shape, dtype, g):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def _ceil(a, b):
    return -(-a // b)


def _tables(shared, own_pages, fam, n_fam, max_pages, g, spare):
    """Tables of rows that hold shared[b] pages with the rest of their family and
    own_pages[b] of their own, at random places of the pool; the pages left over;
    the pool's size."""
    B = len(fam)
    per_fam = torch.zeros(n_fam, dtype=torch.int64, device="cuda").scatter_reduce_(0, fam, shared, "amax")
    n_own = own_pages.sum()
    num = B * max_pages + spare
    perm = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    own0 = torch.cumsum(own_pages, 0) - own_pages
    fam0 = n_own + torch.cumsum(per_fam, 0) - per_fam
    col = torch.arange(max_pages, device="cuda")[None]
    at = torch.where(col < shared[:, None], fam0[fam][:, None] + col, own0[:, None] + col - shared[:, None])
    held = (shared + own_pages)[:, None]
    table = torch.where(col < held, perm[at.clamp(0, num - 1)], -1).int().contiguous()
    n_held = n_own + per_fam.sum()
    free = perm[(torch.arange(num, device="cuda") + n_held) % num].contiguous()
    return table, free, (num - n_held).to(torch.int32).reshape(1), num


def _attn_state(c, g):
    B, page, groups = c["B"], c["page"], c["groups"]
    # members of a group lie anywhere in the batch
    group = (torch.randperm(B, generator=g, device="cuda") % groups).int()
    prefix = _randint(c["p_lo"], c["p_hi"], (groups,), g) // page * page      # whole pages are shared
    mine = prefix[group.long()]
    ctx = mine + _randint(0, c["s_hi"], (B,), g)
    shared = (mine // page).long()
    max_pages = _ceil(c["p_hi"] + c["s_hi"], page)
    table, _, _, _ = _tables(shared, _ceil(ctx, page).long() - shared, group.long(), groups, max_pages, g, 0)
    # the pool holds the pages in use and no more: one number each, in the order of their random places
    used = torch.unique(table)
    used = used[used >= 0]
    num = max(1, len(used))
    at = torch.searchsorted(used, table.clamp(min=0).contiguous()).clamp_(max=num - 1)
    mix = torch.randperm(num, generator=g, device="cuda").int()
    table = torch.where(table >= 0, mix[at], -1).int().contiguous()
    dt, Hkv, D = _dt(c), c["Hkv"], c["D"]
    pool = (num, page, Hkv, D)
    s = {"op": "attn", "q": _normal((B, c["n_q"], c["Hq"], D), dt, g), "k_blk": _normal((B, c["n_q"], Hkv, D), dt, g),
         "v_blk": _normal((B, c["n_q"], Hkv, D), dt, g), "k_pool": _normal(pool, dt, g), "v_pool": _normal(pool, dt, g)}
    return dict(s, page_table=table, ctx_len=ctx.int(), group=group, prefix_len=prefix, causal=c["causal"])


def _families(c, g):
    """(family of each row, number of families, head row of each family); rows in random order."""
    B = c["B"]
    n = _ceil(B, c["family"])
    at = torch.randperm(B, generator=g, device="cuda")
    fam = torch.empty(B, dtype=torch.int64, device="cuda")
    fam[at] = torch.arange(B, device="cuda") % n
    return fam, n, at[:n]


def _pools(c, num, g):
    return [_normal((num, c["page"], c["row"]), torch.bfloat16, g) for _ in range(2 * c["layers"])]


def _fork_state(c, g):
    B, page, top = c["B"], c["page"], c["max_len"]
    fam, n, head = _families(c, g)
    max_pages = _ceil(top + 32, page)
    is_head = torch.zeros(B, dtype=torch.bool, device="cuda")
    is_head[head] = True
    length = torch.where(is_head, _randint((top + 1) // 2, top, (B,), g), 0).int()
    held = _ceil(length, page).long()
    parent = torch.where(is_head, -1, head[fam]).int()
    # one family in sixteen is not sampled again
    parent = torch.where((fam % 16 == 15), -1, parent).int()
    table, free, n_free, num = _tables(torch.zeros_like(held), held, fam, n, max_pages, g, 0)
    # a pool with room for what the heads hold and one page a row
    keep = n * max_pages + B
    used = torch.sort(table.view(-1)).values
    order = torch.argsort((~torch.isin(torch.arange(num, device="cuda", dtype=torch.int32), used)).int(), stable=True)
    new = torch.empty(num, dtype=torch.int32, device="cuda")
    mix = torch.randperm(keep, generator=g, device="cuda").int()
    new[order] = torch.cat([mix, torch.arange(keep, max(keep, num), dtype=torch.int32, device="cuda")])[:num]
    table = torch.where(table >= 0, new[table.clamp(min=0).long()], -1).int().contiguous()
    total = held.sum()
    free = mix[(torch.arange(keep, device="cuda") + total) % keep].contiguous()
    return {"op": "fork", "parent": parent, "length": length, "page_table": table, "n_pages": held.int(),
            "shares": torch.zeros(keep, dtype=torch.int32, device="cuda"), "free_pages": free,
            "n_free": (keep - total).to(torch.int32).reshape(1), "pools": _pools(c, keep, g), "page": page}


def _forest(c, g):
    """Sequences of which those of a family share the pages of their prompt."""
    B, page, top = c["B"], c["page"], c["max_len"]
    fam, n, _ = _families(c, g)
    size = torch.bincount(fam, minlength=n)
    prompt = _randint(1, top, (n,), g).long()
    shared = torch.where(size > 1, prompt // page, 0)[fam]
    length = prompt[fam] + _randint(0, max(1, top // 8), (B,), g).long()
    max_pages = _ceil(top + max(1, top // 8) + 32, page)
    held = _ceil(length + 32, page)                     # with the headroom of a round
    table, free, n_free, num = _tables(shared, held - shared, fam, n, max_pages, g, 0)
    shares = torch.zeros(num, dtype=torch.int32, device="cuda")
    live = torch.arange(max_pages, device="cuda")[None] < held[:, None]
    shares.index_add_(0, table.clamp(min=0).view(-1).long(), live.view(-1).int())
    shares = (shares - 1).clamp_(min=0)
    ended = torch.rand(B, generator=g, device="cuda") < c["ended"]
    return dict(length=torch.where(ended, 0, length).int(), page_table=table, n_pages=held.int(), shares=shares,
                free_pages=free, n_free=n_free, page=page), ended, num


def _release_state(c, g):
    s, _, _ = _forest(c, g)
    return dict(s, op="release")


def _compact_state(c, g):
    s, ended, num = _forest(c, g)
    # the rows that have ended hold nothing any more
    n_pages = torch.where(ended, 0, s["n_pages"])
    live = torch.arange(s["page_table"].shape[1], device="cuda")[None] < n_pages[:, None]
    held = torch.zeros(num, dtype=torch.int32, device="cuda")
    held.index_add_(0, s["page_table"].clamp(min=0).view(-1).long(), live.view(-1).int())
    return {"op": "compact", "page_table": s["page_table"], "n_pages": n_pages, "shares": (held - 1).clamp_(min=0),
            "pools": _pools(c, num, g), "page": c["page"]}


def _hidden(T, d, dtype, g):
    """Rows as hidden states are: a few channels far larger than the rest."""
    x = torch.randn((T, d), generator=g, device="cuda")
    x *= torch.where(torch.rand(d, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(dtype)


def _norm_state(c, g):
    T, d, dt = c["T"], c["d"], _dt(c)
    return {"op": "norm", "x": _hidden(T, d, dt, g), "residual": _hidden(T, d, dt, g) if c["residual"] else None,
            "weight": (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt), "fp8": c["fp8"]}


def prepare(case, seed):
    g = _gen(seed)
    return {"attn": _attn_state, "fork": _fork_state, "release": _release_state, "compact": _compact_state,
            "norm": _norm_state}[case["op"]](case, g)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _attn_plain(s):
    q, table, ctx = s["q"], s["page_table"], s["ctx_len"].long()
    B, n_q, Hq, D = q.shape
    page, Hkv = s["k_pool"].shape[1], s["k_pool"].shape[2]
    n_kv, C = s["k_blk"].shape[1], table.shape[1] * page
    at = table.clamp(min=0).long()

    def rows(pool, blk):
        ctx_rows = pool[at].view(B, C, Hkv, D)
        return torch.cat([ctx_rows, blk], 1).float().permute(0, 2, 1, 3)          # [B, Hkv, C + n_kv, D]

    k, v = rows(s["k_pool"], s["k_blk"]), rows(s["v_pool"], s["v_blk"])
    key = torch.arange(C + n_kv, device=q.device)
    seen = (key[None] < ctx[:, None]) | (key[None] >= C)                         # [B, C + n_kv]
    seen = seen[:, None].expand(B, n_q, -1)
    if s["causal"]:
        i = torch.arange(n_q, device=q.device)
        seen = seen & ((key[None] < C) | (key[None] - C <= i[:, None] + n_kv - n_q))[None]
    qh = q.float().view(B, n_q, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    z = (qh @ k.transpose(2, 3)) * D ** -0.5                                     # [B, Hkv, G n_q, C + n_kv]
    z = z.view(B, Hkv, Hq // Hkv, n_q, -1).masked_fill_(~seen[:, None, None], float("-inf"))
    z = torch.exp(z - z.amax(-1, keepdim=True))
    z = (z / z.sum(-1, keepdim=True)).view(B, Hkv, -1, C + n_kv)
    o = (z @ v).view(B, Hkv, Hq // Hkv, n_q, D).permute(0, 3, 1, 2, 4)
    return o.reshape(B, n_q, Hq, D).to(q.dtype)


def _fork_plain(s):
    table, parent, page = s["page_table"], s["parent"].long(), s["page"]
    B, max_pages = table.shape
    num = len(s["free_pages"])
    p = parent.clamp(min=0)
    child = parent >= 0
    full = torch.where(child, s["length"].long()[p] // page, 0)
    rest = torch.where(child, s["length"].long()[p] % page, 0)
    want = (rest > 0).long()
    upto = torch.cumsum(want, 0)
    granted = child & ((want == 0) | (upto <= s["n_free"].long()))
    col = torch.arange(max_pages, device=table.device)[None]
    both = granted[:, None] & (col < full[:, None])
    new = s["free_pages"][(s["n_free"].long() - upto).clamp(0, num - 1)]
    begun = granted & (rest > 0)
    mine = torch.where(both, table[p], table)
    mine = torch.where(begun[:, None] & (col == full[:, None]), new[:, None], mine)
    shares = s["shares"].clone()
    shares.index_add_(0, mine.clamp(min=0).view(-1).long(), both.view(-1).int())
    src, dst, n = table[p, full.clamp(max=max_pages - 1)][begun].long(), new[begun].long(), rest[begun]
    first = torch.arange(page, device=table.device)[None, :, None] < n[:, None, None]
    for pool in s["pools"]:
        pool[dst] = torch.where(first, pool[src], pool[dst])
    table.copy_(mine)
    n_pages = torch.where(granted, full + want, s["n_pages"].long()).int()
    return {"page_table": table, "n_pages": n_pages, "shares": shares, "pools": s["pools"],
            "n_free": (s["n_free"] - (want * granted).sum()).int(), "short": (child & ~granted).to(torch.uint8)}


def _release_plain(s):
    table, have, page, free = s["page_table"], s["n_pages"].long(), s["page"], s["free_pages"]
    max_pages, num = table.shape[1], len(free)
    need = torch.minimum(_ceil(s["length"].long(), page), have)
    col = torch.arange(max_pages, device=table.device)[None]
    gone = (col >= need[:, None]) & (col < have[:, None])
    n = torch.zeros(num, dtype=torch.int32, device=table.device)
    n.index_add_(0, table.clamp(min=0).view(-1).long(), gone.view(-1).int())
    freed = n > s["shares"]
    at = s["n_free"].long() + torch.cumsum(freed, 0) - 1
    pages = torch.arange(num, dtype=torch.int32, device=table.device)
    grown = torch.cat([free, free[:1]]).scatter_(0, torch.where(freed, at, num), pages)[:num]
    free.copy_(grown)
    return {"free_pages": free, "n_pages": need.int(), "n_free": (s["n_free"] + freed.sum()).int(),
            "shares": torch.where(freed, 0, s["shares"] - n)}


def _compact_plain(s):
    table, have = s["page_table"], s["n_pages"].long()
    num, max_pages = len(s["shares"]), table.shape[1]
    dev = table.device
    live = torch.arange(max_pages, device=dev)[None] < have[:, None]
    used = torch.zeros(num, dtype=torch.int32, device=dev)
    used = used.index_add_(0, table.clamp(min=0).view(-1).long(), live.view(-1).int()) > 0
    n_used = used.sum()
    page = torch.arange(num, device=dev)
    moving, hole = used & (page >= n_used), ~used & (page < n_used)
    src, dst = moving.nonzero()[:, 0], hole.nonzero()[:, 0]
    to = page.clone()
    to[src] = dst
    out = torch.where(live, to[table.clamp(min=0).long()].int(), table)
    shares = torch.where(used, s["shares"], 0)
    shares[dst] = shares[src]
    shares[src] = 0
    for pool in s["pools"]:
        pool[dst] = pool[src]
    return {"page_table": out, "shares": shares, "pools": s["pools"], "free_pages": (num - 1 - page).int(),
            "n_free": (num - n_used).int().reshape(1)}


def _norm_plain(s):
    x = s["x"].float()
    out = {}
    if s["residual"] is not None:
        x = x + s["residual"].float()
        out["sum"] = x.to(s["x"].dtype)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if not s["fp8"]:
        return dict(out, y=y.to(s["x"].dtype))
    T, d = y.shape
    G = _ceil(d, GROUP)
    pad = torch.nn.functional.pad(y.abs(), (0, G * GROUP - d))
    scale = torch.clamp(pad.view(T, G, GROUP).amax(2) / E4M3_MAX, min=NORMAL_MIN)
    q = y / scale.repeat_interleave(GROUP, 1)[:, :d]
    return dict(out, q=q.to(torch.float8_e4m3fn), scale=scale)


def run(state):
    op = state["op"]
    s = state
    if own:
        from block_diffusion_speculative_fusion_gb300 import api
        if op == "attn":
            return api.prefix_attn(s["q"], s["k_blk"], s["v_blk"], s["k_pool"], s["v_pool"], s["page_table"],
                                   s["ctx_len"], s["group"], s["prefix_len"], causal=s["causal"])
        if op == "fork":
            r = api.pages_fork(s["parent"], s["length"], s["page_table"], s["n_pages"], s["shares"], s["free_pages"],
                               s["n_free"], s["page"], s["pools"])
            return dict(r, page_table=s["page_table"], pools=s["pools"])
        if op == "release":
            r = api.pages_release(s["length"], s["page_table"], s["n_pages"], s["shares"], s["free_pages"],
                                  s["n_free"], s["page"])
            return dict(r, free_pages=s["free_pages"])
        if op == "compact":
            return dict(api.pages_compact(s["page_table"], s["n_pages"], s["shares"], s["page"], s["pools"]),
                        pools=s["pools"])
        return api.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], fp8=s["fp8"])
    return {"attn": _attn_plain, "fork": _fork_plain, "release": _release_plain, "compact": _compact_plain,
            "norm": _norm_plain}[op](s)


# ---------------------------------------------------------------------------
# the least work of one pass
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "attn":
        el = 2 if case["dtype"] == "bf16" else 4
        B, n_q, Hq, Hkv, D, page = (case[k] for k in ("B", "n_q", "Hq", "Hkv", "D", "page"))
        prefix = (case["p_lo"] + case["p_hi"]) / 2 // page * page
        rows = case["groups"] * prefix + B * (case["s_hi"] / 2 + n_q)            # K/V rows, each once
        keys = B * (prefix + case["s_hi"] / 2 + n_q)                             # that the queries see
        return {"bytes": int(rows * Hkv * D * 2 * el + 2 * B * n_q * Hq * D * el + B * prefix / page * 4),
                "flops": int(4 * keys * n_q * Hq * D)}
    if op == "norm":
        el = 2 if case["dtype"] == "bf16" else 4
        T, d = case["T"], case["d"]
        n = T * d * el * (3 if case["residual"] else 1) + d * el
        n += T * d + T * _ceil(d, GROUP) * 4 if case["fp8"] else T * d * el
        return {"bytes": n, "flops": T * d * 5}
    B, page, top, fam = case["B"], case["page"], case["max_len"], case["family"]
    heads = _ceil(B, fam)
    if op == "fork":
        pages = 0.75 * top / page
        num = heads * _ceil(top + 32, page) + B
        copied = (B - heads) * page / 2 * case["row"] * 2 * 2 * case["layers"]   # rows of the pages begun
        return {"bytes": int(heads * pages * 4 + (B - heads) * pages * 4 + num * 8 + 2 * copied + B * 17),
                "flops": int(B)}
    # the pages of a family's prompt, and each row's own
    prompt, mine = top / 2 / page, (top / 16 + 48) / page
    num = B * _ceil(top + max(1, top // 8) + 32, page)
    if op == "release":
        gone = B * (case["ended"] * (prompt + mine) + (1 - case["ended"]) * 32 / page)
        return {"bytes": int(gone * 8 + num * 8 + B * 12), "flops": int(gone)}
    left = 1 - case["ended"]
    used = heads * (1 - case["ended"] ** fam) * prompt + B * left * mine if fam > 1 else B * left * (prompt + mine)
    used = min(used, num)
    moved = used * (1 - used / num) * page * case["row"] * 2 * 2 * case["layers"]
    table = B * _ceil(top + max(1, top // 8) + 32, page) * 8
    return {"bytes": int(2 * moved + table + num * 12), "flops": int(num)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _grid_e4m3(v):
    """The nearest value of the e4m3 grid, ties to the even one, by magnitude at most 448."""
    a = v.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -20))).clamp(min=-6)
    e = torch.where(a >= torch.exp2(e + 1), e + 1, e)        # log2 may land below a power of two
    step = torch.exp2(e - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _attn_exact(s):
    q = s["q"]
    B, n_q, Hq, D = q.shape
    page, Hkv = s["k_pool"].shape[1], s["k_pool"].shape[2]
    n_kv = s["k_blk"].shape[1]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    for b in range(B):
        C = int(s["ctx_len"][b])
        slot = torch.arange(C, device=q.device)
        slot = s["page_table"][b].long()[slot // page] * page + slot % page
        k = torch.cat([s["k_pool"].view(-1, Hkv, D)[slot], s["k_blk"][b]]).double()
        v = torch.cat([s["v_pool"].view(-1, Hkv, D)[slot], s["v_blk"][b]]).double()
        for h in range(Hq):
            z = q[b, :, h].double() @ k[:, h // (Hq // Hkv)].t() / math.sqrt(D)
            if s["causal"]:
                for i in range(n_q):
                    z[i, C + i + n_kv - n_q + 1:] = -math.inf
            w = torch.exp(z - z.max(1, keepdim=True).values)
            out[b, :, h] = (w @ v[:, h // (Hq // Hkv)]) / w.sum(1, keepdim=True)
    return out


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def _fork_exact(s):
    table, shares, free = (s[k].cpu().tolist() for k in ("page_table", "shares", "free_pages"))
    parent, length, have = (s[k].cpu().tolist() for k in ("parent", "length", "n_pages"))
    left, page = int(s["n_free"]), s["page"]
    short, asked = [0] * len(parent), 0
    for b, p in enumerate(parent):
        if p < 0:
            continue
        full, rest = divmod(length[p], page)
        asked += rest > 0
        if rest and asked > int(s["n_free"]):
            short[b] = 1
            continue
        for j in range(full):
            table[b][j] = table[p][j]
            shares[table[p][j]] += 1
        have[b] = full
        if rest:
            left -= 1
            table[b][full] = free[left]
            have[b] += 1
            for pool in s["pools"]:
                pool[free[left], :rest] = pool[table[p][full], :rest]
    return {"page_table": _i32(table), "n_pages": _i32(have), "shares": _i32(shares), "pools": s["pools"],
            "n_free": _i32([left]), "short": torch.tensor(short, dtype=torch.uint8)}


def _release_exact(s):
    table, shares, free = (s[k].cpu().tolist() for k in ("page_table", "shares", "free_pages"))
    length, have = s["length"].cpu().tolist(), s["n_pages"].cpu().tolist()
    at, freed = int(s["n_free"]), []
    for b, n in enumerate(length):
        keep = min(have[b], -(-n // s["page"]))
        for page in table[b][keep:have[b]]:
            if shares[page]:
                shares[page] -= 1
            else:
                freed.append(page)
        have[b] = keep
    free[at:at + len(freed)] = sorted(freed)
    return {"free_pages": _i32(free), "n_pages": _i32(have), "n_free": _i32([at + len(freed)]), "shares": _i32(shares)}


def _compact_exact(s):
    table, shares, have = (s[k].cpu().tolist() for k in ("page_table", "shares", "n_pages"))
    num = len(shares)
    used = sorted({p for row, n in zip(table, have) for p in row[:n]})
    holes = sorted(set(range(len(used))) - set(used))
    to = dict(zip([p for p in used if p >= len(used)], holes))
    count = [0] * num
    for p in used:
        count[to.get(p, p)] = shares[p]
    for row, n in zip(table, have):
        row[:n] = [to.get(p, p) for p in row[:n]]
    for a, b in to.items():
        for pool in s["pools"]:
            pool[b] = pool[a]
    return {"page_table": _i32(table), "shares": _i32(count), "pools": s["pools"],
            "free_pages": _i32(list(range(num - 1, -1, -1))), "n_free": _i32([num - len(used)])}


def _norm_exact(s):
    x = s["x"].double()
    out = {}
    if s["residual"] is not None:
        x = x + s["residual"].double()
        out["sum"] = x
    y = x / torch.sqrt((x ** 2).sum(1, keepdim=True) / x.shape[1] + EPS) * s["weight"].double()
    if not s["fp8"]:
        return dict(out, y=y)
    scale = torch.stack([y[:, j:j + GROUP].abs().amax(1) for j in range(0, y.shape[1], GROUP)], 1)
    scale = (scale / E4M3_MAX).clamp(min=NORMAL_MIN)
    q = _grid_e4m3(y / scale[:, torch.arange(y.shape[1], device=y.device) // GROUP])
    return dict(out, q=q, scale=scale)


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _attn_exact, "fork": _fork_exact, "release": _release_exact, "compact": _compact_exact,
            "norm": _norm_exact}[case["op"]](s)
