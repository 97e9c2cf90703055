"""The operators around a serving round's draft and verify, as cases to measure.

Five operators, each in its plain form (elementary torch operations) and through
the library's binding (``own``):

  rules     penalties for repeated tokens, sparse biases and grammar masks on the
            logits of every verify row, whose history grows along the candidates
  resize    every sequence's paged-cache block table grown or shrunk to a length,
            pages taken from and given back to a free list
  slots     the slot map (sequence, position, pool slot) of a ragged batch of rows
  quant     rows to 8-bit floating point (e4m3) with one scale per 128 values
  product   x w^T of 8-bit operands, x scaled per 1 x 128 and w per 128 x 128 block

Sizes are those of the workloads (Llama-3.1-8B and Qwen3-4B draft shapes: d =
4096 / 2560, five captured layers, K/V projections of 10240 columns, vocabularies
of 128256 and 151936) or generic odd ones.
"""
import math

import torch

own = False

GROUP = 128           # values per scale
E4M3_MAX = 448.0
NORMAL_MIN = 2.0 ** -126
PAGE = 16
WORKLOAD_KN = ((20480, 4096), (4096, 10240), (12800, 2560), (2560, 10240))


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # plain sampling of one sequence, one row: the latency of a call
        dict(name="rules_b1_r1", op="rules", dtype="bf16", B=1, R=1, V=128256, hist=2048, n_bias=16, mask="none"),
        # a small fp32 batch over an odd vocabulary: rows start at any alignment
        dict(name="rules_b8_r10_f32_odd", op="rules", dtype="f32", B=8, R=10, V=100003, hist=1021, n_bias=100,
             mask="half"),
        # the throughput workload's verify: 64 sequences, 16 rows, half of them under a grammar
        dict(name="rules_b64_r16", op="rules", dtype="bf16", B=64, R=16, V=128256, hist=8192, n_bias=64, mask="half"),
        # headroom of one decode round of 64 sequences
        dict(name="resize_b64_round", op="resize", B=64, max_len=8192, fresh=0.0),
        # a thousand sequences, a quarter of them admitted whole, some finished
        dict(name="resize_b1024_admit", op="resize", B=1024, max_len=8192, fresh=0.25),
        # the block rows of one decode round
        dict(name="slots_b64_block", op="slots", B=64, rows=16, max_len=8192, whole=False),
        # whole prompts of 512 sequences
        dict(name="slots_b512_prefill", op="slots", B=512, rows=8192, max_len=8192, whole=True),
        # captured hidden rows of one sequence's commit
        dict(name="quant_t10", op="quant", dtype="bf16", T=10, K=20480, block=1),
        # captured hidden rows of a prefill
        dict(name="quant_t8190", op="quant", dtype="bf16", T=8190, K=20480, block=1),
        # context fusion of one sequence's commit: the weights' bytes bound it
        dict(name="product_t10_k20480", op="product", dtype="bf16", T=10, K=20480, N=4096),
        # K/V projection of the throughput workload's commit (271 rows)
        dict(name="product_t271_k4096", op="product", dtype="f32", T=271, K=4096, N=10240),
        # context fusion of a prefill: the matrix rate bounds it
        dict(name="product_t8190_k20480", op="product", dtype="bf16", T=8190, K=20480, N=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rules", "rules", "resize", "slots", "quant", "product", "product"])
    if op == "rules":
        B, R = _log(rng, 1, 64), rng.randint(1, 16)
        V = rng.choice([128256, 151936, _log(rng, 1000, 128256), _log(rng, 1000, 128256) | 1])
        while B * R * V > 64 * 16 * 128256:
            B = max(1, B // 2)
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]) if B <= 32 else "bf16", B=B, R=R, V=V,
                    hist=_log(rng, 1, 8192), n_bias=rng.choice([0, 1, _log(rng, 2, 300)]),
                    mask=rng.choice(["none", "half", "all"]))
    if op == "resize":
        return dict(op=op, B=_log(rng, 1, 1024), max_len=_log(rng, 17, 8192), fresh=rng.choice([0.0, 0.1, 0.25]))
    if op == "slots":
        return dict(op=op, B=_log(rng, 1, 512), rows=_log(rng, 1, 8192), max_len=8192, whole=rng.random() < 0.5)
    if op == "quant":
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), T=_log(rng, 1, 4095), K=16 * _log(rng, 1, 1280),
                    block=rng.choice([1, 1, 128]))
    K, N = rng.choice(WORKLOAD_KN) if rng.random() < 0.5 else (16 * _log(rng, 1, 1280), _log(rng, 1, 10240))
    return dict(op=op, dtype=rng.choice(["bf16", "f32"]), T=_log(rng, 1, 8190), K=K, N=min(N, 10240))


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


def _rules_state(c, g):
    B, R, V, H = c["B"], c["R"], c["V"], c["hist"]
    # peaked rows, as a target model gives them
    logits = torch.randn((B, R, V), generator=g, device="cuda").mul_(2.5)
    logits.scatter_(2, torch.randint(0, V, (B, R, 4), generator=g, device="cuda"), 14.0)
    s = {"op": "rules", "logits": logits.to(_dt(c)), "out": torch.zeros((B, R, V), dtype=_dt(c), device="cuda")}
    # text repeats itself: tokens by a skewed law over the vocabulary
    skew = lambda shape: (torch.rand(shape, generator=g, device="cuda").pow(4) * V).long().clamp_(0, V - 1)  # noqa: E731
    s["hist"] = skew((B, H))
    s["hist_len"] = _randint(max(1, H // 8), H, (B,), g)
    s["prompt_len"] = (s["hist_len"].float() * torch.rand(B, generator=g, device="cuda")).int()
    s["cand"] = skew((B, R))
    s["n_draft"] = _randint(R // 2, R - 1, (B,), g)
    s["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device="cuda")
    s["presence"] = 0.8 * torch.rand(B, generator=g, device="cuda")
    s["frequency"] = 0.5 * torch.rand(B, generator=g, device="cuda")
    s["bias_tok"] = s["bias_val"] = None
    if c["n_bias"]:
        n = c["n_bias"]
        # distinct tokens, the last eighth of a list unused
        first = torch.randint(0, V, (B, 1), generator=g, device="cuda")
        tok = (first + torch.arange(n, device="cuda") * max(1, V // n)) % V
        s["bias_tok"] = torch.where(torch.arange(n, device="cuda") < n - n // 8, tok, -1).contiguous()
        s["bias_val"] = torch.randn((B, n), generator=g, device="cuda") * 4
    s["mask"] = s["mask_on"] = None
    if c["mask"] != "none":
        W = (V + 31) // 32
        bits = torch.tensor([1 << i for i in range(31)] + [-(1 << 31)], dtype=torch.int32, device="cuda")
        mask = torch.empty((B, R, W), dtype=torch.int32, device="cuda")
        for b in range(B):
            # inside free text nearly every token is allowed, at a structural place few are
            keep = torch.where(torch.rand((R, 1), generator=g, device="cuda") < 0.5, 0.98, 0.003)
            ok = torch.rand((R, W * 32), generator=g, device="cuda") < keep
            mask[b] = (ok.view(R, W, 32) * bits).sum(-1, dtype=torch.int32)
        s["mask"] = mask
        if c["mask"] == "half":
            s["mask_on"] = (torch.arange(B, device="cuda") % 2 == 0).to(torch.uint8)
    return s


def _pages_of(n):
    return (n + PAGE - 1) // PAGE


def _table(B, max_pages, have, spare, g):
    """Pages of every sequence at random places of the pool, and the free list of the rest."""
    num = B * max_pages + spare
    perm = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(max_pages, device="cuda")
    first = torch.cumsum(have.long(), 0) - have
    held = col[None] < have[:, None]
    table = torch.where(held, perm[(first[:, None] + col[None]).clamp_(max=num - 1)], -1).int().contiguous()
    n_held = have.long().sum()
    free = perm[(torch.arange(num, device="cuda") + n_held) % num].contiguous()
    return table, free, (num - n_held).to(torch.int32).reshape(1), num


def _resize_state(c, g):
    B, top = c["B"], c["max_len"]
    max_pages = _pages_of(top + 64)
    was = _randint(1, top, (B,), g)
    admit = torch.rand(B, generator=g, device="cuda") < c["fresh"]
    done = torch.rand(B, generator=g, device="cuda") < c["fresh"] / 2
    # a round holds headroom of two blocks past the commit: some of it goes back, more is taken
    have = torch.where(admit, 0, _pages_of(was + 32)).int()
    now = was + _randint(1, 32, (B,), g)
    now = torch.where(done & ~admit, 0, now).int()
    table, free, n_free, num = _table(B, max_pages, have, 0, g)
    return {"op": "resize", "length": now, "n_pages": have, "page_table": table, "free_pages": free,
            "n_free": n_free, "num_pages": num}


def _slots_state(c, g):
    B = c["B"]
    max_pages = _pages_of(c["max_len"] + c["rows"])
    if c["whole"]:
        n_rows = _randint((c["rows"] + 1) // 2, c["rows"], (B,), g)
        start = torch.zeros(B, dtype=torch.int32, device="cuda")
    else:
        n_rows = _randint(1, c["rows"], (B,), g)
        start = _randint(0, c["max_len"], (B,), g)
    table, _, _, num = _table(B, max_pages, _pages_of(start + n_rows).int(), 0, g)
    return {"op": "slots", "start_pos": start, "n_rows": n_rows, "page_table": table, "num_pages": num,
            "rows_max": B * c["rows"]}


def _hidden(T, K, dtype, g):
    """Rows as captured hidden states are: a few channels far larger than the rest."""
    x = torch.randn((T, K), generator=g, device="cuda")
    x *= torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(dtype)


def _quant_plain(x, block):
    """(values on the e4m3 grid, scales) of x [T, K] by blocks of `block` rows x 128 columns."""
    T, K = x.shape
    G, S = (K + GROUP - 1) // GROUP, (T + block - 1) // block
    x = x.float()
    pad = torch.nn.functional.pad(x.abs(), (0, G * GROUP - K, 0, S * block - T))
    amax = pad.view(S, block, G, GROUP).amax(dim=(1, 3))
    scale = torch.clamp(amax / E4M3_MAX, min=NORMAL_MIN)
    q = x / _spread(scale, block, T, K)
    return q.to(torch.float8_e4m3fn), scale


def _spread(scale, block, T, K):
    """scale [S, G] over the elements it belongs to."""
    if block > 1:
        scale = scale.repeat_interleave(block, 0)[:T]
    return scale.repeat_interleave(GROUP, 1)[:, :K]


def _product_state(c, g):
    T, K, N = c["T"], c["K"], c["N"]
    xq, xs = _quant_plain(_hidden(T, K, torch.bfloat16, g), 1)
    wq, ws = _quant_plain(torch.randn((N, K), generator=g, device="cuda") * 0.02, 128)
    bias = torch.randn(N, generator=g, device="cuda").to(_dt(c))
    return {"op": "product", "x": xq, "x_scale": xs, "w": wq, "w_scale": ws, "bias": bias, "dtype": _dt(c)}


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "rules":
        return _rules_state(case, g)
    if op == "resize":
        return _resize_state(case, g)
    if op == "slots":
        return _slots_state(case, g)
    if op == "quant":
        return {"op": op, "x": _hidden(case["T"], case["K"], _dt(case), g), "block": case["block"]}
    return _product_state(case, g)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rules_plain(s):
    logits, out = s["logits"], s["out"]
    B, R, V = logits.shape
    dev = logits.device
    z = logits.float()
    at = torch.arange(s["hist"].shape[1], device=dev)[None]
    in_prompt = at < s["prompt_len"][:, None]
    in_output = (at < s["hist_len"][:, None]) & ~in_prompt
    prompt = torch.zeros((B, V), device=dev).scatter_add_(1, s["hist"], in_prompt.float())
    count = torch.zeros((B, V), device=dev).scatter_add_(1, s["hist"], in_output.float())
    # row r also follows the candidates 1 .. r
    one = torch.ones((B, R, 1), device=dev)
    one[:, 0] = 0
    more = torch.zeros((B, R, V), device=dev).scatter_(2, s["cand"][:, :, None], one).cumsum_(1)
    count = more.add_(count[:, None])
    seen = (count > 0) | (prompt > 0)[:, None]
    theta = s["repetition"][:, None, None]
    z = torch.where(seen, torch.where(z > 0, z / theta, z * theta), z)
    z = z - s["frequency"][:, None, None] * count
    z = z - s["presence"][:, None, None] * (count > 0).float()
    if s["bias_tok"] is not None:
        used = s["bias_tok"] >= 0
        bias = torch.zeros((B, V), device=dev)
        bias.scatter_add_(1, s["bias_tok"].clamp(min=0), torch.where(used, s["bias_val"], 0.0))
        z = z + bias[:, None]
    if s["mask"] is not None:
        bit = torch.arange(32, dtype=torch.int32, device=dev)
        ok = ((s["mask"][..., None] >> bit) & 1).view(B, R, -1)[..., :V].bool()
        if s["mask_on"] is not None:
            ok = ok | (s["mask_on"] == 0)[:, None, None]
        z = torch.where(ok, z, float("-inf"))
    live = (torch.arange(R, device=dev)[None] <= s["n_draft"][:, None])[..., None]
    out.copy_(torch.where(live, z.to(out.dtype), out))
    return out


def _resize_plain(s):
    table, free, have = s["page_table"], s["free_pages"], s["n_pages"].long()
    B, max_pages = table.shape
    num = s["num_pages"]
    need = _pages_of(s["length"].long())
    beyond = need > max_pages
    need = torch.where(beyond, have, need)
    give, want = (have - need).clamp(min=0), (need - have).clamp(min=0)
    pool = s["n_free"].long() + give.sum()
    upto = torch.cumsum(want, 0)
    granted = torch.where(upto <= pool, want, 0)
    col = torch.arange(max_pages, device=table.device)[None]
    # pages given back follow the free list in sequence order
    back = (col >= need[:, None]) & (col < have[:, None])
    at = s["n_free"].long() + (torch.cumsum(give, 0) - give)[:, None] + col - need[:, None]
    grown = torch.cat([free, free[:1]]).scatter_(0, torch.where(back, at, num).view(-1), table.view(-1))[:num]
    # pages are taken from the list's end
    taken = (col >= have[:, None]) & (col < (have + granted)[:, None])
    frm = pool - 1 - ((upto - want)[:, None] + col - have[:, None])
    table.copy_(torch.where(taken, grown[frm.clamp(0, num - 1)], table))
    free.copy_(grown)
    return {"page_table": table, "free_pages": free, "n_pages": (have - give + granted).int(),
            "n_free": (pool - granted.sum()).int().reshape(1),
            "short": (beyond | (granted < want)).to(torch.uint8)}


def _slots_plain(s):
    table, start = s["page_table"], s["start_pos"].long()
    B, max_pages = table.shape
    T = s["rows_max"]
    n = s["n_rows"].long()
    ends = torch.cumsum(n, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=table.device), ends])
    t = torch.arange(T, device=table.device)
    live = t < ends[-1]
    seq = torch.searchsorted(ends, t, right=True).clamp_(max=B - 1)
    pos = start[seq] + t - cu[seq]
    lp = pos // PAGE
    page = table[seq, lp.clamp(max=max_pages - 1)].long()
    ok = live & (lp < max_pages) & (page >= 0) & (page < s["num_pages"])
    return {"cu_rows": cu.int(), "row_seq": torch.where(live, seq, -1).int(),
            "positions": torch.where(live, pos, -1).int(), "slots": torch.where(ok, page * PAGE + pos % PAGE, -1)}


def _product_plain(s):
    x = s["x"].float() * _spread(s["x_scale"], 1, *s["x"].shape)
    w = s["w"].float() * _spread(s["w_scale"], 128, *s["w"].shape)
    return (x @ w.t() + s["bias"].float()).to(s["dtype"])


def run(state):
    op = state["op"]
    if own:
        from block_diffusion_speculative_fusion_gb300 import api
        s = state
        if op == "rules":
            return api.logits_rules(
                s["logits"], cand=s["cand"], n_draft=s["n_draft"], hist=s["hist"], hist_len=s["hist_len"],
                prompt_len=s["prompt_len"], repetition=s["repetition"], presence=s["presence"],
                frequency=s["frequency"], bias_tok=s["bias_tok"], bias_val=s["bias_val"], mask=s["mask"],
                mask_on=s["mask_on"], out=s["out"])
        if op == "resize":
            r = api.pages_resize(s["length"], s["page_table"], s["n_pages"], s["free_pages"], s["n_free"], PAGE)
            return {"page_table": s["page_table"], "free_pages": s["free_pages"], "n_pages": r["n_pages"],
                    "n_free": r["n_free"], "short": r["short"]}
        if op == "slots":
            return api.slot_map(s["start_pos"], s["n_rows"], s["page_table"], PAGE, s["num_pages"], s["rows_max"])
        if op == "quant":
            q, scale = api.fp8_quant(s["x"], block_rows=s["block"])
            return {"q": q, "scale": scale}
        return api.fp8_gemm(s["x"], s["x_scale"], s["w"], s["w_scale"], bias=s["bias"], out_dtype=s["dtype"])
    if op == "rules":
        return _rules_plain(state)
    if op == "resize":
        return _resize_plain(state)
    if op == "slots":
        return _slots_plain(state)
    if op == "quant":
        q, scale = _quant_plain(state["x"], state["block"])
        return {"q": q, "scale": scale}
    return _product_plain(state)


# ---------------------------------------------------------------------------
# the least work of one pass
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "rules":
        B, R, V = case["B"], case["R"], case["V"]
        el = 2 if case["dtype"] == "bf16" else 4
        rows = B * (R // 2 + R - 1 + 2) / 2                 # n_draft is uniform on R // 2 .. R - 1
        masked = {"none": 0.0, "half": (B + 1) // 2 / B, "all": 1.0}[case["mask"]]
        # at a structural place nearly no logit is read: nothing of it comes through the mask
        read = rows * V * el * (1 - 0.5 * masked)
        small = B * (case["hist"] * 8 * 0.56 + case["n_bias"] * 12 + R * 8)
        return {"bytes": int(read + rows * V * el + rows * masked * V / 8 + small), "flops": int(rows * V)}
    if op == "resize":
        B = case["B"]
        pages = _pages_of(case["max_len"]) / 2
        moved = B * (case["fresh"] * 1.5 * pages + 1)
        return {"bytes": int(B * 17 + moved * 8), "flops": int(B * 4)}
    if op == "slots":
        B = case["B"]
        rows = B * case["rows"] * (0.75 if case["whole"] else 0.5)
        pages = B * ((0.75 if case["whole"] else 0.5) * case["rows"] / PAGE + 1)
        return {"bytes": int(B * case["rows"] * 16 + pages * 4 + B * 12), "flops": int(rows * 4)}
    if op == "quant":
        T, K = case["T"], case["K"]
        el = 2 if case["dtype"] == "bf16" else 4
        scales = -(-T // case["block"]) * -(-K // GROUP)
        return {"bytes": T * K * (el + 1) + scales * 4, "flops": T * K * 2}
    T, K, N = case["T"], case["K"], case["N"]
    el = 2 if case["dtype"] == "bf16" else 4
    G = -(-K // GROUP)
    return {"bytes": T * K + N * K + T * N * el + N * el + (T + -(-N // GROUP)) * G * 4, "flops": 2 * T * K * N}


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


def _rules_exact(s):
    logits = s["logits"]
    B, R, V = logits.shape
    out = s["out"].double()
    hist, cand = s["hist"].cpu().tolist(), s["cand"].cpu().tolist()
    for b in range(B):
        n, p = int(s["hist_len"][b]), int(s["prompt_len"][b])
        prompt = torch.zeros(V, dtype=torch.bool, device=logits.device)
        prompt[torch.tensor(hist[b][:p], dtype=torch.int64, device=logits.device)] = True
        count = torch.bincount(torch.tensor(hist[b][p:n], dtype=torch.int64), minlength=V).double().to(logits.device)
        theta, pres, freq = (float(s[k][b]) for k in ("repetition", "presence", "frequency"))
        for r in range(int(s["n_draft"][b]) + 1):
            if r:
                count[cand[b][r]] += 1
            z = logits[b, r].double()
            seen = prompt | (count > 0)
            z[seen] = torch.where(z[seen] > 0, z[seen] / theta, z[seen] * theta)
            z = z - freq * count - pres * (count > 0)
            if s["bias_tok"] is not None:
                used = s["bias_tok"][b] >= 0
                z.index_add_(0, s["bias_tok"][b][used], s["bias_val"][b][used].double())
            if s["mask"] is not None and (s["mask_on"] is None or int(s["mask_on"][b])):
                words = s["mask"][b, r].long() & 0xFFFFFFFF
                tok = torch.arange(V, device=logits.device)
                z[(words[tok // 32] >> (tok % 32)) % 2 == 0] = -math.inf
            out[b, r] = z
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rules":
        return _rules_exact(s)
    if op == "quant":
        x, block = s["x"].double(), case["block"]
        T, K = x.shape
        scale = torch.stack([torch.stack([x[i:i + block, j:j + GROUP].abs().amax() for j in range(0, K, GROUP)])
                             for i in range(0, T, block)]) if block > 1 else \
            torch.stack([x[:, j:j + GROUP].abs().amax(1) for j in range(0, K, GROUP)], 1)
        scale = (scale / E4M3_MAX).clamp(min=NORMAL_MIN)
        rows = torch.arange(T, device=x.device) // block
        cols = torch.arange(K, device=x.device) // GROUP
        q = torch.empty_like(x)
        for i in range(0, T, 512):                            # in pieces: 64-bit copies are large
            q[i:i + 512] = _grid_e4m3(x[i:i + 512] / scale[rows[i:i + 512]][:, cols])
        return {"q": q, "scale": scale}
    if op == "product":
        w = s["w"].double()
        G, out = s["x_scale"].shape[1], s["bias"].double().expand(case["T"], -1).clone()
        rows = torch.arange(case["N"], device=w.device) // 128
        for k in range(G):
            part = slice(k * GROUP, (k + 1) * GROUP)
            xk = s["x"][:, part].double() * s["x_scale"][:, k:k + 1].double()
            out += xk @ (w[:, part] * s["w_scale"][rows, k:k + 1].double()).t()
        return out
    if op == "slots":
        start, n, table = (s[k].cpu().tolist() for k in ("start_pos", "n_rows", "page_table"))
        if sum(n) > 1 << 20:
            return None                                       # whole numbers: a loop over rows takes too long
        seq, pos, slot, cu = [], [], [], [0]
        for b, k in enumerate(n):
            cu.append(cu[-1] + k)
            for p in range(start[b], start[b] + k):
                page = table[b][p // PAGE] if p // PAGE < len(table[b]) else -1
                seq.append(b)
                pos.append(p)
                slot.append(page * PAGE + p % PAGE if 0 <= page < s["num_pages"] else -1)
        pad = [-1] * (s["rows_max"] - len(seq))
        return {"cu_rows": torch.tensor(cu, dtype=torch.int32), "row_seq": torch.tensor(seq + pad, dtype=torch.int32),
                "positions": torch.tensor(pos + pad, dtype=torch.int32), "slots": torch.tensor(slot + pad)}
    length, have, table, free = (s[k].cpu().tolist() for k in ("length", "n_pages", "page_table", "free_pages"))
    stack = free[:int(s["n_free"])]
    need = [-(-v // PAGE) for v in length]
    short = [int(k > len(table[0])) for k in need]
    need = [h if bad else k for k, h, bad in zip(need, have, short)]
    now = list(have)
    for b, k in enumerate(need):
        if k < have[b]:
            stack += table[b][k:have[b]]
            now[b] = k
    whole = stack + free[len(stack):]
    asked = 0
    for b, k in enumerate(need):
        want = max(0, k - have[b])
        asked += want
        if want and (asked > len(whole[:int(s["n_free"])]) + sum(max(0, h - j) for h, j in zip(have, need))):
            short[b] = 1
            continue
        for i in range(want):
            table[b][have[b] + i] = stack.pop()
        now[b] += want
    return {"page_table": torch.tensor(table, dtype=torch.int32), "free_pages": torch.tensor(whole, dtype=torch.int32),
            "n_pages": torch.tensor(now, dtype=torch.int32), "n_free": torch.tensor([len(stack)], dtype=torch.int32),
            "short": torch.tensor(short, dtype=torch.uint8)}
