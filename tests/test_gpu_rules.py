"""GPU parity of the rules on the verify rows' logits (dflash_logits_rules)
against the oracle in 64 bits.

Tolerance: a value takes at most five fp32 roundings (the division or product
by the repetition penalty, frequency * count, two subtractions, the bias), each
at most half a step (2^-24) of a quantity no larger than the sum of the terms'
magnitudes, so 6 * 2^-24 of that sum covers them; the one rounding to the I/O
type adds 2^-8 (bf16) of the value. A logit without a rule keeps its bits."""
import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_speculative_fusion_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_fusion_gb300 import build
    build.build()
    api.lib()


def _case(B, R, V, dtype, H=37, nb=5, mask=True, seed=0):
    g = np.random.default_rng(seed)
    s = {}
    s["logits"] = torch.from_numpy(g.normal(0, 3, (B, R, V)).astype(np.float32)).to(DT[dtype])
    few = max(1, V // 4)                       # tokens repeat
    s["cand"] = torch.from_numpy(g.integers(-1, few, (B, R)))
    s["n_draft"] = torch.from_numpy(g.integers(0, R, B).astype(np.int32))
    if H:
        s["hist"] = torch.from_numpy(g.integers(-1, V + 2, (B, H)) % np.where(g.random((B, 1)) < .5, V + 2, few + 2))
        s["hist_len"] = torch.from_numpy(g.integers(0, H + 1, B).astype(np.int32))
        s["prompt_len"] = torch.from_numpy(g.integers(0, H + 1, B).astype(np.int32))
    s["repetition"] = torch.from_numpy((0.7 + g.random(B)).astype(np.float32))
    s["presence"] = torch.from_numpy(g.normal(0, 1, B).astype(np.float32))
    s["frequency"] = torch.from_numpy(g.normal(0, 1, B).astype(np.float32))
    if nb:
        s["bias_tok"] = torch.from_numpy(g.integers(-1, V + 1, (B, nb)))
        s["bias_val"] = torch.from_numpy(g.normal(0, 5, (B, nb)).astype(np.float32))
    if mask:
        W = (V + 31) // 32
        dense = g.random((B, R, W * 32)) < g.choice([0.02, 0.5, 1.0], (B, R, 1))
        bits = dense.reshape(B, R, W, 32) * (1 << np.arange(32, dtype=np.int64))
        s["mask"] = torch.from_numpy(bits.sum(-1).astype(np.uint32).view(np.int32))
        s["mask_on"] = torch.from_numpy((g.random(B) < 0.7).astype(np.uint8))
    return s


def _host(s):
    return {k: (v.float() if k == "logits" or k == "out" else v).numpy() for k, v in s.items()}


def _check(s, inplace=False, out0=None):
    dev = {k: v.to(DEV) for k, v in s.items()}
    if inplace:
        out = dev["logits"]
        got = api.logits_rules(**dev, out=out)
        ref, size = O.logits_rules(**_host(s), out=s["logits"].float().numpy())
    else:
        out = torch.full_like(dev["logits"], 7.0)
        got = api.logits_rules(**dev, out=out)
        ref, size = O.logits_rules(**_host(s), out=torch.full_like(s["logits"], 7.0).float().numpy())
    assert got.data_ptr() == out.data_ptr() and api.last_launch_count() == 1
    with np.errstate(over="ignore"):
        ref[np.isinf(ref.astype(np.float32))] *= np.inf      # past the range of the fp32 arithmetic
    y = got.float().cpu().numpy().astype(np.float64)
    z = s["logits"].float().numpy().astype(np.float64)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isneginf(ref), np.isneginf(y))
    eps = 2.0 ** -8 if s["logits"].dtype == torch.bfloat16 else 0.0
    tol = 6 * 2.0 ** -24 * size[fin] * (1 + eps) + eps * np.abs(ref[fin])
    assert np.all(np.abs(y[fin] - ref[fin]) <= tol)
    same = fin & (ref == z)
    assert np.array_equal(y[same], z[same])
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 7, 31, 32, 33, 1000, 1023, 2048 + 5, 8192 + 8, 20011])
def test_vocabulary_sizes(V, dtype):
    s = _case(3, 4, V, dtype, seed=V)
    _check(s)
    _check(s, inplace=True)


@pytest.mark.parametrize("B,R,H,nb,mask", [(1, 1, 0, 0, False), (1, 1, 1, 1, False), (2, 16, 300, 0, True),
                                           (5, 1, 64, 40, True), (1, 256, 20, 3, False), (70, 3, 9, 2, True),
                                           (4, 7, 0, 3, True), (3, 2, 5000, 300, False)])
def test_batches_and_lists(B, R, H, nb, mask):
    s = _case(B, R, 517, "bf16", H=H, nb=nb, mask=mask, seed=B * 100 + R)
    _check(s)
    _check(s, inplace=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [2051, 4099])
def test_many_masked_rows_at_any_alignment(V, dtype):
    # more rows than one pass over their unaligned ends takes
    s = _case(2, 75, V, dtype, nb=30, seed=V)
    s["n_draft"][0] = 74
    s["mask_on"][:] = 1
    _check(s)
    _check(s, inplace=True)
    only_mask = {k: s[k] for k in ("logits", "n_draft", "mask")}
    _check(only_mask)
    _check(only_mask, inplace=True)


def test_one_token_repeated_everywhere():
    # the history and the candidates are one token: its count passes 4000
    s = _case(2, 6, 300, "f32", H=4096, nb=4, seed=5)
    s["hist"][:] = 123
    s["hist_len"][:] = 4096
    s["prompt_len"][:] = torch.tensor([0, 4095])
    s["cand"][:] = 123
    s["n_draft"][:] = 5
    s["bias_tok"][:] = 123        # the same token in every entry: the last counts
    _check(s)


def test_non_finite_logits_and_lowest_values():
    s = _case(2, 3, 640, "bf16", seed=6)
    s["n_draft"][:] = 2
    low = torch.finfo(torch.bfloat16).min
    s["logits"][:, :, 0::5] = float("-inf")
    s["logits"][:, :, 1::5] = low
    s["mask_on"][:] = 1
    got = _check(s)
    # a masked place is -inf whatever it held; an unmasked NaN or infinity without a rule stays
    s["logits"][:, :, 2::5] = float("nan")
    s["logits"][:, :, 3::5] = float("inf")
    dev = {k: v.to(DEV) for k, v in s.items()}
    y = api.logits_rules(**dev).float().cpu().numpy()
    words = s["mask"].numpy().astype(np.int64) & 0xFFFFFFFF
    t = np.arange(640)
    ok = (words[:, :, t // 32] >> (t % 32)) & 1
    assert np.all(np.isneginf(y[ok == 0]))
    assert np.all(np.isnan(y[:, :, 2::5][ok[:, :, 2::5] == 1]))
    assert got is not None


def test_row_without_an_allowed_token_through_verify():
    # an empty mask row: -inf everywhere; both verify rules still answer inside the vocabulary
    B, R, V = 3, 4, 1003
    s = _case(B, R, V, "bf16", seed=7)
    s["n_draft"][:] = R - 1
    s["mask"][:] = -1
    s["mask"][:, 1] = 0
    s["mask_on"][:] = 1
    dev = {k: v.to(DEV) for k, v in s.items()}
    z = api.logits_rules(**dev)
    assert bool(torch.isneginf(z[:, 1].float()).all())
    cand = torch.zeros((B, R), dtype=torch.int64, device=DEV)
    cand[:, 1] = z[:, 0].float().argmax(-1)        # row 0 accepts, row 1 is empty
    cand[:, 2] = 5
    g = api.verify_greedy(z, cand, dev["n_draft"])
    assert g["accept_len"].tolist() == [1] * B and g["bonus"].tolist() == [0] * B
    u = torch.zeros((B, R - 1), device=DEV)
    dl = torch.zeros((B, R - 1, V), dtype=torch.bfloat16, device=DEV)
    r = api.verify_sample(z, dl, cand, u, torch.full((B,), 0.5, device=DEV), 1.0, dev["n_draft"])
    assert r["accept_len"].tolist() == [1] * B
    assert all(0 <= x < V for x in r["bonus"].tolist())
    assert all(f & api.FLAG_DEGENERATE for f in r["flags"].tolist())


def test_masked_candidate_is_rejected_and_never_drawn():
    # grammar-masked rows through both verify rules, against the oracle on the same masked logits
    B, R, V = 8, 5, 2003
    s = _case(B, R, V, "f32", seed=8)
    s["n_draft"][:] = R - 1
    s["mask_on"][:] = 1
    s["mask"][:, :, 0] |= 3
    dev = {k: v.to(DEV) for k, v in s.items()}
    z = api.logits_rules(**dev)
    g = np.random.default_rng(9)
    dl = torch.from_numpy(g.normal(0, 3, (B, R - 1, V)).astype(np.float32))
    cand = torch.from_numpy(g.integers(0, V, (B, R)))
    cand[::2, 1] = z[::2, 0].cpu().argmax(-1)
    ua = torch.from_numpy(g.random((B, R - 1)).astype(np.float32))
    uf = torch.from_numpy(g.random(B).astype(np.float32))
    got = api.verify_sample(z, dl.to(DEV), cand.to(DEV), ua.to(DEV), uf.to(DEV), 1.0, dev["n_draft"], want_probs=True)
    ref = O.verify_sample(z.cpu().numpy().astype(np.float64), dl.numpy().astype(np.float64), cand.numpy(),
                          s["n_draft"].numpy(), ua.numpy(), uf.numpy(), 1.0)
    ok = (ref["flags"] == 0) & (got["flags"].cpu().numpy() == 0)
    assert ok.any()
    for k in ("accept_len", "bonus"):
        assert np.array_equal(got[k].cpu().numpy()[ok], np.asarray(ref[k])[ok]), k
    assert not torch.isnan(got["probs"]).any()
    rows = got["accept_len"].long()
    assert not torch.isneginf(z[torch.arange(B, device=DEV), rows, got["bonus"]]).any()


def test_neutral_parameters_copy():
    s = _case(2, 3, 999, "bf16", nb=0, mask=False, seed=10)
    s["repetition"][:] = 1
    s["presence"][:] = 0
    s["frequency"][:] = 0
    s["n_draft"][:] = 2
    y = api.logits_rules(**{k: v.to(DEV) for k, v in s.items()})
    assert torch.equal(y.cpu(), s["logits"])
    z = s["logits"].to(DEV)
    assert torch.equal(api.logits_rules(z).cpu(), s["logits"])     # no rule at all


def test_views_at_odd_offsets():
    # logits and out that start at different alignments inside larger buffers
    s = _case(2, 3, 997, "bf16", seed=11)
    dev = {k: v.to(DEV) for k, v in s.items()}
    ref = api.logits_rules(**dev)
    n = dev["logits"].numel()
    for off_in, off_out in ((1, 0), (3, 3), (0, 5)):
        src = torch.zeros(n + 16, dtype=torch.bfloat16, device=DEV)[off_in:off_in + n].view(dev["logits"].shape)
        src.copy_(dev["logits"])
        dst = torch.zeros(n + 16, dtype=torch.bfloat16, device=DEV)[off_out:off_out + n].view(src.shape)
        api.logits_rules(**{**dev, "logits": src}, out=dst)
        assert torch.equal(dst, ref)


def test_large_offsets_pass_32_bits():
    # rows that start past 2^31 elements and 2^32 bytes
    B, R, V = 70, 256, 128256
    free = torch.cuda.mem_get_info()[0]
    if free < 12 << 30:
        pytest.skip("needs 12 GB")
    z = torch.zeros((B, R, V), dtype=torch.bfloat16, device=DEV)
    assert z.numel() > 2 ** 31
    bias_tok = torch.full((B, 1), V - 1, dtype=torch.int64, device=DEV)
    bias_val = torch.arange(B, dtype=torch.float32, device=DEV)[:, None].contiguous()
    api.logits_rules(z, bias_tok=bias_tok, bias_val=bias_val, out=z)
    assert torch.equal(z[:, :, V - 1].float(), bias_val.expand(B, R))
    assert float(z[:, :, :V - 1].abs().max()) == 0.0


def test_side_stream_and_graph_replay():
    s = _case(4, 5, 3001, "bf16", seed=12)
    dev = {k: v.to(DEV) for k, v in s.items()}
    ref = api.logits_rules(**dev)
    out = torch.zeros_like(dev["logits"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        api.logits_rules(**dev, out=out)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.logits_rules(**dev, out=out)
    t = _case(4, 5, 3001, "bf16", seed=13)
    for k in dev:
        dev[k].copy_(t[k])
    out.zero_()
    graph.replay()
    assert torch.equal(out, api.logits_rules(**dev))
