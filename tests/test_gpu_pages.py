"""GPU parity of the block tables (dflash_pages_resize) and slot maps
(dflash_slot_map) against the oracle: whole numbers, compared exactly."""
import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_speculative_fusion_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_fusion_gb300 import build
    build.build()
    api.lib()


def _state(B, max_pages, spare, seed, fill=None):
    g = np.random.default_rng(seed)
    have = g.integers(0, max_pages + 1, B) if fill is None else np.full(B, fill)
    num = int(have.sum()) + spare
    perm = g.permutation(num)
    table = np.full((B, max_pages), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    free = np.full(max(num, 1), -1, dtype=np.int32)
    free[:spare] = perm[at:]
    return g, table, have.astype(np.int32), free, spare


def _resize(length, table, have, free, n_free, page):
    d = [torch.from_numpy(np.ascontiguousarray(x)).to(DEV) for x in
         (length.astype(np.int32), table, have, free, np.array([n_free], dtype=np.int32))]
    got = []
    for _ in range(2):          # a repeated call gives the same result
        o = api.pages_resize(d[0], d[1], d[2], d[3], d[4], page)
        got.append([d[1].cpu().numpy(), o["n_pages"].cpu().numpy(), d[3].cpu().numpy(), int(o["n_free"]),
                    o["short"].cpu().numpy()])
    for a, b in zip(*got):
        assert np.array_equal(a, b)
    ref = O.pages_resize(length, table, have, free, n_free, page)
    for name, a, b in zip(("page_table", "n_pages", "free_pages", "n_free", "short"), got[0], ref):
        assert np.array_equal(a, b), name
    return got[0]


@pytest.mark.parametrize("B,max_pages,spare,page", [(1, 1, 0, 16), (1, 7, 3, 1), (3, 5, 40, 16), (64, 40, 700, 16),
                                                    (64, 40, 60, 16), (515, 9, 100, 3), (1025, 33, 4000, 16),
                                                    (4096, 3, 50, 64)])
@pytest.mark.parametrize("seed", [0, 1])
def test_resize(B, max_pages, spare, page, seed):
    g, table, have, free, n_free = _state(B, max_pages, spare, seed)
    length = g.integers(-3, max_pages * page + 1, B)
    length[g.random(B) < 0.2] = 0
    if seed:
        length[g.random(B) < 0.1] = max_pages * page + 1     # longer than a row: left as it is
    t, now, f, n, short = _resize(length, table, have, free, n_free, page)
    # no page is lost or given twice
    owned = np.concatenate([t[b, :now[b]] for b in range(B)] + [f[:n]])
    assert np.array_equal(np.sort(owned), np.arange(len(owned)))


def test_resize_runs_dry_and_recovers():
    g, table, have, free, n_free = _state(8, 4, 5, 3, fill=0)
    length = np.array([32, 48, 16, 0, 16, 16, 16, 0])
    t, now, f, n, short = _resize(length, table, have, free, n_free, 16)
    # 2 + 3 pages fit, the others come after the list is used up
    assert now.tolist() == [2, 3, 0, 0, 0, 0, 0, 0] and n == 0
    assert short.tolist() == [0, 0, 1, 0, 1, 1, 1, 0]
    # a sequence ends and its pages serve the others in the same call
    length = np.array([0, 48, 16, 0, 16, 16, 16, 0])
    t2, now2, f2, n2, short2 = _resize(length, t, now, f, n, 16)
    assert now2.tolist() == [0, 3, 1, 0, 1, 0, 0, 0] and n2 == 0
    assert short2.tolist() == [0, 0, 0, 0, 0, 1, 1, 0]


def test_resize_clamps_bad_counts():
    # counts outside their ranges are clamped: nothing is read or written out of range
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    free = np.array([12, 13, 14], dtype=np.int32)
    d = [torch.from_numpy(x).to(DEV) for x in (np.array([0, 0, 64], np.int32), table,
                                               np.array([9, -5, 4], np.int32), free, np.array([99], np.int32))]
    o = api.pages_resize(*d, 16)
    assert o["n_pages"].tolist() == [0, 0, 4] and o["n_free"].tolist() == [3]
    assert d[3].tolist() == [12, 13, 14]          # the list is full: what comes back past it is dropped


@pytest.mark.parametrize("B,rows_max,page,max_pages", [(1, 1, 16, 1), (1, 5, 1, 9), (3, 64, 16, 40), (64, 1024, 16, 40),
                                                       (700, 4093, 16, 12), (4096, 9001, 64, 3)])
@pytest.mark.parametrize("seed", [0, 1])
def test_slot_map(B, rows_max, page, max_pages, seed):
    g = np.random.default_rng(seed)
    num = B * max_pages
    table = g.permutation(num).reshape(B, max_pages).astype(np.int32)
    table[g.random((B, max_pages)) < 0.05] = -1
    table[g.random((B, max_pages)) < 0.02] = num
    n = g.integers(-1, max(2, 2 * rows_max // B + 1), B).astype(np.int32)
    n[g.random(B) < 0.3] = 0
    start = g.integers(-2, max_pages * page + 2, B).astype(np.int32)
    got = api.slot_map(torch.from_numpy(start).to(DEV), torch.from_numpy(n).to(DEV),
                       torch.from_numpy(table).to(DEV), page, num, rows_max)
    ref = O.slot_map(start, n, table, page, num, rows_max)
    for name, r in zip(("cu_rows", "row_seq", "positions", "slots"), ref):
        assert np.array_equal(got[name].cpu().numpy(), r), name


def test_slot_map_without_rows_and_cut_off():
    z = torch.zeros(3, dtype=torch.int32, device=DEV)
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(3, 2)
    got = api.slot_map(z, z, table, 16, 6, 10)
    assert got["cu_rows"].tolist() == [0] * 4 and got["slots"].tolist() == [-1] * 10
    big = torch.full((3,), 2 ** 31 - 1, dtype=torch.int32, device=DEV)    # the sum passes 32 bits
    got = api.slot_map(z, big, table, 16, 6, 10)
    assert got["cu_rows"].tolist() == [0, 10, 10, 10] and got["row_seq"].tolist() == [0] * 10
    assert got["slots"].tolist() == list(range(10))


def test_slot_map_into_unaligned_rows():
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    start = torch.tensor([3, 0], dtype=torch.int32, device=DEV)
    n = torch.tensor([9, 6], dtype=torch.int32, device=DEV)
    ref = api.slot_map(start, n, table, 4, 8, 17)
    out = {"row_seq": torch.zeros(18, dtype=torch.int32, device=DEV)[1:],
           "positions": torch.zeros(18, dtype=torch.int32, device=DEV)[1:],
           "slots": torch.zeros(18, dtype=torch.int64, device=DEV)[1:]}
    got = api.slot_map(start, n, table, 4, 8, 17, out=out)
    for k in ref:
        assert torch.equal(got[k], ref[k]), k


def test_round_of_pages_slots_and_materialisation():
    """Headroom reserved, the block's rows mapped, the commit given back: the
    pages that the rows were mapped to hold what the materialisation writes."""
    B, page, max_pages, R, Hkv, D, d = 3, 16, 8, 6, 2, 128, 128
    num = 14
    ctx = torch.tensor([30, 0, 17], dtype=torch.int32, device=DEV)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(num, dtype=torch.int32, device=DEV).flip(0).contiguous()
    n0 = torch.tensor([num], dtype=torch.int32, device=DEV)
    held = torch.zeros(B, dtype=torch.int32, device=DEV)
    r1 = api.pages_resize(ctx + R, table, held, free, n0, page)
    assert r1["short"].tolist() == [0, 0, 0]
    n_rows = torch.tensor([R, R, R], dtype=torch.int32, device=DEV)
    sm = api.slot_map(ctx, n_rows, table, page, num, B * R)
    assert int((sm["slots"] >= 0).sum()) == B * R
    g = torch.Generator().manual_seed(3)
    hidden = torch.randn((B, R, d), generator=g).to(torch.bfloat16).to(DEV)
    W_f = torch.randn((d, d), generator=g).mul(0.1).to(torch.bfloat16).to(DEV)
    W_kv = torch.randn((1, 2, Hkv * D, d), generator=g).mul(0.1).to(torch.bfloat16).to(DEV)
    kp = torch.full((num, page, Hkv, D), 9.0, dtype=torch.bfloat16, device=DEV)
    vp = kp.clone()
    commit = torch.tensor([6, 2, 1], dtype=torch.int32, device=DEV)
    new_len = torch.empty_like(ctx)
    api.materialize_ctx_kv(hidden, commit, ctx, W_f, None, W_kv, None, 1e-6, 0.0, [kp], [vp], table, new_len=new_len)
    flat = vp.view(num * page, -1)
    written = (flat != 9.0).any(1)
    want = torch.zeros(num * page, dtype=torch.bool, device=DEV)
    for b in range(B):
        lo = int(sm["cu_rows"][b])
        want[sm["slots"][lo:lo + int(commit[b])]] = True
    assert torch.equal(written, want)
    r2 = api.pages_resize(new_len, table, r1["n_pages"], free, r1["n_free"], page)
    assert r2["n_pages"].tolist() == [-(-x // page) for x in new_len.tolist()]
    assert int(r2["n_free"]) == num - sum(r2["n_pages"].tolist())


def test_slots_end_where_positions_end():
    # pages that reach past the last int32 position: the rows behind it have no slot
    page, last = 1 << 20, 2 ** 31 - 1
    table = torch.full((2, 2050), -1, dtype=torch.int32, device=DEV)
    table[1, 2047:2049] = torch.tensor([1, 0], dtype=torch.int32)
    start = torch.tensor([0, last - 5], dtype=torch.int32, device=DEV)
    n_rows = torch.tensor([0, 10], dtype=torch.int32, device=DEV)
    sm = api.slot_map(start, n_rows, table, page, 2, 12)
    assert sm["slots"].tolist() == [page + page - 6 + i for i in range(6)] + [-1] * 6
    assert sm["positions"].tolist()[:6] == list(range(last - 5, last + 1))
    assert sm["row_seq"].tolist() == [1] * 10 + [-1] * 2


def test_graph_replay():
    g, table, have, free, n_free = _state(16, 8, 40, 5)
    length = g.integers(0, 8 * 16 + 1, 16).astype(np.int32)
    d = [torch.from_numpy(x).to(DEV) for x in (length, table, have, free, np.array([n_free], np.int32))]
    api.pages_resize(*d, 16)                       # loads the kernels before the capture
    out = {"n_pages": torch.empty(16, dtype=torch.int32, device=DEV)}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.pages_resize(*d, 16, out=out)
        sm = api.slot_map(d[2], d[0], d[1], 16, len(free), 500)
    g, table, have, free2, n_free = _state(16, 8, 40, 5)
    length = g.integers(0, 8 * 16 + 1, 16).astype(np.int32)[::-1].copy()
    d[0].copy_(torch.from_numpy(length))
    d[1].copy_(torch.from_numpy(table))
    d[3].copy_(torch.from_numpy(free2))
    graph.replay()
    ref = O.pages_resize(length, table, have, free2, n_free, 16)
    assert np.array_equal(d[1].cpu().numpy(), ref[0]) and np.array_equal(out["n_pages"].cpu().numpy(), ref[1])
    assert np.array_equal(sm["slots"].cpu().numpy(), O.slot_map(have, length, ref[0], 16, len(free), 500)[3])
