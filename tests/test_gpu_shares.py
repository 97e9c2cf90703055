"""GPU parity of the pages that rows of the block table hold together
(dflash_pages_fork, _release, _compact) against the oracle: whole numbers and
copied bytes, compared exactly."""
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


def _dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=dtype)).to(DEV)


def _pools(num, page, shape, n, g, dtype=torch.bfloat16):
    return [torch.from_numpy(g.integers(-64, 64, (num, page, *shape)).astype(np.float32)).to(dtype).to(DEV)
            for _ in range(n)]


def _host(pools):
    return [p.float().cpu().numpy() for p in pools]


def _forest(B, max_pages, page, num, g, full=False):
    """Rows that hold pages, some of them together with rows before; the free list."""
    perm = list(map(int, g.permutation(num)))
    table = np.full((B, max_pages), -1, dtype=np.int32)
    have = np.zeros(B, dtype=np.int32)
    holds = np.zeros(num, dtype=np.int64)
    for b in range(B):
        n = max_pages if full else int(g.integers(0, max_pages + 1))
        k = 0
        if b and g.random() < 0.6:
            a = int(g.integers(0, b))
            k = int(g.integers(0, min(n, have[a]) + 1))
            table[b, :k] = table[a, :k]
        while k < n and perm:
            table[b, k] = perm.pop()
            k += 1
        have[b] = k
        for p in table[b, :k]:
            holds[p] += 1
    free = np.full(num, -1, dtype=np.int32)
    free[:len(perm)] = perm
    return table, have, np.maximum(holds - 1, 0).astype(np.int32), free, len(perm)


SHAPES = [(1, 1, 1, 2), (2, 3, 16, 8), (9, 7, 16, 70), (64, 40, 16, 1500), (64, 40, 16, 60), (515, 9, 3, 4100),
          (1030, 130, 8, 60000), (4096, 3, 1, 9000)]


@pytest.mark.parametrize("B,max_pages,page,num", SHAPES)
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_fork(B, max_pages, page, num, seed):
    g = np.random.default_rng(seed)
    table, have, shares, free, n_free = _forest(B, max_pages, page, num, g)
    # two rows in three are empty; some parents are not allowed: no row, the row itself, a child, too short
    empty = g.random(B) < 0.66
    length = np.maximum(have * page - g.integers(0, page + 1, B), 0)
    length[g.random(B) < 0.05] = max_pages * page
    length[g.random(B) < 0.05] = -3
    for b in np.flatnonzero(empty):
        have[b] = 0
    parent = np.where(empty | (g.random(B) < 0.1), g.integers(-B // 4 - 1, B + 1, B), -1)
    if seed == 2:
        n_free = min(n_free, B // 8)
        parent[g.random(B) < 0.5] = 0
    pools = _pools(num, page, (2, 8), 3, g)
    before = _host(pools)
    d = [_dev(x) for x in (parent, length, table, have, shares, free, [n_free])]
    ref = O.pages_fork(parent, length, table, have, shares, free, n_free, page, before)
    for _ in range(2):              # a repeated call gives the same result
        o = api.pages_fork(*d, page, pools)
        for name, got, want in zip(("page_table", "n_pages", "shares", "n_free", "short"),
                                   (d[2], o["n_pages"], o["shares"], o["n_free"], o["short"]), ref):
            assert np.array_equal(got.cpu().numpy().reshape(np.shape(want)), want), name
        for got, want in zip(_host(pools), ref[5]):
            assert np.array_equal(got, want)
        assert np.array_equal(d[4].cpu().numpy(), shares) and np.array_equal(d[5].cpu().numpy(), free)


@pytest.mark.parametrize("shape,dtype,offset", [((8, 128), torch.bfloat16, 0), ((3,), torch.bfloat16, 0),
                                                ((1,), torch.float32, 0), ((16,), torch.bfloat16, 1)])
def test_fork_copies_rows_of_any_width(shape, dtype, offset):
    # rows that are no multiple of 16 bytes, and a pool that starts two bytes past one
    num, page = 9, 16
    g = np.random.default_rng(5)
    n = num * page * int(np.prod(shape))
    flat = torch.from_numpy(g.integers(-64, 64, n + offset).astype(np.float32)).to(dtype).to(DEV)
    pool = flat[offset:].view(num, page, *shape)
    before = pool.float().cpu().numpy()
    table = np.array([[3, 8, -1], [-1, -1, -1], [-1, -1, -1]])
    o = api.pages_fork(_dev([-1, 0, 0]), _dev([16 + 5, 0, 0]), t := _dev(table), _dev([2, 0, 0]), _dev(np.zeros(num)),
                       _dev([0, 1, 2, 4, 5, 6, 7, -1, -1]), _dev([7]), page, [pool])
    assert t.cpu().tolist() == [[3, 8, -1], [3, 7, -1], [3, 6, -1]] and o["n_free"].tolist() == [5]
    assert o["shares"].tolist() == [0, 0, 0, 2, 0, 0, 0, 0, 0] and o["n_pages"].tolist() == [2, 2, 2]
    after = pool.float().cpu().numpy()
    want = before.copy()
    want[7, :5] = want[6, :5] = before[8, :5]
    assert np.array_equal(after, want)


@pytest.mark.parametrize("B,max_pages,page,num", SHAPES)
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_release(B, max_pages, page, num, seed):
    g = np.random.default_rng(10 + seed)
    table, have, shares, free, n_free = _forest(B, max_pages, page, num, g, full=seed == 2)
    length = g.integers(-2, max_pages * page + page, B)
    length[g.random(B) < 0.6] = 0
    if seed == 1:
        table[g.random(table.shape) < 0.02] = num + 5     # entries outside the pool are passed over
        table[g.random(table.shape) < 0.02] = -7
    d = [_dev(x) for x in (length, table, have, shares, free, [n_free])]
    ref = O.pages_release(length, table, have, shares, free, n_free, page)
    for _ in range(2):
        o = api.pages_release(*d, page)
        for name, got, want in zip(("n_pages", "shares", "free_pages", "n_free"),
                                   (o["n_pages"], o["shares"], d[4], o["n_free"]), ref):
            assert np.array_equal(got.cpu().numpy().reshape(np.shape(want)), want), name
        assert np.array_equal(d[1].cpu().numpy(), table) and np.array_equal(d[3].cpu().numpy(), shares)


@pytest.mark.parametrize("B,max_pages,page,num", SHAPES + [(3, 5, 16, 2048), (40, 60, 16, 2049)])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_compact(B, max_pages, page, num, seed):
    g = np.random.default_rng(20 + seed)
    table, have, shares, _, _ = _forest(B, max_pages, page, num, g, full=seed == 2)
    if seed < 2:
        have[g.random(B) < 0.5] = 0
    if seed == 1:
        table[g.random(table.shape) < 0.02] = num
    pools = _pools(num, page, (3,), 2, g) if seed else _pools(num, page, (8,), 4, g, torch.float32)
    ref = O.pages_compact(table, have, shares, _host(pools))
    d = [_dev(x) for x in (table, have, shares)]
    for _ in range(2):
        o = api.pages_compact(*d, page, pools)
        for name, want in zip(("page_table", "shares", "free_pages", "n_free"), ref):
            assert np.array_equal(o[name].cpu().numpy().reshape(np.shape(want)), want), name
        for got, want in zip(_host(pools), ref[4]):
            assert np.array_equal(got, want)
        assert np.array_equal(d[0].cpu().numpy(), table)


def test_life_of_a_pool():
    """Prompts admitted (resize), sampled (fork), grown (resize), ended (release) and
    compacted, until nothing is left: every page is held or free at all times, a row's
    tokens read the same through every table, and the pool comes back whole."""
    B, max_pages, page, num = 24, 12, 16, 200
    g = np.random.default_rng(3)
    pool = torch.zeros((num, page, 4), dtype=torch.float32, device=DEV)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    free = _dev(g.permutation(num))
    held, n_free, shares = _dev(np.zeros(B)), _dev([num]), _dev(np.zeros(num))
    length = np.zeros(B, dtype=np.int64)
    text = [[] for _ in range(B)]

    def check():
        t, h, s = table.cpu().numpy(), held.cpu().numpy(), shares.cpu().numpy()
        n = np.zeros(num, dtype=np.int64)
        for b in range(B):
            np.add.at(n, t[b, :h[b]], 1)
        f = free.cpu().numpy()[:int(n_free)]
        assert len(set(f.tolist())) == len(f) and not n[f].any() and (n > 0).sum() + len(f) == num
        assert np.array_equal(s, np.maximum(n - 1, 0))
        p = pool.cpu().numpy()
        for b in range(B):
            got = [p[t[b, i // page], i % page, 0] for i in range(length[b])]
            assert got == text[b], b

    def write(b, k):
        for i in range(length[b], length[b] + k):
            v = float(g.integers(1, 1 << 20))
            pool[int(table[b, i // page]), i % page] = v
            text[b].append(v)
        length[b] += k

    for step in range(30):
        # a prompt in a free row
        empty = np.flatnonzero(length == 0)
        if len(empty) and step % 2 == 0:
            b, k = int(empty[0]), int(g.integers(1, 60))
            want = length.copy()
            want[b] = k
            r = api.pages_resize(_dev(np.maximum(want, held.cpu().numpy() * page)), table, held, free, n_free, page)
            if not int(r["short"][b]):
                held, n_free = r["n_pages"], r["n_free"]
                write(b, k)
                check()
        # samples of a row
        empty, live = np.flatnonzero(length == 0), np.flatnonzero(length)
        if len(live) and len(empty) > 3:
            parent = np.full(B, -1)
            parent[empty[:3]] = g.choice(live)
            r = api.pages_fork(_dev(parent), _dev(length), table, held, shares, free, n_free, page, [pool])
            held, n_free, shares = r["n_pages"], r["n_free"], r["shares"]
            for b in empty[:3]:
                if not int(r["short"][b]):
                    text[b], length[b] = list(text[parent[b]]), length[parent[b]]
            check()
        # every row writes on
        grow = np.minimum(length + (length > 0) * g.integers(0, 9, B), max_pages * page)
        r = api.pages_resize(_dev(np.maximum(grow, held.cpu().numpy() * page)), table, held, free, n_free, page)
        held, n_free = r["n_pages"], r["n_free"]
        # (a page begun is held by one row alone: a fork copies it)
        for b in np.flatnonzero(length):
            if not int(r["short"][b]):
                write(b, int(grow[b] - length[b]))
        check()
        # some end
        done = (g.random(B) < 0.2) | (step == 29)
        length[done] = 0
        for b in np.flatnonzero(done):
            text[b] = []
        r = api.pages_release(_dev(length), table, held, shares, free, n_free, page)
        held, n_free, shares = r["n_pages"], r["n_free"], r["shares"]
        check()
        if step % 5 == 4:
            r = api.pages_compact(table, held, shares, page, [pool])
            table, shares, free, n_free = r["page_table"], r["shares"], r["free_pages"], r["n_free"]
            check()
            used = num - int(n_free)
            assert int(shares[used:].abs().sum()) == 0
    assert int(n_free) == num and int(held.sum()) == 0 and int(shares.sum()) == 0


def test_captured_and_on_another_stream():
    B, max_pages, page, num = 40, 20, 16, 900
    g = np.random.default_rng(4)
    table, have, shares, free, n_free = _forest(B, max_pages, page, num, g)
    have[::3] = 0
    parent = np.full(B, -1)
    parent[::3] = 1
    length = have * page - 5
    pools = _pools(num, page, (2, 8), 4, g)
    d = [_dev(x) for x in (parent, length, table, have, shares, free, [n_free])]

    def run(out):
        f = api.pages_fork(*d, page, pools, out=out[0])
        r = api.pages_release(d[1], d[2], f["n_pages"], f["shares"], d[5], f["n_free"], page, out=out[1])
        return f, r, api.pages_compact(d[2], r["n_pages"], r["shares"], page, pools, out=out[2])

    keep = [t.clone() for t in d]
    base = [p.clone() for p in pools]
    want = [t.clone() for x in run([{}, {}, {}]) for t in x.values()] + [p.clone() for p in pools]
    out = [{}, {}, {}]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for t, k in zip(d + pools, keep + base):
            t.copy_(k)
        run(out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out)
    for _ in range(3):
        for t, k in zip(d + pools, keep + base):
            t.copy_(k)
        for x in out:
            for t in x.values():
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([t for x in out for t in x.values()] + pools, want):
            assert torch.equal(a, b)


def test_pages_past_four_gigabytes():
    # pools of 140,000 pages of 32 KB: a begun page copied from the last one to one near it, then
    # the pages in use moved from there to the pool's start
    num, page = 140000, 16
    pool = torch.zeros((num, page, 1024), dtype=torch.bfloat16, device=DEV)
    pool[num - 3:] = torch.arange(3 * page, device=DEV).view(3, page, 1) + 1
    table = _dev([[num - 3, num - 1], [-1, -1]])
    n_pages, shares, n_free = _dev([2, 0]), _dev(np.zeros(num)), _dev([1])
    free = _dev(np.full(num, num - 2))
    o = api.pages_fork(_dev([-1, 0]), _dev([21, 0]), table, n_pages, shares, free, n_free, page, [pool])
    assert table.tolist() == [[num - 3, num - 1], [num - 3, num - 2]] and o["n_pages"].tolist() == [2, 2]
    want = [pool[num - 3].clone(), pool[num - 2].clone(), pool[num - 1].clone()]
    assert torch.equal(want[1][:5], want[2][:5]) and int(want[1][5, 0]) == 16 + 6
    c = api.pages_compact(table, o["n_pages"], o["shares"], page, [pool])
    assert c["page_table"].tolist() == [[0, 2], [0, 1]] and int(c["n_free"]) == num - 3
    assert all(torch.equal(pool[i], w) for i, w in enumerate(want)) and c["shares"][:3].tolist() == [1, 0, 0]
