"""Refusals of the pages held together, the residual norm and the shared-prefix
attention, before a launch, and the oracle's own checks of them (no GPU)."""
import ctypes

import numpy as np
import pytest

import oracle as O
from block_diffusion_speculative_fusion_gb300 import api, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


B, PAGES, NUM, PAGE, ROW = 4, 8, 64, 16, 32
BASE = 0x1000000
SEQ, TAB, ALL, POOL = 4 * B, 4 * B * PAGES, 4 * NUM, NUM * PAGE * ROW
WS = 1 << 20


def _p(x):
    return ctypes.c_void_p(x) if x else None


def _fork(L, ptrs, dims=None, row=ROW, n_pools=2):
    d = dims or api.PagesDims(B, PAGE, PAGES, NUM)
    pools = (ctypes.c_void_p * 2)(*ptrs[11:13])
    return L.dflash_pages_fork(ctypes.byref(d), *map(_p, ptrs[:7]), n_pools, row, ctypes.cast(pools, ctypes.c_void_p),
                               *map(_p, ptrs[7:11]), None)


def _release(L, ptrs, dims=None):
    d = dims or api.PagesDims(B, PAGE, PAGES, NUM)
    return L.dflash_pages_release(ctypes.byref(d), *map(_p, ptrs[:9]), _p(ptrs[9]), WS, None)


def _compact(L, ptrs, dims=None, row=ROW, n_pools=2):
    d = dims or api.PagesDims(B, PAGE, PAGES, NUM)
    pools = (ctypes.c_void_p * 2)(*ptrs[8:10])
    return L.dflash_pages_compact(ctypes.byref(d), *map(_p, ptrs[:3]), n_pools, row,
                                  ctypes.cast(pools, ctypes.c_void_p), *map(_p, ptrs[3:7]), _p(ptrs[7]), WS, None)


# bytes of each buffer, and which ones the call writes
CALLS = {
    "fork": (_fork, [SEQ, SEQ, TAB, SEQ, ALL, ALL, 4, SEQ, 4, ALL, B, POOL, POOL], {2, 7, 8, 9, 10, 11, 12}),
    "release": (_release, [SEQ, TAB, SEQ, ALL, ALL, 4, SEQ, 4, ALL, 16384 + 256], {4, 6, 7, 8, 9}),
    "compact": (_compact, [TAB, SEQ, ALL, TAB, ALL, ALL, 4, 16384 + 256, POOL, POOL], {3, 4, 5, 6, 7, 8, 9}),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_overlapping_buffers_are_refused(L, name):
    call, sizes, written = CALLS[name]
    for i in written:
        for j in range(len(sizes)):
            if i == j:
                continue
            for at in (0, sizes[j] - 4, 4 - sizes[i]):
                ptrs = [BASE * (k + 1) for k in range(len(sizes))]
                ptrs[i] = ptrs[j] + at
                # a workspace off its alignment is refused for that; pools may stand at even addresses
                assert call(L, ptrs) in (api.ERR_INVALID_ARG, api.ERR_WORKSPACE), (i, j, at)
                assert "overlap" in api.last_error() or "aligned" in api.last_error()


@pytest.mark.parametrize("name", sorted(CALLS))
def test_bad_dims_and_missing_buffers_are_refused(L, name):
    call, sizes, _ = CALLS[name]
    ptrs = [BASE * (k + 1) for k in range(len(sizes))]
    for d in ((0, PAGE, PAGES, NUM), (B, 0, PAGES, NUM), (B, PAGE, 0, NUM), (B, PAGE, PAGES, 0)):
        assert call(L, ptrs, api.PagesDims(*d)) == api.ERR_INVALID_ARG, d
    for d in ((5000, PAGE, PAGES, NUM), (B, PAGE, PAGES, (1 << 30) + 1)):
        assert call(L, ptrs, api.PagesDims(*d)) == api.ERR_UNSUPPORTED, d
    optional = {10} if name == "fork" else set()
    for i in range(len(sizes)):
        if i in optional:
            continue
        missing = list(ptrs)
        missing[i] = 0
        assert call(L, missing) in (api.ERR_INVALID_ARG, api.ERR_WORKSPACE), i
        assert "NULL" in api.last_error()
    if name != "release":
        assert call(L, ptrs, row=0) == api.ERR_INVALID_ARG and "row_bytes" in api.last_error()
        assert call(L, ptrs, row=3) == api.ERR_INVALID_ARG
        assert call(L, ptrs, n_pools=33) == api.ERR_UNSUPPORTED and "n_pools" in api.last_error()
        assert call(L, ptrs, n_pools=-1) == api.ERR_UNSUPPORTED
        odd = list(ptrs)
        odd[-1] += 1
        assert call(L, odd) == api.ERR_INVALID_ARG and "aligned" in api.last_error()


def _norm(L, T=4, d=64, dtype=api.BF16, eps=1e-6, **kw):
    p = dict(x=0x10000, residual=0x20000, weight=0x30000, sum=0x40000, y=0x50000, q=0x60000, scale=0x70000)
    p.update(kw)
    dims = api.RmsNormDims(T, d, dtype)
    return L.dflash_rms_norm(ctypes.byref(dims), _p(p["x"]), _p(p["residual"]), _p(p["weight"]), eps, _p(p["sum"]),
                             _p(p["y"]), _p(p["q"]), _p(p["scale"]), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(T=-1), api.ERR_INVALID_ARG, "dims"), (dict(d=0), api.ERR_INVALID_ARG, "dims"),
    (dict(dtype=7), api.ERR_INVALID_ARG, "dtype"), (dict(T=(1 << 23) + 1), api.ERR_UNSUPPORTED, "2^23"),
    (dict(d=(1 << 23) + 16), api.ERR_UNSUPPORTED, "2^23"), (dict(eps=-1e-6), api.ERR_INVALID_ARG, "eps"),
    (dict(eps=float("nan")), api.ERR_INVALID_ARG, "eps"), (dict(eps=float("inf")), api.ERR_INVALID_ARG, "eps"),
    (dict(q=0), api.ERR_INVALID_ARG, "together"), (dict(scale=0), api.ERR_INVALID_ARG, "together"),
    (dict(d=40), api.ERR_UNSUPPORTED, "multiple of 16"), (dict(x=0), api.ERR_INVALID_ARG, "NULL"),
    (dict(weight=0), api.ERR_INVALID_ARG, "NULL"), (dict(y=0, q=0, scale=0), api.ERR_INVALID_ARG, "NULL"),
    (dict(x=0x10001), api.ERR_INVALID_ARG, "aligned"), (dict(q=0x60008), api.ERR_INVALID_ARG, "aligned"),
    (dict(scale=0x70002), api.ERR_INVALID_ARG, "aligned"), (dict(y=0x40000), api.ERR_INVALID_ARG, "same buffer"),
    (dict(y=0x10020), api.ERR_INVALID_ARG, "overlap"), (dict(sum=0x20010), api.ERR_INVALID_ARG, "overlap"),
    (dict(q=0x10000), api.ERR_INVALID_ARG, "overlap"), (dict(scale=0x60000), api.ERR_INVALID_ARG, "overlap"),
    (dict(y=0x30000), api.ERR_INVALID_ARG, "overlap"), (dict(sum=0x10000, y=0x10020), api.ERR_INVALID_ARG, "overlap"),
])
def test_norm_refusals(L, kw, code, word):
    assert _norm(L, **kw) == code
    assert word in api.last_error()


def test_norm_without_rows_needs_no_buffer(L):
    assert _norm(L, T=0, x=0, residual=0, weight=0, sum=0, y=0, q=0, scale=0) == api.OK
    assert L.dflash_last_launch_count() == 0


def test_prefix_attention_refusals(L):
    def call(n_groups, group=0x8000, prefix=0x9000, dims=None):
        d = dims or api.AttnDims(4, 16, 16, 32, 8, 128, 16, 64, 256, 1024, api.BF16, 0)
        p = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(7)]
        return L.dflash_prefix_attn(ctypes.byref(d), n_groups, *p, _p(group), _p(prefix), 0.1,
                                    ctypes.c_void_p(0x900000), None, 0, None)

    assert call(-1) == api.ERR_INVALID_ARG and "n_groups" in api.last_error()
    assert call(5) == api.ERR_INVALID_ARG and "n_groups" in api.last_error()
    assert call(2, group=0) == api.ERR_INVALID_ARG and "NULL" in api.last_error()
    assert call(2, prefix=0) == api.ERR_INVALID_ARG and "NULL" in api.last_error()
    assert call(2) == api.ERR_WORKSPACE
    bad = api.AttnDims(4, 16, 15, 32, 8, 128, 16, 64, 256, 1024, api.BF16, 1)
    assert call(2, dims=bad) == api.ERR_INVALID_ARG and "n_kv_blk" in api.last_error()
    d = api.AttnDims(4, 16, 16, 32, 8, 128, 16, 64, 256, 1024, api.BF16, 0)
    assert L.dflash_prefix_attn_workspace_size(ctypes.byref(d), 2) > api.WS_COUNTER_BYTES
    assert L.dflash_prefix_attn_workspace_size(ctypes.byref(d), 5) == 0


def test_a_pool_that_is_missing_or_unlike_the_first_is_refused():
    import torch

    good = torch.zeros((4, 2, 8))
    for bad in (None, torch.zeros((4, 2, 9)), torch.zeros((4, 2, 8), dtype=torch.bfloat16),
                torch.zeros((4, 2, 16))[:, :, ::2], 7):
        for pools in ([good, bad], [bad, good]):
            with pytest.raises((ValueError, TypeError)):
                api._pools(pools, good.get_device(), 4, 2)


def test_oracle_fork_release_compact_by_hand():
    table = np.array([[4, 2, 7], [-1, -1, -1], [-1, -1, -1]])
    pool = np.arange(8 * 4, dtype=np.float64).reshape(8, 4, 1)
    t, n, s, left, short, (p,) = O.pages_fork([-1, 0, 0], [10, 0, 0], table, [3, 0, 0], [0] * 8, [0, 1, 3, 5, 6, -1, -1, -1],
                                              5, 4, [pool])
    assert t.tolist() == [[4, 2, 7], [4, 2, 6], [4, 2, 5]] and n.tolist() == [3, 3, 3] and left == 3
    assert s.tolist() == [0, 0, 2, 0, 2, 0, 0, 0] and not short.any()
    assert p[6, :2, 0].tolist() == [28, 29] and p[6, 2:, 0].tolist() == [26, 27]
    n2, s2, f2, left2 = O.pages_release([0, 9, 0], t, n, s, [0, 1, 3, 5, 6, -1, -1, -1], 3, 4)
    assert n2.tolist() == [0, 3, 0] and s2.tolist() == [0] * 8 and f2.tolist() == [0, 1, 3, 5, 7, -1, -1, -1] and left2 == 5
    t3, s3, f3, left3, (p3,) = O.pages_compact(t, n2, s2, [p])
    assert t3[1].tolist() == [0, 2, 1] and left3 == 5 and f3.tolist() == [7, 6, 5, 4, 3, 2, 1, 0]
    assert p3[0].tolist() == p[4].tolist() and p3[1].tolist() == p[6].tolist()


def test_oracle_norm_closed_forms():
    s, y, scale = O.residual_norm(np.full((1, 256), 3.0), np.full(256, 2.0), 0.0)
    assert np.allclose(y, 2.0) and np.allclose(scale, 2 / 448)
    s, y, _ = O.residual_norm(np.eye(4), np.ones(4), 0.0, residual=-np.eye(4) + 1)
    assert np.allclose(s, 1) and np.allclose(y, 1)
