"""GPU parity of the 8-bit quantisation, the product with block scales and the
materialisation with 8-bit weights.

Quantisation: the definition's fp32 steps are correctly rounded on both sides,
so values and scales are compared exactly.

Product: products of two e4m3 values are exact in fp32. A group's 128 of them
are added in fp32 (at most one step, 2^-23, of the running magnitude lost an
addition, whatever the order and the rounding), the product of the two scales,
the groups' and the split parts' sums and the bias round by half a step (2^-24)
each: 128 * 2^-23 + (groups + 12) * 2^-24 of the sum of the magnitudes of all
terms covers it, and bf16 adds 2^-8 of the value. An error in a scale, a group
or a lane is of the order of the value itself."""
import ctypes
import dataclasses

import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_speculative_fusion_gb300 import api, synth
from block_diffusion_speculative_fusion_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_fusion_gb300 import build
    build.build()
    api.lib()
    yield
    api.set_wait_limit_ns(0)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _rows(T, K, dtype, seed):
    g = np.random.default_rng(seed)
    x = g.normal(0, 1, (T, K)) * np.where(g.random(K) < 0.02, 30.0, 1.0) * np.exp2(g.integers(-20, 20, (T, 1)))
    x[g.random((T, K)) < 0.05] = 0.0
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("T,K", [(1, 16), (3, 128), (7, 144), (128, 112), (129, 272), (300, 1040), (1, 20480)])
def test_quant(T, K, dtype, block):
    x = _rows(T, K, dtype, T * 1000 + K)
    q, s = api.fp8_quant(x.to(DEV), block_rows=block)
    assert api.last_launch_count() == 1 and q.dtype == torch.float8_e4m3fn
    rq, rs = O.fp8_quant(x.float().numpy(), block)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(f64(q), rq)


def test_quant_many_rows():
    # several passes of the grid
    x = _rows(4099, 2064, "bf16", 1)
    q, s = api.fp8_quant(x.to(DEV))
    pick = np.random.default_rng(0).choice(4099, 64, replace=False)
    rq, rs = O.fp8_quant(x.float().numpy()[pick])
    assert np.array_equal(s.cpu().numpy()[pick], rs) and np.array_equal(f64(q)[pick], rq)


def test_quant_zeros_tiny_and_non_finite():
    x = torch.zeros((6, 256), dtype=torch.float32)
    x[1, 5] = 2.0 ** -140                      # a subnormal's block: the scale stops at 2^-126
    x[2, :] = 3e38
    x[3, 7] = float("nan")
    x[3, 9] = 2.0
    x[4, 200] = float("inf")
    x[4, 201] = 1.0
    q, s = api.fp8_quant(x.to(DEV))
    v, s = f64(q), s.cpu().numpy()
    assert s[0, 0] == np.float32(2.0 ** -126) and not v[0].any()
    assert s[1, 0] == np.float32(2.0 ** -126) and not v[1].any()
    assert np.all(v[2] == 448)
    assert np.isnan(v[3, 7]) and v[3, 9] == 448 and s[3, 0] == np.float32(2) / np.float32(448)
    assert np.isinf(s[4, 1]) and np.isnan(v[4, 200]) and v[4, 201] == 0
    assert np.isfinite(s[4, 0]) and not v[4, :128].any()


def _operands(T, N, K, seed, dtype="bf16"):
    g = torch.Generator().manual_seed(seed)
    x, xs = api.fp8_quant(_rows(T, K, "bf16", seed).to(DEV) if T else torch.empty((0, K), dtype=torch.bfloat16, device=DEV))
    w, ws = api.fp8_quant((torch.randn((N, K), generator=g) * torch.rand((N, 1), generator=g)).to(DEV), block_rows=128)
    bias = torch.randn(N, generator=g).to(DT[dtype]).to(DEV)
    return x, xs, w, ws, bias


def _check_gemm(T, N, K, dtype, seed=0, bias=True, out=None):
    x, xs, w, ws, b = _operands(T, N, K, seed, dtype)
    work = torch.zeros(api.WS_COUNTER_BYTES, dtype=torch.uint8, device=DEV)
    got = api.fp8_gemm(x, xs, w, ws, bias=b if bias else None, out_dtype=DT[dtype], ws=work, out=out)
    assert api.device_error_word(work) == 0
    ref, size = O.fp8_gemm(f64(x), f64(xs), f64(w), f64(ws), f64(b) if bias else None)
    groups = -(-K // 128)
    tol = (128 * 2.0 ** -23 + (groups + 12) * 2.0 ** -24) * size * (1 + 2.0 ** -8)
    if dtype == "bf16":
        tol += 2.0 ** -8 * np.abs(ref)
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), (err.max(), (err / np.maximum(tol, 1e-300)).max())
    return got


@pytest.mark.parametrize("T,N,K", [
    (1, 1, 16), (1, 128, 128), (2, 7, 144), (8, 100, 400), (9, 129, 2064), (10, 256, 4096), (127, 127, 128),
    (128, 128, 256), (129, 257, 272), (130, 1000, 112), (271, 640, 1040), (64, 2560, 2560),      # split over K
    (17, 10240, 640), (600, 2560, 384), (1500, 2560, 272), (1537, 2500, 144), (2100, 2600, 256),  # whole tiles
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_product(T, N, K, dtype):
    _check_gemm(T, N, K, dtype, seed=T + N + K, bias=(T + N) % 2 == 0)


def test_product_llama8b_fusion_and_projection():
    # one sequence's commit through W_f, the throughput workload's through W_kv
    _check_gemm(10, 4096, 20480, "bf16", seed=1)
    _check_gemm(271, 10240, 4096, "f32", seed=2)


@pytest.mark.parametrize("T,N,K", [(290, 4000, 8016), (300, 2500, 12048),
                                   (1500, 2600, 4112), (271, 3900, 20496),    # wide tiles, whole and split over K
                                   (20000, 100, 144)])                        # several narrow tiles a CTA
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_product_other_tilings(T, N, K, dtype):
    _check_gemm(T, N, K, dtype, seed=T, bias=dtype == "bf16")


def test_product_of_a_prefill_on_picked_rows():
    # persistent CTAs over several waves of wide tiles
    T, N, K = 8190, 4096, 1024
    x, xs, w, ws, b = _operands(T, N, K, 3)
    got = api.fp8_gemm(x, xs, w, ws, bias=b, out_dtype=torch.bfloat16)
    pick = torch.from_numpy(np.random.default_rng(4).choice(T, 200, replace=False)).to(DEV)
    ref, size = O.fp8_gemm(f64(x)[pick.cpu()], f64(xs)[pick.cpu()], f64(w), f64(ws), f64(b))
    tol = (128 * 2.0 ** -23 + 20 * 2.0 ** -24) * size * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(f64(got[pick]) - ref) <= tol)


def test_product_repeats_bit_for_bit_on_any_stream_and_in_a_graph():
    x, xs, w, ws, b = _operands(33, 900, 2064, 5)
    ref = api.fp8_gemm(x, xs, w, ws, bias=b)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        side = api.fp8_gemm(x, xs, w, ws, bias=b)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(side, ref)
    out = torch.zeros_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.fp8_gemm(x, xs, w, ws, bias=b, out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, ref)


def test_product_into_an_odd_view_and_no_rows():
    x, xs, w, ws, b = _operands(5, 131, 272, 6)
    ref = api.fp8_gemm(x, xs, w, ws, bias=b)
    buf = torch.full((5 * 131 + 9,), 7.0, dtype=torch.bfloat16, device=DEV)
    api.fp8_gemm(x, xs, w, ws, bias=b, out=buf[3:3 + 5 * 131].view(5, 131))
    assert torch.equal(buf[3:3 + 5 * 131].view(5, 131), ref)
    assert float(buf[:3].min()) == 7.0 and float(buf[3 + 5 * 131:].min()) == 7.0    # nothing written outside
    none = api.fp8_gemm(x[:0], xs[:0], w, ws, bias=b)
    assert none.shape == (0, 131) and api.last_launch_count() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", [(130, 256, 272), (1500, 2608, 4112)])     # narrow and wide tiles
def test_product_alignments_of_out_and_bias(T, N, K, dtype):
    x, xs, w, ws, b = _operands(T, N, K, 11, dtype)
    ref = api.fp8_gemm(x, xs, w, ws, bias=b, out_dtype=DT[dtype])
    el = ref.element_size()
    for skip_out, skip_bias in ((0, 1), (16 // el, 0), (8 // el, 3)):    # elements past a 256-byte boundary
        buf = torch.full((T * N + 32,), 7.0, dtype=DT[dtype], device=DEV)
        bias = torch.zeros(N + 8, dtype=DT[dtype], device=DEV)
        bias[skip_bias:skip_bias + N] = b
        out = buf[skip_out:skip_out + T * N].view(T, N)
        api.fp8_gemm(x, xs, w, ws, bias=bias[skip_bias:skip_bias + N], out=out)
        assert torch.equal(out, ref)
        assert bool((buf[:skip_out] == 7.0).all()) and bool((buf[skip_out + T * N:] == 7.0).all())


def test_product_keeps_nan_and_infinity_to_their_rows():
    T, N, K = 6, 70, 256
    x, xs, w, ws, _ = _operands(T, N, K, 7)
    src = torch.randn((T, K), device=DEV)
    src[2, 3] = float("nan")
    src[4, 200] = float("inf")
    x, xs = api.fp8_quant(src)
    y = api.fp8_gemm(x, xs, w, ws, out_dtype=torch.float32)
    assert torch.isnan(y[2]).all() and torch.isnan(y[4]).all()
    assert torch.isfinite(y[[0, 1, 3, 5]]).all()


def test_product_wait_limit_runs_out_then_recovers():
    x, xs, w, ws, b = _operands(40, 2560, 4096, 8)
    work = torch.zeros(api.WS_COUNTER_BYTES, dtype=torch.uint8, device=DEV)
    ref = api.fp8_gemm(x, xs, w, ws, bias=b, ws=work)
    torch.cuda.synchronize()
    api.set_wait_limit_ns(200)              # far below the first copy of any launch
    try:
        api.fp8_gemm(x, xs, w, ws, bias=b, ws=work)
        torch.cuda.synchronize()            # the kernel returned: no hang
    finally:
        api.set_wait_limit_ns(0)
    assert 1 <= api.device_error_word(work) <= 99
    api.clear_counters(work)
    assert torch.equal(api.fp8_gemm(x, xs, w, ws, bias=b, ws=work), ref)
    assert api.device_error_word(work) == 0


def _mat_case(d, m, L, Hkv, D, commit, start, seed, page=16, k_norm=True, theta=10000.0):
    """Small whole numbers: every sum before h_ctx's quantisation is exact, so
    the oracle's h_ctx, and with it every 8-bit value, is the kernel's."""
    B, rows = len(commit), max(max(commit), 1)
    g = np.random.default_rng(seed)
    hidden = torch.from_numpy(g.choice([-2.0, -1.0, 0.0, 0.5, 1.0, 2.0], (B, rows, m * d)).astype(np.float32))
    hidden[:, :, ::128] = 2.0                  # every group's largest value: 448 / 2^k are on the grid
    W_f = torch.from_numpy(g.choice([-1.0, 0.0, 0.0, 0.0, 1.0], (d, m * d)).astype(np.float32))
    W_kv = torch.from_numpy(g.normal(0, 0.05, (L, 2, Hkv * D, d)).astype(np.float32))
    b_f = torch.from_numpy(g.integers(-3, 4, d).astype(np.float32))
    kn = torch.from_numpy((1 + 0.1 * g.normal(0, 1, (L, D))).astype(np.float32)).to(torch.bfloat16) if k_norm else None
    n_pg = [(s + rows + page - 1) // page for s in start]
    pt = torch.full((B, max(n_pg)), -1, dtype=torch.int32)
    perm = g.permutation(sum(n_pg)).astype(np.int32)
    at = 0
    for b in range(B):
        pt[b, :n_pg[b]] = torch.from_numpy(perm[at:at + n_pg[b]])
        at += n_pg[b]
    pools = [torch.from_numpy(g.normal(0, 1, (sum(n_pg), page, Hkv, D)).astype(np.float32)).to(torch.bfloat16)
             for _ in range(2 * L)]
    fq, fs = api.fp8_quant(W_f.to(torch.bfloat16).to(DEV), block_rows=128)
    kq, ks = api.fp8_quant(W_kv.to(DEV).view(-1, d), block_rows=128)
    kd, vd = [t.to(DEV) for t in pools[:L]], [t.to(DEV) for t in pools[L:]]
    new_len = torch.empty(B, dtype=torch.int32, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    args = (hidden.to(torch.bfloat16).to(DEV), torch.tensor(commit, **i32), torch.tensor(start, **i32), fq, fs,
            b_f.to(torch.bfloat16).to(DEV), kq.view(L, 2, Hkv * D, d), ks, None if kn is None else kn.to(DEV), 1e-6, theta)
    api.materialize_ctx_kv_fp8(*args, kd, vd, pt.to(DEV), new_len=new_len)
    assert api.last_launch_count() == 6 and set(api.error_words().values()) == {0}
    assert new_len.tolist() == [s + c for s, c in zip(start, commit)]
    # the oracle's chain on the dequantised weights and the quantised rows
    wf = f64(fq) * O.fp8_spread(f64(fs), 128, d, m * d)
    wkv = (f64(kq) * O.fp8_spread(f64(ks), 128, L * 2 * Hkv * D, d)).reshape(L, 2, Hkv * D, d)
    q, s = O.fp8_quant(hidden.reshape(-1, m * d).numpy())
    h = (q * O.fp8_spread(s, 1, *q.shape)) @ wf.T + f64(b_f)
    exact = hidden.reshape(-1, m * d).double().numpy() @ W_f.double().numpy().T + f64(b_f)
    assert np.abs(h - exact).max() < 1e-3 and np.abs(exact).max() <= 256 and np.all(exact * 2 == np.rint(exact * 2))
    h = torch.from_numpy(exact).to(torch.bfloat16).float().numpy()
    hq, hs = O.fp8_quant(h)
    h = (hq * O.fp8_spread(hs, 1, *hq.shape)).reshape(B, rows, d)
    eye = np.eye(d)
    rk, rv = O.materialize_ctx_kv(h, commit, start, eye, np.zeros(d), wkv, None if kn is None else f64(kn), 1e-6,
                                  theta, [f64(t) for t in pools[:L]], [f64(t) for t in pools[L:]], pt.numpy(), page)
    for got, ref in zip(kd + vd, rk + rv):
        # one rounding to bf16 and fp32 sums; the rotation and the norm mix a head's values
        big = np.abs(ref).max(axis=-1, keepdims=True)
        assert np.all(np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -14 * big)
    return args, pt, pools


@pytest.mark.parametrize("d,m,L,Hkv,D,commit,start", [
    (128, 2, 1, 2, 128, [3, 0, 5], [0, 7, 30]),
    (256, 1, 2, 1, 64, [1], [100]),
    (144, 2, 3, 2, 32, [4, 2], [15, 16]),           # groups and blocks that end early
    (512, 1, 2, 2, 128, [16] * 20, list(range(0, 200, 10))),
    # far fewer rows committed than the call is sized for, tiles of many K/V columns
    (128, 1, 5, 8, 128, [16, 3] + [0] * 40 + [1] * 30 + [0, 9] * 4, list(range(80))),
])
def test_materialize_fp8(d, m, L, Hkv, D, commit, start):
    _mat_case(d, m, L, Hkv, D, commit, start, seed=d + m, k_norm=D == 128, theta=10000.0 if D != 64 else 0.0)


def test_materialize_fp8_without_committed_rows():
    _mat_case(128, 1, 1, 1, 128, [0, 0], [4, 5], seed=9)


def test_materialize_fp8_follows_the_bf16_materialisation():
    # the throughput shape: 8-bit K/V within the quantisation's error of the bf16 ones.
    # Each factor is off by at most 2^-4 relative, independently: the four
    # quantisations of the chain leave a relative error of the whole below 0.1.
    wl = dataclasses.replace(W.LLAMA8B_B64, B=4)
    w = synth.ctx_weights(wl, 21)
    hidden = synth.captured_hidden(wl, wl.k, 21, B=wl.B).to(DEV)
    start = torch.tensor([5, 100, 0, 33], dtype=torch.int32)
    cache = synth.paged_cache(wl, headroom=wl.k, seed=21, layers=wl.L, ctx_len=start, device=DEV)
    commit = torch.tensor([16, 9, 1, 12], dtype=torch.int32, device=DEV)
    pt, st = cache.page_table.to(DEV), start.to(DEV)
    zero = [torch.zeros_like(t) for t in cache.k_pools]
    k1, v1 = [t.clone() for t in zero], [t.clone() for t in zero]
    k2, v2 = [t.clone() for t in zero], [t.clone() for t in zero]
    bf = w["b_f"].to(DEV)
    kn = w["k_norm_w"].to(DEV)
    api.materialize_ctx_kv(hidden, commit, st, w["W_f"].to(DEV), bf, w["W_kv"].to(DEV), kn, wl.rms_eps, wl.rope_theta,
                           k1, v1, pt)
    fq, fs = api.fp8_quant(w["W_f"].to(DEV), block_rows=128)
    kq, ks = api.fp8_quant(w["W_kv"].to(DEV).view(-1, wl.d), block_rows=128)
    api.materialize_ctx_kv_fp8(hidden, commit, st, fq, fs, bf, kq.view(w["W_kv"].shape), ks, kn, wl.rms_eps,
                               wl.rope_theta, k2, v2, pt)
    for a, b in zip(k1 + v1, k2 + v2):
        assert torch.equal(a != 0, b != 0) or float(((a != 0) ^ (b != 0)).float().mean()) < 1e-3
        rel = float((a.float() - b.float()).norm() / a.float().norm())
        assert rel < 0.1, rel


def test_captured_materialisation_outlives_a_larger_call():
    # the cached workspace is outgrown after a capture: the graph keeps the one it was captured with
    api.reset_workspaces()
    args, pt, pools = _mat_case(128, 2, 1, 2, 128, [3, 0, 5], [0, 7, 30], seed=11)
    kd, vd = [pools[0].to(DEV)], [pools[1].to(DEV)]
    table = pt.to(DEV)
    api.materialize_ctx_kv_fp8(*args, kd, vd, table)
    ref = kd[0].clone(), vd[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.materialize_ctx_kv_fp8(*args, kd, vd, table)
    _mat_case(256, 2, 1, 2, 128, [16] * 40, [0] * 40, seed=12)         # a larger workspace
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in range(64)]
    kd[0].zero_()
    vd[0].zero_()
    graph.replay()
    rows = (kd[0] != 0).flatten(2).any(2)
    assert rows.any() and torch.equal(kd[0][rows], ref[0][rows]) and torch.equal(vd[0][rows], ref[1][rows])
    assert all(int(j.min()) == 255 for j in junk)
