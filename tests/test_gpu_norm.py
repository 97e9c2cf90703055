"""GPU parity of the root-mean-square norm (dflash_rms_norm) against the oracle.

Tolerances, from the roundings of the definition (u = 2^-24, the fp32 half step): a
sum of squares errs by at most the longest chain of additions, c = (elements a thread
adds) + 12 of the tree, times u, relative, which its root halves; the sum with the
residual, the division, the root's reciprocal and two products add 6 u. y is then
within (c / 2 + 6) u, plus its type's half step (2^-8 for bf16); q times its scale
within half an e4m3 step of y (2^-4 relative, 2^-10 of the scale below the normal
range), plus the same. Below the normal range (2^-126) a type's steps stop shrinking:
bf16's 7 fraction bits leave steps of 2^-133, so y, rounded to nearest, may be off by
2^-134 there beside an element of 3e38 (fp32's 2^-150 is in the 1e-44)."""
import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_speculative_fusion_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_fusion_gb300 import build
    build.build()
    api.lib()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _tol(d):
    return (max(32, -(-d // 256)) + 12) / 2 * U + 6 * U


def _check(o, x, w, eps, residual, dtype):
    s, y, scale = O.residual_norm(_f64(x), _f64(w), eps, None if residual is None else _f64(residual))
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    t = _tol(s.shape[1])
    if residual is not None:
        assert np.all(np.abs(_f64(o["sum"]) - s) <= np.abs(s) * (half + U))
    if "y" in o:
        least = 2.0 ** -134 if dtype == torch.bfloat16 else 0.0
        assert np.all(np.abs(_f64(o["y"]) - y) <= np.abs(y) * (half + t * 1.01) + least + 1e-44)
    if "q" in o:
        sc = _f64(o["scale"])
        assert sc.shape == scale.shape and np.all(np.abs(sc - scale) <= scale * (t + 2 * U) + 1e-44)
        wide = np.repeat(sc, 128, 1)[:, :s.shape[1]]
        err = np.abs(_f64(o["q"]) * wide - y)
        assert np.all(err <= np.maximum(np.abs(y) * 2.0 ** -4, wide * 2.0 ** -10) * (1 + 1e-5) + np.abs(y) * t)


def _rows(T, d, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, d), generator=g) * size
    x[:, torch.rand(d, generator=g) < 0.02] *= 30
    return x.to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(1, 16), (1, 4096), (3, 128), (7, 144), (10, 4096), (5, 2560), (200, 272), (271, 2560),
                                 (1000, 4096), (2, 16384), (3, 20480), (200, 8192), (1, 65536), (2, 70000), (513, 64)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_and_e4m3(dtype, T, d, residual):
    x, r = _rows(T, d, dtype, 1), _rows(T, d, dtype, 2) if residual else None
    w = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(3))).to(dtype).to(DEV)
    o = api.rms_norm(x, w, 1e-6, residual=r, fp8=True, want_y=True)
    assert set(o) == ({"sum"} if residual else set()) | {"y", "q", "scale"}
    _check(o, x, w, 1e-6, r, dtype)
    again = api.rms_norm(x, w, 1e-6, residual=r, fp8=True)
    assert "y" not in again and torch.equal(again["q"].view(torch.uint8), o["q"].view(torch.uint8))
    assert torch.equal(again["scale"], o["scale"])
    plain = api.rms_norm(x, w, 1e-6, residual=r)
    assert set(plain) == ({"sum"} if residual else set()) | {"y"} and torch.equal(plain["y"], o["y"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(1, 1), (4, 7), (3, 129), (9, 1001), (2, 4095)])
def test_odd_widths(dtype, T, d):
    x, r, w = _rows(T, d, dtype, 4), _rows(T, d, dtype, 5), _rows(1, d, dtype, 6)[0].contiguous()
    _check(api.rms_norm(x, w, 1e-5, residual=r), x, w, 1e-5, r, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", range(4))
def test_tensors_off_a_vector(dtype, which):
    # one tensor of four starts an element past a multiple of 16 bytes
    T, d = 6, 256
    x, r, w = _rows(T, d, dtype, 7), _rows(T, d, dtype, 8), _rows(1, d, dtype, 9)[0].contiguous()

    def off(t):
        buf = torch.empty(t.numel() + 1, dtype=dtype, device=DEV)
        buf[1:].copy_(t.flatten())
        return buf[1:].view(t.shape)

    a = [x, r, w, torch.empty_like(x)]
    a[which] = off(a[which])
    o = api.rms_norm(a[0], a[2], 1e-6, residual=a[1], fp8=True, out={"y": a[3]})
    _check(o, x, w, 1e-6, r, dtype)


@pytest.mark.parametrize("T,d", [(2500, 4096), (5001, 144), (1500, 12288)])
def test_in_place_where_a_team_takes_several_rows(T, d):
    x, r, w = _rows(T, d, torch.bfloat16, 13), _rows(T, d, torch.bfloat16, 14), _rows(1, d, torch.bfloat16, 15)[0]
    w = w.contiguous()
    x[T // 2, :] = 0
    r[T // 2, :] = 0
    x[T - 1, 3] = 3e38
    x0, r0 = x.clone(), r.clone()
    o = api.rms_norm(x, w, 1e-6, residual=r, fp8=True, out={"sum": x, "y": r})
    _check(o, x0, w, 1e-6, r0, torch.bfloat16)


@pytest.mark.parametrize("d", [512, 4096, 20480, 70000])
def test_in_place(d):
    for alias in ("sum=x", "sum=residual", "y=x", "sum=residual,y=x", "sum=x,y=residual"):
        x, r, w = _rows(5, d, torch.bfloat16, 10), _rows(5, d, torch.bfloat16, 11), _rows(1, d, torch.bfloat16, 12)[0]
        w = w.contiguous()
        want = api.rms_norm(x, w, 1e-6, residual=r, fp8=True, want_y=True)
        t = {"x": x.clone(), "residual": r.clone()}
        out = {k: t[v] for k, v in (e.split("=") for e in alias.split(","))}
        got = api.rms_norm(t["x"], w, 1e-6, residual=t["residual"], fp8=True, want_y=True, out=out)
        for k in ("sum", "y", "scale"):
            assert torch.equal(got[k], want[k]), (alias, k)
        assert torch.equal(got["q"].view(torch.uint8), want["q"].view(torch.uint8))


@pytest.mark.parametrize("d", [256, 4096, 40000])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-18])
def test_rows_whose_squares_leave_the_range(d, eps):
    sizes = [1e30, 1e22, 1e15, 1.0, 1e-15, 1e-20, 1e-30, 1e-38]
    x = torch.cat([_rows(1, d, torch.float32, 20 + i, 1.0) * s for i, s in enumerate(sizes)])
    w = _rows(1, d, torch.float32, 30)[0].contiguous()
    o = api.rms_norm(x, w, eps, fp8=True, want_y=True)
    eps32 = float(np.float32(eps))
    _, y, _ = O.residual_norm(_f64(x), _f64(w), eps32)
    live = np.abs(y) > 1e-37                       # below it the result itself is subnormal
    assert np.all(np.abs(_f64(o["y"]) - y)[live] <= np.abs(y)[live] * _tol(d) * 1.5)


def test_zero_rows_infinities_and_nan():
    d = 384
    x = _rows(6, d, torch.float32, 40)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    w = torch.ones(d, device=DEV)
    o = api.rms_norm(x, w, 1e-6, fp8=True, want_y=True)
    y, q, s = o["y"], o["q"].float(), o["scale"]
    assert torch.equal(y[1], torch.zeros(d, device=DEV)) and torch.equal(q[1], torch.zeros(d, device=DEV))
    assert bool((s[1] == 2.0 ** -126).all())
    assert bool(y[2, 5].isnan()) and bool((y[2, :5] == 0).all()) and bool(q[2, 5].isnan())
    assert bool(y[3].isnan().all()) and bool(q[3].isnan().all())
    keep = [0, 4, 5]
    _check({k: v[keep] for k, v in o.items()}, x[keep], w, 1e-6, None, torch.float32)


def test_no_rows_and_a_million():
    w = torch.ones(32, dtype=torch.bfloat16, device=DEV)
    o = api.rms_norm(torch.empty((0, 32), dtype=torch.bfloat16, device=DEV), w, 1e-6, fp8=True)
    assert o["q"].shape == (0, 32) and o["scale"].shape == (0, 1)
    x = _rows(1 << 20, 32, torch.bfloat16, 50)
    o = api.rms_norm(x, w, 1e-6, fp8=True, want_y=True)
    pick = torch.tensor([0, 1, 77777, (1 << 20) - 1], device=DEV)
    _check({k: v[pick] for k, v in o.items()}, x[pick], w, 1e-6, None, torch.bfloat16)


def test_feeds_the_8_bit_product():
    # the normed rows in e4m3 through the product, against the definition in 64 bits of the same operands
    T, d, N = 33, 4096, 640
    x, r = _rows(T, d, torch.bfloat16, 60), _rows(T, d, torch.bfloat16, 61)
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    Wq, Ws = api.fp8_quant(_rows(N, d, torch.bfloat16, 62, 0.02), block_rows=128)
    o = api.rms_norm(x, w, 1e-6, residual=r, fp8=True)
    got = api.fp8_gemm(o["q"], o["scale"], Wq, Ws, out_dtype=torch.float32)
    ref, size = O.fp8_gemm(_f64(o["q"]), _f64(o["scale"]), _f64(Wq), _f64(Ws))
    assert np.all(np.abs(_f64(got) - ref) <= 2e-5 * size)


def test_captured_and_on_another_stream():
    x, r = _rows(50, 4096, torch.bfloat16, 70), _rows(50, 4096, torch.bfloat16, 71)
    w = _rows(1, 4096, torch.bfloat16, 72)[0].contiguous()
    want = api.rms_norm(x, w, 1e-6, residual=r, fp8=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out = api.rms_norm(x, w, 1e-6, residual=r, fp8=True)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.rms_norm(x, w, 1e-6, residual=r, fp8=True, out=out)
    for t in out.values():
        t.view(torch.uint8).zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(out[k].view(torch.uint8), want[k].view(torch.uint8)), k


def test_elements_past_two_to_the_31():
    T, d = 530000, 4096
    x = torch.zeros((T, d), dtype=torch.bfloat16, device=DEV)
    tail, w = _rows(40, d, torch.bfloat16, 16), _rows(1, d, torch.bfloat16, 17)[0].contiguous()
    x[-40:] = tail
    o = api.rms_norm(x, w, 1e-6, residual=x, fp8=True, want_y=True, out={"sum": x})
    # (against the definition: how a row's squares are added depends on the number of rows)
    _check({k: o[k][-40:] for k in ("sum", "y", "q", "scale")}, tail, w, 1e-6, tail, torch.bfloat16)
    assert not bool(o["y"][:-40].any())
