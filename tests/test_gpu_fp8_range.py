"""The 8-bit product where the two scales' product leaves fp32's normal range and
the terms do not.

Tolerance: a group's 128 products of e4m3 values are added in fp32 (at most a step,
2^-23, of the running magnitude lost an addition); each scale's multiplication, and
each addition of the groups, of the split parts and of the result, rounds by half a
step (2^-24): 128 * 2^-23 + (groups + 12) * 2^-24 of the sum of the terms' magnitudes.
Every term in the cases is 0 or in the normal range."""
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


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _case(T, N, K, seed):
    """Rows and weight blocks of three kinds in turn, whose scales are about 1, small
    and large: where small meets small the product is subnormal or rounds to 0, and
    sums of up to 448 * 448 * 128 lift the terms to 2^-126 and more; where large meets
    large it is infinite, and one product of 2^-9 * 2^-9 a group brings them to 2^122."""
    g = np.random.default_rng(seed)
    G, NB = -(-K // 128), -(-N // 128)
    xe, we = np.array([0, -76, 68])[np.arange(T) % 3], np.array([-75, 0, 70])[np.arange(NB) % 3]
    xs = (g.uniform(1.5, 2, (T, G)) * np.exp2(xe[:, None])).astype(np.float32)
    ws = (g.uniform(1.5, 2, (NB, G)) * np.exp2(we[:, None])).astype(np.float32)
    x, w = g.choice([1.0, 1.25, 0.5], (T, K)), g.choice([1.0, 1.5, 2.0], (N, K))     # one sign: no sum cancels
    x[xe < 0] = 448.0
    x[xe > 0] = 0.0
    x[np.ix_(xe > 0, np.arange(0, K, 128))] = 2.0 ** -9
    kind = np.repeat(we, 128)[:N]
    w[kind < 0] = 448.0
    w[kind > 0] = 2.0 ** -9
    to8 = lambda a: torch.from_numpy(a).float().to(torch.float8_e4m3fn).to(DEV)
    return to8(x), torch.from_numpy(xs).to(DEV), to8(w), torch.from_numpy(ws).to(DEV)


@pytest.mark.parametrize("T,N,K", [
    (3, 384, 128), (7, 390, 384), (100, 300, 1168), (30, 512, 5120),       # narrow tiles, whole and split over K
    (1500, 2600, 528), (271, 3900, 5136), (400, 10240, 640),               # wide ones among them
])
def test_scales_whose_product_leaves_the_range(T, N, K):
    x, xs, w, ws = _case(T, N, K, T + K)
    with np.errstate(over="ignore"):
        f = xs.cpu().numpy()[:, None, :] * ws.cpu().numpy()[None]
    assert (f < 2.0 ** -126).any() and (np.isinf(f).any() or N < 384)
    got = _f64(api.fp8_gemm(x, xs, w, ws, out_dtype=torch.float32))
    ref, size = O.fp8_gemm(_f64(x), xs.cpu().numpy().astype(np.float64), _f64(w), ws.cpu().numpy().astype(np.float64))
    assert size.max() < 2.0 ** 128 and np.all((ref == 0) | (np.abs(ref) > 2.0 ** -126))
    tol = (128 * 2.0 ** -23 + (-(-K // 128) + 12) * 2.0 ** -24) * size
    err = np.abs(got - ref)
    assert np.isfinite(got).all() and np.all(err <= tol), (err / np.maximum(tol, 1e-300)).max()


def test_one_group_each_way():
    # terms that stand alone: 2^-140 x 2^21 and 2^145 x 2^-18, signs and all, and 2^130 x 0
    q = lambda v: torch.full((1, 128), 0.0).index_fill_(1, torch.tensor([5]), v).to(torch.float8_e4m3fn).to(DEV)
    s = lambda v: torch.full((1, 1), v, dtype=torch.float32, device=DEV)
    for xv, wv, a, b in [(448.0, 448.0, 1.37 * 2.0 ** -120, 1.21 * 2.0 ** -20),
                         (-448.0, 448.0, 1.21 * 2.0 ** -20, 1.37 * 2.0 ** -120),
                         (448.0, 448.0, 1.9 * 2.0 ** -126, 1.1 * 2.0 ** -16),
                         (2.0 ** -9, 2.0 ** -9, 1.37 * 2.0 ** 75, 1.21 * 2.0 ** 68),
                         (2.0 ** -9, -2.0 ** -9, 1.21 * 2.0 ** 18, 1.9 * 2.0 ** 125),
                         (0.0, 448.0, 6e35, 1e3)]:
        y = float(api.fp8_gemm(q(xv), s(a), q(wv), s(b), out_dtype=torch.float32))
        want = xv * wv * float(np.float32(a)) * float(np.float32(b))
        assert abs(y - want) <= 2 * 2.0 ** -24 * abs(want), (y, want)


@pytest.mark.parametrize("T,N,K", [(64, 128, 256), (40, 256, 2944), (1500, 2600, 528)])
def test_rows_whose_products_differ_in_kind(T, N, K):
    """Beside rows whose scales' product leaves the range, rows whose product is in the
    middle of it while one scale times the sum would overflow, and rows of scale 0."""
    g = np.random.default_rng(T)
    kind = np.arange(T) % 3
    xs = g.uniform(1.5, 2, (T, -(-K // 128))) * np.exp2(np.array([-76, 115, 0])[kind][:, None])
    xs[kind == 2] = 0.0
    ws = g.uniform(1.5, 2, (-(-N // 128), -(-K // 128))) * 2.0 ** -75
    x, w = np.full((T, K), 448.0), np.full((N, K), 448.0)
    to8 = lambda a: torch.from_numpy(a).float().to(torch.float8_e4m3fn).to(DEV)
    xs, ws = xs.astype(np.float32), ws.astype(np.float32)
    got = _f64(api.fp8_gemm(to8(x), torch.from_numpy(xs).to(DEV), to8(w), torch.from_numpy(ws).to(DEV),
                            out_dtype=torch.float32))
    ref, size = O.fp8_gemm(x, xs.astype(np.float64), w, ws.astype(np.float64))
    assert size.max() < 2.0 ** 128 and np.all((ref == 0) == (kind == 2)[:, None])
    tol = (128 * 2.0 ** -23 + (-(-K // 128) + 12) * 2.0 ** -24) * size
    assert np.all(np.abs(got - ref) <= tol)
