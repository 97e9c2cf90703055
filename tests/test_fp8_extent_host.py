"""Refusals of the 8-bit calls at the ends of their extents and alignments, before a launch."""
import ctypes

import pytest

from block_diffusion_speculative_fusion_gb300 import api, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


@pytest.mark.parametrize("T,K,rows", [((1 << 23) + 1, 16, 128), (16, (1 << 23) + 16, 128), (1 << 23, 1 << 23, 128)])
def test_quant_refuses_more_blocks_than_a_grid_holds(L, T, K, rows):
    p = ctypes.c_void_p(0x10000)
    d = api.Fp8QuantDims(T, K, api.BF16, rows)
    assert L.dflash_fp8_quant(ctypes.byref(d), p, p, p, None) == api.ERR_UNSUPPORTED
    assert "2^23" in api.last_error() or "blocks" in api.last_error()


@pytest.mark.parametrize("dtype,off", [(api.BF16, 1), (api.F32, 2), (api.F32, 1)])
def test_product_refuses_out_and_bias_between_elements(L, dtype, off):
    d = api.Fp8GemmDims(4, 8, 128, dtype)
    for i in (4, 5):                            # bias, out
        p = [ctypes.c_void_p(0x10000)] * 7
        p[i] = ctypes.c_void_p(0x10000 + off)
        assert L.dflash_fp8_gemm(ctypes.byref(d), *p, api.WS_COUNTER_BYTES, None) == api.ERR_INVALID_ARG
        assert "aligned to its type" in api.last_error()
