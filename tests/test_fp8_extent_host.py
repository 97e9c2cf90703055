"""Refusals at the ends of the 8-bit quantisation's extents, before a launch."""
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
