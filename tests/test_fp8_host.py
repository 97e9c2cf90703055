"""Host checks of the 8-bit quantisation, product and materialisation: every
refusal happens before a launch, and the oracle's e4m3 rounding against torch's."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_speculative_fusion_gb300 import api, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def _p(x=0x10000):
    return ctypes.c_void_p(x)


@pytest.mark.parametrize("dims,code,word", [
    (api.Fp8QuantDims(-1, 128, api.BF16, 1), api.ERR_INVALID_ARG, "T=-1"),
    (api.Fp8QuantDims(4, 0, api.BF16, 1), api.ERR_INVALID_ARG, "K=0"),
    (api.Fp8QuantDims(4, 128, 9, 1), api.ERR_INVALID_ARG, "dtype"),
    (api.Fp8QuantDims(4, 128, api.BF16, 64), api.ERR_INVALID_ARG, "block_rows"),
    (api.Fp8QuantDims(4, 120, api.BF16, 1), api.ERR_UNSUPPORTED, "multiple of 16"),
    (api.Fp8QuantDims((1 << 23) + 1, 128, api.BF16, 1), api.ERR_UNSUPPORTED, "2^23"),
    (api.Fp8QuantDims(4, (1 << 23) + 16, api.BF16, 1), api.ERR_UNSUPPORTED, "2^23"),
])
def test_quant_refusals(L, dims, code, word):
    assert L.dflash_fp8_quant(ctypes.byref(dims), _p(), _p(), _p(), None) == code and word in api.last_error()


def test_quant_refuses_pointers(L):
    d = api.Fp8QuantDims(4, 128, api.BF16, 1)
    for args in ((None, _p(), _p()), (_p(), None, _p()), (_p(), _p(), None)):
        assert L.dflash_fp8_quant(ctypes.byref(d), *args, None) == api.ERR_INVALID_ARG
    for args in ((_p(0x10008), _p(), _p()), (_p(), _p(0x10004), _p())):
        assert L.dflash_fp8_quant(ctypes.byref(d), *args, None) == api.ERR_INVALID_ARG
        assert "16-byte" in api.last_error()
    assert L.dflash_fp8_quant(None, _p(), _p(), _p(), None) == api.ERR_INVALID_ARG
    # no rows: nothing is launched, whatever the pointers
    assert L.dflash_fp8_quant(ctypes.byref(api.Fp8QuantDims(0, 128, api.BF16, 1)), None, None, None, None) == api.OK


@pytest.mark.parametrize("dims,code,word", [
    (api.Fp8GemmDims(-1, 8, 128, api.BF16), api.ERR_INVALID_ARG, "T=-1"),
    (api.Fp8GemmDims(4, 0, 128, api.BF16), api.ERR_INVALID_ARG, "N=0"),
    (api.Fp8GemmDims(4, 8, 128, 5), api.ERR_INVALID_ARG, "dtype"),
    (api.Fp8GemmDims(4, 8, 136, api.BF16), api.ERR_UNSUPPORTED, "multiple of 16"),
    (api.Fp8GemmDims(4, (1 << 23) + 1, 128, api.BF16), api.ERR_UNSUPPORTED, "2^23"),
    (api.Fp8GemmDims(1 << 23, 1 << 23, 128, api.BF16), api.ERR_UNSUPPORTED, "tiles"),
])
def test_product_refusals(L, dims, code, word):
    assert L.dflash_fp8_gemm_workspace_size(ctypes.byref(dims)) == 0 and word in api.last_error()
    ptrs = [_p()] * 7
    assert L.dflash_fp8_gemm(ctypes.byref(dims), *ptrs, 1 << 20, None) == code and word in api.last_error()


def test_product_refuses_pointers_and_workspaces(L):
    d = api.Fp8GemmDims(4, 8, 128, api.BF16)
    need = L.dflash_fp8_gemm_workspace_size(ctypes.byref(d))
    assert need == api.WS_COUNTER_BYTES
    # x, x_scale, w, w_scale, bias, out, workspace
    for i in (0, 1, 2, 3, 5):
        ptrs = [_p()] * 7
        ptrs[i] = None
        assert L.dflash_fp8_gemm(ctypes.byref(d), *ptrs, need, None) == api.ERR_INVALID_ARG
    for i in (0, 2):
        ptrs = [_p()] * 7
        ptrs[i] = _p(0x10008)
        assert L.dflash_fp8_gemm(ctypes.byref(d), *ptrs, need, None) == api.ERR_INVALID_ARG
        assert "16-byte" in api.last_error()
    ptrs = [_p()] * 7
    assert L.dflash_fp8_gemm(ctypes.byref(d), *ptrs, need - 1, None) == api.ERR_WORKSPACE
    ptrs[6] = None
    assert L.dflash_fp8_gemm(ctypes.byref(d), *ptrs, need, None) == api.ERR_WORKSPACE
    assert L.dflash_fp8_gemm(ctypes.byref(api.Fp8GemmDims(0, 8, 128, api.BF16)), *([None] * 7), 0, None) == api.OK


def test_materialize_fp8_refusals(L):
    ok = api.CtxKvDims(2, 4, 5, 256, 2, 2, 128, 16, 8, 64, api.BF16)
    need = L.dflash_materialize_fp8_workspace_size(ctypes.byref(ok))
    assert need > api.WS_COUNTER_BYTES
    f32 = api.CtxKvDims(2, 4, 5, 256, 2, 2, 128, 16, 8, 64, api.F32)
    assert L.dflash_materialize_fp8_workspace_size(ctypes.byref(f32)) == 0 and "bf16" in api.last_error()
    odd = api.CtxKvDims(2, 4, 5, 264, 2, 2, 128, 16, 8, 64, api.BF16)
    assert L.dflash_materialize_fp8_workspace_size(ctypes.byref(odd)) == 0 and "multiple of 16" in api.last_error()
    pools = ctypes.cast((ctypes.c_void_p * 2)(0x10000, 0x20000), ctypes.c_void_p)
    eps, theta = ctypes.c_float(1e-6), ctypes.c_float(1e4)

    def call(W_f=_p(), W_f_scale=_p(), new_len=None, size=need):
        return L.dflash_materialize_ctx_kv_fp8(ctypes.byref(ok), _p(), _p(), _p(0x30000), W_f, W_f_scale, None, _p(),
                                               _p(), None, eps, theta, pools, pools, _p(), new_len, _p(), size, None)
    assert call(W_f_scale=None) == api.ERR_INVALID_ARG and "NULL" in api.last_error()
    assert call(W_f=_p(0x10008)) == api.ERR_INVALID_ARG and "16-byte" in api.last_error()
    assert call(new_len=_p(0x30000)) == api.ERR_INVALID_ARG and "alias" in api.last_error()
    assert call(size=need - 1) == api.ERR_WORKSPACE


def test_oracle_rounding_is_torchs():
    g = np.random.default_rng(0)
    v = np.concatenate([g.normal(0, 1, 4000) * np.exp2(g.integers(-12, 8, 4000)), [0, 448, -448, 2.0 ** -9, 2.0 ** -10,
                        1.5 * 2.0 ** -9, 17, 17.0001, 19, 0.0625 * 17]]).astype(np.float32)
    v = np.clip(v, -448, 448)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(O.e4m3_round(v), want)
