"""The 8-bit product when a wait runs out: it returns, with every copy of its own
landed, and the next call on the same workspace is right. Few groups a CTA: all of
its copies are issued before any other role gives up."""
import pytest
import torch

from block_diffusion_speculative_fusion_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_fusion_gb300 import build
    build.build()
    api.lib()
    yield
    api.set_wait_limit_ns(0)


@pytest.mark.parametrize("T,N,K", [
    (17, 10240, 512),                           # whole narrow tiles of four groups
    (40, 256, 2944),                            # three groups in each part of a split tile
    (20000, 100, 144),                          # two groups a tile, several tiles a CTA
    (1500, 2600, 4112), (290, 4000, 8016),      # wide tiles, whole and split
])
def test_wait_limit_runs_out_then_recovers(T, N, K):
    g = torch.Generator().manual_seed(T)
    x, xs = api.fp8_quant(torch.randn((T, K), generator=g).to(DEV))
    w, ws = api.fp8_quant(torch.randn((N, K), generator=g).to(DEV), block_rows=128)
    work = torch.zeros(api.WS_COUNTER_BYTES, dtype=torch.uint8, device=DEV)
    out = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    ref = api.fp8_gemm(x, xs, w, ws, ws=work)
    torch.cuda.synchronize()
    for _ in range(3):
        api.set_wait_limit_ns(200)              # far below the first copy of any launch
        try:
            api.fp8_gemm(x, xs, w, ws, ws=work, out=out)
            torch.cuda.synchronize()            # the kernel returned: no hang
        finally:
            api.set_wait_limit_ns(0)
        assert 1 <= api.device_error_word(work) <= 99
        api.clear_counters(work)
        # another kernel's shared memory and tensor memory right behind it
        assert torch.equal(api.fp8_gemm(x, xs, w, ws, ws=work, out=out), ref)
        assert api.device_error_word(work) == 0
