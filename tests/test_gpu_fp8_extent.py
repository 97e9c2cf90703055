"""8-bit quantisation in blocks at the largest extents that the call takes."""
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


@pytest.mark.parametrize("T,K", [(65535 * 128, 16), (65535 * 128 + 1, 16), (1 << 23, 16),
                                 (3, 65535 * 128 + 16), (130, 1 << 23)])
def test_quant_blocks_of_long_sides(T, K):
    # more than 65535 blocks along either side; the ends and some places between, exactly
    g = torch.Generator(device=DEV).manual_seed(T + K)
    x = torch.randn((T, K), generator=g, device=DEV).to(torch.bfloat16)
    q, s = api.fp8_quant(x, block_rows=128)
    assert s.shape == (-(-T // 128), -(-K // 128))
    rng = np.random.default_rng(0)
    row_blocks = sorted({0, s.shape[0] - 1, max(s.shape[0] - 2, 0), *rng.integers(0, s.shape[0], 5).tolist()})
    groups = sorted({0, s.shape[1] - 1, max(s.shape[1] - 2, 0), *rng.integers(0, s.shape[1], 5).tolist()})
    for i in row_blocks:
        for k in groups:
            blk = x[128 * i:128 * i + 128, 128 * k:128 * k + 128]
            rq, rs = O.fp8_quant(blk.float().cpu().numpy(), 128)
            assert float(s[i, k]) == rs[0, 0]
            assert np.array_equal(q[128 * i:128 * i + 128, 128 * k:128 * k + 128].float().cpu().numpy(), rq)
