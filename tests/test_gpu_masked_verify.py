"""The sampled accept rule on rows that a grammar mask has been through."""
import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_speculative_fusion_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NEG = float("-inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_fusion_gb300 import build
    build.build()
    api.lib()


def _lse(z):
    return torch.logsumexp(z.float(), -1)


def _verify(zt, zd, cand, ua, uf, lse):
    return api.verify_sample(zt.to(DEV), zd.to(DEV), cand.to(DEV), ua.to(DEV), uf.to(DEV), 1.0, want_probs=True,
                             draft_row_lse=_lse(zd).to(DEV) if lse else None)


def _f64(t):
    return t.float().numpy().astype(np.float64)


@pytest.mark.parametrize("lse", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [37, 2003, 40000])
def test_target_row_without_a_token(V, dtype, lse):
    """The row that the bonus is drawn from is -inf alone: after every candidate
    was accepted, and after a rejection."""
    B, n = 3, 3
    g = torch.Generator().manual_seed(V)
    zt = torch.randn((B, n + 1, V), generator=g).to(DT[dtype])
    zd = torch.randn((B, n, V), generator=g).to(DT[dtype])
    cand = torch.randint(0, V, (B, n + 1), generator=g)
    ua = torch.zeros((B, n))
    uf = torch.tensor([0.0, 0.5, 1 - 2.0 ** -24])
    zt[0, n] = NEG                             # all accepted (u = 0)
    zt[1, 1] = NEG                             # its candidate has p = 0
    zt[2, 0] = NEG
    got = _verify(zt, zd, cand, ua, uf, lse)
    ref = O.verify_sample(_f64(zt), _f64(zd), cand.numpy(), [n] * B, ua.numpy(), uf.numpy())
    assert got["accept_len"].tolist() == [n, 1, 0] == ref["accept_len"].tolist()
    assert torch.isfinite(got["probs"]).all(), got["probs"]
    assert got["probs"][:, 2 * n].tolist() == [0.0] * B      # the mass drawn from
    assert all(f & api.FLAG_DEGENERATE for f in got["flags"].tolist())
    assert all(f & O.FLAG_DEGENERATE for f in ref["flags"].tolist())
    assert not any(f & api.FLAG_INVALID for f in got["flags"].tolist())
    assert all(0 <= y < V for y in got["bonus"].tolist())
