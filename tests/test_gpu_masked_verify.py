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


@pytest.mark.parametrize("lse", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q", ["-inf", "underflows", "row of -inf"])
def test_forbidden_candidate_is_rejected_where_q_is_zero(q, dtype, lse):
    """p(x) = 0 by the mask and q(x) = 0: not accepted, whatever u (0 included)."""
    B, n, V = 4, 2, 1003
    g = torch.Generator().manual_seed(5)
    zt = torch.randn((B, n + 1, V), generator=g).to(DT[dtype])
    zd = torch.randn((B, n, V), generator=g).to(DT[dtype])
    cand = torch.randint(1, V, (B, n + 1), generator=g)
    bad = cand[:, 1]                           # forbidden in row 0
    zt[torch.arange(B), 0, bad] = NEG
    if q == "row of -inf":
        zd[:, 0] = NEG
    else:
        zd[torch.arange(B), 0, bad] = NEG if q == "-inf" else -1000.0
    ua = torch.tensor([[0.0, 0.5], [0.25, 0.5], [0.5, 0.5], [1 - 2.0 ** -24, 0.5]])
    uf = torch.tensor([0.1, 0.4, 0.7, 0.95])
    got = _verify(zt, zd, cand, ua, uf, lse)
    ref = O.verify_sample(_f64(zt), _f64(zd), cand.numpy(), [n] * B, ua.numpy(), uf.numpy())
    assert got["accept_len"].tolist() == [0] * B == ref["accept_len"].tolist()
    assert all(f & api.FLAG_INVALID for f in got["flags"].tolist())
    assert torch.isfinite(got["probs"]).all()
    assert got["probs"][:, 0].tolist() == [0.0] * B and got["probs"][:, n].tolist() == [0.0] * B
    y = got["bonus"].cpu()
    assert not torch.isneginf(zt[torch.arange(B), 0, y].float()).any()
    # fp32 and 64 bits may differ within 1e-6 of a step, which is flagged
    sure = (got["flags"].cpu().numpy() | ref["flags"]) & api.FLAG_CDF_BOUNDARY == 0
    assert np.array_equal(y.numpy()[sure], ref["bonus"][sure])
    if q == "row of -inf":                     # the draft has no law: the residual is p itself
        assert torch.allclose(got["probs"][:, 2 * n].cpu(), torch.ones(B), atol=1e-5)


@pytest.mark.parametrize("reject", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,keep", [(9000, 4000), (20011, 17000), (128256, 30000)])
def test_last_uniform_draws_an_allowed_token(V, keep, dtype, reject):
    """u_final next to 1 puts the target at the end of the allowed tokens, past
    the sum of the steps as it was rounded for some rows: the token drawn is the
    last one with weight, or one of those before it, never a forbidden one."""
    B, n = 64, 1
    g = torch.Generator().manual_seed(V + keep)
    zt = (2 * torch.randn((B, n + 1, V), generator=g)).to(DT[dtype])
    zt[:, :, keep:] = NEG
    zd = (2 * torch.randn((B, n, V), generator=g)).to(DT[dtype])
    cand = torch.zeros((B, n + 1), dtype=torch.int64)
    cand[:, 1] = V - 1 if reject else zt[:, 0].float().argmax(-1)
    ua = torch.zeros((B, n))
    uf = torch.full((B,), 1 - 2.0 ** -24)
    got = _verify(zt, zd, cand, ua, uf, False)
    assert got["accept_len"].tolist() == [0 if reject else 1] * B
    y = got["bonus"].cpu()
    assert (y < keep).all(), y[y >= keep].tolist()
    row = zt[:, 0 if reject else 1].float()
    assert (torch.softmax(row.double(), -1)[torch.arange(B), y] > 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sparse_masks_at_every_step_of_the_law(dtype):
    """Every other token forbidden, and u_final at, just below and just above the steps
    of the law: the token drawn is one that the mask allows."""
    B, V = 64, 300
    g = torch.Generator().manual_seed(3)
    row = (2 * torch.randn((1, 1, V), generator=g)).to(DT[dtype])
    row[..., 1::2] = NEG
    zt = row.expand(B, 1, V).contiguous()
    zd = torch.zeros((B, 0, V), dtype=DT[dtype])
    steps = torch.softmax(row[0, 0].double(), -1).cumsum(-1)[::2].float()
    us = torch.cat([steps, torch.nextafter(steps, torch.zeros(())), torch.nextafter(steps, torch.ones(()))])
    us = us.clamp(0, 1 - 2.0 ** -24)
    us = torch.cat([us, us.new_zeros(-len(us) % B)])
    cand = torch.zeros((B, 1), dtype=torch.int64)
    for u in us.split(B):
        got = _verify(zt, zd, cand, torch.zeros((B, 0)), u.contiguous(), False)
        assert (got["bonus"] % 2 == 0).all() and got["accept_len"].tolist() == [0] * B


@pytest.mark.parametrize("dtype,u", [("f32", float.fromhex("0x1.d1970ep-1")), ("bf16", float.fromhex("0x1.515a64p-2"))])
def test_uniform_between_a_token_and_its_forbidden_neighbour(dtype, u):
    """The one uniform of each row's 2^24 whose target fp32 sums put behind an allowed
    token and before the step of the forbidden one next to it."""
    V = 300
    row = (2 * torch.randn((1, 1, V), generator=torch.Generator().manual_seed(0))).to(DT[dtype])
    row[..., 1::2] = NEG
    got = _verify(row, torch.zeros((1, 0, V), dtype=DT[dtype]), torch.zeros((1, 1), dtype=torch.int64),
                  torch.zeros((1, 0)), torch.tensor([u]), False)
    assert int(got["bonus"]) % 2 == 0 and int(got["flags"]) & api.FLAG_CDF_BOUNDARY
