"""Logit rules in place give the bits that a second buffer gets."""
import numpy as np
import pytest
import torch

from block_diffusion_speculative_fusion_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_fusion_gb300 import build
    build.build()
    api.lib()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [4096, 20000, 20011])
@pytest.mark.parametrize("masked", [False, True])
def test_biases_in_place(V, dtype, masked):
    # entries all over the chunks, some of value 0 (and -0), some tokens named twice
    B, R, nb = 3, 9, 1500
    g = np.random.default_rng(V)
    z = torch.from_numpy(g.normal(0, 3, (B, R, V)).astype(np.float32)).to(DT[dtype]).to(DEV)
    tok = torch.from_numpy(g.integers(-1, V, (B, nb))).to(DEV)
    val = torch.from_numpy(g.choice([0.0, -0.0, 1.5, -4.0], (B, nb)).astype(np.float32)).to(DEV)
    kw = dict(bias_tok=tok, bias_val=val)
    if masked:
        kw["mask"] = torch.from_numpy(g.integers(-2 ** 31, 2 ** 31, (B, R, (V + 31) // 32)).astype(np.int32)).to(DEV)
    ref = api.logits_rules(z, out=torch.empty_like(z), **kw)
    want = z.float().clone()
    for b in range(B):                          # the last entry of a token counts
        last = {int(t): float(v) for t, v in zip(tok[b].tolist(), val[b].tolist()) if t >= 0}
        want[b][:, list(last)] += torch.tensor(list(last.values()), device=DEV)
    want = want.to(z.dtype)
    if masked:
        t = torch.arange(V, device=DEV)
        want[(kw["mask"].long()[:, :, t // 32] >> (t % 32)) & 1 == 0] = float("-inf")
    assert torch.equal(ref, want)
    for _ in range(5):
        y = z.clone()
        api.logits_rules(y, out=y, **kw)
        assert torch.equal(y, ref)
