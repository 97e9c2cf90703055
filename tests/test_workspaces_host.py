"""The binding's cached workspaces, on CPU tensors in place of device ones."""
import pytest
import torch

from block_diffusion_speculative_fusion_gb300 import api


@pytest.fixture
def cache(monkeypatch):
    real = torch.zeros
    monkeypatch.setattr(api, "_WS", {})
    monkeypatch.setattr(api, "_WS_OUTGROWN", [])
    monkeypatch.setattr(api.torch, "zeros", lambda n, dtype=None, device=None: real(n, dtype=dtype))
    return api


def _fail(ws, code):
    ws[api.WS_ERROR_WORD_OFFSET:api.WS_COUNTER_BYTES].view(torch.int32)[0] = code


def test_error_word_of_an_outgrown_workspace_is_reported(cache):
    dev = torch.device("cuda:0")
    small = api.workspace(dev, 1 << 16, slot=4)
    large = api.workspace(dev, 1 << 20, slot=4)
    other = api.workspace(dev, 1 << 16, slot=2)
    assert large is not small and api.workspace(dev, 1 << 19, slot=4) is large
    assert api.error_words() == {(0, 4): 0, (0, 2): 0}
    _fail(small, 23)                            # a graph captured with it replays and runs out of a wait
    assert api.error_words() == {(0, 4): 23, (0, 2): 0}
    _fail(other, 5)
    assert api.error_words() == {(0, 4): 23, (0, 2): 5}
    assert any(w is small for _, w in api.cached_workspaces())
    api.reset_workspaces()
    assert api.error_words() == {}
