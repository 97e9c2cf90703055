"""The binding's cached workspaces, on CPU tensors in place of device ones."""
import pytest
import torch

from block_diffusion_speculative_fusion_gb300 import api


@pytest.fixture
def cache(monkeypatch):
    real = torch.zeros
    monkeypatch.setattr(api, "_WS", {})
    monkeypatch.setattr(api, "_WS_OUTGROWN", [])
    monkeypatch.setattr(api.torch, "zeros", lambda n, dtype=None, device=None: real(1, dtype=dtype).expand(n)
                        if n > 1 << 20 else real(n, dtype=dtype))
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


@pytest.mark.parametrize("step", [1, 256, 4096, 1 << 20])
def test_outgrown_workspaces_take_no_more_than_the_current_one(cache, step):
    # calls that grow by small steps
    dev = torch.device("cuda:0")
    first = 1 << 16
    for i in range(300):
        need = first + i * step
        ws = api.workspace(dev, need, slot=2)
        assert need <= ws.numel() <= max(first, 2 * need)
        kept = sum(w.numel() for _, w in api.cached_workspaces() if w is not ws)
        assert kept <= ws.numel()
    # a call that needs far more gets that
    assert api.workspace(dev, 1 << 31, slot=2).numel() == 1 << 31
