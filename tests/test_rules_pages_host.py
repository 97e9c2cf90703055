"""Host checks of the logit rules, block tables and slot maps: every refusal
happens before a launch, and the oracle of each agrees with hand-worked cases."""
import ctypes

import numpy as np
import pytest

import oracle as O
from block_diffusion_speculative_fusion_gb300 import api, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def _p(x=0x10000):
    return ctypes.c_void_p(x)


def _rules(L, dims, logits=_p(0x1000000), hist=None, hist_len=None, tok=None, val=None, out=_p(0x9000000)):
    return L.dflash_logits_rules(ctypes.byref(dims) if dims else None, logits, None, None, hist, hist_len, None, None,
                                 None, None, tok, val, None, None, out, None)


@pytest.mark.parametrize("dims,code,word", [
    (api.RulesDims(0, 4, 100, api.BF16, 0, 0), api.ERR_INVALID_ARG, "bad dims"),
    (api.RulesDims(2, 4, 0, api.BF16, 0, 0), api.ERR_INVALID_ARG, "bad dims"),
    (api.RulesDims(2, 4, 100, 7, 0, 0), api.ERR_INVALID_ARG, "dtype"),
    (api.RulesDims(2, 257, 100, api.BF16, 0, 0), api.ERR_UNSUPPORTED, "n_rows"),
    (api.RulesDims(2, 4, 100, api.BF16, 1 << 18, 0), api.ERR_UNSUPPORTED, "hist_max"),
    (api.RulesDims(2, 4, 100, api.BF16, 0, 2048), api.ERR_UNSUPPORTED, "n_bias"),
    (api.RulesDims(65536, 1, 100, api.BF16, 0, 0), api.ERR_UNSUPPORTED, "B="),
    (api.RulesDims(2, 4, 100, api.BF16, 5, 0), api.ERR_INVALID_ARG, "NULL"),
    (api.RulesDims(2, 4, 100, api.BF16, 0, 5), api.ERR_INVALID_ARG, "NULL"),
])
def test_rules_refusals(L, dims, code, word):
    assert _rules(L, dims) == code and word in api.last_error()


def test_rules_refuses_missing_and_overlapping_buffers(L):
    d = api.RulesDims(2, 4, 100, api.BF16, 0, 0)
    assert _rules(L, None) == api.ERR_INVALID_ARG
    assert _rules(L, d, logits=None) == api.ERR_INVALID_ARG
    assert _rules(L, d, out=None) == api.ERR_INVALID_ARG
    for off in (2, 1598, -1598):               # 1600 bytes of logits
        assert _rules(L, d, out=_p(0x1000000 + off)) == api.ERR_INVALID_ARG and "overlap" in api.last_error()
    assert _rules(L, d, out=_p(0x9000001)) == api.ERR_INVALID_ARG and "aligned" in api.last_error()


@pytest.mark.parametrize("dims,code,word", [
    (api.PagesDims(0, 16, 8, 64), api.ERR_INVALID_ARG, "bad dims"),
    (api.PagesDims(2, 0, 8, 64), api.ERR_INVALID_ARG, "bad dims"),
    (api.PagesDims(4097, 16, 8, 64), api.ERR_UNSUPPORTED, "4096"),
    (api.PagesDims(4096, 16, 1 << 20, 64), api.ERR_UNSUPPORTED, "max_pages"),
])
def test_pages_refusals(L, dims, code, word):
    p = [_p(0x10000 * (i + 1)) for i in range(8)]
    assert L.dflash_pages_resize(ctypes.byref(dims), *p, None) == code and word in api.last_error()
    assert L.dflash_slot_map(ctypes.byref(dims), 16, *p[:7], None) == code and word in api.last_error()


def test_pages_refuses_aliases_and_missing_pointers(L):
    d = api.PagesDims(2, 16, 8, 64)
    p = [_p(0x10000 * (i + 1)) for i in range(8)]   # length, table, n_pages, free, n_free, n_pages_out, n_free_out, short
    q = list(p)
    q[5] = p[2]
    assert L.dflash_pages_resize(ctypes.byref(d), *q, None) == api.ERR_INVALID_ARG and "alias" in api.last_error()
    q = list(p)
    q[6] = p[4]
    assert L.dflash_pages_resize(ctypes.byref(d), *q, None) == api.ERR_INVALID_ARG and "alias" in api.last_error()
    for i in range(7):
        q = list(p)
        q[i] = None
        assert L.dflash_pages_resize(ctypes.byref(d), *q, None) == api.ERR_INVALID_ARG and "NULL" in api.last_error()
        q = list(p[:7])
        q[i] = None
        assert L.dflash_slot_map(ctypes.byref(d), 16, *q, None) == api.ERR_INVALID_ARG and "NULL" in api.last_error()
    for rows in (0, -1, (1 << 30) + 1):
        assert L.dflash_slot_map(ctypes.byref(d), rows, *p[:7], None) == api.ERR_INVALID_ARG
        assert "rows_max" in api.last_error()


def test_binding_refuses_half_given_lists(L):
    import torch
    with pytest.raises(ValueError):
        api.logits_rules(torch.zeros(1, 2, 8))              # not a CUDA tensor


# ---- the oracle itself, by hand -------------------------------------------------
def test_oracle_rules_by_hand():
    z = np.array([[[2.0, -2.0, 4.0, 1.0], [2.0, -2.0, 4.0, 1.0]]])
    kw = dict(cand=np.array([[9, 3]]), hist=np.array([[0, 1, 1]]), hist_len=[3], prompt_len=[1], repetition=[2.0],
              presence=[0.5], frequency=[0.25], bias_tok=np.array([[2, 2]]), bias_val=np.array([[1.0, 10.0]]),
              mask=np.array([[[0b1111], [0b0111]]]))
    y, _ = O.logits_rules(z, **kw)
    # token 0 in the prompt, token 1 twice in the output, token 2 biased, token 3 from row 1 on (then masked)
    assert y[0, 0].tolist() == [1.0, -4.0 - 0.5 - 0.5, 14.0, 1.0]
    assert y[0, 1].tolist() == [1.0, -5.0, 14.0, -np.inf]
    kw["mask"] = None
    y, _ = O.logits_rules(z, **kw)
    assert y[0, 1, 3] == 0.5 - 0.25 - 0.5


def test_oracle_resize_by_hand():
    # sequence 0 gives page 7 back, sequence 1 takes it first (the list's end), then 9
    t, n, f, k, s = O.pages_resize([16, 33, 16], [[5, 7, -1], [6, -1, -1], [-1, -1, -1]], [2, 1, 0],
                                   [8, 9, -1, -1, -1, -1], 2, 16)
    assert t[1].tolist() == [6, 7, 9] and n.tolist() == [1, 3, 1] and t[2][0] == 8 and k == 0
    assert f.tolist()[:3] == [8, 9, 7] and s.tolist() == [0, 0, 0]


def test_oracle_slot_map_by_hand():
    cu, seq, pos, slot = O.slot_map([15, 0], [2, 1], [[3, 1], [2, -1]], 16, 4, 5)
    assert cu.tolist() == [0, 2, 3] and seq.tolist() == [0, 0, 1, -1, -1]
    assert pos.tolist() == [15, 16, 0, -1, -1] and slot.tolist() == [63, 16, 32, -1, -1]
