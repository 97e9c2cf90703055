"""The oracle's sampled accept rule on rows that a grammar mask has been through."""
import numpy as np

import oracle as O


def test_rows_that_allow_no_token():
    # after every candidate was accepted, and after a rejection: no mass to draw from
    z = np.zeros((2, 2, 4))
    z[0, 1] = z[1, 0] = -np.inf
    ref = O.verify_sample(z, np.zeros((2, 1, 4)), [[0, 1], [0, 1]], [1, 1], np.full((2, 1), 0.5), [0.3, 0.3])
    assert ref["accept_len"].tolist() == [1, 0] and all(f & O.FLAG_DEGENERATE for f in ref["flags"])
    for d in ref["debug"]:
        assert d["Z"] == 0.0 and not d["final_dist"].any()
    assert ref["debug"][1]["p_x"].tolist() == [0.0] and not np.isnan(O.softmax(z)).any()


def test_forbidden_candidate_is_rejected_where_q_is_zero():
    z = np.zeros((3, 2, 4))
    zd = np.zeros((3, 1, 4))
    z[:2, 0, 1] = -np.inf
    zd[1:, 0, 1] = -np.inf                     # q(x) = 0 for the last two, allowed in the last alone
    u = np.zeros((3, 1))
    ref = O.verify_sample(z, zd, np.ones((3, 2), dtype=np.int64), [1] * 3, u, [0.3] * 3)
    assert ref["accept_len"].tolist() == [0, 0, 1]
    assert [bool(f & O.FLAG_INVALID) for f in ref["flags"]] == [False, True, True]
    assert 1 not in ref["bonus"][:2]
