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
