"""Block tables and slot maps refuse buffers that share bytes, before a launch."""
import ctypes

import pytest

from block_diffusion_speculative_fusion_gb300 import api, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


B, PAGES, NUM, ROWS = 4, 8, 64, 16
BASE = 0x10000


def _call(L, name, ptrs):
    d = api.PagesDims(B, 16, PAGES, NUM)
    p = [ctypes.c_void_p(x) for x in ptrs]
    if name == "pages_resize":
        return L.dflash_pages_resize(ctypes.byref(d), *p, None)
    return L.dflash_slot_map(ctypes.byref(d), ROWS, *p, None)


# bytes of each argument, and which ones the call writes
RESIZE = [4 * B, 4 * B * PAGES, 4 * B, 4 * NUM, 4, 4 * B, 4, B]     # length, table, n_pages, free, n_free, outputs
SLOTS = [4 * B, 4 * B, 4 * B * PAGES, 4 * B + 4, 4 * ROWS, 4 * ROWS, 8 * ROWS]


@pytest.mark.parametrize("name,sizes,written", [("pages_resize", RESIZE, {1, 3, 5, 6, 7}),
                                                ("slot_map", SLOTS, {3, 4, 5, 6})])
def test_overlapping_buffers_are_refused(L, name, sizes, written):
    for i in written:
        for j in range(len(sizes)):
            if i == j:
                continue
            # the first and the last bytes of buffer j
            for at in (0, sizes[j] - 1, 1 - sizes[i]):
                ptrs = [BASE * (k + 1) for k in range(len(sizes))]
                ptrs[i] = ptrs[j] + at
                assert _call(L, name, ptrs) == api.ERR_INVALID_ARG, (i, j, at)
                assert "overlap" in api.last_error()
