"""Refusals at the edges of the calls for drafted tokens, on the host (nothing is launched)."""
import ctypes

import pytest

import entropy_bounded_denoising_gb300 as dg
from test_serving_validation import _kv


@pytest.mark.parametrize("name,words", [("kv_len", 4), ("page_table", 4 * 3), ("cu", 5), ("path", 9), ("na", 4)])
def test_keep_new_lengths_over_an_input(name, words):
    """new_len over anything that other blocks still read is refused, from its first word to its last; beside it the next
    check (an odd address) answers."""
    lib = dg.load()
    at = dict(kv_len=0x10000, page_table=0x20000, cu=0x30000, path=0x40000, na=0x50000)

    def call(new, cu=at["cu"] + 2):
        kv = _kv(kv_len=at["kv_len"], page_table=at["page_table"], max_pages=3)
        return lib.dg_kv_keep(ctypes.byref(kv), 1, 0, cu, 4, 9, 1, 128, at["path"], at["na"], new, None)

    here = at[name]
    cu = here if name == "cu" else at["cu"] + 2
    for new in (here, here + 4, here + 4 * (words - 1), here - 4, here - 12):
        assert call(new, cu) == dg.DG_ERR_INVALID_ARG, new
    if name != "cu":
        for new in (here + 4 * words, here - 16):
            assert call(new) == dg.DG_ERR_ALIGNMENT, new
