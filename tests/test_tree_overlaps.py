"""Outputs of the draft-tree calls that lie over an input another part of the call still reads are
refused on the host (pointers that are never dereferenced)."""
import ctypes

import pytest

from test_tree_refusals import FAKE, INVALID, keep, rmm  # noqa: F401 (a fixture)

B, T = 2, 4
LENS, PATH, KEPT, OUT = ((1 << 20) + (i << 12) for i in range(4))


@pytest.mark.parametrize("out", [KEPT, KEPT + 4 * (B - 1), KEPT - 4 * (B - 1), PATH, PATH + 4 * (B * T - 1),
                                 PATH - 4 * (B - 1), LENS + 4])
def test_cache_keep_new_lengths_over_an_input(rmm, out):  # noqa: F811
    """The lengths leave with one part of the call while others read the counts and paths."""
    a = keep(lens=ctypes.c_void_p(LENS), path=ctypes.c_void_p(PATH), kept=ctypes.c_void_p(KEPT), B=B, T=T,
             out=ctypes.c_void_p(out))
    assert rmm.lib().rmm_cache_keep(*a) == INVALID
