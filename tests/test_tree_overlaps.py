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


BYTES = B * 2 * 128 * 64 * 2  # of a cache of keep()'s sizes


def caches(*k, v):
    return dict(n=len(k), Kts=(ctypes.c_void_p * len(k))(*k), Vs=(ctypes.c_void_p * len(k))(*v))


@pytest.mark.parametrize("kt,v", [
    ((1 << 24, (1 << 24) + BYTES - 16), (1 << 26, 1 << 27)),           # two layers' keys
    (((1 << 24) + 4096, 1 << 24), (1 << 26, 1 << 27)),
    ((1 << 24, 1 << 25), ((1 << 26) + BYTES // 2, 1 << 26)),           # two layers' values
    ((1 << 24, 1 << 25), (1 << 26, 1 << 24)),                          # one layer's keys as another's values
    ((1 << 24,), ((1 << 24) + 16,)),                                   # one layer's keys and values
    ((1 << 24, 1 << 25, (1 << 24) + BYTES), (1 << 26, 1 << 27, (1 << 27) - 16)),
])
def test_cache_keep_of_caches_that_overlap(rmm, kt, v):  # noqa: F811
    """Each cache is moved by itself, at the same time: rows of two of them would move twice."""
    assert rmm.lib().rmm_cache_keep(*keep(**caches(*kt, v=v))) == INVALID


def test_cache_keep_of_caches_side_by_side_passes_the_checks(rmm):  # noqa: F811
    import torch

    if torch.cuda.is_available():
        pytest.skip("the call would be made")
    at = [(1 << 24) + i * BYTES for i in (3, 0, 5, 1, 4, 2)]
    a = keep(**caches(*at[:3], v=at[3:]))
    a[7], a[8], a[9] = (ctypes.c_void_p(p) for p in (LENS, PATH, KEPT))
    assert rmm.lib().rmm_cache_keep(*a) == rmm.RMM_ERR_CUDA  # no device here
