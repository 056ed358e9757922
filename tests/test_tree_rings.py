"""The tree attention's key and value rings, on the CPU: the depths that the library takes and
what the kernel's waits need of them.

A full barrier counts rounds (tile copies landed in its slot) and a wait knows its round by
the parity alone: waiting for round r passes when the barrier is at round r + 1, and also at
round r - 1, when the copy of the round before has not landed yet.  So whoever waits for a
block must know that the block before it in the same slot has landed: because it waited for
it too, or because its P.V is done.  With one row tile two groups take alternate blocks."""
import ctypes

import pytest


class Rings(ctypes.Structure):
    _fields_ = [("nk", ctypes.c_int), ("nv", ctypes.c_int), ("smem", ctypes.c_int)]


@pytest.fixture(scope="module")
def rings():
    from input_adaptive_reduced_rmm_b200 import build as b

    b.build()
    from input_adaptive_reduced_rmm_b200 import rmm

    fn = ctypes.CDLL(rmm.LIB_PATH)["_ZN3rmm15attn_tree_ringsEii"]  # rmm::attn_tree_rings(int, int)
    fn.restype, fn.argtypes = Rings, [ctypes.c_int, ctypes.c_int]
    return lambda tiles, kp: (lambda r: (r.nk, r.nv, r.smem))(fn(tiles, kp))


TILES = [1, 2, 3, 4, 5, 16, 17, 1024, 2048]
KEPT = list(range(16, 129, 16))


def passes_early(depth, groups, ahead=1, blocks=40):
    """Whether a wait for a block of a piece can pass before the block has landed, with copies that
    land in any order: group g of `groups` takes every groups-th block; its waits for full barriers
    come in order, and it knows of the other group's blocks nothing.  The blocks before the last
    `ahead` of its own have been used."""
    for p in range(depth, blocks):  # the first round of a slot has none before it
        before = p - depth  # the block of the round before in this slot
        mine = before % groups == p % groups
        # a group's own earlier block that is not among the last `ahead` has landed
        if not (mine and (p - before) // groups >= ahead):
            return True
    return False


def test_the_model_of_a_ring():
    assert passes_early(5, 2) and passes_early(7, 2) and passes_early(3, 2)
    assert not any(passes_early(n, 2) for n in (2, 4, 6, 8))
    assert not any(passes_early(n, 1) for n in range(2, 9))
    assert passes_early(2, 2, ahead=2) and not passes_early(4, 2, ahead=2)


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("kp", KEPT)
def test_no_wait_passes_before_its_block_has_landed(rings, tiles, kp):
    nk, nv, smem = rings(tiles, kp)
    assert 2 <= nk <= 8 and 2 <= nv <= 8 and smem <= 227 * 1024
    for groups in {1 if tiles > 1 else 2, 2 if tiles % 2 else 1}:  # two row tiles; the last one alone
        # the MMA warp of a group waits for each of its blocks in order
        assert not passes_early(nk, groups) and not passes_early(nv, groups), (nk, nv)
        # its softmax warps wait for values only near the end of a piece: S of a block is there once
        # the P.V of the block two before it in the group is done
        assert not passes_early(nv, groups, ahead=2), nv
