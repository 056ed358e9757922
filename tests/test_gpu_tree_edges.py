"""Tree attention where its work is cut and staged in the rarer ways: an odd number of row tiles,
more row pairs per head than go side by side, kept sets whose rings would be of odd depth.
Tolerances as in test_gpu_tree.py."""
import pytest
import torch

from test_gpu_tree import D, attn_inputs, check_attn, cuda, rmm  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

CUTS = [  # B, T, Hq, Hkv, lens, ldL, r, tree
    (1, 40, 8, 1, [2000], 2040, 1.0, "full"),               # 320 rows: three tiles, the last alone
    (3, 40, 8, 1, [2000, 100, 900], 2040, 1.0, "padded"),
    (1, 40, 8, 1, [2000], 2040, 0.875, "full"),
    (2, 36, 8, 1, [1500, 700], 1536, 0.6, "padded"),        # 288 rows
    (1, 64, 12, 1, [700], 768, 1.0, "full"),                # 768 rows: three pairs side by side
    (1, 64, 10, 1, [700], 768, 0.5, "full"),                # 640 rows: three pairs, the last of one tile
    (1, 64, 64, 1, [300], 368, 1.0, "full"),                # 4096 rows: sixteen pairs in a row
    (1, 64, 33, 1, [300], 368, 0.5, "padded"),              # 2112 rows: nine pairs, the last of one tile
    (2, 64, 66, 2, [300, 700], 768, 1.0, "full"),           # the same, two heads of two sequences
    (1, 16, 8, 2, [5000], 5016, 0.75, "full"),              # one tile, 96 kept dims, many blocks
    (2, 25, 8, 2, [3000, 4100], 4128, 0.6, "padded"),       # 80 kept
    (1, 16, 8, 1, [9000], 9016, 0.875, "full"),             # 112 kept
]


@pytest.mark.parametrize("B,T,Hq,Hkv,lens,ldL,r,tree", CUTS)
def test_attn_tree_cuts(rmm, B, T, Hq, Hkv, lens, ldL, r, tree):  # noqa: F811
    check_attn(rmm, *attn_inputs(B, T, Hq, Hkv, lens, ldL, tree, 300 + T), r)


@pytest.mark.parametrize("B,T,Hq,Hkv,lens,ldL,r", [(2, 40, 8, 1, [6000, 2500], 6040, 1.0),
                                                   (4, 16, 16, 4, [4000, 100, 2222, 3000], 4024, 0.75),
                                                   (1, 64, 66, 2, [900], 968, 1.0)])
def test_attn_tree_repeats_its_bits(rmm, B, T, Hq, Hkv, lens, ldL, r):  # noqa: F811
    """Two groups at the same keys, whatever order their copies land in: 200 calls, one result."""
    Q, Kt, V, lens, parents = attn_inputs(B, T, Hq, Hkv, lens, ldL, "padded", 31, junk=False)
    q, kt, v, ln, pr = cuda(Q, Kt, V, lens, parents)
    ws = rmm.new_workspace(rmm.rmm_attn_tree_workspace_bytes(B, Hq, Hkv, T, ldL))
    want = rmm.rmm_attn_tree(q, kt, v, ln, r, parents=pr, workspace=ws)
    O = torch.zeros(B, Hq, T, D, dtype=torch.bfloat16, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        rmm.rmm_attn_tree(q, kt, v, ln, r, parents=pr, O=O, workspace=ws)
        wrong += (O != want).sum()
    assert int(wrong) == 0
    assert rmm.rmm_get_status(ws) == rmm.RMM_OK
