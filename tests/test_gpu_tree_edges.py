"""Tree attention where its work is cut and staged in the rarer ways: an odd number of row tiles,
more row pairs per head than go side by side, kept sets whose rings would be of odd depth.
Tolerances as in test_gpu_tree.py."""
import pytest
import torch

import tree_ref as ref
from test_gpu_tree import D, H16, H32, attn_inputs, check_attn, cuda, rmm  # noqa: F401 (a fixture)

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


BAD = [  # B, T, Hq, Hkv, lens, ldL: whole units and cut ones, of one row tile and of two
    (90, 1, 8, 2, [3 + i for i in range(90)], 96),
    (90, 20, 8, 2, [3 + i for i in range(90)], 120),
    (1, 16, 8, 2, [5000], 5016),
    (90, 33, 8, 2, [3 + i for i in range(90)], 128),
    (2, 64, 16, 2, [900, 61], 968),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,lens,ldL", BAD)
@pytest.mark.parametrize("where,value,r", [("query", "nan", 1.0), ("query row", "nan", 1.0), ("query row", "inf", 1.0),
                                           ("key", "nan", 1.0), ("key", "nan", 0.5), ("key", "inf", 0.5),
                                           ("node's key", "nan", 1.0), ("value", "nan", 0.5), ("value", "inf", 1.0)])
def test_attn_tree_nan_stays_nan(rmm, B, T, Hq, Hkv, lens, ldL, where, value, r):  # noqa: F811
    """NaN and infinite queries, keys and values reach exactly the outputs that the formula gives them
    (a query's its own row, a key's the rows that see it), however the work is cut."""
    Q, Kt, V, lens, parents = attn_inputs(B, T, Hq, Hkv, lens, ldL, "full", 40, junk=False)
    bad, G, t = float(value), Hq // Hkv, T // 2
    for b in range(0, B, 2):
        n = int(lens[b])
        if where == "query":
            Q[b, 1, t, 5] = bad
        elif where == "query row":
            Q[b, G, t] = bad
        elif where == "key":
            Kt[b, 1, :, n // 2] = bad
        elif where == "node's key":
            Kt[b, 0, :, n + t] = bad
        else:
            V[b, 1, n // 2, 7] = bad
    wo, wi, A, X = ref.attn_tree(Q, Kt, V, lens, parents, r)
    q, kt, v, ln, pr = cuda(Q, Kt, V, lens, parents)
    idx = torch.full((B, Hkv, rmm.rmm_k_for(D, r)), -1, dtype=torch.int32, device="cuda")
    O = rmm.rmm_attn_tree(q, kt, v, ln, r, parents=pr, idx_out=idx).double().cpu()
    if where not in ("query", "query row"):
        assert torch.equal(idx.cpu(), wi)
    assert bool(torch.isnan(wo).any()) or value == "inf"
    assert torch.equal(torch.isnan(O), torch.isnan(wo))
    assert torch.equal(torch.isinf(O), torch.isinf(wo))
    fine = torch.isfinite(wo)
    tol = H16 * wo.abs() + (H16 + 2e-4 + 2 * (idx.shape[-1] + 2) * H32 * X[..., None]) * A
    assert bool(((O - wo).abs() <= tol)[fine].all())


@pytest.mark.parametrize("B,T,Hq,Hkv,lens,ldL", BAD)
def test_attn_tree_rows_of_minus_infinity(rmm, B, T, Hq, Hkv, lens, ldL):  # noqa: F811
    """Nothing but -inf logits: 0, beside a head whose rows are as ever."""
    Q, Kt, V, lens, parents = attn_inputs(B, T, Hq, Hkv, lens, ldL, "full", 41, junk=False)
    Q = Q.abs() + 0.125
    Kt[:, 0] = -float("inf")
    O = rmm.rmm_attn_tree(*cuda(Q, Kt, V, lens), 1.0, parents=parents.cuda()).cpu()
    G = Hq // Hkv
    assert not bool(O[:, :G].any())
    wo, _, A, X = ref.attn_tree(Q[:, G:], Kt[:, 1:], V[:, 1:], lens, parents, 1.0)
    assert bool(((O[:, G:].double() - wo).abs() <= H16 * wo.abs() + (H16 + 2e-4 + 260 * H32 * X[..., None]) * A).all())


@pytest.mark.parametrize("B,T,Hq,Hkv,lens,ldL,r", [(3, 5, 8, 2, [700, 30, -1], 1024, 1.0), (3, 5, 8, 2, [700, 30, -1], 1024, 0.5),
                                                   (2, 64, 16, 2, [900, 61], 968, 1.0), (2, 64, 16, 2, [900, 61], 968, 0.5),
                                                   (1, 40, 8, 1, [2000], 2040, 0.75)])
def test_attn_tree_watchdog(rmm, B, T, Hq, Hkv, lens, ldL, r):  # noqa: F811
    """A wait that runs out (50 ms) is reported, the call ends, and the next one on the same workspace is as ever."""
    Q, Kt, V, lens, parents = attn_inputs(B, T, Hq, Hkv, lens, ldL, "padded", 43, junk=False)
    args, pr = cuda(Q, Kt, V, lens), parents.cuda()
    want = rmm.rmm_attn_tree(*args, r, parents=pr)
    ws = rmm.new_workspace(rmm.rmm_attn_tree_workspace_bytes(B, Hq, Hkv, T, ldL))
    for _ in range(2):
        rmm.rmm_attn_tree(*args, r, parents=pr, workspace=ws, opts=rmm.options(debug_timeout_test=True))
        assert rmm.rmm_get_status(ws) == rmm.RMM_ERR_TIMEOUT
        got = rmm.rmm_attn_tree(*args, r, parents=pr, workspace=ws)
        assert rmm.rmm_get_status(ws) == rmm.RMM_OK
        assert torch.equal(got, want)
