"""Draft-tree decoding on the GPU against the formulas in 64 bits (tree_ref.py).

Tolerances, with h = eps / 2 a type's half step (bf16 2^-8, fp32 2^-24):
  q/k rows   one rounding to bf16 of a value off by less than 32 h32 of its rotated pair's
             length: the norm (16 sums, the mean, eps, rsqrtf's 2 ulp, two products) 24 h32 at
             most, sine and cosine and the angle's rounding 14 h32 of which the two products
             of a pair see a half each, their sum 2
  attention  P is rounded to bf16 before P.V and O after it: 2^-8 (|O| + sum p |v|); the
             exponentials' relative error (6e-5 for the polynomial, 2^-22 else) counts twice
             (numerator and sum), 2e-4 with the fp32 sums over up to 16384 keys (16 sums of
             2^-24 each a tile); a logit of k products is off by (k + 2) h32 sum |q k|, twice
  softmax    (x - M) c: three roundings of |z|, exp2f 2 ulp, a sum of at most 81 steps, the
             same |z| weighted by p in the sum, two more products
Whole numbers (kept sets, tokens, paths) and moved data are equal.
"""
import math

import pytest
import torch

import tree_ref as ref

pytestmark = pytest.mark.gpu
D = 128
H16, H32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def rmm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from input_adaptive_reduced_rmm_b200 import rmm as _rmm

    _rmm.lib()
    return _rmm


def normal(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def within(got, want, tol, what):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, the worst by {float((err - tol).max()):.3e}"


# ---------------------------------------------------------------- q/k norms and rotation

QKV = [  # B, T, Hq, Hkv, lens, ldL, rot, interleaved, norm, tree
    (1, 1, 4, 1, [0], 8, 128, False, True, False),
    (3, 1, 8, 2, [5, -1, 17], 32, 128, True, True, False),
    (2, 2, 9, 3, [0, 30], 32, 64, False, True, True),       # the second fills its cache to the last slot
    (3, 7, 16, 16, [3, 26, 11], 32, 128, False, True, True),  # the second has no room: skipped
    (2, 25, 8, 4, [1000, 7], 1048, 32, True, False, True),
    (2, 64, 12, 9, [13, 64], 128, 16, False, True, True),
    (1, 65, 4, 2, [62], 128, 128, False, True, False),      # two token tiles, odd start
    (2, 200, 5, 1, [1, 40], 240, 96, True, True, False),
    (75, 1, 40, 9, list(range(-1, 74)), 80, 128, False, True, False),  # single tokens, more than the GPU takes at once
    (150, 1, 8, 8, list(range(150)), 152, 64, True, False, True),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,lens,ldL,rot,inter,norm,tree", QKV)
def test_qkv_rope(rmm, B, T, Hq, Hkv, lens, ldL, rot, inter, norm, tree):
    Yq, Yk, Yv = (normal(i, B * T, h * D, std=3.0) for i, h in ((1, Hq), (2, Hkv), (3, Hkv)))
    Q, Kt, V = normal(4, B, Hq, T, D), normal(5, B, Hkv, D, ldL), normal(6, B, Hkv, ldL, D)
    qn, kn = (normal(7, D), normal(8, D)) if norm else (None, None)
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float32) / rot)
    lens = torch.tensor(lens, dtype=torch.int32)
    parents = ref.random_trees(B, T, 9, roots=True) if tree else None
    wq, wk, wv, mq, mk = ref.qkv_rope(Yq, Yk, Yv, Q, Kt, V, lens, parents, qn, kn, 1e-6, freq, inter)
    yq, yk, yv, q, kt, v, ln, pr, a, b, f = cuda(Yq, Yk, Yv, Q, Kt, V, lens, parents, qn, kn, freq)
    out = rmm.rmm_qkv_rope(yq, yk, yv, q, kt, v, lens=ln, parents=pr, q_norm=a, k_norm=b, inv_freq=f, interleaved=inter)
    assert out is q
    # what is not written keeps its bits: there the reference holds the old value and m = 0
    within(q, wq, torch.where(mq > 0, H16 * wq.abs() + 32 * H32 * mq, 0.0), "Q")
    within(kt, wk, torch.where(mk > 0, H16 * wk.abs() + 32 * H32 * mk, 0.0), "Kt")
    within(v, wv, torch.zeros(()), "V")


def test_qkv_rope_far_positions(rmm):
    """Angles of positions near 130000 in full: an fp32 angle would be off by 0.004."""
    T, ldL = 3, 131072
    Yq, Yk, Yv = (normal(i, T, D) for i in (1, 2, 3))
    freq = 500000.0 ** (-torch.arange(0, D, 2, dtype=torch.float32) / D)
    Q, lens = torch.zeros(1, 1, T, D, dtype=torch.bfloat16), torch.tensor([ldL - 4], dtype=torch.int32)
    kt = torch.zeros(1, 1, D, ldL, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(1, 1, ldL, D, dtype=torch.bfloat16, device="cuda")
    wq, wk, _, mq, mk = ref.qkv_rope(Yq, Yk, Yv, Q, kt.cpu(), v.cpu(), lens, None, None, None, 0.0, freq, False)
    q = rmm.rmm_qkv_rope(*cuda(Yq, Yk, Yv, Q), kt, v, lens=lens.cuda(), inv_freq=freq.cuda())
    within(q, wq, H16 * wq.abs() + 32 * H32 * mq, "Q")
    within(kt, wk, H16 * wk.abs() + 32 * H32 * mk, "Kt")


def test_qkv_rope_without_norm_or_rotation_is_the_plain_layout(rmm):
    T, Hq, Hkv, ldL, L0 = 70, 8, 2, 160, 37
    ys = cuda(*(normal(i, T, h * D) for i, h in ((1, Hq), (2, Hkv), (3, Hkv))))
    outs = []
    for batched in (False, True):
        Q = torch.zeros(1, Hq, T, D, dtype=torch.bfloat16, device="cuda")
        Kt = torch.zeros(1, Hkv, D, ldL, dtype=torch.bfloat16, device="cuda")
        V = torch.zeros(1, Hkv, ldL, D, dtype=torch.bfloat16, device="cuda")
        if batched:
            rmm.rmm_qkv_rope(*ys, Q, Kt, V, L0=L0)
        else:
            rmm.rmm_qkv_heads(*ys, Q[0], Kt[0], V[0], L0)
        outs.append((Q, Kt, V))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_qkv_rope_one_norm_alone(rmm):
    B, T, Hq, Hkv, ldL = 1, 5, 2, 2, 16
    Y = [normal(i, B * T, 2 * D) for i in (1, 2, 3)]
    Q, Kt, V = normal(4, B, Hq, T, D), normal(5, B, Hkv, D, ldL), normal(6, B, Hkv, ldL, D)
    kn, lens = normal(8, D), torch.tensor([2], dtype=torch.int32)
    wq, wk, wv, mq, mk = ref.qkv_rope(*Y, Q, Kt, V, lens, None, None, kn, 1e-5, None, False)
    q, kt, v = cuda(Q, Kt, V)
    rmm.rmm_qkv_rope(*cuda(*Y), q, kt, v, lens=lens.cuda(), k_norm=kn.cuda(), eps=1e-5)
    within(q, wq, torch.zeros(()), "Q")
    within(kt, wk, torch.where(mk > 0, H16 * wk.abs() + 32 * H32 * mk, 0.0), "Kt")


# ---------------------------------------------------------------- tree attention

def attn_inputs(B, T, Hq, Hkv, lens, ldL, tree, seed, junk=True):
    Q = (normal(seed, B, Hq, T, D, dtype=torch.float32) * torch.exp(0.5 * normal(seed + 1, D, dtype=torch.float32))).bfloat16()
    Kt, V = normal(seed + 2, B, Hkv, D, ldL), normal(seed + 3, B, Hkv, ldL, D)
    lens = torch.tensor(lens, dtype=torch.int32)
    if junk:  # what no node may see: NaN and infinities past every sequence's slots
        for b in range(B):
            n = max(0, int(lens[b]) + T) if 0 <= int(lens[b]) <= ldL - T else 0
            Kt[b, :, :, n:], V[b, :, n:] = float("nan"), float("inf")
    parents = ref.random_trees(B, T, seed, padded=tree != "full", roots=tree == "roots") if tree else None
    return Q, Kt, V, lens, parents


def check_attn(rmm, Q, Kt, V, lens, parents, r, scale=None):
    B, Hq, T, _ = Q.shape
    Hkv, ldL = Kt.shape[1], Kt.shape[3]
    k = rmm.rmm_k_for(D, r)
    wo, wi, A, X = ref.attn_tree(Q, Kt, V, lens, parents, r, scale)
    idx = torch.full((B, Hkv, k), -1, dtype=torch.int32, device="cuda")
    O = torch.full((B, Hq, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = rmm.new_workspace(rmm.rmm_attn_tree_workspace_bytes(B, Hq, Hkv, T, ldL))
    q, kt, v, ln, pr = cuda(Q, Kt, V, lens, parents)
    rmm.rmm_attn_tree(q, kt, v, ln, r, parents=pr, scale=scale, O=O, idx_out=idx, workspace=ws)
    full = bool((lens > ldL - T).any())
    assert rmm.rmm_get_status(ws) == (rmm.RMM_ERR_INVALID_ARG if full else rmm.RMM_OK)
    assert torch.equal(idx.cpu(), wi), "kept sets"
    tol = H16 * wo.abs() + (H16 + 2e-4 + 2 * (k + 2) * H32 * X[..., None]) * A
    within(O, wo, tol, "O")
    return O


ATTN = [  # B, T, Hq, Hkv, lens, ldL, r, tree
    (1, 1, 4, 1, [0], 8, 1.0, None),                       # a first token: it sees itself alone
    (1, 1, 1, 1, [1], 16, 0.1, None),
    (4, 1, 8, 2, [0, 127, 128, 300], 312, 0.5, None),      # block borders, ragged
    (3, 1, 32, 8, [-1, 700, 5], 704, 1.0, None),           # an empty slot
    (2, 2, 10, 2, [126, 127], 136, 0.3, "full"),           # the tree's own slots cross a block border
    (2, 5, 16, 2, [250, 1000], 1008, 1.0, "padded"),
    (3, 25, 8, 2, [3, 1015, 600], 1040, 0.5, "padded"),
    (3, 25, 8, 2, [3, 1017, 600], 1040, 0.5, "padded"),    # the second has no room for its tree
    (2, 32, 16, 4, [0, 0], 40, 0.75, "roots"),             # nothing cached
    (2, 32, 20, 4, [511, 90], 552, 1.0, "roots"),          # 160 rows: more than one row tile
    (2, 33, 8, 2, [400, 222], 440, 0.5, None),             # chains; 132 rows
    (1, 63, 8, 1, [2000], 2064, 0.25, "padded"),           # 504 rows
    (2, 64, 64, 8, [900, 61], 968, 1.0, "full"),           # 512 rows
    (2, 64, 12, 4, [1, 130], 200, 0.9, "padded"),          # 192 rows
    (1, 48, 8, 1, [900], 952, 0.5, "full"),                # 384 rows: three row tiles
    (1, 4, 32, 1, [333], 344, 1.0, "full"),                # one KV head for 32 query heads
    (40, 1, 8, 2, list(range(0, 160, 4)), 168, 1.0, None),  # many short sequences
    (1, 16, 32, 8, [5000], 5016, 0.5, "full"),             # one long sequence over the whole GPU
    (40, 3, 8, 4, list(range(10, 410, 10)), 416, 0.4, "padded"),  # more heads of keys than the GPU has SMs
    (2, 25, 10, 1, [77, 900], 960, 0.6, "padded"),         # 250 rows: two tiles, the dims of one unit
]


@pytest.mark.parametrize("B,T,Hq,Hkv,lens,ldL,r,tree", ATTN)
def test_attn_tree(rmm, B, T, Hq, Hkv, lens, ldL, r, tree):
    check_attn(rmm, *attn_inputs(B, T, Hq, Hkv, lens, ldL, tree, 100 + T), r)


def test_attn_tree_every_node_absent(rmm):
    Q, Kt, V, lens, parents = attn_inputs(2, 9, 8, 2, [50, 20], 64, "full", 3)
    parents[0] = -2
    parents[1, 0] = 5  # the root itself is no root: everything below it is absent
    O = check_attn(rmm, Q, Kt, V, lens, parents, 0.5)
    assert not bool(O[0].any())


def test_attn_tree_ties_and_large_logits(rmm):
    """Equal magnitudes (ties to the lower dim), and logits far apart (sharp softmax; the
    reference maximum moves by more than the rescale threshold)."""
    Q, Kt, V, lens, parents = attn_inputs(1, 6, 4, 1, [777], 800, "full", 5, junk=False)
    Q = torch.where(Q > 0, 1.0, -1.0).bfloat16()
    check_attn(rmm, Q, Kt, V, lens, parents, 0.5)
    Kt = (Kt.float() * torch.linspace(0.1, 30.0, 800)).bfloat16()
    check_attn(rmm, Q, Kt, V, lens, parents, 0.5, scale=1.0)


def test_attn_tree_matches_the_chunk_attention(rmm):
    """A chain over one length is a causal chunk: the same kept sets as rmm_attn_qk, and outputs
    within both kernels' roundings."""
    B, T, Hq, Hkv, L = 2, 24, 8, 2, 530
    Q, Kt, V, _, _ = attn_inputs(B, T, Hq, Hkv, [L - T] * B, 536, None, 11, junk=False)
    q, kt, v = cuda(Q, Kt, V)
    lens = torch.full((B,), L - T, dtype=torch.int32, device="cuda")
    i1, i2 = (torch.empty(B, Hkv, 64, dtype=torch.int32, device="cuda") for _ in range(2))
    a = rmm.rmm_attn_tree(q, kt, v, lens, 0.5, idx_out=i1)
    b = rmm.rmm_attn_qk(q, kt, v, L, 0.5, idx_out=i2)
    assert torch.equal(i1, i2)
    _, _, A, X = ref.attn_tree(Q, Kt, V, lens.cpu(), None, 0.5)
    within(a, b.double().cpu(), 2 * (H16 * b.double().cpu().abs() + (H16 + 2e-4 + 2 * 66 * H32 * X[..., None]) * A), "O")


def test_attn_tree_twice_gives_the_same_bits(rmm):
    Q, Kt, V, lens, parents = attn_inputs(2, 40, 16, 2, [3000, 1000], 3048, "padded", 13)
    args = cuda(Q, Kt, V, lens)
    a, b = (rmm.rmm_attn_tree(*args, 0.5, parents=parents.cuda()) for _ in range(2))
    assert torch.equal(a, b)


def test_attn_tree_captured_and_replayed_with_other_lengths(rmm):
    """One graph serves every step: lengths and trees are device data."""
    B, T, Hq, Hkv, ldL = 3, 12, 8, 2, 512
    Q, Kt, V, lens, parents = attn_inputs(B, T, Hq, Hkv, [100, 200, 300], ldL, "padded", 17, junk=False)
    q, kt, v, ln, pr = cuda(Q, Kt, V, lens, parents)
    O = torch.zeros(B, Hq, T, D, dtype=torch.bfloat16, device="cuda")
    idx = torch.full((B, Hkv, 64), -1, dtype=torch.int32, device="cuda")
    ws = rmm.new_workspace(rmm.rmm_attn_tree_workspace_bytes(B, Hq, Hkv, T, ldL))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rmm.rmm_attn_tree(q, kt, v, ln, 0.5, parents=pr, O=O, idx_out=idx, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rmm.rmm_attn_tree(q, kt, v, ln, 0.5, parents=pr, O=O, idx_out=idx, workspace=ws)
    for step, new in enumerate(([100, 200, 300], [0, 500, 499], [-1, 17, 128])):
        lens = torch.tensor(new, dtype=torch.int32)
        parents = ref.random_trees(B, T, 50 + step)
        ln.copy_(lens)
        pr.copy_(parents)
        idx.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        wo, wi, A, X = ref.attn_tree(Q, Kt, V, lens, parents, 0.5)
        assert torch.equal(idx.cpu(), wi)
        within(O, wo, H16 * wo.abs() + (H16 + 2e-4 + 2 * 66 * H32 * X[..., None]) * A, f"step {step}")
    assert rmm.rmm_get_status(ws) == rmm.RMM_OK


def test_attn_tree_many_calls_with_inputs_just_written(rmm):
    """Lengths, trees, queries and caches written by the kernels directly before each call, into the buffers of
    the call before, kept sets into a buffer of -1: every call sees its own."""
    B, T, Hq, Hkv, ldL, k = 24, 4, 16, 4, 1024, 48
    ws = rmm.new_workspace(rmm.rmm_attn_tree_workspace_bytes(B, Hq, Hkv, T, ldL))
    g = torch.Generator(device="cuda").manual_seed(1)
    Q, O = (torch.zeros(B, Hq, T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Kt, V = torch.zeros(B, Hkv, D, ldL, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, Hkv, ldL, D, dtype=torch.bfloat16, device="cuda")
    lens, idx = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, Hkv, k, dtype=torch.int32, device="cuda")
    Kt.normal_(generator=g)
    for i in range(300):
        Q.normal_(generator=g)
        v = 1.0 + i % 7  # equal values: so is every output that has seen only this call's
        V.fill_(v)
        idx.fill_(-1)
        lens.random_(-1, ldL - T + 1, generator=g)
        rmm.rmm_attn_tree(Q, Kt, V, lens, k / D, O=O, idx_out=idx, workspace=ws)
        s = Q.view(B, Hkv, -1, D).abs().amax(2)
        want = torch.sort(torch.sort(s, dim=-1, descending=True, stable=True).indices[..., :k], -1).values.int()
        there = lens >= 0
        assert torch.equal(idx, torch.where(there[:, None, None], want, -1)), i
        # a weighted mean of v with weights P / l, P rounded to bf16 (2^-8), then O rounded (2^-8)
        want = torch.where(there, v, 0.0)[:, None, None, None]
        assert bool(((O.float() - want).abs() <= 2.1 * H16 * v).all()), i


def test_attn_tree_on_two_streams_with_their_own_workspaces(rmm):
    cases = [attn_inputs(2, 10, 8, 2, [700, 300], 1024, "padded", s, junk=False) for s in (21, 22)]
    want = [rmm.rmm_attn_tree(*cuda(*c[:4]), 0.5, parents=c[4].cuda()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    dev = [cuda(*c) for c in cases]
    torch.cuda.synchronize()
    got = []
    for s, c in zip(streams, dev):
        got.append(rmm.rmm_attn_tree(*c[:4], 0.5, parents=c[4], stream=s))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- probabilities

def softmax_tol(x, t, p):
    z = torch.where(torch.isfinite(x), (x - x.amax(-1, keepdim=True)).abs() / t, 0.0)
    return (4 * z + 4 * (p * z).sum(-1, keepdim=True) + 96) * H32 * p + 1e-37


@pytest.mark.parametrize("rows,V", [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 1000), (2, 4096), (2, 4097), (3, 8200),
                                    (2, 32000), (2, 50021), (1, 131072), (1, 262144)])
@pytest.mark.parametrize("t", [1.0, 0.3])
def test_softmax(rmm, rows, V, t):
    X = normal(V, rows, V, std=4.0)
    if V > 8:
        X[0, 1::3] = -math.inf
    x = X.double()
    want = torch.softmax(x / t, -1)
    within(rmm.rmm_softmax(X.cuda(), t), want, softmax_tol(x, t, want), "Y")


@pytest.mark.parametrize("rows,V,ldx,ldy", [(32, 16384, 16384, 16384), (33, 16391, 16392, 16396), (40, 20000, 20008, 20008),
                                            (32, 65543, 65544, 65544), (35, 131072, 131072, 131076),
                                            (32, 262144, 262144, 262144),
                                            # rows that start anywhere, the outputs' like the logits' or not
                                            (9, 2049, 2049, 2049), (17, 2051, 2051, 2059), (5, 50257, 50257, 50257),
                                            (33, 65537, 65537, 65537), (3, 131069, 131069, 131069), (9, 4099, 4099, 4100)])
def test_softmax_many_long_rows(rmm, rows, V, ldx, ldy):
    X = normal(V, rows, ldx, std=3.0)
    X[1, : V - 4] = -math.inf  # mass in the last part alone
    X[2, 5:V] = -math.inf
    Y = torch.full((rows, ldy), 5.0, device="cuda")
    rmm.rmm_softmax(X.cuda()[:, :V], 0.9, Y=Y[:, :V])
    x = X[:, :V].double()
    want = torch.softmax(x / 0.9, -1)
    within(Y[:, :V], want, softmax_tol(x, 0.9, want), "Y")
    assert bool((Y[:, V:] == 5.0).all())


@pytest.mark.parametrize("off,ldx,ldy", [(0, 1008, 1004), (0, 1001, 1001), (1, 1008, 1003), (3, 1007, 1008)])
def test_softmax_strides(rmm, off, ldx, ldy):
    """Rows of padded logits and padded outputs, aligned and not; the padding is neither read
    into the sum nor written."""
    rows, V = 5, 999
    buf = torch.full((off + rows * ldx,), math.inf, dtype=torch.bfloat16)
    X = buf.as_strided((rows, V), (ldx, 1), off)
    X.copy_(normal(3, rows, V, std=3.0))
    xb = buf.cuda()
    out = torch.full((off + rows * ldy,), 5.0, device="cuda")
    Y = out.as_strided((rows, V), (ldy, 1), off)
    rmm.rmm_softmax(xb.as_strided((rows, V), (ldx, 1), off), 0.8, Y=Y)
    x = X.double()
    want = torch.softmax(x / 0.8, -1)
    within(Y, want, softmax_tol(x, 0.8, want), "Y")
    touched = torch.zeros(out.numel(), dtype=torch.bool)
    touched.as_strided((rows, V), (ldy, 1), off).fill_(True)
    assert bool((out.cpu()[~touched] == 5.0).all())


@pytest.mark.parametrize("V", [1, 5, 4100, 40000])
def test_softmax_greedy_and_empty_rows(rmm, V):
    X = normal(V, 4, V)
    X[1] = -math.inf                       # nothing to choose from
    X[2, V // 2:] = X[2].max()             # a tie: the lowest index
    X[3] = 0.25
    for t in (0.0, 1.0):
        Y = rmm.rmm_softmax(X.cuda(), t).cpu()
        assert not bool(Y[1].any())
        if t == 0.0:
            for i in (0, 2, 3):
                first = int((X[i] == X[i].max()).nonzero()[0])
                assert float(Y[i].sum()) == 1.0 and float(Y[i, first]) == 1.0
        else:
            within(Y[3], torch.full((V,), 1.0 / V, dtype=torch.float64), 96 * H32 / V, "equal logits")


@pytest.mark.parametrize("rows,V,ldx", [(5, 10, 16), (3, 4096, 4096), (2, 40000, 40000), (33, 16389, 16392),
                                        (33, 20480, 20480)])
def test_softmax_nan_and_infinity_reach_the_whole_row(rmm, rows, V, ldx):
    """Wherever they stand, and with nothing but -inf beside them."""
    X = torch.full((rows, ldx), float("nan"), dtype=torch.bfloat16)
    X[:, :V] = normal(V, rows, V)
    bad = {0: (float("nan"), V - 1), 1: (float("inf"), V - 1), 2: (float("inf"), 3)}
    for r, (v, i) in bad.items():
        if r < rows:
            X[r, i] = v
    hidden = [r for r in (3, 4) if r < rows]
    for r in hidden:  # -inf everywhere else
        X[r, :V] = -float("inf")
        X[r, 0 if r == 3 else V - 1] = float("nan")
    Y = torch.zeros(rows, ldx, device="cuda")
    y = rmm.rmm_softmax(X.cuda()[:, :V], 0.7, Y=Y[:, :V]).cpu()
    assert not bool(Y[:, V:].any())
    for r in range(rows):
        assert bool(torch.isnan(y[r]).all()) == (r in bad or r in hidden), r
        assert not bool(torch.isnan(y[r]).any()) or r in bad or r in hidden, r


# ---------------------------------------------------------------- verification

def verify_inputs(B, T, V, seed, draft=True, fan=4, noise=1.0, padded=True, roots=True):
    g = torch.Generator().manual_seed(seed)
    a = 2.0 * torch.randn(B, T, V, generator=g)
    P = torch.softmax(a, -1)
    Qd = torch.softmax(a + noise * torch.randn(B, T, V, generator=g), -1)
    parents = ref.random_trees(B, T, seed, fan=fan, padded=padded, roots=roots)
    tokens = torch.empty(B, T, dtype=torch.int32)
    for b in range(B):
        for t in range(T):
            p = int(parents[b, t])
            tokens[b, t] = torch.multinomial(Qd[b, p if 0 <= p < t else 0], 1, generator=g)
    u = torch.rand(B, T, generator=g)
    return P, tokens, parents, u, Qd if draft else None


def check_verify(rmm, P, tokens, parents, u, Qd):
    want = ref.verify(P, tokens, parents, u, Qd)
    p, t, pr, uu, q = cuda(P, tokens, parents, u, Qd)
    got = rmm.rmm_tree_verify(p, t, pr, uu, Qd=q)
    for name, a, b in zip(("path", "emitted", "count"), got, want):
        assert torch.equal(a.cpu(), b), name
    return want


@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (2, 1, 50), (3, 2, 2), (4, 5, 7), (5, 8, 129), (6, 16, 1000),
                                   (2, 33, 4099), (2, 64, 17000), (1, 9, 50021), (300, 6, 40)])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("fan,noise", [(1, 0.3), (8, 1.5)])
def test_tree_verify(rmm, B, T, V, draft, fan, noise):
    check_verify(rmm, *verify_inputs(B, T, V, 31 * T + V, draft, fan, noise))


@pytest.mark.parametrize("V", [131071, 131072, 131073, 300007])
@pytest.mark.parametrize("draft", [True, False])
def test_tree_verify_large_vocabularies(rmm, V, draft):
    """Rows that just fill the registers of a sequence's CTAs and rows that do not fit there: rejections one
    after the other at a node, the next token at both ends, mass in the last few tokens only."""
    P, tokens, parents, u, Qd = verify_inputs(4, 6, V, V, draft, 5, 2.0, padded=False, roots=False)
    parents[1:, 1:] = 0
    u[1:, 1:] = 0.999
    u[2, 0], u[3, 0] = 0.0, 1.0 - 2.0 ** -24
    P[3, 0, : V - 3] = 0.0
    want = check_verify(rmm, P, tokens, parents, u, Qd)
    assert int(want[1][3, 0]) >= V - 3


def test_tree_verify_walks_deep_and_rejects_often(rmm):
    """The inputs reach what they are for: long accepted paths and several rejections at a node."""
    *_, count = check_verify(rmm, *verify_inputs(64, 32, 100, 5, True, 2, 0.2, padded=False))
    assert int(count.max()) > 8
    P, tokens, parents, u, Qd = verify_inputs(32, 24, 60, 6, True, 24, 3.0, padded=False, roots=False)
    parents[:, 1:] = 0  # 23 siblings under the root
    check_verify(rmm, P, tokens, parents, u, Qd)
    check_verify(rmm, P, tokens, parents, u, None)
    check_verify(rmm, P, tokens, parents, torch.full_like(u, 0.999), Qd)


def test_tree_verify_borders(rmm):
    """Random numbers at 0 and next to 1, certain and impossible tokens, equal rows, tokens
    outside the vocabulary, the same token twice, an absent root, a row with no mass, NaN."""
    B, T, V = 12, 6, 33
    P, tokens, parents, u, Qd = verify_inputs(B, T, V, 77, True, 3, 0.5, padded=False, roots=False)
    u[0], u[1] = 0.0, 1.0 - 2.0 ** -24
    P[2] = 0.0
    P[2, :, 9] = 1.0                    # certain
    Qd[3] = P[3]                        # the draft is the target: everything is accepted
    tokens[4, 1:] = torch.tensor([-1, V, 2 ** 31 - 1, -5, 3])
    parents[5, 1:] = 0
    tokens[5, 1:] = 7                   # one token five times
    u[5] = 0.99
    parents[6, 0] = -2                  # an empty slot
    P[7] = 0.0                          # no mass at all
    P[8, :, 4], Qd[8, :, 5] = float("nan"), float("nan")
    P[9, :, 4] = -0.5
    Qd[10] = 2.0                        # covers everything: a rejection would leave nothing
    u[10] = 0.99
    u[11] = float("nan")
    for q in (Qd, None):
        _, emitted, count = check_verify(rmm, P, tokens, parents, u, q)
        assert int(count[6]) == 0 and int(emitted[7, 0]) == -1
        assert int(emitted[2, int(count[2]) - 1]) == 9


@pytest.mark.parametrize("ldp,ldq,off", [(1004, 1000, 0), (1001, 1000, 0), (1000, 1003, 0), (1000, 1000, 1)])
def test_tree_verify_strides(rmm, ldp, ldq, off):
    B, T, V = 3, 7, 1000
    P, tokens, parents, u, Qd = verify_inputs(B, T, V, 91)
    want = ref.verify(P, tokens, parents, u, Qd)

    def strided(x, ld):
        buf = torch.full((off + B * T * ld,), float("nan"), device="cuda")
        y = buf.as_strided((B * T, V), (ld, 1), off)
        y.copy_(x.view(B * T, V))
        return y

    got = rmm.rmm_tree_verify(strided(P, ldp), *cuda(tokens, parents, u), Qd=strided(Qd, ldq))
    for a, b in zip(got, want):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("draft", [True, False])
def test_tree_verify_emits_the_targets_distribution(rmm, draft):
    """Over many sequences the first emitted token is distributed as the target's root row,
    whatever the draft: each frequency within 6 standard deviations.  (Certain picks leave the
    distribution alone for any tokens chosen without looking at u.)"""
    n, T, V = 4096, 5, 12
    g = torch.Generator().manual_seed(2)
    p = torch.softmax(torch.randn(V, generator=g), -1)
    q = torch.softmax(torch.randn(V, generator=g), -1)
    rows = 8
    freq = torch.zeros(V, dtype=torch.float64)
    for i in range(rows):
        tokens = torch.multinomial(q, n * T, True, generator=g).view(n, T).int()
        if not draft:
            tokens = torch.argsort(torch.rand(n, V, generator=g), 1)[:, :T].int()
        parents = torch.zeros(n, T, dtype=torch.int32)
        parents[:, 0] = -1
        u = torch.rand(n, T, generator=g)
        P = p.expand(n, T, V).contiguous().cuda()
        Qd = q.expand(n, T, V).contiguous().cuda() if draft else None
        _, emitted, count = rmm.rmm_tree_verify(P, *cuda(tokens, parents, u), Qd=Qd)
        assert int(count.min()) >= 1
        freq += torch.bincount(emitted[:, 0].long().cpu(), minlength=V).double()
    N = n * rows
    pd = p.double()
    assert bool(((freq / N - pd).abs() <= 6 * torch.sqrt(pd * (1 - pd) / N)).all())


# ---------------------------------------------------------------- kept nodes

def keep_inputs(B, T, Hkv, ldL, n, seed):
    g = torch.Generator().manual_seed(seed)
    caches = [(normal(seed + 2 * i, B, Hkv, D, ldL), normal(seed + 2 * i + 1, B, Hkv, ldL, D)) for i in range(n)]
    lens = torch.randint(0, ldL - T + 1, (B,), generator=g).int()
    path, count = torch.full((B, T), -1, dtype=torch.int32), torch.empty(B, dtype=torch.int32)
    for b in range(B):
        c = int(torch.randint(1, T + 1, (1,), generator=g))
        path[b, :c] = torch.sort(torch.randperm(T, generator=g)[:c]).values.int()
        count[b] = c
    return caches, lens, path, count


@pytest.mark.parametrize("B,T,Hkv,ldL,n", [(1, 1, 1, 8, 1), (3, 2, 2, 16, 2), (5, 7, 3, 40, 1), (4, 33, 2, 64, 3),
                                           (6, 64, 4, 136, 2), (2, 64, 1, 64, 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_cache_keep(rmm, B, T, Hkv, ldL, n, in_place):
    caches, lens, path, count = keep_inputs(B, T, Hkv, ldL, n, 7 * T + B)
    if B > 3:
        lens[1] = -1                     # an empty slot
        lens[2] = ldL - T + 1            # no room: such a sequence had no tree
        count[3] = 0
        path[0, : int(count[0])] = torch.arange(int(count[0]))  # already in place
    if B > 4:
        path[4, 0], path[4, 1], count[4] = 3, 2, 2  # not ascending
    dev = [tuple(cuda(*c)) for c in caches]
    ln, pt, ct = cuda(lens, path, count)
    out = rmm.rmm_cache_keep(dev, ln, pt, ct, lens_out=ln if in_place else None)
    for (Kt, V), (kt, v) in zip(caches, dev):
        wk, wv, wl = ref.keep(Kt, V, lens, path, count)
        assert torch.equal(kt.cpu(), wk) and torch.equal(v.cpu(), wv)
    assert torch.equal(out.cpu(), wl)
    assert (out is ln) == in_place
    if not in_place:
        assert torch.equal(ln.cpu(), lens)


# ---------------------------------------------------------------- the calls themselves

def test_the_short_way_and_the_long_way_agree(rmm, monkeypatch):
    """The compiled module in front of the calls and the binding's own marshalling: the same results and the
    same refusals, on the current stream and a given one."""
    B, T, Hq, Hkv, ldL, V = 2, 6, 4, 2, 64, 500
    ys = cuda(*(normal(i, B * T, h * D) for i, h in ((1, Hq), (2, Hkv), (3, Hkv))))
    lens = torch.tensor([3, 40], dtype=torch.int32, device="cuda")
    parents = ref.random_trees(B, T, 3).cuda()
    freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float32) / D)).cuda()
    P, tokens, _, u, Qd = cuda(*verify_inputs(B, T, V, 5))
    X = normal(9, B * T, V).cuda()
    new = lambda *s, dtype=torch.int32: torch.full(s, -7, device="cuda").to(dtype)

    def run(stream):
        Q, O = new(B, Hq, T, D, dtype=torch.bfloat16), new(B, Hq, T, D, dtype=torch.bfloat16)
        caches = [(new(B, Hkv, D, ldL, dtype=torch.bfloat16), new(B, Hkv, ldL, D, dtype=torch.bfloat16)) for _ in range(3)]
        idx, Y = new(B, Hkv, 64), new(B * T, V, dtype=torch.float32)
        path, emitted, count, grown = new(B, T), new(B, T), new(B), new(B)
        ws = rmm.new_workspace(rmm.rmm_attn_tree_workspace_bytes(B, Hq, Hkv, T, ldL))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        kw = dict(stream=stream)
        for kt, v in caches:
            rmm.rmm_qkv_rope(*ys, Q, kt, v, lens=lens, parents=parents, inv_freq=freq, interleaved=True, **kw)
        rmm.rmm_attn_tree(Q, *caches[0], lens, 0.5, parents=parents, O=O, idx_out=idx, workspace=ws, **kw)
        rmm.rmm_softmax(X, 0.8, Y=Y, **kw)
        rmm.rmm_tree_verify(Y, tokens, parents, u, Qd=Qd, path=path, emitted=emitted, count=count, **kw)
        rmm.rmm_cache_keep(caches, lens, path, count, lens_out=grown, **kw)
        torch.cuda.synchronize()
        with pytest.raises(ValueError, match="emitted"):
            rmm.rmm_tree_verify(Y, tokens, parents, u, Qd=Qd, path=path, emitted=emitted[:, :-1], count=count)
        with pytest.raises(ValueError, match="Kt"):
            rmm.rmm_cache_keep([(caches[0][0][..., :-8], caches[0][1])], lens, path, count, lens_out=grown)
        with pytest.raises(ValueError, match="Yk"):
            rmm.rmm_qkv_rope(ys[0], ys[1].float(), ys[2], Q, *caches[0], lens=lens)
        with pytest.raises(rmm.RmmError):
            rmm.rmm_softmax(X, -1.0, Y=Y)
        with pytest.raises(rmm.RmmError):
            rmm.rmm_attn_tree(Q, *caches[0], lens, 0.5, O=O, workspace=ws[:256])
        return [Q, O, idx, Y, path, emitted, count, grown] + [t for c in caches for t in c]

    want = run(None)
    assert int(want[6].min()) >= 0 and bool((want[7] != -7).all())
    got = [run(torch.cuda.Stream())]

    class Nothing:
        def __getattr__(self, name):
            return lambda *a: None

    monkeypatch.setattr(rmm, "_short", Nothing)
    got += [run(None), run(torch.cuda.Stream())]
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


def test_calls_from_several_threads(rmm):
    """Each thread on its own stream, with rows that need different amounts of shared memory: the same bits as
    one after the other."""
    import threading

    xs = [normal(n, 32, n).cuda() for n in (16384, 24576, 65536, 131072)]
    want = [rmm.rmm_softmax(x, 0.9) for x in xs]
    torch.cuda.synchronize()
    got, wrong = [None] * len(xs), []

    def work(i):
        try:
            s = torch.cuda.Stream()
            y = torch.zeros_like(want[i])
            s.wait_stream(torch.cuda.default_stream())
            for _ in range(50):
                rmm.rmm_softmax(xs[i], 0.9, Y=y, stream=s)
            s.synchronize()
            got[i] = y
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong
    for a, b in zip(got, want):
        assert torch.equal(a, b)
