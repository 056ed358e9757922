"""Decoding with drafts through the decoder layer: the tree operators run together.

Each operator gets the GPU's own inputs, so a last-bit difference before it cannot flip a
kept set or a token behind it.  Where two runs with different kernels are compared over
two layers, every tensor between two operators is rounded to bf16, off by at most 2^-8 of
its elements and so of its norm; a residual row passes 10 such tensors per layer, whose
differences arrive with a gain of at most 1 (the weights' gain is 0.02 sqrt(512) = 0.45 on
normed rows, the norms and the softmax average): less than 2 * 10 * 2^-8 of the row's norm.
"""
import pytest
import torch

import rmm_synth
import tree_ref as ref
from parity import assert_close
from test_gpu_layer import check_step, make_weights

pytestmark = pytest.mark.gpu
D = 128
H16, H32 = 2.0 ** -8, 2.0 ** -24
H, HQ, HKV, F, V = 512, 4, 2, 1024, 320
TWO_LAYERS = 2 * 10 * H16


@pytest.fixture(scope="module")
def rmm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from input_adaptive_reduced_rmm_b200 import rmm as _rmm

    _rmm.lib()
    return _rmm


def normal(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).bfloat16()


FREQ = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float32) / D)
TURNED = dict(q_norm=1.0 + normal(70, D, std=0.1).float(), k_norm=1.0 + normal(71, D, std=0.1).float(), inv_freq=FREQ)
TURNED = {k: v if k == "inv_freq" else v.bfloat16() for k, v in TURNED.items()}


def make_layer(seed, r, max_len=64, **kw):
    from input_adaptive_reduced_rmm_b200.layer import DecoderLayer, LayerDims

    W = make_weights(H, HQ, HKV, F, seed)
    return DecoderLayer(LayerDims(H=H, Hq=HQ, Hkv=HKV, F=F), W, max_len=max_len, r=r, device=torch.device("cuda"), **kw), W


def within(got, want, tol, what):
    assert bool(((got.double().cpu() - want).abs() <= tol).all()), what


def check_rotated(tr, T, L0, parents=None):
    """q, k and v of a traced call against the formulas, and nothing else written to the caches."""
    c = {n: tr[n].cpu() for n in ("yq", "yk", "yv", "Q", "Kt", "V")}
    Q0, K0, V0 = c["Q"][None], c["Kt"][None].clone(), c["V"][None].clone()
    K0[..., L0:L0 + T], V0[:, :, L0:L0 + T] = 0, 0
    lens = torch.tensor([L0], dtype=torch.int32)
    wq, wk, wv, mq, mk = ref.qkv_rope(c["yq"], c["yk"], c["yv"], Q0, K0, V0, lens, parents, TURNED["q_norm"],
                                      TURNED["k_norm"], 1e-5, FREQ, False)
    within(c["Q"][None], wq, H16 * wq.abs() + 32 * H32 * mq, "Q")
    within(c["Kt"][None], wk, H16 * wk.abs() + 32 * H32 * mk, "Kt")
    within(c["V"][None], wv, 0.0, "V")


def test_layer_with_norms_and_rotation(rmm):
    layer, _ = make_layer(1, 0.5, **TURNED)
    for T in (20, 1):
        tr, L0 = {}, layer.pos
        layer.forward(rmm_synth.activations(T, H, rmm_synth.seed_for(3, 5, T)).cuda(), trace=tr)
        assert layer.pos == L0 + T
        check_rotated(tr, T, L0)


@pytest.mark.parametrize("T", [1, 7, 40])
def test_a_chain_is_the_causal_layer(rmm, T):
    layer, W = make_layer(2, 0.5)
    layer.forward(rmm_synth.activations(21, H, rmm_synth.seed_for(3, 6, 0)).cuda())
    x = rmm_synth.activations(T, H, rmm_synth.seed_for(3, 6, 1)).cuda()
    for parents in (None, (torch.arange(T, dtype=torch.int32) - 1).cuda()):
        tr = {}
        layer.forward_tree(x, parents, trace=tr)
        assert layer.pos == 21
        check_step(tr, W, 0.5, HQ, HKV)


def test_a_tree_against_the_formulas(rmm):
    T, L0 = 24, 21
    layer, _ = make_layer(3, 0.5, **TURNED)
    layer.forward(rmm_synth.activations(L0, H, rmm_synth.seed_for(3, 7, 0)).cuda())
    parents = ref.random_trees(2, T, 5)[1:]  # some nodes are absent
    tr = {}
    layer.forward_tree(rmm_synth.activations(T, H, rmm_synth.seed_for(3, 7, 1)).cuda(), parents[0].cuda(), trace=tr)
    there = [t for t in range(T) if ref.way(parents[0].tolist(), t)]
    assert 0 < len(there) < T
    Q, Kt, Vc, O = (tr[n].cpu()[None] for n in ("Q", "Kt", "V", "O"))
    lens = torch.tensor([L0], dtype=torch.int32)
    wo, wi, A, X = ref.attn_tree(Q, Kt, Vc, lens, parents, 0.5)
    assert torch.equal(tr["idx_attn"].cpu()[None], wi)
    within(O, wo, H16 * wo.abs() + (H16 + 2e-4 + 2 * 66 * H32 * X[..., None]) * A, "O")
    check_rotated(tr, T, L0, parents)


def next_token(P, u):
    run = P.double().cumsum(0)
    return int((run > u * run[-1]).nonzero()[0])


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("draft,temperature", [(True, 1.0), (False, 1.0), (False, 0.0)])
def test_decoding_with_drafts(rmm, turned, draft, temperature):
    """Six steps of trees: every step's tokens are the rule's for its probabilities, the caches hold exactly the
    accepted nodes' keys and values, and both agree with layers that were given the emitted tokens in order."""
    from input_adaptive_reduced_rmm_b200.layer import OutputHead, decode_tree

    kw = TURNED if turned else {}
    layers, plain = ([make_layer(s, 1.0, max_len=96, **kw)[0] for s in (11, 12)] for _ in range(2))
    head = OutputHead(normal(20, V, H, std=0.05), 1.0, "cuda")
    embed = normal(21, V, H).cuda()
    g = torch.Generator().manual_seed(5)
    text = torch.randint(0, V, (9,), generator=g).tolist()
    for stack in (layers, plain):
        x = embed[text]
        for layer in stack:
            x = layer.forward(x)
    text.append(next_token(head.probabilities(x[-1:].contiguous())[0].cpu(), 0.5))
    counts = []
    for step in range(6):
        T = [1, 5, 12, 12, 33, 64][step]
        start = layers[0].pos
        parents = ref.random_trees(1, T, step, fan=3, padded=False)
        Qd = torch.softmax(2.0 * torch.randn(T, V, generator=g), -1)
        tokens = torch.randint(0, V, (1, T), generator=g, dtype=torch.int32)
        tokens[0, 0] = text[-1]
        u = 0.02 * torch.rand(1, T, generator=g)  # small: drafts are accepted often
        if not draft:  # certain picks: make the first child of each node likely
            tr = {}
            probe(layers, head, embed, tokens, parents, tr)
            best = tr["P"].argmax(-1).cpu().int()
            for t in range(1, min(T, 4)):
                parents[0, t] = t - 1
            for t in range(1, min(T, 4)):
                tokens[0, t] = best[t - 1]
                probe(layers, head, embed, tokens, parents, tr)
                best = tr["P"].argmax(-1).cpu().int()
        before = [(l.Kt.clone(), l.V.clone()) for l in layers]
        tr = {}
        got = decode_tree(layers, head, embed, tokens[0].cuda(), parents[0].cuda(), u[0].cuda(), temperature,
                          Qd=Qd.cuda() if draft else None, trace=tr)
        path, emitted, count = ref.verify(tr["P"].cpu()[None], tokens, parents, u, Qd[None] if draft else None)
        n = int(count[0])
        assert got == emitted[0, :n].tolist() and torch.equal(tr["path"].cpu(), path)
        counts.append(n)
        assert all(l.pos == start + n for l in layers)
        for l, (k, v) in zip(layers, before):  # what was cached stays
            assert torch.equal(l.Kt[..., :start], k[..., :start]) and torch.equal(l.V[:, :start], v[:, :start])
        # the emitted tokens one call later through the plain layers: the root and the accepted drafts
        x = embed[[text[-1]] + got[:-1]]
        for layer in plain:
            x = layer.forward(x)
        taken = path[0, :n].long()
        rel = (tr["x"][taken].float() - x.float()).norm(dim=1) / x.float().norm(dim=1)
        assert float(rel.max()) <= TWO_LAYERS, float(rel.max())
        for a, b in zip(layers, plain):
            for y, z in ((a.Kt[..., :a.pos], b.Kt[..., :a.pos]), (a.V[:, :a.pos], b.V[:, :a.pos])):
                assert float((y.float() - z.float()).norm() / z.float().norm()) <= TWO_LAYERS
        text += got
    assert max(counts) > 1, counts


def probe(layers, head, embed, tokens, parents, tr):
    """The nodes' probabilities without keeping anything."""
    x = embed[tokens[0].long()]
    for layer in layers:
        x = layer.forward_tree(x, parents[0].cuda())
    tr["P"] = head.probabilities(x)


def test_keep_path_refuses_layers_of_different_lengths(rmm):
    from input_adaptive_reduced_rmm_b200.layer import keep_path

    a, b = make_layer(1, 0.5)[0], make_layer(2, 0.5)[0]
    a.forward(rmm_synth.activations(3, H, 1).cuda())
    with pytest.raises(ValueError, match="different numbers"):
        keep_path([a, b], torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                  torch.ones(1, dtype=torch.int32, device="cuda"))


def test_a_whole_step_captured_and_replayed(rmm):
    """Two layers, the head, the verification and the keeping as one graph over device tensors: replays with other
    lengths, trees, tokens and random numbers give the bits of the same calls made eagerly."""
    from input_adaptive_reduced_rmm_b200.layer import OutputHead

    T, S = 12, torch.cuda.Stream()
    head = OutputHead(normal(20, V, H, std=0.05), 0.5, "cuda")
    embed = normal(21, V, H).cuda()
    stacks = [[make_layer(s, 0.5, max_len=64, **TURNED)[0] for s in (11, 12)] for _ in range(2)]
    prefix = embed[torch.arange(30)]
    for stack in stacks:
        x = prefix
        for layer in stack:
            x = layer.forward(x)
        for layer in stack:
            layer.pos = 0  # lengths come from the device alone
    io = [dict(tokens=torch.zeros(1, T, dtype=torch.int32, device="cuda"),
               parents=(torch.arange(T, dtype=torch.int32, device="cuda") - 1)[None].contiguous(),
               u=torch.zeros(1, T, device="cuda"), lens=torch.zeros(1, dtype=torch.int32, device="cuda"),
               path=torch.zeros(1, T, dtype=torch.int32, device="cuda"),
               emitted=torch.zeros(1, T, dtype=torch.int32, device="cuda"),
               count=torch.zeros(1, dtype=torch.int32, device="cuda")) for _ in range(2)]

    def step(stack, d):
        x = embed.index_select(0, d["tokens"][0])
        for layer in stack:
            x = layer.forward_tree(x, d["parents"], d["lens"])
        P = head.probabilities(x, 0.7)
        rmm.rmm_tree_verify(P, d["tokens"], d["parents"], d["u"], path=d["path"], emitted=d["emitted"], count=d["count"])
        rmm.rmm_cache_keep([(l.Kt[None], l.V[None]) for l in stack], d["lens"], d["path"], d["count"], lens_out=d["lens"])

    S.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(S):
        saved = [(l.Kt.clone(), l.V.clone()) for l in stacks[0]]
        step(stacks[0], io[0])  # workspaces and buffers
        S.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=S):
            step(stacks[0], io[0])
        for l, (k, v) in zip(stacks[0], saved):
            l.Kt.copy_(k), l.V.copy_(v)
    S.synchronize()
    g = torch.Generator().manual_seed(3)
    grew = 0
    for n in (0, 30, 7, -1, 52, 53):  # an empty cache, others, an empty slot, the last slot, one past it
        tokens = torch.randint(0, V, (1, T), generator=g, dtype=torch.int32)
        parents = ref.random_trees(2, T, n + 100)[n % 2][None]
        u = 0.05 * torch.rand(1, T, generator=g)
        for d in io:
            d["tokens"].copy_(tokens), d["parents"].copy_(parents), d["u"].copy_(u), d["lens"].fill_(n)
        torch.cuda.synchronize()
        graph.replay()
        step(stacks[1], io[1])
        torch.cuda.synchronize()
        for k in io[0]:
            assert torch.equal(io[0][k], io[1][k]), (n, k)
        for a, b in zip(*stacks):
            assert torch.equal(a.Kt, b.Kt) and torch.equal(a.V, b.V), n
        grew += int(io[0]["lens"]) != n
    assert grew == 4  # every one with a slot for its tree
