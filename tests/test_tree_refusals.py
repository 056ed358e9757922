"""The draft-tree entry points refuse what they do not handle, on the host: through the C ABI
with pointers that are never dereferenced, and through the binding before the library is called."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def rmm():
    from input_adaptive_reduced_rmm_b200 import build as b

    b.build()
    from input_adaptive_reduced_rmm_b200 import rmm as _rmm

    _rmm.lib()
    return _rmm


FAKE = ctypes.c_void_p(1 << 20)      # 16-byte aligned, never touched
ODD = ctypes.c_void_p((1 << 20) + 2)  # aligned for bf16 only


def qkv(**k):
    a = dict(Yq=FAKE, Yk=FAKE, Yv=FAKE, B=2, T=4, Hq=8, Hkv=2, d=128, qn=FAKE, kn=FAKE, eps=1e-6, freq=FAKE, rot=128,
             inter=0, lens=FAKE, L0=0, parents=FAKE, Q=FAKE, Kt=FAKE, V=FAKE, ldL=64, stream=None)
    a.update(k)
    return list(a.values())


def attn(**k):
    a = dict(Q=FAKE, Kt=FAKE, V=FAKE, lens=FAKE, parents=FAKE, B=2, Hq=8, Hkv=2, T=4, ldL=64, d=128, r=0.5, scale=1.0,
             O=FAKE, idx=None, ws=FAKE, bytes=1 << 40, stream=None, opts=None)
    a.update(k)
    return list(a.values())


def softmax(**k):
    a = dict(X=FAKE, rows=2, V=100, ldx=100, t=1.0, Y=FAKE, ldy=100, stream=None)
    a.update(k)
    return list(a.values())


def verify(**k):
    a = dict(P=FAKE, ldp=100, Qd=FAKE, ldq=100, B=2, T=4, V=100, tokens=FAKE, parents=FAKE, u=FAKE, path=FAKE,
             emitted=FAKE, count=FAKE, stream=None)
    a.update(k)
    return list(a.values())


def keep(n=2, **k):
    ks = (ctypes.c_void_p * 200)(*[(1 << 20) + 4096 * i for i in range(200)])
    vs = (ctypes.c_void_p * 200)(*[(1 << 24) + 4096 * i for i in range(200)])
    a = dict(count=n, Kts=ks, Vs=vs, B=2, Hkv=2, d=128, ldL=64, lens=FAKE, path=FAKE, kept=FAKE, T=4, out=None,
             stream=None)
    a.update(k)
    return list(a.values())


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.mark.parametrize("change,status", [
    (dict(Yq=None), INVALID), (dict(Yk=None), INVALID), (dict(Yv=None), INVALID), (dict(Q=None), INVALID),
    (dict(Kt=None), INVALID), (dict(V=None), INVALID), (dict(B=0), INVALID), (dict(T=0), INVALID),
    (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(ldL=60), INVALID), (dict(T=65, ldL=64), INVALID),
    (dict(lens=None, L0=-1), INVALID), (dict(lens=None, L0=61), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(rot=0), INVALID), (dict(rot=144), INVALID), (dict(Yq=ODD), INVALID),
    (dict(Kt=ODD), INVALID), (dict(qn=ODD), INVALID), (dict(kn=ODD), INVALID), (dict(d=64, rot=64), UNSUPPORTED),
    (dict(rot=72), UNSUPPORTED), (dict(T=65, ldL=128), UNSUPPORTED), (dict(Hq=5000), UNSUPPORTED),
    (dict(B=4097), UNSUPPORTED), (dict(parents=None, T=(1 << 20) + 8, ldL=1 << 21), UNSUPPORTED),
])
def test_qkv_rope_refusals(rmm, change, status):
    assert rmm.lib().rmm_qkv_rope(*qkv(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(Q=None), INVALID), (dict(Kt=None), INVALID), (dict(V=None), INVALID), (dict(lens=None), INVALID),
    (dict(O=None), INVALID), (dict(B=0), INVALID), (dict(Hq=7), INVALID), (dict(Hkv=0), INVALID), (dict(T=0), INVALID),
    (dict(ldL=63), INVALID), (dict(T=72, ldL=64), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID), (dict(r=0.0), INVALID),
    (dict(r=1.5), INVALID), (dict(Q=ODD), INVALID), (dict(V=ODD), INVALID), (dict(O=ODD), INVALID),
    (dict(d=64), UNSUPPORTED), (dict(T=65, ldL=128), UNSUPPORTED), (dict(parents=None, T=65, ldL=128), UNSUPPORTED),
    (dict(B=4097), UNSUPPORTED), (dict(Hq=8192, Hkv=8), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(bytes=100), WORKSPACE), (dict(ws=ODD), WORKSPACE),
])
def test_attn_tree_refusals(rmm, change, status):
    assert rmm.lib().rmm_attn_tree(*attn(**change)) == status


def test_attn_tree_options_and_workspace_sizes(rmm):
    for o, status in ((rmm.options(attn_per_query_head=True), UNSUPPORTED), (rmm.options(attn_path=1), UNSUPPORTED),
                      (rmm.options(attn_path=3), INVALID)):
        assert rmm.lib().rmm_attn_tree(*attn(opts=ctypes.byref(o))) == status
        assert rmm.rmm_attn_tree_workspace_bytes(2, 8, 2, 4, 64, opts=o) == 0
    assert rmm.rmm_attn_tree_workspace_bytes(2, 8, 2, 4, 64) > 0
    for bad in ((0, 8, 2, 4, 64), (2, 8, 3, 4, 64), (2, 8, 2, 65, 128), (2, 8, 2, 4, 60), (2, 8, 2, 8, 4)):
        assert rmm.rmm_attn_tree_workspace_bytes(*bad) == 0
    assert rmm.rmm_attn_tree_workspace_bytes(2, 8, 2, 4, 64, d=64) == 0


@pytest.mark.parametrize("change,status", [
    (dict(X=None), INVALID), (dict(Y=None), INVALID), (dict(rows=0), INVALID), (dict(V=0), INVALID),
    (dict(ldx=99), INVALID), (dict(ldy=99), INVALID), (dict(t=-1.0), INVALID), (dict(t=1e-9), INVALID),
    (dict(t=1e9), INVALID), (dict(t=float("nan")), INVALID), (dict(t=float("inf")), INVALID),
    (dict(X=ctypes.c_void_p((1 << 20) + 1)), INVALID), (dict(Y=ODD), INVALID),
    (dict(V=262145, ldx=262145, ldy=262145), UNSUPPORTED), (dict(rows=(1 << 24) + 1), UNSUPPORTED),
])
def test_softmax_refusals(rmm, change, status):
    assert rmm.lib().rmm_softmax(*softmax(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(P=None), INVALID), (dict(tokens=None), INVALID), (dict(parents=None), INVALID), (dict(u=None), INVALID),
    (dict(path=None), INVALID), (dict(emitted=None), INVALID), (dict(count=None), INVALID), (dict(B=0), INVALID),
    (dict(T=0), INVALID), (dict(V=0), INVALID), (dict(ldp=99), INVALID), (dict(ldq=99), INVALID), (dict(P=ODD), INVALID),
    (dict(Qd=ODD), INVALID), (dict(T=65), UNSUPPORTED), (dict(B=4097), UNSUPPORTED),
    (dict(V=(1 << 24) + 1, ldp=1 << 25, ldq=1 << 25), UNSUPPORTED),
])
def test_tree_verify_refusals(rmm, change, status):
    assert rmm.lib().rmm_tree_verify(*verify(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(Kts=None), INVALID), (dict(Vs=None), INVALID), (dict(lens=None), INVALID), (dict(path=None), INVALID),
    (dict(kept=None), INVALID), (dict(n=0), INVALID), (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(T=0), INVALID),
    (dict(ldL=60), INVALID), (dict(T=65, ldL=64), INVALID), (dict(T=65, ldL=128), UNSUPPORTED),
    (dict(d=64), UNSUPPORTED), (dict(n=129), UNSUPPORTED), (dict(B=4097), UNSUPPORTED),
    (dict(out=ctypes.c_void_p((1 << 20) + 4)), INVALID),  # overlaps lens without being it
    (dict(Kts=(ctypes.c_void_p * 2)(1 << 20, 1 << 20)), INVALID),  # one cache twice
    (dict(Kts=(ctypes.c_void_p * 2)(1 << 20, None)), INVALID),
    (dict(Vs=(ctypes.c_void_p * 2)(1 << 24, (1 << 25) + 2)), INVALID),
])
def test_cache_keep_refusals(rmm, change, status):
    assert rmm.lib().rmm_cache_keep(*keep(**change)) == status


# ---------------------------------------------------------------- the binding

def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def test_binding_names_what_does_not_fit(rmm):
    B, T, Hq, Hkv, d, L = 2, 3, 4, 2, 128, 64
    q, k, v = bf(B * T, Hq * d), bf(B * T, Hkv * d), bf(B * T, Hkv * d)
    Q, Kt, V = bf(B, Hq, T, d), bf(B, Hkv, d, L), bf(B, Hkv, L, d)
    ok = dict(lens=i32(B), parents=i32(B, T))
    with pytest.raises(ValueError, match="must be a CUDA tensor"):  # the shapes are right
        rmm.rmm_qkv_rope(q, k, v, Q, Kt, V, **ok)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        rmm.rmm_attn_tree(Q, Kt, V, i32(B), 0.5, parents=i32(B, T))
    for bad in (dict(lens=i32(B + 1)), dict(parents=i32(B, T + 1)), dict(q_norm=bf(d - 1)),
                dict(inv_freq=torch.zeros(64, dtype=torch.float64)), dict(lens=torch.zeros(B, dtype=torch.int64)),
                dict(k_norm=torch.zeros(d))):
        with pytest.raises(ValueError):
            rmm.rmm_qkv_rope(q, k, v, Q, Kt, V, **{**ok, **bad})
    with pytest.raises(ValueError, match="Yk"):
        rmm.rmm_qkv_rope(q, q, v, Q, Kt, V, **ok)
    with pytest.raises(ValueError, match="batch"):
        rmm.rmm_qkv_rope(q, k, v, Q, Kt[:1], V[:1], **ok)
    with pytest.raises(ValueError, match="contiguous"):
        rmm.rmm_attn_tree(Q, Kt.transpose(2, 3), V.transpose(2, 3), i32(B), 0.5)
    for bad in (dict(O=bf(B, Hq, T + 1, d)), dict(idx_out=i32(B, Hkv, 63)), dict(parents=i32(T))):
        with pytest.raises(ValueError):
            rmm.rmm_attn_tree(Q, Kt, V, i32(B), 0.5, **bad)
    X = bf(4, 100)
    for bad in (X.float(), X.t(), bf(4), X[:, ::2]):
        with pytest.raises(ValueError):
            rmm.rmm_softmax(bad)
    with pytest.raises(ValueError, match="expected"):
        rmm.rmm_softmax(X, Y=torch.zeros(4, 99))
    with pytest.raises(ValueError, match="overlapping"):
        rmm.rmm_softmax(bf(100).expand(4, 100))
    P, u = torch.zeros(B, T, 50), torch.zeros(B, T)
    for a in ((P[:, :2], i32(B, T), i32(B, T), u), (P, i32(B, T), i32(B, T + 1), u), (P.double(), i32(B, T), i32(B, T), u),
              (P, i32(B, T), i32(B, T), u.double()), (P, i32(B * T), i32(B, T), u)):
        with pytest.raises(ValueError):
            rmm.rmm_tree_verify(*a)
    with pytest.raises(ValueError):
        rmm.rmm_tree_verify(P, i32(B, T), i32(B, T), u, Qd=P[..., :49])
    with pytest.raises(ValueError, match="no cache"):
        rmm.rmm_cache_keep([], i32(B), i32(B, T), i32(B))
    with pytest.raises(ValueError):
        rmm.rmm_cache_keep([(Kt, V), (Kt[:1], V[:1])], i32(B), i32(B, T), i32(B))
    with pytest.raises(ValueError):
        rmm.rmm_cache_keep([(Kt, V)], i32(B), i32(B + 1, T), i32(B))
