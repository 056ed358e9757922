"""Draft-tree decoding in 64 bits, one sequence and one node at a time, from the formulas
in include/rmm.h (no code of the library)."""
import math

import torch

D = 128


def way(parents, t):
    """Node t and its ancestors, nothing when it is absent or below an absent node."""
    out = [t]
    while parents[out[-1]] != -1:
        up = parents[out[-1]]
        if not 0 <= up < out[-1]:
            return []
        out.append(up)
    return out


def ways(parents, b, T):
    if parents is None:
        return [list(range(t + 1)) for t in range(T)]
    p = parents[b].tolist()
    return [way(p, t) for t in range(T)]


def random_trees(B, T, seed, fan=4, padded=True, roots=False):
    """Random parents [B, T]; `padded`: some nodes absent (-2 at the tail, one in the middle);
    `roots`: some more nodes are roots."""
    g = torch.Generator().manual_seed(seed)
    p = torch.empty(B, T, dtype=torch.int32)
    for b in range(B):
        for t in range(T):
            p[b, t] = -1 if t == 0 else int(torch.randint(max(0, t - fan), t, (1,), generator=g))
        if roots and T > 3:
            p[b, T // 2] = -1
        if padded and b % 2 == 1 and T > 2:
            p[b, T - T // 4 - 1:] = -2
            if T > 8:
                p[b, 4] = 77  # neither a node nor a root: absent, and all below it
    return p


def qkv_rope(Yq, Yk, Yv, Q, Kt, V, lens, parents, q_norm, k_norm, eps, inv_freq, interleaved):
    """(Q, Kt, V) after the call as fp64 copies, and the size of the rotated pair behind each
    q and k element (0 where nothing is written)."""
    B, Hq, T, d = Q.shape
    Hkv, ldL = Kt.shape[1], Kt.shape[3]
    Q, Kt, V = Q.double().clone(), Kt.double().clone(), V.double().clone()
    Mq, Mk = torch.zeros_like(Q), torch.zeros_like(Kt)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    for b in range(B):
        start = int(lens[b])
        if start < 0 or start > ldL - T:
            continue
        for t, w in enumerate(ways(parents, b, T) if T <= 64 or parents is not None else [[0] * (t + 1) for t in range(T)]):
            if not w:
                continue
            pos = start + len(w) - 1
            for Y, H, nw, kind in ((Yq, Hq, q_norm, "q"), (Yk, Hkv, k_norm, "k"), (Yv, Hkv, None, "v")):
                x = Y[b * T + t].view(H, d).double().clone()
                if nw is not None:
                    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * nw.double()
                m = x.abs().clone()
                if rot and kind != "v":
                    p = torch.arange(rot // 2)
                    i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
                    a = pos * inv_freq.double()
                    c, s = torch.cos(a), torch.sin(a)
                    u, v = x[:, i].clone(), x[:, j].clone()
                    x[:, i], x[:, j] = u * c - v * s, v * c + u * s
                    m[:, i] = m[:, j] = torch.hypot(u, v)
                if kind == "q":
                    Q[b, :, t], Mq[b, :, t] = x, m
                elif kind == "k":
                    Kt[b, :, :, start + t], Mk[b, :, :, start + t] = x, m
                else:
                    V[b, :, start + t] = x
    return Q, Kt, V, Mq, Mk


def attn_tree(Q, Kt, V, lens, parents, r, scale=None):
    """(O, kept sets or -1, A, X): A the outputs with |v| in v's place, X the largest
    scale * sum |q_j k_j| of the row (what the tolerances need)."""
    B, Hq, T, d = Q.shape
    Hkv, ldL = Kt.shape[1], Kt.shape[3]
    G, k = Hq // Hkv, max(1, math.ceil(r * d))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    O = torch.zeros(B, Hq, T, d, dtype=torch.float64)
    A, X = torch.zeros_like(O), torch.zeros(B, Hq, T, dtype=torch.float64)
    idx = torch.full((B, Hkv, k), -1, dtype=torch.int32)
    for b in range(B):
        n = int(lens[b])
        if n < 0 or n > ldL - T:
            continue
        ws = ways(parents, b, T)
        there = [t for t in range(T) if ws[t]]
        for g in range(Hkv):
            q = Q[b, g * G:(g + 1) * G].double()
            s = q[:, there].abs().amax((0, 1)) if there else torch.zeros(d)
            dims = sorted(sorted(range(d), key=lambda j: (-float(s[j]), j))[:k])
            idx[b, g] = torch.tensor(dims, dtype=torch.int32)
            for t in there:
                keys = list(range(n)) + sorted(n + a for a in ws[t])
                kk, vv = Kt[b, g][dims][:, keys].double(), V[b, g, keys].double()
                x = q[:, t, dims] @ kk * scale
                p = torch.softmax(x, -1)
                O[b, g * G:(g + 1) * G, t] = p @ vv
                A[b, g * G:(g + 1) * G, t] = p @ vv.abs()
                X[b, g * G:(g + 1) * G, t] = (q[:, t, dims].abs() @ kk.abs() * scale).amax(-1)
    return O, idx, A, X


def verify(P, tokens, parents, u, Qd=None):
    """path, emitted, count per sequence by the rule in the header, a sequence at a time."""
    B, T, V = P.shape
    path, emitted = torch.full((B, T), -1, dtype=torch.int32), torch.full((B, T), -1, dtype=torch.int32)
    count = torch.zeros(B, dtype=torch.int32)

    def clean(x):
        x = x.double()
        return torch.where(x > 0, x, 0.0)

    for b in range(B):
        par, tok, uu = parents[b].tolist(), tokens[b].tolist(), u[b].double().tolist()
        if par[0] != -1:
            continue
        v, R, Z, taken = 0, clean(P[b, 0]), 1.0, [0]
        for c in range(1, T):
            x = tok[c]
            if par[c] != v or not 0 <= x < V:
                continue
            q = clean(Qd[b, v]) if Qd is not None else None
            if uu[c] * (1.0 if q is None else float(q[x])) * Z < float(R[x]):
                v, R, Z = c, clean(P[b, c]), 1.0
                taken.append(c)
                continue
            if q is None:
                rest = R.clone()
                rest[x] = 0.0
            else:
                rest = torch.clamp(R - Z * q, min=0.0)
            if float(rest.sum()) > 0.0:
                R, Z = rest, float(rest.sum())
        run = torch.cumsum(R, 0)
        if float(run[-1]) > 0.0:
            goal = (uu[0] if uu[0] > 0.0 else 0.0) * float(run[-1])  # NaN counts as 0
            over = torch.nonzero((run > goal) & (R > 0))
            nxt = int(over[0]) if len(over) else int(torch.nonzero(R > 0)[-1])
        else:
            nxt = -1
        path[b, :len(taken)] = torch.tensor(taken, dtype=torch.int32)
        emitted[b, :len(taken)] = torch.tensor([tok[c] for c in taken[1:]] + [nxt], dtype=torch.int32)
        count[b] = len(taken)
    return path, emitted, count


def keep(Kt, V, lens, path, count):
    """(Kt, V, lens) after the call."""
    B, T = path.shape
    ldL = Kt.shape[-1]
    K2, V2, L2 = Kt.clone(), V.clone(), lens.clone()
    for b in range(B):
        n, L = int(count[b]), int(lens[b])
        p = path[b, :max(n, 0)].tolist()
        if not 1 <= n <= T or L < 0 or L > ldL - T or any(not 0 <= x < T for x in p) or p != sorted(set(p)):
            continue
        for i, x in enumerate(p):
            K2[b, :, :, L + i] = Kt[b, :, :, L + x]
            V2[b, :, L + i] = V[b, :, L + x]
        L2[b] = L + n
    return K2, V2, L2
