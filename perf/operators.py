"""The operators of one draft-tree decode step, as they are measured.

A step scores a small tree of drafted tokens in one forward pass and keeps the branch
that the target model agrees with:

  qkv      per-head RMS norms of q and k with the position rotation, laid out as heads and
           appended to the key/value caches at each sequence's own length
  attn     reduced attention of the tree's nodes over the cache and their own ancestors
  softmax  the logits' rows as probabilities at a temperature
  verify   drafted tokens accepted or rejected from given random numbers, and the next token
  keep     the accepted nodes' keys and values moved to the front of the tree's slots

`run` computes them in elementary torch operations, or, where `own` is true, through the
library's binding.
"""
import math

import torch

own = False

D = 128  # head dimension of the library's caches


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token for each of 64 sequences: the smallest append of a serving step
        dict(name="qkv decode 64x1", op="qkv", B=64, T=1, Hq=32, Hkv=8, lo=100, hi=4000, ldL=4096, norm=True, rot=128,
             interleaved=False, tree=False),
        # a prefill chunk of 4096 tokens at the 64/8-head configuration
        dict(name="qkv prefill 4096", op="qkv", B=1, T=4096, Hq=64, Hkv=8, lo=1001, hi=1001, ldL=8192, norm=True,
             rot=128, interleaved=False, tree=False),
        # one sequence, a short context: the latency of a call
        dict(name="attn tree 16, 1 x 2k", op="attn", B=1, T=16, Hq=32, Hkv=8, lo=2029, hi=2029, ldL=2048, r=0.5,
             tree=True),
        # plain decoding of a ragged batch, every head dimension kept
        dict(name="attn decode, 32 x 8k", op="attn", B=32, T=1, Hq=32, Hkv=8, lo=700, hi=8100, ldL=8192, r=1.0,
             tree=False),
        # a ragged batch of padded trees, half of the head dimensions kept
        dict(name="attn tree 25, 8 x 16k", op="attn", B=8, T=25, Hq=32, Hkv=8, lo=3001, hi=16001, ldL=16384, r=0.5,
             tree=True),
        # the largest: wide trees over long contexts at the 64/8-head configuration
        dict(name="attn tree 64, 4 x 32k", op="attn", B=4, T=64, Hq=64, Hkv=8, lo=29999, hi=32700, ldL=32768, r=1.0,
             tree=True),
        # the draft model's own sampling: one row of a small vocabulary
        dict(name="softmax 1 x 32000", op="softmax", rows=1, V=32000, temperature=0.7),
        # the target's rows of 16 trees of 32 nodes
        dict(name="softmax 512 x 131072", op="softmax", rows=512, V=131072, temperature=1.0),
        # one sequence with a chain of drafts
        dict(name="verify chain 8, 1 x 32000", op="verify", B=1, T=8, V=32000, draft=True, fan=1, noise=0.5),
        # a batch of trees with several drafts drawn at every node
        dict(name="verify tree 32, 16 x 131072", op="verify", B=16, T=32, V=131072, draft=True, fan=4, noise=1.0),
        # one layer's cache after one sequence's chain
        dict(name="keep 8, 1 cache", op="keep", B=1, T=8, Hkv=8, caches=1, ldL=2048),
        # every layer's cache of a batch after wide trees
        dict(name="keep 64, 16 caches", op="keep", B=16, T=64, Hkv=8, caches=16, ldL=1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["qkv", "attn", "attn", "softmax", "verify", "keep"])
    if op == "qkv":
        T = _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, max(1, min(64, 4096 // T)))
        Hkv = rng.choice([1, 2, 4, 8])
        hi = _log_int(rng, 1, 8000)
        return dict(op=op, B=B, T=T, Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 8]), lo=rng.randint(0, hi), hi=hi,
                    ldL=(hi + T + 7 + 8 * rng.randint(0, 20)) // 8 * 8, norm=rng.random() < 0.7,
                    rot=rng.choice([128, 128, 64, 32]), interleaved=rng.random() < 0.4,
                    tree=T <= 64 and rng.random() < 0.7)
    if op == "attn":
        T = _log_int(rng, 1, 64)
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 5, 8])
        B = _log_int(rng, 1, 32)
        # no more than the largest listed case's keys and products
        most = min(4 * 8 * 32768 // (B * Hkv), 4 * 8 * 32768 * 512 // (B * Hkv * G * T))
        hi = _log_int(rng, 1, max(1, min(32700, most - T - 8)))
        return dict(op=op, B=B, T=T, Hkv=Hkv, Hq=Hkv * G, lo=rng.randint(0, hi), hi=hi,
                    ldL=(hi + T + 7 + 8 * rng.randint(0, 20)) // 8 * 8, r=rng.choice([0.125, 0.3, 0.5, 0.75, 1.0, 1.0]),
                    tree=rng.random() < 0.8)
    if op == "softmax":
        return dict(op=op, rows=_log_int(rng, 1, 512), V=_log_int(rng, 500, 131072),
                    temperature=rng.choice([1.0, 0.7, 1.3, 0.25]))
    if op == "verify":
        T = _log_int(rng, 1, 64)
        return dict(op=op, B=_log_int(rng, 1, max(1, 512 // T)), T=T, V=_log_int(rng, 500, 131072),
                    draft=rng.random() < 0.6, fan=rng.choice([1, 2, 4, 8]), noise=rng.choice([0.3, 1.0, 2.0]))
    T = _log_int(rng, 1, 64)
    B = _log_int(rng, 1, 16)
    return dict(op=op, B=B, T=T, Hkv=rng.choice([1, 2, 4, 8]), caches=_log_int(rng, 1, 16),
                ldL=8 * rng.randint(max(9, (T + 15) // 8), 128))


# ---------------------------------------------------------------- inputs

def _lens(c):
    """Each sequence's cache length: spread over [lo, hi], the longest at the end."""
    return [c["hi"] if b == c["B"] - 1 else c["lo"] + int((c["hi"] - c["lo"]) * ((b * 0.6180339887) % 1.0))
            for b in range(c["B"])]


def _kept(c):
    """How many nodes of each sequence are kept (the root among them): 1 .. about T / 2 + 1."""
    return [1 + (3 + 5 * b) % (c["T"] // 2 + 1) for b in range(c["B"])]


def _trees(c, g, dev, fan=8):
    """Random trees, parent before child: node t hangs on one of the `fan` nodes before it.
    A batch is padded to its widest tree: every third sequence has fewer nodes (parent -2)."""
    B, T = c["B"], c["T"]
    t = torch.arange(T, device=dev)
    back = 1 + (torch.rand(B, T, device=dev, generator=g) * torch.clamp(t, max=fan)).long().clamp(max=max(fan - 1, 0))
    parents = torch.where(t == 0, -1, t - torch.minimum(back, t))
    nodes = torch.where(torch.arange(B, device=dev) % 3 == 1, (3 * T + 3) // 4, T)
    return torch.where(t < nodes[:, None], parents, -2).int().contiguous()


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.empty(*shape, dtype=dtype, device=dev).normal_(0.0, std, generator=g)

    s = dict(c)
    op = c["op"]
    if op in ("qkv", "attn"):
        B, T, Hq, Hkv, ldL = c["B"], c["T"], c["Hq"], c["Hkv"], c["ldL"]
        s["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device=dev)
        s["parents"] = _trees(c, g, dev) if c["tree"] else None
        s["Kt"] = normal(B, Hkv, D, ldL)
        s["V"] = normal(B, Hkv, ldL, D)
    if op == "qkv":
        for n, h in (("yq", Hq), ("yk", Hkv), ("yv", Hkv)):
            s[n] = normal(B * T, h * D, std=2.0)
        s["qn"] = (1.0 + 0.2 * normal(D, dtype=torch.float32)).bfloat16() if c["norm"] else None
        s["kn"] = (1.0 + 0.2 * normal(D, dtype=torch.float32)).bfloat16() if c["norm"] else None
        s["inv_freq"] = 1.0 / 500000.0 ** (torch.arange(0, c["rot"], 2, device=dev, dtype=torch.float32) / c["rot"])
        s["Q"] = torch.zeros(B, Hq, T, D, dtype=torch.bfloat16, device=dev)
    if op == "attn":
        # a few head dimensions are far larger than the others, as rotated queries have them
        s["Q"] = (normal(B, Hq, T, D, dtype=torch.float32) * torch.exp(0.6 * normal(D, dtype=torch.float32))).bfloat16()
        s["O"] = torch.zeros(B, Hq, T, D, dtype=torch.bfloat16, device=dev)
        s["idx"] = torch.full((B, Hkv, math.ceil(c["r"] * D)), -1, dtype=torch.int32, device=dev)
    if op == "softmax":
        s["X"] = normal(c["rows"], c["V"], std=3.0)
        s["Y"] = torch.empty(c["rows"], c["V"], dtype=torch.float32, device=dev)
    if op == "verify":
        B, T, V = c["B"], c["T"], c["V"]
        s["parents"] = _trees(c, g, dev, fan=c["fan"])
        a = normal(B, T, V, dtype=torch.float32, std=3.0)
        s["P"] = torch.softmax(a, -1)
        # the draft model agrees with the target up to some noise; each node's token is drawn
        # from the draft's row of its parent (the same rows stand in for a draft of greedy picks)
        q = torch.softmax(a.add_(normal(B, T, V, dtype=torch.float32, std=c["noise"])), -1)
        del a
        up = s["parents"].long().clamp(min=0)
        cdf = torch.cumsum(q, -1)
        pick = torch.rand(B, T, 1, device=dev, generator=g) * torch.gather(cdf[..., -1], 1, up)[..., None]
        rows = (torch.arange(B, device=dev)[:, None] * T + up).reshape(-1)
        tok = torch.searchsorted(cdf.reshape(B * T, V)[rows], pick.reshape(-1, 1), right=True)
        s["tokens"] = tok.clamp(max=V - 1).int().reshape(B, T).contiguous()
        s["u"] = torch.rand(B, T, device=dev, generator=g)
        s["Qd"] = q if c["draft"] else None
        s["path"], s["emitted"] = (torch.empty(B, T, dtype=torch.int32, device=dev) for _ in range(2))
        s["count"] = torch.empty(B, dtype=torch.int32, device=dev)
    if op == "keep":
        B, T, Hkv, n, ldL = c["B"], c["T"], c["Hkv"], c["caches"], c["ldL"]
        s["Kt"] = normal(n, B, Hkv, D, ldL)
        s["V"] = normal(n, B, Hkv, ldL, D)
        s["lens"] = torch.randint(0, ldL - T + 1, (B,), device=dev, generator=g).int()
        # the accepted nodes: the root and a random choice of later ones, in order
        count = torch.tensor(_kept(c), dtype=torch.int32, device=dev)
        rank = torch.rand(B, T, device=dev, generator=g)
        rank[:, 0] = -1.0
        place = torch.argsort(torch.argsort(rank, 1), 1)
        i = torch.arange(T, device=dev)
        chosen = torch.where(place < count[:, None], i, T + i)
        path = torch.sort(chosen, 1).values
        s["path"] = torch.where(path < T, path, -1).int().contiguous()
        s["count"] = count
        s["lens_out"] = torch.zeros_like(s["lens"])
        s["layers"] = [(s["Kt"][l], s["V"][l]) for l in range(n)]
    return s


# ---------------------------------------------------------------- plain forms

def _ancestors(parents):
    """[B, T, T]: node t has node a on its way to the root (itself among them); no row for a
    node that is absent or hangs on an absent one."""
    B, T = parents.shape
    t = torch.arange(T, device=parents.device)
    up = (parents[..., None] == t).float()
    way = torch.eye(T, device=parents.device) + up
    for _ in range(6):  # trees of up to 64 nodes
        way = (way @ way > 0).float()
    way = way > 0
    rooted = (way & (parents == -1)[:, None, :]).any(-1)
    return way & rooted[..., None]


def _chain(B, T, dev):
    return torch.ones(T, T, dtype=torch.bool, device=dev).tril().expand(B, T, T)


def _plain_qkv(s):
    B, T, Hq, Hkv, rot = s["B"], s["T"], s["Hq"], s["Hkv"], s["rot"]
    dev = s["yq"].device
    way = _chain(B, T, dev) if s["parents"] is None else _ancestors(s["parents"])
    start = s["lens"].long()
    pos = start[:, None] + way.sum(-1) - 1
    ang = pos.double()[..., None] * s["inv_freq"].double()
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]  # [B, 1, T, rot / 2]

    def heads(y, H, w):
        x = y.view(B, T, H, D).transpose(1, 2).float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        if s["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((turned, x[..., rot:]), -1).bfloat16()

    q, k = heads(s["yq"], Hq, s["qn"]), heads(s["yk"], Hkv, s["kn"])
    v = s["yv"].view(B, T, Hkv, D)
    there = way.any(-1)  # [B, T]
    s["Q"].copy_(torch.where(there[:, None, :, None], q, s["Q"]))
    b, t = there.nonzero(as_tuple=True)
    slot = start[b] + t
    s["Kt"][b, :, :, slot] = k.transpose(1, 2)[b, t]
    s["V"][b, :, slot] = v[b, t]
    return s["Q"], s["Kt"], s["V"]


def _plain_attn(s):
    B, T, Hq, Hkv, ldL = s["B"], s["T"], s["Hq"], s["Hkv"], s["ldL"]
    dev = s["Q"].device
    way = _chain(B, T, dev) if s["parents"] is None else _ancestors(s["parents"])
    k = math.ceil(s["r"] * D)
    q = s["Q"].float().view(B, Hkv, Hq // Hkv, T, D)
    # the kept head dimensions: largest |q| of the set's present rows, ties to the lower index
    there = way.any(-1)
    score = torch.where(there[:, None, None, :, None], q.abs(), 0.0).amax((2, 3))
    idx = torch.sort(torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k], -1).values
    keep = torch.zeros_like(score).scatter_(-1, idx, 1.0)
    logit = (q * keep[:, :, None, None]).reshape(B, Hkv, -1, D) @ s["Kt"].float() * (1.0 / math.sqrt(D))
    # node t sees the cache below the sequence's length, and its own way through the tree's slots
    at = torch.arange(ldL, device=dev) - s["lens"].long()[:, None]  # [B, ldL]: slot of the tree, negative in the cache
    slot = at.clamp(0, T - 1)[:, None, :].expand(B, T, ldL)
    sees = (at < 0)[:, None, :] & there[..., None] | ((at >= 0) & (at < T))[:, None, :] & torch.gather(way, 2, slot)
    logit = torch.where(sees[:, None, None], logit.view(B, Hkv, -1, T, ldL), -math.inf)
    top = logit.amax(-1, keepdim=True)
    e = torch.exp(logit - torch.where(top > -math.inf, top, 0.0))
    total = e.sum(-1, keepdim=True)
    o = (e.view(B, Hkv, -1, ldL) @ s["V"].float()).view(B, Hkv, -1, T, D)
    o = torch.where(total > 0, o / total, 0.0)
    return o.reshape(B, Hq, T, D).bfloat16(), idx.int()


def _plain_softmax(s):
    x = s["X"].float() / s["temperature"]
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_verify(s):
    """In 64 bits: a token changes where a running sum passes a random number."""
    P, tokens, parents, u, Qd = s["P"], s["tokens"].long(), s["parents"], s["u"].double(), s["Qd"]
    B, T, V = P.shape
    b = torch.arange(B, device=P.device)
    t = torch.arange(T, device=P.device)
    at = torch.zeros(B, dtype=torch.long, device=P.device)  # the last accepted node
    left, mass = P[:, 0].double(), torch.ones(B, dtype=torch.float64, device=P.device)
    took = [torch.ones(B, dtype=torch.bool, device=P.device)]
    for n in range(1, T):  # a node comes after its parent and its earlier siblings
        child = parents[:, n] == at
        x = tokens[:, n]
        draft = torch.zeros_like(left).scatter_(1, x[:, None], 1.0) if Qd is None else Qd[b, at].double()
        yes = child & (u[:, n] * draft[b, x] * mass < left[b, x])
        no = child & ~yes
        # what a rejection leaves: the part of the target's row above the draft's
        rest = (left - mass[:, None] * draft).clamp(min=0) if Qd is not None else left * (1.0 - draft)
        total = rest.sum(-1)
        no = no & (total > 0)
        left = torch.where(yes[:, None], P[:, n].double(), torch.where(no[:, None], rest, left))
        mass = torch.where(yes, 1.0, torch.where(no, total, mass))
        at = torch.where(yes, n, at)
        took.append(yes)
    took = torch.stack(took, 1)
    count = took.sum(1)
    order = torch.sort(torch.where(took, t, T + t), 1).values
    path = torch.where(order < T, order, -1)
    run = torch.cumsum(left, -1)
    nxt = torch.searchsorted(run, (u[:, :1] * run[:, -1:]).contiguous(), right=True)[:, 0]
    drafted = torch.gather(tokens, 1, torch.roll(path, -1, 1).clamp(min=0))
    said = torch.where(t < count[:, None] - 1, drafted, torch.where(t == count[:, None] - 1, nxt[:, None], -1))
    return path.int(), said.int(), count.int()


def _plain_keep(s):
    B, T = s["B"], s["T"]
    b, i = (torch.arange(T, device=s["lens"].device) < s["count"][:, None]).nonzero(as_tuple=True)
    src = (s["lens"][b] + s["path"][b, i]).long()
    dst = (s["lens"][b] + i).long()
    s["Kt"][:, b, :, :, dst] = s["Kt"][:, b, :, :, src]
    s["V"][:, b, :, dst] = s["V"][:, b, :, src]
    return s["Kt"], s["V"], s["lens"] + s["count"]


# ---------------------------------------------------------------- one pass

def run(s):
    if not own:
        plain = dict(qkv=_plain_qkv, attn=_plain_attn, softmax=_plain_softmax, verify=_plain_verify, keep=_plain_keep)
        return plain[s["op"]](s)
    from input_adaptive_reduced_rmm_b200 import rmm

    op = s["op"]
    if op == "qkv":
        rmm.rmm_qkv_rope(s["yq"], s["yk"], s["yv"], s["Q"], s["Kt"], s["V"], lens=s["lens"], parents=s["parents"],
                         q_norm=s["qn"], k_norm=s["kn"], eps=1e-6, inv_freq=s["inv_freq"],
                         interleaved=s["interleaved"])
        return s["Q"], s["Kt"], s["V"]
    if op == "attn":
        if "ws" not in s:  # kept by the program, as a decoder layer keeps it
            s["ws"] = rmm.new_workspace(rmm.rmm_attn_tree_workspace_bytes(s["B"], s["Hq"], s["Hkv"], s["T"], s["ldL"]))
        rmm.rmm_attn_tree(s["Q"], s["Kt"], s["V"], s["lens"], s["r"], parents=s["parents"], O=s["O"], idx_out=s["idx"],
                          workspace=s["ws"])
        return s["O"], s["idx"]
    if op == "softmax":
        return rmm.rmm_softmax(s["X"], s["temperature"], Y=s["Y"])
    if op == "verify":
        return rmm.rmm_tree_verify(s["P"], s["tokens"], s["parents"], s["u"], Qd=s["Qd"], path=s["path"],
                                   emitted=s["emitted"], count=s["count"])
    rmm.rmm_cache_keep(s["layers"], s["lens"], s["path"], s["count"], lens_out=s["lens_out"])
    return s["Kt"], s["V"], s["lens_out"]


# ---------------------------------------------------------------- what a pass cannot do without

def work(c):
    op = c["op"]
    if op == "qkv":  # q, k, v read once and written once
        n = c["B"] * c["T"] * D
        return dict(bytes=2 * 2 * n * (c["Hq"] + 2 * c["Hkv"]), flops=8 * n * (c["Hq"] + c["Hkv"]))
    if op == "attn":  # the kept rows of K^T and all of V below each length, queries in, outputs out
        k = math.ceil(c["r"] * D)
        keys = sum(n + c["T"] for n in _lens(c))
        rows = c["B"] * c["Hq"] * c["T"]
        return dict(bytes=2 * keys * c["Hkv"] * (k + D) + 4 * rows * D, flops=2 * keys * c["Hq"] * c["T"] * (k + D))
    if op == "softmax":  # bf16 in, fp32 out
        return dict(bytes=6 * c["rows"] * c["V"], flops=5 * c["rows"] * c["V"])
    if op == "verify":  # the row each sequence's next token is drawn from, and the draft's beside it
        rows = c["B"] * (2 if c["draft"] else 1)
        return dict(bytes=4 * rows * c["V"] + 16 * c["B"] * c["T"], flops=3 * rows * c["V"])
    moved = sum(n - 1 for n in _kept(c)) * c["caches"] * c["Hkv"] * D
    return dict(bytes=2 * 2 * 2 * moved + 8 * c["B"] * c["T"], flops=c["B"] * c["T"])


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _walk(parents, t):
    """Node t's way to its root, or nothing where it meets an absent node."""
    way = [t]
    while parents[way[-1]] != -1:
        up = parents[way[-1]]
        if not 0 <= up < way[-1]:
            return []
        way.append(up)
    return way


def _ways(s, b):
    T = s["T"]
    if s["parents"] is None:
        return [list(range(t + 1)) for t in range(T)]
    parents = s["parents"][b].tolist()
    return [_walk(parents, t) for t in range(T)]


def exact(c, seed):
    s = prepare(c, seed)
    return dict(qkv=_exact_qkv, attn=_exact_attn, softmax=_exact_softmax, verify=_exact_verify,
                keep=_exact_keep)[c["op"]](s)


def _exact_qkv(s):
    B, T, rot = s["B"], s["T"], s["rot"]
    Q, Kt, V = s["Q"].double(), s["Kt"].double(), s["V"].double()
    for b in range(B):
        if T <= 64:
            ways = _ways(s, b)
            there = [t for t in range(T) if ways[t]]
            depth = [len(ways[t]) - 1 for t in there]
        else:
            there = depth = list(range(T))
        L0 = int(s["lens"][b])
        rows = torch.tensor(there, device=Q.device)
        pos = torch.tensor(depth, device=Q.device, dtype=torch.float64) + L0
        turn = torch.polar(torch.ones(1, dtype=torch.float64, device=Q.device), pos[:, None] * s["inv_freq"].double())
        for name, w, H in (("yq", s["qn"], s["Hq"]), ("yk", s["kn"], s["Hkv"]), ("yv", None, s["Hkv"])):
            x = s[name].view(B, T, H, D)[b, rows].double()  # [n, H, D]
            if w is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
            if name != "yv":
                if s["interleaved"]:
                    z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * turn[:, None]
                    x[..., 0:rot:2], x[..., 1:rot:2] = z.real, z.imag
                else:
                    z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn[:, None]
                    x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
            if name == "yq":
                Q[b, :, rows] = x.transpose(0, 1)
            elif name == "yk":
                Kt[b, :, :, L0 + rows] = x.permute(1, 2, 0)
            else:
                V[b, :, L0 + rows] = x.transpose(0, 1)
    return Q, Kt, V


def _exact_attn(s):
    B, T, Hq, Hkv = s["B"], s["T"], s["Hq"], s["Hkv"]
    G, k, dev = Hq // Hkv, math.ceil(s["r"] * D), s["Q"].device
    O = torch.zeros(B, Hq, T, D, dtype=torch.float64, device=dev)
    idx = torch.full((B, Hkv, k), -1, dtype=torch.int32, device=dev)
    for b in range(B):
        ways, n = _ways(s, b), int(s["lens"][b])
        there = [t for t in range(T) if ways[t]]
        own_keys = torch.full((T, T), -math.inf, dtype=torch.float64)
        for t in there:
            own_keys[t, ways[t]] = 0.0
        own_keys = own_keys.to(dev)[there]
        for g in range(Hkv):
            q = s["Q"][b, g * G:(g + 1) * G][:, there].double()  # [G, n, D]
            big = q.abs().amax((0, 1)).tolist()
            dims = sorted(sorted(range(D), key=lambda j: (-big[j], j))[:k])
            idx[b, g] = torch.tensor(dims, dtype=torch.int32, device=dev)
            x = q[..., dims] @ s["Kt"][b, g, dims, :n + T].double() / math.sqrt(D)
            x[..., n:] += own_keys
            O[b, g * G:(g + 1) * G, there] = torch.softmax(x, -1) @ s["V"][b, g, :n + T].double()
    return O, idx


def _exact_softmax(s):
    return torch.exp(torch.log_softmax(s["X"].double() / s["temperature"], -1))


def _exact_verify(s):
    B, T, V = s["P"].shape
    path, said, count = (torch.full(n, -1, dtype=torch.int32) for n in ((B, T), (B, T), (B,)))
    for b in range(B):
        parents, tokens, u = s["parents"][b].tolist(), s["tokens"][b].tolist(), s["u"][b].double().tolist()
        way, left, n = [0], s["P"][b, 0].double(), 1
        left_mass = 1.0
        while n < T:
            if parents[n] == way[-1]:
                q = s["Qd"][b, way[-1]].double() if s["Qd"] is not None else None
                like = 1.0 if q is None else float(q[tokens[n]])
                if u[n] * like * left_mass < float(left[tokens[n]]):
                    way.append(n)
                    left, left_mass = s["P"][b, n].double(), 1.0
                else:
                    rest = left.clone()
                    if q is None:
                        rest[tokens[n]] = 0.0
                    else:
                        rest = (rest - left_mass * q).clamp(min=0.0)
                    if float(rest.sum()) > 0.0:
                        left, left_mass = rest, float(rest.sum())
            n += 1
        run_ = left.cumsum(0)
        nxt = int((run_ <= u[0] * float(run_[-1])).sum())
        path[b, :len(way)] = torch.tensor(way, dtype=torch.int32)
        said[b, :len(way)] = torch.tensor([tokens[w] for w in way[1:]] + [nxt], dtype=torch.int32)
        count[b] = len(way)
    return path, said, count


def _exact_keep(s):
    Kt, V, lens = s["Kt"].clone(), s["V"].clone(), s["lens"].tolist()
    for b, n in enumerate(s["count"].tolist()):
        for i, p in enumerate(s["path"][b].tolist()[:n]):
            Kt[:, b, :, :, lens[b] + i] = s["Kt"][:, b, :, :, lens[b] + p]
            V[:, b, :, lens[b] + i] = s["V"][:, b, :, lens[b] + p]
    return Kt.double(), V.double(), s["lens"] + s["count"]
