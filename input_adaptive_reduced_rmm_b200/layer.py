"""One Llama-style decoder layer built on the reduced products (batch 1).

    x -> RMSNorm -> q, k, v (one kept set: they share their input)
      -> heads + KV-cache append -> reduced attention (head-dim sets) -> o
      -> residual add + RMSNorm -> gate, up (one kept set) -> SwiGLU -> down
      -> residual add
(without a trace, SwiGLU is applied as gate and up are produced)

The anatomy (RMSNorm, a residual stream through every block, a SwiGLU MLP)
follows the 'Numerical Linear Algebra for LLMs' paper digest (ai-feeds.com),
section 'Method: key modules'; the reduced products and the reduced QK^T
follow the reduced-matrix-multiplication pages (input-adaptive slices of the
contraction dimension kept at ratio r).  The norm weights of the blocks are 1;
per-head norms of q and k and the rotation by position are applied where their
weights and frequencies are given.  Every op runs in this package's kernels through the C ABI;
this module only sequences the calls and owns the buffers (PyTorch device
memory).  Intermediates are bf16 between ops.

Decoding with drafts: forward_tree scores a tree of drafted tokens behind the
cache, decode_tree runs it through a stack of layers and an output head, keeps
the branch that the model agrees with and drops the rest of the tree.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import rmm

D_HEAD = 128


@dataclass
class LayerDims:
    H: int = 4096        # hidden size
    Hq: int = 32         # query heads
    Hkv: int = 8         # key/value heads
    F: int = 14336       # MLP width
    eps: float = 1e-5

    @property
    def q_cols(self) -> int:
        return self.Hq * D_HEAD

    @property
    def kv_cols(self) -> int:
        return self.Hkv * D_HEAD


class DecoderLayer:
    """Weights pre-transposed once (W^T [in, out]); KV caches for max_len tokens.

    q_norm, k_norm (bf16 [128], optional): weights of the RMS norms of each query and key head.
    inv_freq (fp32 [rot/2], optional): the angle per position of each rotated pair of dims, (i, i + rot/2)
    or, interleaved, (2i, 2i + 1)."""

    def __init__(self, dims: LayerDims, weights: dict, max_len: int, r: float, device,
                 q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None,
                 inv_freq: torch.Tensor | None = None, interleaved: bool = False):
        self.d = dims
        self.q_norm, self.k_norm, self.inv_freq = (None if t is None else t.to(device)
                                                   for t in (q_norm, k_norm, inv_freq))
        self.interleaved = bool(interleaved)
        self.r = float(r)
        self.dev = device
        self.Wt = {n: rmm.rmm_transpose_weight(weights[n].to(device)) for n in
                   ("q", "k", "v", "o", "gate", "up", "down")}
        self.ldL = (max_len + 7) // 8 * 8
        self.Kt = torch.zeros(dims.Hkv, D_HEAD, self.ldL, dtype=torch.bfloat16, device=device)
        self.V = torch.zeros(dims.Hkv, self.ldL, D_HEAD, dtype=torch.bfloat16, device=device)
        self.pos = 0
        self._ws = {}
        self._bufs = {}
        self._opts_swiglu = rmm.options(swiglu_pair=True)

    # workspaces and activations are kept per token count, so repeated calls
    # (decode steps) allocate nothing
    def _ws_for(self, key, nbytes):
        w = self._ws.get(key)
        if w is None or w.numel() < nbytes:
            w = rmm.new_workspace(nbytes, self.dev)
            self._ws[key] = w
        return w

    def _buf(self, name, shape):
        key = (name, tuple(shape))
        b = self._bufs.get(key)
        if b is None:
            b = torch.empty(*shape, dtype=torch.bfloat16, device=self.dev)
            self._bufs[key] = b
        return b

    def reset(self):
        self.pos = 0

    def forward(self, x: torch.Tensor, trace: dict | None = None, events: list | None = None) -> torch.Tensor:
        """x [T, H] bf16 at cache positions pos .. pos+T-1 (causal).  Returns the layer output.
        trace (optional) receives every intermediate and kept set; events (optional) receives
        (op name, start event, end event) per op."""
        out = self._run(x, None, None, trace, events)
        self.pos += x.shape[0]
        return out

    def forward_tree(self, x: torch.Tensor, parents: torch.Tensor | None = None, lens: torch.Tensor | None = None,
                     trace: dict | None = None, events: list | None = None) -> torch.Tensor:
        """x [T, H] bf16, the T <= 64 nodes of a tree of drafted tokens: parents int32 [T] (None: a chain) gives
        each node's parent, smaller than its own number, -1 for the root.  A node's position is its depth past
        the cache and it attends to the cache and its own ancestors.  Node t's key and value go to cache slot
        pos + t; pos stays, so the next call overwrites them unless keep_path has moved some to their place.
        lens (int32 [1], optional): pos on the device, where the caller has it."""
        if lens is None:
            lens = torch.full((1,), self.pos, dtype=torch.int32, device=self.dev)
        return self._run(x, lens, parents, trace, events)

    def _run(self, x, lens, parents, trace, events):
        """One pass over the layer: causal rows at pos, or with lens the nodes of a tree behind it."""
        dm, T, r = self.d, x.shape[0], self.r
        L0 = self.pos
        if L0 + T > self.ldL:
            raise ValueError("KV cache full")
        H, F = dm.H, dm.F
        tree = lens is not None
        if parents is not None:
            parents = parents.view(1, -1)
        Kt, V = self.Kt.unsqueeze(0), self.V.unsqueeze(0)

        def op(name):
            if events is None:
                return _NullCtx()
            return _EventCtx(events, name)

        with op("rmsnorm"):
            _, xn = rmm.rmm_add_rmsnorm(x, eps=dm.eps, Y=self._buf("xn", (T, H)))
        idx_qkv = self._idx("qkv", H)
        with op("qkv"):
            yq, yk, yv = self._buf("yq", (T, dm.q_cols)), self._buf("yk", (T, dm.kv_cols)), self._buf("yv", (T, dm.kv_cols))
            rmm.rmm_linear_group(xn, [self.Wt["q"], self.Wt["k"], self.Wt["v"]], r, Ys=[yq, yk, yv],
                                 idx_out=idx_qkv,
                                 workspace=self._ws_for(("qkv", T), rmm.rmm_linear_group_workspace_bytes(
                                     T, H, [dm.q_cols, dm.kv_cols, dm.kv_cols])))
        Q = self._buf("Q", (dm.Hq, T, D_HEAD))
        with op("kv_append"):
            if tree or self.q_norm is not None or self.k_norm is not None or self.inv_freq is not None:
                rmm.rmm_qkv_rope(yq, yk, yv, Q.unsqueeze(0), Kt, V, lens=lens, L0=0 if tree else L0, parents=parents,
                                 q_norm=self.q_norm, k_norm=self.k_norm, eps=dm.eps, inv_freq=self.inv_freq,
                                 interleaved=self.interleaved)
            else:
                rmm.rmm_qkv_heads(yq, yk, yv, Q, self.Kt, self.V, L0)
        L = L0 + T
        idx_attn = torch.empty(1, dm.Hkv, rmm.rmm_k_for(D_HEAD, r), dtype=torch.int32, device=self.dev)
        O = self._buf("O", (1, dm.Hq, T, D_HEAD))
        with op("attention"):
            if tree:
                rmm.rmm_attn_tree(Q.unsqueeze(0), Kt, V, lens, r, parents=parents, O=O, idx_out=idx_attn,
                                  workspace=self._ws_for(("attn_tree", T), rmm.rmm_attn_tree_workspace_bytes(
                                      1, dm.Hq, dm.Hkv, T, self.ldL, D_HEAD)))
            else:
                rmm.rmm_attn_qk(Q.unsqueeze(0), Kt, V, L, r, causal=True, O=O, idx_out=idx_attn,
                                workspace=self._ws_for(("attn", T), rmm.rmm_attn_workspace_bytes(
                                    1, dm.Hq, dm.Hkv, T, self.ldL, D_HEAD)))
        with op("heads_to_tokens"):
            a = rmm.rmm_heads_to_tokens(O[0], A=self._buf("a", (T, dm.q_cols)))
        idx_o = self._idx("o", dm.q_cols)
        with op("o"):
            yo = rmm.rmm_linear(a, self.Wt["o"], r, Y=self._buf("yo", (T, H)), idx_out=idx_o,
                                workspace=self._ws_for(("o", T), rmm.rmm_linear_workspace_bytes(T, dm.q_cols, H)))
        with op("add_rmsnorm"):
            h2, xn2 = rmm.rmm_add_rmsnorm(x, yo, eps=dm.eps, Hsum=self._buf("h2", (T, H)),
                                          Y=self._buf("xn2", (T, H)))
        idx_gu = self._idx("gu", H)
        ws_gu = self._ws_for(("gu", T), rmm.rmm_linear_group_workspace_bytes(T, H, [F, F]))
        g, u = self._buf("g", (T, F)), self._buf("u", (T, F))
        if trace is None:
            # SwiGLU applied as gate/up are produced (folded into the decode GEMV's
            # split sums; after the products on the GEMM path): hh directly, the
            # same bits as the two steps below
            with op("gate_up_swiglu"):
                hh = self._buf("hh", (T, F))
                rmm.rmm_linear_group(xn2, [self.Wt["gate"], self.Wt["up"]], r, Ys=[hh, u], idx_out=idx_gu,
                                     workspace=ws_gu, opts=self._opts_swiglu)
        else:
            with op("gate_up"):
                rmm.rmm_linear_group(xn2, [self.Wt["gate"], self.Wt["up"]], r, Ys=[g, u], idx_out=idx_gu,
                                     workspace=ws_gu)
            with op("swiglu"):
                hh = rmm.rmm_swiglu(g, u, out=self._buf("hh", (T, F)))
        idx_d = self._idx("down", F)
        with op("down"):
            yd = rmm.rmm_linear(hh, self.Wt["down"], r, Y=self._buf("yd", (T, H)), idx_out=idx_d,
                                workspace=self._ws_for(("down", T), rmm.rmm_linear_workspace_bytes(T, F, H)))
        out = torch.empty(T, H, dtype=torch.bfloat16, device=self.dev)
        with op("residual"):
            rmm.rmm_add_rmsnorm(h2, yd, eps=dm.eps, Hsum=out, want_y=False)
        if trace is not None:
            # copies: the activation buffers are reused by the next call
            vals = dict(x=x, xn=xn, yq=yq, yk=yk, yv=yv, Q=Q, L0=L0, L=L, O=O[0], a=a, yo=yo, h2=h2, xn2=xn2,
                        g=g, u=u, hh=hh, yd=yd, out=out, idx_qkv=idx_qkv, idx_attn=idx_attn[0], idx_o=idx_o,
                        idx_gu=idx_gu, idx_down=idx_d, Kt=self.Kt, V=self.V)
            for key, v in vals.items():
                trace[key] = v.clone() if torch.is_tensor(v) else v
        return out

    def _idx(self, name, H):
        return torch.empty(H, dtype=torch.int32, device=self.dev)


class OutputHead:
    """Hidden rows to next-token probabilities: RMSNorm, the product with the output weights [V, H] at ratio r,
    softmax at a temperature.  The rows between are kept per row count, so one head serves one stream at a time."""

    def __init__(self, weight: torch.Tensor, r: float, device, eps: float = 1e-5):
        self.Wt = rmm.rmm_transpose_weight(weight.to(device))
        self.r = float(r)
        self.eps = eps
        self._kept = {}  # row count -> (norm, logits, workspace)

    def probabilities(self, x: torch.Tensor, temperature: float = 1.0) -> torch.Tensor:
        """x [T, H] bf16 -> fp32 [T, V]; temperature 0 is greedy."""
        T, (H, V) = x.shape[0], self.Wt.shape
        if T not in self._kept:
            self._kept[T] = (torch.empty(T, H, dtype=torch.bfloat16, device=x.device),
                             torch.empty(T, V, dtype=torch.bfloat16, device=x.device),
                             rmm.new_workspace(rmm.rmm_linear_workspace_bytes(T, H, V), x.device))
        xn, logits, ws = self._kept[T]
        rmm.rmm_add_rmsnorm(x, eps=self.eps, Y=xn)
        rmm.rmm_linear(xn, self.Wt, self.r, Y=logits, workspace=ws)
        return rmm.rmm_softmax(logits, temperature)


def _common_pos(layers) -> int:
    """How many tokens every layer's cache holds."""
    if any(layer.pos != layers[0].pos for layer in layers):
        raise ValueError("the layers' caches hold different numbers of tokens")
    return layers[0].pos


def keep_path(layers, path: torch.Tensor, count: torch.Tensor, lens: torch.Tensor | None = None) -> int:
    """Keep the nodes path[0, :count[0]] (int32 [1, T], ascending) of the tree that forward_tree scored last, in
    every layer's cache: their keys and values move up to the cache, pos grows by their number, which is returned
    (it is read from the device)."""
    pos = _common_pos(layers)
    if lens is None:
        lens = torch.full((1,), pos, dtype=torch.int32, device=path.device)
    grown = rmm.rmm_cache_keep([(layer.Kt.unsqueeze(0), layer.V.unsqueeze(0)) for layer in layers], lens, path, count)
    n = int(grown) - pos
    for layer in layers:
        layer.pos += n
    return n


def decode_tree(layers, head: OutputHead, embed: torch.Tensor, tokens: torch.Tensor, parents: torch.Tensor,
                u: torch.Tensor, temperature: float = 1.0, Qd: torch.Tensor | None = None,
                trace: dict | None = None) -> list[int]:
    """One step of decoding with drafts.  tokens int32 [T] are the tree's, its root the last token that was emitted
    (its key is not in the cache yet); parents int32 [T] the tree; embed bf16 [V, H] the tokens' rows; u fp32 [T] in
    [0, 1), one random number per node, the root's for the next token; Qd fp32 [T, V] the rows that each node's
    children were drawn from (None: certain picks).  Returns the tokens emitted, one more than the drafts that were
    accepted: the last of them is the next tree's root.  For any draft they are distributed as sampling one token
    at a time from the layers would have them, given the kept sets of this pass."""
    pos = _common_pos(layers)  # before the first layer writes its nodes there
    tokens, parents, u = tokens.view(1, -1), parents.view(1, -1), u.view(1, -1)
    lens = torch.full((1,), pos, dtype=torch.int32, device=tokens.device)
    x = embed.index_select(0, tokens[0].clamp(0, embed.shape[0] - 1))  # other tokens are never accepted
    for layer in layers:
        x = layer.forward_tree(x, parents, lens)
    P = head.probabilities(x, temperature)
    path, emitted, count = rmm.rmm_tree_verify(P, tokens, parents, u, Qd=Qd)
    n = keep_path(layers, path, count, lens)
    if trace is not None:
        trace.update(x=x, P=P, path=path, emitted=emitted, count=count)
    return emitted[0, :n].tolist()


class DenseLayer:
    """The same layer with dense products (cuBLAS through torch.matmul) and dense
    attention (torch scaled_dot_product_attention): the comparison, not the product.
    Like the reduced layer, which runs q/k/v and gate/up as one grouped launch each,
    it runs q|k|v and gate|up as one product each over concatenated weights."""

    def __init__(self, dims: LayerDims, weights: dict, max_len: int, device):
        self.d = dims
        self.dev = device
        Wt = {n: weights[n].to(device).t().contiguous() for n in ("q", "k", "v", "o", "gate", "up", "down")}
        self.Wt = {"qkv": torch.cat([Wt["q"], Wt["k"], Wt["v"]], dim=1), "o": Wt["o"],
                   "gate_up": torch.cat([Wt["gate"], Wt["up"]], dim=1), "down": Wt["down"]}
        self.K = torch.zeros(1, dims.Hkv, max_len, D_HEAD, dtype=torch.bfloat16, device=device)
        self.V = torch.zeros(1, dims.Hkv, max_len, D_HEAD, dtype=torch.bfloat16, device=device)
        self.pos = 0

    def reset(self):
        self.pos = 0

    def forward(self, x, events: list | None = None):
        dm, T = self.d, x.shape[0]
        L0, L = self.pos, self.pos + x.shape[0]

        def op(name):
            return _NullCtx() if events is None else _EventCtx(events, name)

        with op("rmsnorm"):
            _, xn = rmm.rmm_add_rmsnorm(x, eps=dm.eps)
        with op("qkv"):
            q, k, v = (xn @ self.Wt["qkv"]).split([dm.q_cols, dm.kv_cols, dm.kv_cols], dim=1)
        with op("kv_append"):
            Q = q.view(T, dm.Hq, D_HEAD).transpose(0, 1).unsqueeze(0)
            self.K[0, :, L0:L] = k.view(T, dm.Hkv, D_HEAD).transpose(0, 1)
            self.V[0, :, L0:L] = v.view(T, dm.Hkv, D_HEAD).transpose(0, 1)
        with op("attention"):
            O = torch.nn.functional.scaled_dot_product_attention(
                Q, self.K[:, :, :L], self.V[:, :, :L], is_causal=(T > 1 and L0 == 0), enable_gqa=True,
                scale=1.0 / math.sqrt(D_HEAD))
        with op("heads_to_tokens"):
            a = O[0].transpose(0, 1).reshape(T, dm.q_cols)
        with op("o"):
            yo = a @ self.Wt["o"]
        with op("add_rmsnorm"):
            h2, xn2 = rmm.rmm_add_rmsnorm(x, yo, eps=dm.eps)
        with op("gate_up"):
            g, u = (xn2 @ self.Wt["gate_up"]).split([dm.F, dm.F], dim=1)
        with op("swiglu"):
            hh = torch.nn.functional.silu(g) * u
        with op("down"):
            yd = hh @ self.Wt["down"]
        with op("residual"):
            out, _ = rmm.rmm_add_rmsnorm(h2, yd, eps=dm.eps, want_y=False)
        self.pos = L
        return out


class _NullCtx:
    def __enter__(self):
        return self

    def __exit__(self, *a):
        return False


class _EventCtx:
    """Timing events around one op; recorded as graph nodes when the call is being
    captured (external events), so a replayed graph reports per-op device time."""

    def __init__(self, events, name):
        self.events, self.name = events, name

    def __enter__(self):
        ext = torch.cuda.is_current_stream_capturing()
        self.e0 = torch.cuda.Event(enable_timing=True, external=ext)
        self.e1 = torch.cuda.Event(enable_timing=True, external=ext)
        self.e0.record()
        return self

    def __exit__(self, *a):
        self.e1.record()
        self.events.append((self.name, self.e0, self.e1))
        return False
