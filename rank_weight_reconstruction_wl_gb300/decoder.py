"""A weightless decoder with its cache: projections, rotary positions, quantised
cache, tree attention and norms run together.

Per layer and step (x: the fp32 residual stream, h: its normed bf16 form):

    q, k, v = wl_qkv_fused(h)
    q       = wl_rope_append(q, k, v)        k and v into the layer's cache
    o       = wl_linear(wl_tree_attention(q))
    x, h    = wl_norm_residual(o, x)         norm after, residual, norm before the MLP
    m       = wl_mlp_geglu_fused(h)
    x, h    = wl_norm_residual(m, x)         ... and before the next layer

A step takes the newest tokens of every sequence: one each (decoding), a
drafted tree, or up to 64 of a prompt; ``prompt`` feeds longer ones in chunks.
``accept`` keeps a root-to-node path of the tree that a step put into the cache.
All work runs on the current stream.  Nothing synchronises but a step that might
not fit: the host knows a bound of the lengths, and reads them where the bound
does not tell.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (CacheSeqs, KVCache, RopeTable, wl_linear, wl_mlp_geglu_fused, wl_norm_residual, wl_qkv_fused, wl_rope_append,
               wl_tree_attention)
from .stack import LayerTheta

MAX_STEP = 64  # tokens of one sequence in a step (wl_tree_attention)


@dataclass
class BlockNorms:
    """fp32 weights [hidden] of a layer's four norms (None: no norm after the block)."""

    attn_pre: torch.Tensor
    attn_post: torch.Tensor | None
    mlp_pre: torch.Tensor
    mlp_post: torch.Tensor | None


class Decoder:
    """layers: theta bundles (stack.LayerTheta); norms: one BlockNorms each;
    final: the last norm's weight.  batch sequences of up to max_len positions
    in pages of page_size; head dim = k.out / kv_heads.  len (int32 [batch], on
    the GPU) holds the lengths; beside accept(), write to it only to lower them."""

    def __init__(self, layers: list[LayerTheta], norms: list[BlockNorms], final: torch.Tensor, kv_heads: int, rope: RopeTable | None,
                 batch: int, max_len: int, page_size: int = 64, cache_dtype=torch.float8_e4m3fn, eps: float = 1e-6,
                 w_offset: float = 1.0, scale: float | None = None):
        if len(layers) != len(norms):
            raise ValueError("one BlockNorms per layer")
        self.layers, self.norms, self.final = layers, norms, final
        self.hidden = int(layers[0].q.W0.shape[1])
        self.kv_heads, self.dim = kv_heads, int(layers[0].k.W0.shape[0]) // kv_heads
        self.rope, self.batch, self.eps, self.w_offset, self.scale = rope, batch, eps, w_offset, scale
        dev = self.device = layers[0].q.W0.device
        per = -(-max_len // page_size)
        self.max_len = per * page_size
        self.caches = [KVCache.empty(batch * per, kv_heads, page_size, self.dim, cache_dtype, dev) for _ in layers]
        self.pages = torch.arange(batch * per, dtype=torch.int32, device=dev).view(batch, per).contiguous()
        self.len = torch.zeros(batch, dtype=torch.int32, device=dev)
        self._most = 0  # no sequence is longer ...
        self._known = True  # ... unless a captured step may have been replayed
        self._drafted = None

    def _fits(self, n: int, count: torch.Tensor | None):
        if torch.cuda.is_current_stream_capturing():
            self._known = False
            return
        if self._known and self._most + n <= self.max_len:
            return
        new = n if count is None else count.clamp(0, n)
        self._most, most = torch.stack((self.len.max(), (self.len + new).max())).tolist()
        if most > self.max_len:
            raise ValueError(f"the step would fill a sequence to {most} of {self.max_len} positions")

    def step(self, x: torch.Tensor, n: int, mask: torch.Tensor | None = None, depth: torch.Tensor | None = None,
             count: torch.Tensor | None = None) -> torch.Tensor:
        """x [batch * n, hidden] fp32: the embeddings of each sequence's newest n
        tokens (count[b] of them; rows beyond mean nothing).  A tree gives mask
        (int64 [batch, n], bit j of row i: node j is i or an ancestor of it) and
        depth (int32 [batch, n]).  The tokens are in the cache afterwards but
        not counted in len: accept() does that.  Returns the normed final
        states, bf16 [batch * n, hidden].  Raises ValueError where a sequence
        would pass max_len (a captured step cannot tell: wl_device_status()
        reports positions past the table)."""
        if not 1 <= n <= MAX_STEP:
            raise ValueError(f"a step takes 1 to {MAX_STEP} tokens of each sequence, got {n}")
        self._fits(n, count)
        seqs = CacheSeqs(self.pages, self.len, n, count)
        positions = None if depth is None else (self.len[:, None] + depth).to(torch.int32).contiguous()
        norm = dict(eps=self.eps, w_offset=self.w_offset)
        kept = []
        _, h = wl_norm_residual(None, x, w_pre=self.norms[0].attn_pre, **norm)
        for l, (th, nm, cache) in enumerate(zip(self.layers, self.norms, self.caches)):
            q, k, v = wl_qkv_fused(h, th.q, th.k, th.v)
            kept.append((k, v))
            q = wl_rope_append(q, k, v, positions, self.rope, cache, seqs)
            a = wl_tree_attention(q, cache, seqs, mask=mask, scale=self.scale)
            o = wl_linear(a, th.o.W0, th.o.s, th.o.U, th.o.V)
            x, h = wl_norm_residual(o, x, w_post=nm.attn_post, w_pre=nm.mlp_pre, **norm)
            m = wl_mlp_geglu_fused(h, th.gate, th.up, th.down)
            pre = self.norms[l + 1].attn_pre if l + 1 < len(self.layers) else self.final
            x, h = wl_norm_residual(m, x, w_post=nm.mlp_post, w_pre=pre, **norm)
        self._drafted = (n, count, positions, kept)
        return h

    def accept(self, path: torch.Tensor | None = None, count: torch.Tensor | None = None):
        """Counts tokens of the last step into the sequences.  path None: the
        first count[b] (those of the step) as they lie.  Else path [batch, m]
        int: the nodes of a root-to-node path, count[b] <= m of them (entries
        beyond mean nothing); their k and v, kept from the step, are written
        again at the positions that follow len."""
        if self._drafted is None:
            raise ValueError("accept() needs a step before it")
        n, had, positions, kept = self._drafted
        m = n if path is None else int(path.shape[-1])
        if path is not None and (tuple(path.shape) != (self.batch, m) or not 1 <= m <= n):
            raise ValueError(f"path must be [{self.batch}, 1..{n}], got {tuple(path.shape)}")
        self._drafted = None
        if path is not None:
            rows = (torch.arange(self.batch, device=self.device)[:, None] * n + path.clamp(0, n - 1)).view(-1)
            seqs = CacheSeqs(self.pages, self.len, m, count)
            pos = None if positions is None else positions.view(-1)[rows].contiguous()
            for cache, (k, v) in zip(self.caches, kept):
                wl_rope_append(None, k[rows], v[rows], pos, self.rope, cache, seqs)
        elif had is not None:
            count = had if count is None else torch.minimum(count, had)
        self.len += m if count is None else count.clamp(0, m)
        self._most += m

    def prompt(self, x: torch.Tensor) -> torch.Tensor:
        """x [batch, T, hidden] fp32, T tokens of each sequence; returns the last
        token's normed state, bf16 [batch, hidden]."""
        B, T, H = x.shape
        if T < 1:
            raise ValueError("a prompt has at least one token")
        self._fits(T, None)
        h = None
        for t in range(0, T, MAX_STEP):
            part = x[:, t:t + MAX_STEP]
            n = part.shape[1]
            h = self.step(part.reshape(B * n, H).contiguous(), n).view(B, n, H)[:, -1]
            self.accept()
        return h
