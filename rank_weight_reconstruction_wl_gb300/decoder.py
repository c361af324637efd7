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
With a head, ``logits`` are the step's and ``verify`` decides which drafted tokens
hold, keeps them and draws the next (node 0 of the next step is in ``next``):

    h = dec.step(x, n, mask, depth)            x: embeddings of the drafted tree
    path, accepted, token = dec.verify(dec.logits(h), tokens, uniforms, mask)
    tokens[:, 0] = dec.next                    ... and drafts behind it

With pool_pages the sequences share that many cache pages instead of owning
max_len positions each: a step takes the pages that it needs, gives back what the
last one's rejected drafts had, and ``release`` gives back ended sequences'.
All work runs on the current stream.  Nothing synchronises but a step that might
not fit, and a prompt with shared pages: the host knows a bound of the lengths,
and reads them where the bound does not tell.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (CacheSeqs, F8Weight, KVCache, PagePool, RopeTable, wl_linear, wl_linear_f8, wl_mlp_geglu_fused, wl_norm_residual,
               wl_page_plan, wl_qkv_fused, wl_quant_f8, wl_rope_append, wl_tree_attention, wl_verify)
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
    the GPU) holds the lengths; beside accept(), write to it only to lower them.
    head: the vocabulary's projection (F8Weight [vocab, hidden]).  pool_pages: how
    many pages the sequences share (None: enough for max_len each); where they
    run out, sequences in order get all the pages that a step needs or none, and
    take the first room[b] tokens (nodes) of the step: those for which there is
    space, in the last page that they have too; room is int32 [batch], on the GPU.  next
    (int32 [batch], on the GPU, after verify()): node 0 of the next step."""

    def __init__(self, layers: list[LayerTheta], norms: list[BlockNorms], final: torch.Tensor, kv_heads: int, rope: RopeTable | None,
                 batch: int, max_len: int, page_size: int = 64, cache_dtype=torch.float8_e4m3fn, eps: float = 1e-6,
                 w_offset: float = 1.0, scale: float | None = None, head: F8Weight | None = None, pool_pages: int | None = None):
        if len(layers) != len(norms):
            raise ValueError("one BlockNorms per layer")
        if head is not None and head.inp != layers[0].q.W0.shape[1]:
            raise ValueError(f"the head must take {layers[0].q.W0.shape[1]} inputs, got {head.inp}")
        if pool_pages is not None and pool_pages < 1:
            raise ValueError(f"pool_pages must be at least 1, got {pool_pages}")
        self.layers, self.norms, self.final = layers, norms, final
        self.hidden = int(layers[0].q.W0.shape[1])
        self.kv_heads, self.dim = kv_heads, int(layers[0].k.W0.shape[0]) // kv_heads
        self.rope, self.batch, self.eps, self.w_offset, self.scale = rope, batch, eps, w_offset, scale
        dev = self.device = layers[0].q.W0.device
        per = -(-max_len // page_size)
        self.max_len = per * page_size
        held = batch * per if pool_pages is None else pool_pages
        self.caches = [KVCache.empty(held, kv_heads, page_size, self.dim, cache_dtype, dev) for _ in layers]
        self.len = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.head, self.pool, self.held, self.room, self.next = head, None, None, None, None
        if pool_pages is None:
            self.pages = torch.arange(batch * per, dtype=torch.int32, device=dev).view(batch, per).contiguous()
        else:
            self.pool = PagePool.full(pool_pages, page_size, dev)
            self.pages = torch.full((batch, per), -1, dtype=torch.int32, device=dev)
            self.held = torch.zeros(batch, dtype=torch.int32, device=dev)
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
        if self.pool is not None:
            count, _ = wl_page_plan(self.pool, self.pages, self.held, self.len, n, count)
            self.room = count
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
        self._drafted = (n, count, positions, kept, mask)
        return h

    def accept(self, path: torch.Tensor | None = None, count: torch.Tensor | None = None):
        """Counts tokens of the last step into the sequences.  path None: the
        first count[b] (those of the step) as they lie.  Else path [batch, m]
        int: the nodes of a root-to-node path, count[b] <= m of them (entries
        beyond mean nothing); their k and v, kept from the step, are written
        again at the positions that follow len."""
        if self._drafted is None:
            raise ValueError("accept() needs a step before it")
        n, had, positions, kept, _ = self._drafted
        m = n if path is None else int(path.shape[-1])
        if path is not None and (tuple(path.shape) != (self.batch, m) or not 1 <= m <= n):
            raise ValueError(f"path must be [{self.batch}, 1..{n}], got {tuple(path.shape)}")
        self._drafted = None
        if path is not None and self.pool is not None:  # no more than there were pages for
            count = had if count is None else torch.minimum(count, had)
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

    def logits(self, h: torch.Tensor, ydt=torch.bfloat16) -> torch.Tensor:
        """The head's logits [rows, vocab] of h [rows, hidden], a step's normed states."""
        if self.head is None:
            raise ValueError("logits() needs a head")
        return wl_linear_f8(*wl_quant_f8(h), self.head, ydt=ydt)

    def verify(self, logits: torch.Tensor, tokens: torch.Tensor, uniforms: torch.Tensor, mask: torch.Tensor | None = None,
               draft: torch.Tensor | None = None, temperature=1.0):
        """Which of the last step's drafted tokens hold (wl_verify: logits
        [batch * n, vocab], tokens and uniforms [batch, n]; mask: the step's, where
        it is not given), counted into the sequences as accept() does; returns (path,
        accepted, token) as wl_verify: token is -1 where none was drawn.  self.next
        is what the next step begins with: the token drawn, or, for a sequence that
        took no token in the step (its count or room was 0), its node 0 again, which
        is not in the cache yet; -1 where the model's row had no distribution."""
        if self._drafted is None:
            raise ValueError("verify() needs a step before it")
        n, had = self._drafted[:2]
        if tuple(tokens.shape) != (self.batch, n):
            raise ValueError(f"tokens must be [{self.batch}, {n}] as the step's, got {tuple(tokens.shape)}")
        if mask is None:
            mask = self._drafted[4]
        path, accepted, token = wl_verify(logits, tokens, uniforms, mask, had, draft, temperature)
        self.accept(None if mask is None else path, accepted)  # a chain's path lies as it is
        self.next = token if had is None else torch.where(had > 0, token, tokens[:, 0])
        return path, accepted, token

    def release(self, done: torch.Tensor):
        """Ends the sequences with done[b] (bool [batch]): their lengths become 0
        and their shared pages go back.  An open step is dropped."""
        if tuple(done.shape) != (self.batch,) or done.dtype != torch.bool:
            raise ValueError(f"done must be bool [{self.batch}], got {done.dtype} {tuple(done.shape)}")
        self._drafted = None
        self.len.masked_fill_(done, 0)
        if self.pool is not None:
            wl_page_plan(self.pool, self.pages, self.held, self.len)

    def prompt(self, x: torch.Tensor) -> torch.Tensor:
        """x [batch, T, hidden] fp32, T tokens of each sequence; returns the last
        token's normed state, bf16 [batch, hidden]."""
        B, T, H = x.shape
        if T < 1:
            raise ValueError("a prompt has at least one token")
        self._fits(T, None)
        if self.pool is not None and not torch.cuda.is_current_stream_capturing():
            page = self.pool.page_size
            need, have = torch.stack((((self.len + T + page - 1) // page).sum(), self.held.sum() + self.pool.top[0])).tolist()
            if need > have:
                raise ValueError(f"the sequences would need {need} pages of {have}")
        h = None
        for t in range(0, T, MAX_STEP):
            part = x[:, t:t + MAX_STEP]
            n = part.shape[1]
            h = self.step(part.reshape(B * n, H).contiguous(), n).view(B, n, H)[:, -1]
            self.accept()
        return h
