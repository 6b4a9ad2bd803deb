"""Decode-step composition: the per-token sequence of library calls for a
dense 8B-class decoder and for a MoE decoder, ready to be captured in one
CUDA graph.

Each layer is pre-norm with a weightless RMS norm (folded into the GEMVs'
prologue).  Attention is either
* the one-token-context stand-in (attn_ctx=None): softmax over a single key
  is 1, so each query head's output is the value head it reads (grouped
  heads share one value head); q and k are still computed, so the weight
  traffic is that of a real decode step; or
* epq_attention_decode over a Q8_0 key/value cache per layer (attn_ctx = the
  number of cached positions before the step, filled with seeded synthetic
  keys and values): the step appends its key and value and attends over the
  cache with the ln(1e-4) skip threshold.
Every step below is one C-ABI call; this module holds device buffers and the
order of the calls, nothing else.

TreeDecoder verifies a tree of drafted tokens in one dense step over a paged
Q8_0 cache: the drafted tokens are the GEMVs' columns, every layer appends
their keys and values and attends over the cache and the tree, and the walk
over the logits and the commit of the accepted rows end the step -- all of it
queued (or captured in one graph) without a host synchronisation.  Its prompt
method brings any number of tokens into the cache first; with a RopeTable the
queries and keys of both are turned by their positions (a drafted token's is its
depth in the tree), and a step can be given penalties, biases and a grammar.

`timers` (optional) brackets each call of the first layer with a pair of
CUDA events, so that per-kernel durations can be read after a graph replay.
"""
from __future__ import annotations

import contextlib
import math

import torch

from . import _lib as L

SKIP_LOG = math.log(1e-4)


def kv_caches(n_layers, n_kv, head_dim, ctx, max_pos, device, seed):
    """One KVCache per layer with positions 0..ctx-1 filled: seeded N(0,1)
    keys and values quantized by epq_quantize (Q8_0) and laid out as the
    cache rows (block factors, then codes)."""
    gen = torch.Generator(device=device)
    caches = []
    nblk = head_dim // 32
    for li in range(n_layers):
        c = L.KVCache(n_kv, head_dim, max_pos, device)
        if ctx > 0:
            for dst in (c.k, c.v):
                gen.manual_seed(seed * 1000 + li * 2 + (dst is c.v))
                n = n_kv * ctx * head_dim
                x = torch.zeros(-(-n // 256) * 256, device=device, dtype=torch.float32)
                x[:n] = torch.randn(n, generator=gen, device=device, dtype=torch.float32)
                # Q8_0 blocks are independent 32-runs: pack as rows of 256 and drop the padding
                b = L.epq_quantize(L.EPQ_Q8_0, x.view(-1, 256)).view(-1)[:n // 32 * 34].view(n_kv, ctx, nblk, 34)
                dst[:, :ctx, :2 * nblk] = b[..., :2].reshape(n_kv, ctx, 2 * nblk)
                dst[:, :ctx, 2 * nblk:] = b[..., 2:].reshape(n_kv, ctx, head_dim)
        caches.append(c)
    return caches


@contextlib.contextmanager
def _timed(timers, name, stream, on):
    if timers is None or not on:
        yield
        return
    a, b = timers.pair(name)
    a.record(stream)
    yield
    b.record(stream)


class DenseDecoder:
    """32-layer dense decoder + LM head, Q-format weights, nvec columns
    (one library call per matrix, or the whole step as one epq_gemv_chain).

    Per layer (h: [nvec, H] residual stream):
      qkv = Wqkv rms(h)                 (q, k, v rows concatenated)
      h   = h + Wo v                    (v heads repeated heads/kv_heads times)
      m   = silu(Wg rms(h)) * (Wu rms(h))
      h   = h + Wd m
    then logits = Whead rms(h).
    """

    def __init__(self, cfg, fmt, layers, head, device, nvec=1, chain=False, attn_ctx=None):
        self.cfg, self.fmt, self.layers, self.head, self.nvec = cfg, fmt, layers, head, nvec
        H = cfg.hidden
        self.qkv = torch.empty((nvec, cfg.q_rows + 2 * cfg.kv_rows), dtype=torch.float32, device=device)
        # KV-cache attention (one vector): caches of attn_ctx positions, the step at position attn_ctx
        self.attn_ctx = attn_ctx if (attn_ctx is not None and nvec == 1 and not chain) else None
        if self.attn_ctx is not None:
            self.caches = kv_caches(len(layers), cfg.kv_heads, cfg.head_dim, self.attn_ctx, self.attn_ctx + 64,
                                    device, seed=7)
            self.attn = torch.empty((1, cfg.q_rows), dtype=torch.float32, device=device)
            self.pos = self.attn_ctx
        self.m = torch.empty((nvec, cfg.inter), dtype=torch.float32, device=device)
        self.h = torch.empty((nvec, H), dtype=torch.float32, device=device)
        self.logits = torch.empty((nvec, cfg.vocab), dtype=torch.float32, device=device)
        # chain mode: the whole step is one epq_gemv_chain launch (Q4_K, nvec <= 2)
        self.chain = chain and fmt == L.EPQ_Q4_K and nvec <= 2
        self.ws = torch.zeros(L.epq_gemv_chain_workspace_bytes() if self.chain else 16, dtype=torch.uint8,
                              device=device)
        self._ops = {}

    def chain_ops(self, x):
        """The step's ops for epq_gemv_chain (same sequence as step())."""
        c, H = self.cfg, self.cfg.hidden
        nq, nkv = c.q_rows, c.kv_rows
        h = self.h
        ops = []
        for li, (wqkv, wo, wgu, wd) in enumerate(self.layers):
            src = x if li == 0 else h
            ops.append(L.gemv_op(wqkv, src, self.qkv, nq + 2 * nkv, H, rms_prenorm=True, rms_eps=c.rms_eps))
            ops.append(L.gemv_op(wo, self.qkv[:, nq + nkv:], h, H, nq, residual=src, x_group=c.heads // c.kv_heads,
                                 x_head_dim=c.head_dim))
            ops.append(L.gemv_op(wgu, h, self.m, 2 * c.inter, H, swiglu=True, rms_prenorm=True, rms_eps=c.rms_eps))
            ops.append(L.gemv_op(wd, self.m, h, H, c.inter, residual=h))
        ops.append(L.gemv_op(self.head, h, self.logits, c.vocab, H, rms_prenorm=True, rms_eps=c.rms_eps))
        return ops

    def step(self, x, stream=None, timers=None):
        """x [nvec, H] (read only) -> self.logits."""
        c, f, H = self.cfg, self.fmt, self.cfg.hidden
        if self.chain:
            key = x.data_ptr()
            if key not in self._ops:
                self._ops[key] = self.chain_ops(x)
            with _timed(timers, "gemv_chain", stream, True):
                L.epq_gemv_chain(f, self._ops[key], self.nvec, self.ws, stream=stream)
            return self.logits
        nq, nkv = c.q_rows, c.kv_rows
        h = self.h
        for li, (wqkv, wo, wgu, wd) in enumerate(self.layers):
            src = x if li == 0 else h
            on = li == 0
            with _timed(timers, "gemv_qkv", stream, on):
                L.epq_gemv_ex(f, wqkv, src, nq + 2 * nkv, H, y=self.qkv, rms_prenorm=True, rms_eps=c.rms_eps,
                              weights_ready=True, stream=stream)
            if self.attn_ctx is not None:
                q = self.qkv[0]
                L.epq_attention_decode(q[:nq], q[nq:nq + nkv], q[nq + nkv:], self.caches[li], c.heads, self.pos,
                                       1.0 / math.sqrt(c.head_dim), SKIP_LOG, out=self.attn[0], stream=stream)
                L.epq_gemv_ex(f, wo, self.attn, H, nq, y=h, residual=src, weights_ready=True, stream=stream)
            else:
                v = self.qkv[:, nq + nkv:]
                with _timed(timers, "gemv_o", stream, on):
                    L.epq_gemv_ex(f, wo, v, H, nq, y=h, residual=src, x_group=c.heads // c.kv_heads,
                                  x_head_dim=c.head_dim, weights_ready=True, stream=stream)
            with _timed(timers, "gemv_gateup", stream, on):
                L.epq_gemv_ex(f, wgu, h, 2 * c.inter, H, y=self.m, rms_prenorm=True, rms_eps=c.rms_eps,
                              swiglu=True, weights_ready=True, stream=stream)
            with _timed(timers, "gemv_down", stream, on):
                L.epq_gemv_ex(f, wd, self.m, H, c.inter, y=h, residual=h, weights_ready=True, stream=stream)
        L.epq_gemv_ex(f, self.head, h, c.vocab, H, y=self.logits, rms_prenorm=True, rms_eps=c.rms_eps,
                      weights_ready=True, stream=stream)
        return self.logits


class MoEDecoder:
    """MoE decoder, batch 1.

    Per layer: qkv = Wqkv rms(h); h = h + Wo v; h = h + MoE(rms(h)).
    """

    def __init__(self, cfg, fmt, layers, device, attn_ctx=None, max_new=64):
        self.cfg, self.fmt, self.layers = cfg, fmt, layers
        H = cfg.hidden
        self.qkv = torch.empty((1, 3 * H), dtype=torch.float32, device=device)
        self.h = torch.empty((1, H), dtype=torch.float32, device=device)
        # KV-cache attention (q, k and v each H = heads * head_dim: one key/value head per query head)
        self.attn_ctx = attn_ctx
        if attn_ctx is not None:
            self.caches = kv_caches(len(layers), cfg.heads, cfg.head_dim, attn_ctx, attn_ctx + max_new, device,
                                    seed=11)
            self.attn = torch.empty((1, H), dtype=torch.float32, device=device)
        ws = max(layer.workspace_bytes(1, cfg.topk) for (_, _, layer) in layers)
        self.ws = torch.empty(ws, dtype=torch.uint8, device=device)

    def token(self, x, out, stream=None, timers=None, idx_out=None, pos=None):
        """x [1, H] (read only) -> out [1, H], the hidden state after the last layer.

        idx_out (optional, int32 [layers, topk]): each layer's selected experts.
        pos: the token's position in the key/value caches (attention mode)."""
        c, f, H = self.cfg, self.fmt, self.cfg.hidden
        h = self.h
        n = len(self.layers)
        for li, (wqkv, wo, moe) in enumerate(self.layers):
            src = x if li == 0 else h
            on = li == 0
            with _timed(timers, "gemv_qkv", stream, on):
                L.epq_gemv_ex(f, wqkv, src, 3 * H, H, y=self.qkv, rms_prenorm=True, rms_eps=c.rms_eps,
                              weights_ready=True, stream=stream)
            if self.attn_ctx is not None:
                q = self.qkv[0]
                L.epq_attention_decode(q[:H], q[H:2 * H], q[2 * H:], self.caches[li], c.heads, pos,
                                       1.0 / math.sqrt(c.head_dim), SKIP_LOG, out=self.attn[0], stream=stream)
                L.epq_gemv_ex(f, wo, self.attn, H, H, y=h, residual=src, weights_ready=True, stream=stream)
            else:
                with _timed(timers, "gemv_o", stream, on):
                    L.epq_gemv_ex(f, wo, self.qkv[:, 2 * H:], H, H, y=h, residual=src, weights_ready=True,
                                  stream=stream)
            y = out if li == n - 1 else h
            if timers is not None and on:
                for name, st in (("moe_router", L.EPQ_MOE_ROUTE), ("moe_gateup", L.EPQ_MOE_GATE_UP),
                                 ("moe_down", L.EPQ_MOE_DOWN)):
                    with _timed(timers, name, stream, True):
                        L.epq_moe_forward(moe, h, c.topk, y=y, workspace=self.ws, rms_prenorm=True,
                                          rms_eps=c.rms_eps, stages=st, stream=stream)
            else:
                L.epq_moe_forward(moe, h, c.topk, y=y, workspace=self.ws, rms_prenorm=True, rms_eps=c.rms_eps,
                                  topk_idx=None if idx_out is None else idx_out[li:li + 1], stream=stream)
        return out


def paged_cache(caches, ctx, n_seq=1, room=128, spare_pages=0, page_size=64):
    """A PagedKVCache of all layers whose sequence 0 holds positions 0..ctx-1
    of `caches` (one KVCache per layer); `room`: further positions of every
    sequence, for which the pool has pages (plus spare_pages)."""
    c0 = caches[0]
    dev = c0.k.device
    have, each = -(-ctx // page_size), -(-(ctx + room) // page_size)
    pages = L.PagedKVCache(len(caches), each + (n_seq - 1) * (each - ctx // page_size) + spare_pages, c0.n_kv_heads,
                           c0.head_dim, n_seq, each, page_size, dev)
    for li, c in enumerate(caches):
        for plane, rows in enumerate((c.k, c.v)):
            x = torch.zeros((c.n_kv_heads, have * page_size, rows.shape[2]), dtype=torch.uint8, device=dev)
            x[:, :ctx] = rows[:, :ctx]
            pages.pool[li, :have, :, plane] = x.view(c.n_kv_heads, have, page_size, -1).transpose(0, 1)
    pages.table[0, :have] = torch.arange(have, dtype=torch.int32, device=dev)
    pages.refs[:have] = 1
    pages.length[0] = ctx
    return pages


class TreeDecoder:
    """A dense decoder that verifies ntok (1..8) drafted tokens per step.

    layers, head: packed weights as in DenseDecoder; cache: a PagedKVCache of
    all layers (one sequence); rope: None or a RopeTable.  Token 0 of a step is
    the last committed token, the others its drafted continuations; parent names
    their tree."""

    def __init__(self, cfg, fmt, layers, head, cache, ntok, device, rope=None):
        if not 1 <= ntok <= 8 or cache.n_seq != 1:
            raise ValueError("1..8 drafted tokens of one sequence")
        self.cfg, self.fmt, self.layers, self.head, self.cache, self.ntok = cfg, fmt, layers, head, cache, ntok
        self.rope = rope
        f32 = dict(dtype=torch.float32, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        self.qkv = torch.empty((1, ntok, cfg.q_rows + 2 * cfg.kv_rows), **f32)
        self.attn = torch.empty((1, ntok, cfg.q_rows), **f32)
        self.m = torch.empty((ntok, cfg.inter), **f32)
        self.h = torch.empty((ntok, cfg.hidden), **f32)
        self.logits = torch.empty((1, ntok, cfg.vocab), **f32)
        self.mask = torch.empty((1, ntok), dtype=torch.int64, device=device)
        self.extra = torch.full((1,), ntok, **i32)
        self.status = torch.zeros(1, **i32)
        self.n_tok = torch.zeros(1, **i32)  # ntok, or 0 when the cache has no room
        self.path, self.n_accept, self.next_token = (torch.empty(n, **i32) for n in ((1, ntok), (1,), (1,)))
        self.lse = torch.empty((1, ntok), **f32)
        self.attn_ws = L.epq_attention_tree_workspace(cache, cfg.heads, ntok)
        self.verify_ws = L.epq_verify_tree_workspace(self.logits)

    def _reserve(self, extra, n_tok, stream):
        """Room for extra rows; n_tok: as many, or 0 where there is none (status is nonzero then)."""
        L.epq_pages_reserve(self.cache, extra, self.status, stream=stream)
        with torch.cuda.stream(None if stream is None else L._stream_object(stream)):
            torch.mul(extra, self.status == 0, out=n_tok)

    def prompt(self, x, stream=None):
        """x float32 [n, H], contiguous, any n >= 1 (the tokens' embeddings): their rows are appended
        and committed -> logits [1, vocab] behind the last one (logits[None] is
        what epq_logits_adjust and epq_verify_tree take).  The weights are read
        once for every 8 tokens, which is most of a prompt's time; its attention
        has no window, as the steps behind it have none.  status is nonzero when
        the cache had no room: it stays as it is then, and the logits mean
        nothing."""
        c, f, H, nq, nkv, cache = self.cfg, self.fmt, self.cfg.hidden, self.cfg.q_rows, self.cfg.kv_rows, self.cache
        n, new = x.shape[0], L._allocator(stream)
        if n < 1:
            raise ValueError("a prompt has at least one token")
        L._need(x, "x", torch.float32, (n, H), cache._at)
        f32, i32 = dict(dtype=torch.float32, device=x.device), dict(dtype=torch.int32, device=x.device)
        qkv, attn = new((1, n, nq + 2 * nkv), **f32), new((1, n, nq), **f32)
        h, m, logits = new((n, H), **f32), new((n, c.inter), **f32), new((1, c.vocab), **f32)
        extra, n_tok = new(1, **i32), new(1, **i32)
        ws = L.epq_attention_prompt_workspace(cache, c.heads, n, stream)
        with torch.cuda.stream(None if stream is None else L._stream_object(stream)):
            extra.fill_(n)
        self._reserve(extra, n_tok, stream)
        q, k, v = qkv[..., :nq], qkv[..., nq:nq + nkv], qkv[..., nq + nkv:]
        eight = [slice(i, min(i + 8, n)) for i in range(0, n, 8)]
        for li, (wqkv, wo, wgu, wd) in enumerate(self.layers):
            src = x if li == 0 else h
            for r in eight:
                L.epq_gemv_ex(f, wqkv, src[r], nq + 2 * nkv, H, y=qkv[0, r], rms_prenorm=True, rms_eps=c.rms_eps,
                              weights_ready=True, stream=stream)
            if self.rope is not None:
                L.epq_rope(q, self.rope, c.heads, start=cache.length, n_tok=n_tok, out=q, stream=stream)
            L.epq_pages_append(k, v, cache, li, rope=self.rope, n_tok=n_tok, stream=stream)
            L.epq_attention_prompt(q, cache, li, c.heads, 1.0 / math.sqrt(c.head_dim), n_tok=n_tok, out=attn,
                                   workspace=ws, stream=stream)
            for r in eight:
                L.epq_gemv_ex(f, wo, attn[0, r], H, nq, y=h[r], residual=src[r], weights_ready=True, stream=stream)
                L.epq_gemv_ex(f, wgu, h[r], 2 * c.inter, H, y=m[r], rms_prenorm=True, rms_eps=c.rms_eps, swiglu=True,
                              weights_ready=True, stream=stream)
                L.epq_gemv_ex(f, wd, m[r], H, c.inter, y=h[r], residual=h[r], weights_ready=True, stream=stream)
        L.epq_gemv_ex(f, self.head, h[n - 1:], c.vocab, H, y=logits, rms_prenorm=True, rms_eps=c.rms_eps,
                      weights_ready=True, stream=stream)
        L.epq_pages_advance(cache, n_tok, stream=stream)
        return logits

    def forward(self, x, parent, stream=None):
        """x [ntok, H] (the tokens' embeddings), parent int32 [1, ntok] ->
        logits [1, ntok, vocab]; the tokens' rows lie behind the committed
        positions.  status is nonzero when the cache had no room: nothing is
        stored then, and the logits mean nothing."""
        c, f, H, nq, nkv = self.cfg, self.fmt, self.cfg.hidden, self.cfg.q_rows, self.cfg.kv_rows
        h, qkv, attn = self.h, self.qkv, self.attn
        self._reserve(self.extra, self.n_tok, stream)
        L.epq_tree_mask(parent, self.mask, stream=stream)
        q, k, v = qkv[..., :nq], qkv[..., nq:nq + nkv], qkv[..., nq + nkv:]
        for li, (wqkv, wo, wgu, wd) in enumerate(self.layers):
            src = x if li == 0 else h
            L.epq_gemv_ex(f, wqkv, src, nq + 2 * nkv, H, y=qkv[0], rms_prenorm=True, rms_eps=c.rms_eps,
                          weights_ready=True, stream=stream)
            if self.rope is not None:  # query and key heads lie side by side
                qk = qkv[..., :nq + nkv]
                L.epq_rope(qk, self.rope, c.heads + c.kv_heads, start=self.cache.length, mask=self.mask,
                           n_tok=self.n_tok, out=qk, stream=stream)
            L.epq_attention_tree(q, k, v, self.cache, li, c.heads, 1.0 / math.sqrt(c.head_dim), mask=self.mask,
                                 n_tok=self.n_tok, out=attn, workspace=self.attn_ws, stream=stream)
            L.epq_gemv_ex(f, wo, attn[0], H, nq, y=h, residual=src, weights_ready=True, stream=stream)
            L.epq_gemv_ex(f, wgu, h, 2 * c.inter, H, y=self.m, rms_prenorm=True, rms_eps=c.rms_eps, swiglu=True,
                          weights_ready=True, stream=stream)
            L.epq_gemv_ex(f, wd, self.m, H, c.inter, y=h, residual=h, weights_ready=True, stream=stream)
        L.epq_gemv_ex(f, self.head, h, c.vocab, H, y=self.logits[0], rms_prenorm=True, rms_eps=c.rms_eps,
                      weights_ready=True, stream=stream)
        return self.logits

    def step(self, x, tokens, parent, u, draft=None, temperature=1.0, constraints=None, stream=None):
        """One verification step: forward, the walk, the commit.  tokens,
        parent int32 and u float32 [1, ntok], draft None or float32 [1, ntok,
        vocab] -> (path, n_accept, next_token); the cache then holds the
        accepted tokens, and next_token is the root of the next step.
        constraints: None or arguments of epq_logits_adjust (penalties, history
        and its lengths, biases, allowed), applied to the logits first; tokens,
        mask and n_tok are the step's.  A cache without room stays as it is: n_accept 0, next_token -1, status nonzero."""
        self.forward(x, parent, stream=stream)
        if constraints:
            L.epq_logits_adjust(self.logits, tokens=tokens, mask=self.mask, n_tok=self.n_tok, out=self.logits,
                                stream=stream, **constraints)
        L.epq_verify_tree(self.logits, tokens, parent, u, draft=draft, n_tok=self.n_tok, temperature=temperature,
                          path=self.path, n_accept=self.n_accept, next_token=self.next_token, lse=self.lse, workspace=self.verify_ws,
                          stream=stream)
        L.epq_pages_compact(self.cache, self.path, self.n_accept, stream=stream)
        return self.path, self.n_accept, self.next_token
