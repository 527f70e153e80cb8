"""A paged latent-attention layer on the device, on top of the C ABI (``v4a_rope``,
``v4a_latent_*``): the counterpart of ``layer.Layer`` for layers whose cache holds one shared
latent and rotary key a token.

torch owns the memory and the stream; every computation is a library call. Decode and short
chunks (absorbed form, the projections applied around the call by the caller)::

    lay.insert(cu, start, c, k_pe)                   # cache rows of the new tokens
    rope(cfg.rope, q[..., C:], pos, out=q[..., C:])  # q = [q_nope W_uk | q_pe]
    o = lay.attention(cu, start, max_pos, q)         # then out = o W_uv

Prompts, after a cached prefix or none (expanded form)::

    lay.insert(cu, start, c, k_pe)
    rows = lay.gather(cu_k, zeros, n_k)              # every cached row of the sequences
    kv = project(rows[:, :C])                        # [n_k, H, nope + v]
    o = lay.attention_expanded(cu, cu_k, q, kv[..., :nope], rows[:, C:], kv[..., nope:])
"""
from __future__ import annotations

from contextlib import nullcontext

import torch

from . import (BF16, FP32, LatentCfg, RopeCfg, v4a_latent_attn, v4a_latent_attn_expanded,
               v4a_latent_attn_workspace_size, v4a_latent_gather, v4a_latent_insert, v4a_rope)
from .layer import PagedPool

_TYPES = {BF16: torch.bfloat16, FP32: torch.float32}


def _need(t, name, dtype, shape, contiguous=True):
    """A tensor of this type and shape (None: any size) on the current device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s: expected a CUDA tensor" % name)
    if t.device.index != torch.cuda.current_device():
        raise ValueError("%s is on %s, the current device is cuda:%d"
                         % (name, t.device, torch.cuda.current_device()))
    if t.dtype != dtype:
        raise ValueError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != len(shape) or any(w is not None and w != g for w, g in zip(shape, t.shape)):
        raise ValueError("%s: expected shape %s, got %s" % (name, shape, tuple(t.shape)))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if not contiguous and t.numel() and t.stride(-1) != 1:
        raise ValueError("%s: its last dimension must have stride 1" % name)
    return t


def _stride(t, d):
    """Elements between neighbours along d (any aligned value where there are none)."""
    return t.stride(d) if t.shape[d] > 1 else -(-t.shape[-1] // 8) * 8


def _on(stream):
    """Allocations of a call belong to the stream that it runs on."""
    return nullcontext() if stream is None or isinstance(stream, int) else torch.cuda.stream(stream)


def rope(cfg: RopeCfg, x: torch.Tensor, pos: torch.Tensor, out: torch.Tensor | None = None,
         inverse: bool = False, dev_err=None, stream=None) -> torch.Tensor:
    """Rotate x [n, H, dim] or [n, dim] (bf16 or fp32, any strides with a dense last dimension:
    a slice of wider heads, say) at positions pos [n] int64. ``out`` is a new tensor unless
    given; ``out=x`` rotates in place. ``inverse`` turns back; it is also the gradient's map."""
    kinds = {torch.bfloat16: BF16, torch.float32: FP32}
    if not isinstance(x, torch.Tensor) or x.dtype not in kinds or x.dim() not in (2, 3):
        raise ValueError("x: expected a bfloat16 or float32 tensor [n, H, dim] or [n, dim]")
    _need(x, "x", x.dtype, (None,) * (x.dim() - 1) + (cfg.dim,), contiguous=False)
    _need(pos, "pos", torch.int64, (x.shape[0],))
    if out is None:
        with _on(stream):
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _need(out, "out", x.dtype, tuple(x.shape), contiguous=False)
    heads, xh, oh = (1, 0, 0) if x.dim() == 2 else (x.shape[1], _stride(x, 1), _stride(out, 1))
    v4a_rope(cfg, kinds[x.dtype], x.shape[0], heads, pos, x, _stride(x, 0), xh, out,
             _stride(out, 0), oh, inverse, dev_err, stream)
    return out


class LatentLayer:
    """A latent-attention layer's configuration, cache and norm weight.

    pool: PagedPool of [n_pages * 256, latent_dim + rope dim] rows, or None for a layer that
    is only used in the expanded form; gamma: fp32 [latent_dim] or None (no norm at insert).
    """

    def __init__(self, cfg: LatentCfg, pool: PagedPool | None, gamma: torch.Tensor | None = None):
        if cfg.dtype not in _TYPES:
            raise ValueError("dtype: expected BF16 or FP32")
        self.cfg, self.pool, self.gamma = cfg, pool, gamma
        self.dtype = _TYPES[cfg.dtype]
        self.width = cfg.latent_dim + cfg.rope.dim
        if pool is not None:
            _need(pool.data, "pool.data", self.dtype, (None, self.width))
            _need(pool.block_table, "pool.block_table", torch.int32, (None, None))
        if gamma is not None:
            _need(gamma, "gamma", torch.float32, (cfg.latent_dim,))
        self._ws = {}

    def _batch(self, cu, start):
        _need(cu, "cu", torch.int32, (None,))
        n_seq = cu.numel() - 1
        if n_seq < 0:
            raise ValueError("cu: expected the sequences' first rows and the end")
        if self.pool is None:
            raise ValueError("this layer has no cache")
        if n_seq > self.pool.block_table.shape[0]:
            raise ValueError("cu has %d sequences, the block table %d"
                             % (n_seq, self.pool.block_table.shape[0]))
        _need(start, "start", torch.int64, (n_seq,))
        return n_seq

    def _workspace(self, nbytes, device, stream):
        """Kept per stream, so calls on two streams never share one; a call being captured
        into a graph gets memory of that graph's own."""
        if nbytes == 0:
            return None
        with _on(stream):
            if torch.cuda.is_current_stream_capturing():
                return torch.empty(nbytes, dtype=torch.uint8, device=device)
            key = stream if isinstance(stream, int) else torch.cuda.current_stream().cuda_stream
            ws = self._ws.get(key)
            if ws is None or ws.numel() < nbytes:
                ws = self._ws[key] = torch.empty(nbytes, dtype=torch.uint8, device=device)
            return ws

    def insert(self, cu, start, c, k_pe, dev_err=None, stream=None):
        """Write the cache rows of new tokens: c [n, latent_dim], k_pe [n, rope dim] (rows may
        be strided: two slices of one projection's output)."""
        n_seq = self._batch(cu, start)
        _need(c, "c", self.dtype, (None, self.cfg.latent_dim), contiguous=False)
        _need(k_pe, "k_pe", self.dtype, (c.shape[0], self.cfg.rope.dim), contiguous=False)
        v4a_latent_insert(self.cfg, n_seq, c.shape[0], cu, start, c, _stride(c, 0), k_pe,
                          _stride(k_pe, 0), self.gamma, self.pool.c, dev_err, stream)

    def gather(self, cu, start, n_rows, out=None, dev_err=None, stream=None):
        """Copy cached rows out: sequence b's rows cu[b] .. cu[b+1]-1 of the result are its
        cache rows from position start[b] on. n_rows is cu's last value (rows of a larger
        result behind it are left as they are)."""
        n_seq = self._batch(cu, start)
        if out is None:
            with _on(stream):
                out = torch.empty((n_rows, self.width), dtype=self.dtype, device=cu.device)
        else:
            _need(out, "out", self.dtype, (n_rows, self.width))
        v4a_latent_gather(self.cfg, n_seq, n_rows, cu, start, self.pool.c, out, dev_err, stream)
        return out

    def attention(self, cu, start, max_pos, q, out=None, dev_err=None, stream=None):
        """Absorbed attention of q [n, H, latent_dim + rope dim] over the cache: one new token
        a sequence (decode) or chunks; returns [n, H, latent_dim]."""
        n_seq = self._batch(cu, start)
        h = self.cfg.n_heads
        _need(q, "q", self.dtype, (None, h, self.width))
        shape = (q.shape[0], h, self.cfg.latent_dim)
        if out is None:
            with _on(stream):
                out = torch.empty(shape, dtype=self.dtype, device=q.device)
        else:
            _need(out, "out", self.dtype, shape)
        nb = v4a_latent_attn_workspace_size(self.cfg, n_seq, q.shape[0], max_pos)
        v4a_latent_attn(self.cfg, n_seq, q.shape[0], cu, start, max_pos, q, self.pool.c, out,
                        self._workspace(nb, q.device, stream), dev_err, stream)
        return out

    def attention_expanded(self, cu_q, cu_k, q, k, k_pe, v, causal=True, out=None, dev_err=None,
                           stream=None):
        """Expanded attention: q [n_q, H, nope + rope], k [n_k, H, nope], k_pe [n_k, rope]
        (shared by the heads), v [n_k, H, v_dim]; k, k_pe and v may be strided slices of wider
        rows. Returns [n_q, H, v_dim]."""
        c = self.cfg
        _need(cu_q, "cu_q", torch.int32, (None,))
        _need(cu_k, "cu_k", torch.int32, (cu_q.numel(),))
        if cu_q.numel() == 0:
            raise ValueError("cu_q: expected the sequences' first rows and the end")
        _need(q, "q", self.dtype, (None, c.n_heads, c.nope_dim + c.rope.dim))
        _need(k, "k", self.dtype, (None, c.n_heads, c.nope_dim), contiguous=False)
        _need(k_pe, "k_pe", self.dtype, (k.shape[0], c.rope.dim), contiguous=False)
        _need(v, "v", self.dtype, (k.shape[0], c.n_heads, c.v_dim), contiguous=False)
        shape = (q.shape[0], c.n_heads, c.v_dim)
        if out is None:
            with _on(stream):
                out = torch.empty(shape, dtype=self.dtype, device=q.device)
        else:
            _need(out, "out", self.dtype, shape)
        v4a_latent_attn_expanded(c, cu_q.numel() - 1, q.shape[0], cu_q, k.shape[0], cu_k, q, k,
                                 _stride(k, 0), _stride(k, 1), k_pe, _stride(k_pe, 0), v,
                                 _stride(v, 0), _stride(v, 1), causal, out, dev_err, stream)
        return out

    def step(self, cu, start, max_pos, pos, c, k_pe, q, out=None, dev_err=None, stream=None):
        """One decode or chunk step: insert the new tokens, rotate the queries' rotary part in
        place (pos [n]: the new tokens' positions), attend."""
        self.insert(cu, start, c, k_pe, dev_err, stream)
        rot = q[..., self.cfg.latent_dim:]
        rope(self.cfg.rope, rot, pos, out=rot, dev_err=dev_err, stream=stream)
        return self.attention(cu, start, max_pos, q, out=out, dev_err=dev_err, stream=stream)
