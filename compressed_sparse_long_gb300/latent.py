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

from ctypes import byref

import torch

from . import (BF16, FP32, Cache, LatentCfg, RopeCfg, _check, library)
from .layer import PagedPool, current_raw as _current_raw, on_stream, scratch

_TYPES = {BF16: torch.bfloat16, FP32: torch.float32}
_KINDS = {torch.bfloat16: BF16, torch.float32: FP32}


def _fits(t, dev, dtype, shape):
    """t is a contiguous tensor of exactly this type and shape on device `dev`. (At decode sizes
    a call is a few microseconds of GPU time: the usual case is checked in one expression, and
    _need says what is wrong otherwise.)"""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous())


def _rows(t, dev, dtype, shape):
    """The same for rows that may lie apart: dense in the last dimension only."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.stride(-1) == 1)


def _need(t, name, dev, dtype, shape, contiguous=True):
    """Check that t is a tensor of this type and shape (None: any size) on device `dev`, the
    current one."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s: expected a CUDA tensor" % name)
    if t.get_device() != dev:
        raise ValueError("%s is on %s, the current device is cuda:%d" % (name, t.device, dev))
    if t.dtype is not dtype:
        raise ValueError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if len(t.shape) != len(shape) or any(w is not None and w != g for w, g in zip(shape, t.shape)):
        raise ValueError("%s: expected shape %s, got %s" % (name, shape, tuple(t.shape)))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.shape[-1] > 1 and t.numel() and t.stride(-1) != 1:
        raise ValueError("%s: its last dimension must have stride 1" % name)


def _stride(t, d):
    """Elements between neighbours along d (any aligned value where there are none)."""
    return t.stride(d) if t.shape[d] > 1 else -(-t.shape[-1] // 8) * 8


def _strides(t):
    """The same along the first two of three dimensions."""
    n, h, _ = t.shape
    if n > 1 and h > 1:
        return t.stride()[:2]
    return _stride(t, 0), _stride(t, 1)


def _raw(stream, dev):
    return stream if isinstance(stream, int) else stream.cuda_stream


def _new(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with on_stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _zeros(shape, dtype, device, stream):
    with on_stream(stream):
        return torch.zeros(shape, dtype=dtype, device=device)


def _word(dev_err, dev):
    _need(dev_err, "dev_err", dev, torch.int32, (1,))
    return dev_err.data_ptr()


def _rope(cfg, x, pos, out, inverse, dev_err, stream, new=_new):
    """rope() without a graph; `new` makes the result where none is given."""
    kind = _KINDS.get(x.dtype) if isinstance(x, torch.Tensor) else None
    shape = x.shape if kind is not None else ()
    if len(shape) not in (2, 3):
        raise ValueError("x: expected a bfloat16 or float32 tensor [n, H, dim] or [n, dim]")
    dev = torch.cuda.current_device() if x.is_cuda else -2
    if not (shape[-1] == cfg.dim and _rows(x, dev, x.dtype, shape)
            and _fits(pos, dev, torch.int64, shape[:1])):
        _need(x, "x", dev, x.dtype, (None,) * (len(shape) - 1) + (cfg.dim,), contiguous=False)
        _need(pos, "pos", dev, torch.int64, (shape[0],))
    if out is None:
        out = new(shape, x.dtype, x.device, stream)
    elif not _rows(out, dev, x.dtype, shape):
        _need(out, "out", dev, x.dtype, shape, contiguous=False)
    heads, xh, oh = (1, 0, 0) if len(shape) == 2 else (shape[1], _stride(x, 1), _stride(out, 1))
    _check("v4a_rope", library().v4a_rope(
        byref(cfg), kind, shape[0], heads, pos.data_ptr(), x.data_ptr(), _stride(x, 0),
        xh, out.data_ptr(), _stride(out, 0), oh, inverse,
        None if dev_err is None else _word(dev_err, dev),
        _current_raw(dev) if stream is None else _raw(stream, dev)))
    return out


class _Rope(torch.autograd.Function):
    """A recorded call: its gradient is the turn the other way, itself such a call."""

    @staticmethod
    def forward(ctx, x, pos, cfg, inverse, dev_err, stream):
        # a token at a bad position is not written: its result and its gradient are zeros here
        y = _rope(cfg, x, pos, None, inverse, dev_err, stream, _zeros)
        ctx.save_for_backward(pos)
        ctx.cfg, ctx.inverse = RopeCfg.from_buffer_copy(cfg), inverse
        return y

    @staticmethod
    def backward(ctx, g):
        g = g if g.stride(-1) == 1 else g.contiguous()
        turned = _Rope.apply(g, ctx.saved_tensors[0], ctx.cfg, not ctx.inverse, None, None)
        return turned, None, None, None, None, None


def rope(cfg: RopeCfg, x: torch.Tensor, pos: torch.Tensor, out: torch.Tensor | None = None,
         inverse: bool = False, dev_err=None, stream=None) -> torch.Tensor:
    """Rotate x [n, H, dim] or [n, dim] (bf16 or fp32, any strides with a dense last dimension:
    a slice of wider heads, say) at positions pos [n] int64. ``out`` is a new tensor unless
    given; ``out=x`` rotates in place. ``inverse`` turns back; it is also the gradient's map,
    and the gradient of a call without ``out`` on an x that requires grad."""
    if isinstance(x, torch.Tensor) and x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out: a call that writes it is not recorded, but x requires grad")
        return _Rope.apply(x, pos, cfg, inverse, dev_err, stream)
    return _rope(cfg, x, pos, out, inverse, dev_err, stream)


class LatentLayer:
    """A latent-attention layer's configuration, cache and norm weight.

    Forward only: the methods' results are outside any graph, whatever their inputs require.

    pool: PagedPool of [n_pages * 256, latent_dim + rope dim] rows, or None for a layer that
    is only used in the expanded form; gamma: fp32 [latent_dim] or None (no norm at insert).
    """

    def __init__(self, cfg: LatentCfg, pool: PagedPool | None, gamma: torch.Tensor | None = None):
        if cfg.dtype not in _TYPES:
            raise ValueError("dtype: expected BF16 or FP32")
        self.cfg, self.pool, self.gamma = cfg, pool, gamma
        self.dtype = _TYPES[cfg.dtype]
        self.width = cfg.latent_dim + cfg.rope.dim
        self._desc = None, None
        dev = torch.cuda.current_device() if torch.cuda.is_available() else -2
        if pool is not None:
            _need(pool.data, "pool.data", dev, self.dtype, (None, self.width))
            _need(pool.block_table, "pool.block_table", dev, torch.int32, (None, None))
        if gamma is not None:
            _need(gamma, "gamma", dev, torch.float32, (cfg.latent_dim,))

    def _describe(self, dev):
        """(sequences of the block table, C descriptor) of the layer's pool as it is now."""
        pool = self.pool
        if pool is None:
            raise ValueError("this layer has no cache")
        data, bt, rows = pool.data, pool.block_table, pool.rows_per_block
        shape, table = data.shape, bt.shape
        if not (data.dtype is self.dtype and bt.dtype is torch.int32
                and len(shape) == len(table) == 2 and shape[1] == self.width
                and data.get_device() == dev == bt.get_device()
                and data.is_contiguous() and bt.is_contiguous()):
            _need(data, "pool.data", dev, self.dtype, (None, self.width))
            _need(bt, "pool.block_table", dev, torch.int32, (None, None))
        # (the structure is kept for as long as a new one would say the same)
        key = (data.data_ptr(), bt.data_ptr(), table[1], rows, shape[0])
        d = self._desc
        if d[0] != key:
            d = self._desc = key, Cache(key[0], None, key[1], table[1], rows, shape[0] // rows,
                                        self.width, 0)
        return table[0], d[1]

    def _batch(self, cu, start):
        """(device, sequences, cache descriptor) of a call over the cache."""
        dev = torch.cuda.current_device() if torch.cuda.is_initialized() else -2
        known, cache = self._describe(dev)
        n_seq = cu.numel() - 1 if isinstance(cu, torch.Tensor) else -1
        # (_fits of both, written out)
        if n_seq < 0 or not (isinstance(start, torch.Tensor)
                             and cu.dtype is torch.int32 and start.dtype is torch.int64
                             and cu.dim() == 1 and start.shape == (n_seq,)
                             and cu.get_device() == dev == start.get_device()
                             and cu.is_contiguous() and start.is_contiguous()):
            _need(cu, "cu", dev, torch.int32, (None,))
            if n_seq < 0:
                raise ValueError("cu: expected the sequences' first rows and the end")
            _need(start, "start", dev, torch.int64, (n_seq,))
        if n_seq > known:
            raise ValueError("cu has %d sequences, the block table %d" % (n_seq, known))
        return dev, n_seq, cache

    def insert(self, cu, start, c, k_pe, dev_err=None, stream=None):
        """Write the cache rows of new tokens: c [n, latent_dim], k_pe [n, rope dim] (rows may
        be strided: two slices of one projection's output)."""
        dev, n_seq, cache = self._batch(cu, start)
        n = c.shape[0] if isinstance(c, torch.Tensor) and c.dim() else 0
        dc, dr, gamma = self.cfg.latent_dim, self.cfg.rope.dim, self.gamma
        if not (_rows(c, dev, self.dtype, (n, dc)) and _rows(k_pe, dev, self.dtype, (n, dr))):
            _need(c, "c", dev, self.dtype, (None, dc), contiguous=False)
            _need(k_pe, "k_pe", dev, self.dtype, (n, dr), contiguous=False)
        if gamma is not None and not _fits(gamma, dev, torch.float32, (dc,)):
            _need(gamma, "gamma", dev, torch.float32, (dc,))
        cs, ks = (c.stride(0), k_pe.stride(0)) if n > 1 else (dc, dr)
        _check("v4a_latent_insert", library().v4a_latent_insert(
            byref(self.cfg), n_seq, n, cu.data_ptr(), start.data_ptr(), c.data_ptr(),
            cs, k_pe.data_ptr(), ks, None if gamma is None else gamma.data_ptr(), byref(cache),
            None if dev_err is None else _word(dev_err, dev),
            _current_raw(dev) if stream is None else _raw(stream, dev)))

    def gather(self, cu, start, n_rows, out=None, dev_err=None, stream=None):
        """Copy cached rows out: sequence b's rows cu[b] .. cu[b+1]-1 of the result are its
        cache rows from position start[b] on. n_rows is cu's last value (rows of a larger
        result behind it are left as they are)."""
        dev, n_seq, cache = self._batch(cu, start)
        if out is None:
            out = _new((n_rows, self.width), self.dtype, cu.device, stream)
        elif not _fits(out, dev, self.dtype, (n_rows, self.width)):
            _need(out, "out", dev, self.dtype, (n_rows, self.width))
        _check("v4a_latent_gather", library().v4a_latent_gather(
            byref(self.cfg), n_seq, n_rows, cu.data_ptr(), start.data_ptr(), byref(cache),
            out.data_ptr(), None if dev_err is None else _word(dev_err, dev),
            _current_raw(dev) if stream is None else _raw(stream, dev)))
        return out

    def attention(self, cu, start, max_pos, q, out=None, dev_err=None, stream=None):
        """Absorbed attention of q [n, H, latent_dim + rope dim] over the cache: one new token
        a sequence (decode) or chunks; returns [n, H, latent_dim]."""
        dev, n_seq, cache = self._batch(cu, start)
        h = self.cfg.n_heads
        n = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() else 0
        if not _fits(q, dev, self.dtype, (n, h, self.width)):
            _need(q, "q", dev, self.dtype, (None, h, self.width))
        if out is None:
            out = _new((n, h, self.cfg.latent_dim), self.dtype, q.device, stream)
        elif not _fits(out, dev, self.dtype, (n, h, self.cfg.latent_dim)):
            _need(out, "out", dev, self.dtype, (n, h, self.cfg.latent_dim))
        lib, cfg = library(), byref(self.cfg)
        nb = lib.v4a_latent_attn_workspace_size(cfg, n_seq, n, max_pos)
        ws = scratch(nb, q.device, stream)
        _check("v4a_latent_attn", lib.v4a_latent_attn(
            cfg, n_seq, n, cu.data_ptr(), start.data_ptr(), max_pos, q.data_ptr(), byref(cache),
            out.data_ptr(), None if ws is None else ws.data_ptr(), nb,
            None if dev_err is None else _word(dev_err, dev),
            _current_raw(dev) if stream is None else _raw(stream, dev)))
        return out

    def attention_expanded(self, cu_q, cu_k, q, k, k_pe, v, causal=True, out=None, dev_err=None,
                           stream=None):
        """Expanded attention: q [n_q, H, nope + rope], k [n_k, H, nope], k_pe [n_k, rope]
        (shared by the heads), v [n_k, H, v_dim]; k, k_pe and v may be strided slices of wider
        rows. Returns [n_q, H, v_dim]."""
        c = self.cfg
        dev = torch.cuda.current_device() if torch.cuda.is_initialized() else -2
        n_seq = cu_q.numel() - 1 if isinstance(cu_q, torch.Tensor) else -1
        n_q = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() else 0
        n_k = k.shape[0] if isinstance(k, torch.Tensor) and k.dim() else 0
        if n_seq < 0 or not (
                _fits(cu_q, dev, torch.int32, (n_seq + 1,))
                and _fits(cu_k, dev, torch.int32, (n_seq + 1,))
                and _fits(q, dev, self.dtype, (n_q, c.n_heads, c.nope_dim + c.rope.dim))
                and _rows(k, dev, self.dtype, (n_k, c.n_heads, c.nope_dim))
                and _rows(k_pe, dev, self.dtype, (n_k, c.rope.dim))
                and _rows(v, dev, self.dtype, (n_k, c.n_heads, c.v_dim))):
            _need(cu_q, "cu_q", dev, torch.int32, (None,))
            if n_seq < 0:
                raise ValueError("cu_q: expected the sequences' first rows and the end")
            _need(cu_k, "cu_k", dev, torch.int32, (n_seq + 1,))
            _need(q, "q", dev, self.dtype, (None, c.n_heads, c.nope_dim + c.rope.dim))
            _need(k, "k", dev, self.dtype, (None, c.n_heads, c.nope_dim), contiguous=False)
            _need(k_pe, "k_pe", dev, self.dtype, (n_k, c.rope.dim), contiguous=False)
            _need(v, "v", dev, self.dtype, (n_k, c.n_heads, c.v_dim), contiguous=False)
        shape = (n_q, c.n_heads, c.v_dim)
        if out is None:
            out = _new(shape, self.dtype, q.device, stream)
        elif not _fits(out, dev, self.dtype, shape):
            _need(out, "out", dev, self.dtype, shape)
        lib, cfg = library(), byref(c)
        nb = lib.v4a_latent_attn_expanded_workspace_size(cfg, n_seq, n_q, n_k)
        ws = scratch(nb, q.device, stream)
        _check("v4a_latent_attn_expanded", lib.v4a_latent_attn_expanded(
            cfg, n_seq, n_q, cu_q.data_ptr(), n_k, cu_k.data_ptr(), q.data_ptr(),
            k.data_ptr(), *_strides(k), k_pe.data_ptr(), _stride(k_pe, 0), v.data_ptr(),
            *_strides(v), causal, out.data_ptr(),
            None if ws is None else ws.data_ptr(), nb,
            None if dev_err is None else _word(dev_err, dev),
            _current_raw(dev) if stream is None else _raw(stream, dev)))
        return out

    def step(self, cu, start, max_pos, pos, c, k_pe, q, out=None, dev_err=None, stream=None):
        """One decode or chunk step: insert the new tokens, rotate the queries' rotary part in
        place (pos [n]: the new tokens' positions), attend."""
        self.insert(cu, start, c, k_pe, dev_err, stream)
        rot = q[..., self.cfg.latent_dim:]
        _rope(self.cfg.rope, rot, pos, rot, False, dev_err, stream)
        return self.attention(cu, start, max_pos, q, out=out, dev_err=dev_err, stream=stream)
