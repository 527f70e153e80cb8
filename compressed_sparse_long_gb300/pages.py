"""Pages of the pools that share one block table, on top of the C ABI (``v4a_pages_*``): growing,
freeing, forking, copying and compacting, on the device and in stream order.

    table = PageTable([lay.pool for lay in layers], block_table)
    table.grow(first, last)                       # blocks that the next tokens need
    table.fork(src, dst, length)                  # beams, samples, a shared prompt
    table.free(first, last)                       # ended sequences, blocks behind a window
    n_used = table.compact()                      # then the pools' first n_used pages hold all
"""
from __future__ import annotations

from ctypes import byref

import torch

from . import MAX_POOLS, PageTableDesc, Pool, _check, library
from .latent import _fits, _need, _new, _raw, _word
from .layer import current_raw as _current_raw, scratch

_I32, _I64 = torch.int32, torch.int64


class PageTable:
    """A block table, its pages' reference counts, and the pools whose rows they name.

    pools: PagedPool list (may be empty) of the same number of pages, whose block_table is this one
    (a compressed layer's are lay.attn, lay.idx, lay.swa and lay.state);
    block_table: int32 [n_seq, max_blocks], -1 = no page; refs: int32 [n_pages], how many entries of
    the table name each page (0 = free). Without refs they are counted from the table, and the pools
    say how many pages there are. Nothing here waits for the device.
    """

    def __init__(self, pools, block_table: torch.Tensor, refs: torch.Tensor | None = None):
        self.pools, self.block_table = list(pools), block_table
        dev = torch.cuda.current_device() if torch.cuda.is_available() else -2
        _need(block_table, "block_table", dev, _I32, (None, None))
        if len(self.pools) > MAX_POOLS:
            raise ValueError("pools: at most %d share a table" % MAX_POOLS)
        if refs is None:
            if not self.pools:
                raise ValueError("refs: needed where there is no pool")
            n = self.pools[0].data.shape[0] // self.pools[0].rows_per_block
            named = torch.where((block_table >= 0) & (block_table < n), block_table, n).long().flatten()
            refs = torch.zeros(n + 1, dtype=_I32, device=block_table.device)
            refs = refs.index_add_(0, named, torch.ones_like(named, dtype=_I32))[:n].clone()
        _need(refs, "refs", dev, _I32, (None,))
        self.refs = refs
        self._desc = None, None, 0
        self._pools = None, None
        self._describe()

    def _describe(self):
        """(device, table descriptor, workspace bytes) as the tensors are now."""
        dev = torch.cuda.current_device() if torch.cuda.is_initialized() else -2
        bt, refs = self.block_table, self.refs
        if not (len(bt.shape) == 2 and _fits(bt, dev, _I32, bt.shape)
                and len(refs.shape) == 1 and _fits(refs, dev, _I32, refs.shape)):
            _need(bt, "block_table", dev, _I32, (None, None))
            _need(refs, "refs", dev, _I32, (None,))
        n = refs.shape[0]
        # (the structure is kept for as long as a new one would say the same)
        key = (bt.data_ptr(), refs.data_ptr(), *bt.shape, n)
        d = self._desc
        if d[0] != key:
            desc = PageTableDesc(*key)
            d = self._desc = key, desc, library().v4a_pages_workspace_size(byref(desc))
        return dev, d[1], d[2]

    def _describe_pools(self, dev):
        table, n = self.block_table, self.refs.shape[0]
        at = table.data_ptr()
        # (all that the checks below look at: where it says the same, so would they)
        key = [at, table.shape, n, dev]
        for p in self.pools:
            d, s, t = p.data, p.scale, p.block_table
            key += (d.data_ptr(), d.shape, d.dtype, d.get_device(), d.is_contiguous(),
                    p.rows_per_block, p.late)
            key += (None,) if s is None else (s.data_ptr(), s.shape, s.dtype, s.get_device(),
                                              s.is_contiguous())
            key += (None,) if t is table else (t.data_ptr(), t.shape)
        kept = self._pools
        if kept[0] != key:
            for i, p in enumerate(self.pools):
                name = "pools[%d]" % i
                _need(p.data, name + ".data", dev, p.data.dtype, (n * p.rows_per_block, None))
                if p.scale is not None:
                    _need(p.scale, name + ".scale", dev, torch.float32, (n * p.rows_per_block,))
                if p.block_table.data_ptr() != at or p.block_table.shape != table.shape:
                    raise ValueError("%s has another block table" % name)
                if not 0 <= p.late < 256:
                    raise ValueError("%s.late: 0 .. 255 is needed" % name)
                if p.data.shape[1] * p.data.element_size() % 16:
                    raise ValueError("%s: rows of a multiple of 16 bytes are needed" % name)
            kept = self._pools = key, (Pool * len(self.pools))(*[
                Pool(p.data.data_ptr(), None if p.scale is None else p.scale.data_ptr(),
                     p.data.shape[1] * p.data.element_size(), p.rows_per_block, p.late, 0)
                for p in self.pools])
        return kept[1], len(kept[1])

    def _list(self, t, name, dev, dtype, n):
        if not _fits(t, dev, dtype, (n,)):
            _need(t, name, dev, dtype, (n,))
        return t.data_ptr()

    @staticmethod
    def _end(dev, dev_err, stream):
        return (None if dev_err is None else _word(dev_err, dev),
                _current_raw(dev) if stream is None else _raw(stream, dev))

    def free(self, first, last, dev_err=None, stream=None):
        """Give back blocks first[b] .. last[b] - 1 (int32 [n_seq]) of every row b."""
        dev, desc, _ = self._describe()
        n = self.block_table.shape[0]
        _check("v4a_pages_free", library().v4a_pages_free(
            byref(desc), self._list(first, "first", dev, _I32, n),
            self._list(last, "last", dev, _I32, n), *self._end(dev, dev_err, stream)))

    def grow(self, first, last, dev_err=None, stream=None):
        """Give the lowest free pages to those of blocks first[b] .. last[b] - 1 that have none."""
        dev, desc, nb = self._describe()
        n = self.block_table.shape[0]
        a, b = self._list(first, "first", dev, _I32, n), self._list(last, "last", dev, _I32, n)
        ws = scratch(nb, self.refs.device, stream)
        _check("v4a_pages_grow", library().v4a_pages_grow(
            byref(desc), a, b, None if ws is None else ws.data_ptr(), nb,
            *self._end(dev, dev_err, stream)))

    def fork(self, src, dst, length, dev_err=None, stream=None):
        """Row dst[i] takes over the first length[i] positions of row src[i] (int32, int32, int64
        [n]): blocks that are complete there are shared, the block that length[i] cuts is copied to
        a page of its own, in every pool, and so is the one before it where some pool's ``late``
        says that tokens behind length[i] still write into it. dst's row must hold no page."""
        dev, desc, nb = self._describe()
        n = src.shape[0] if isinstance(src, torch.Tensor) and src.dim() else 0
        a, b = self._list(src, "src", dev, _I32, n), self._list(dst, "dst", dev, _I32, n)
        c = self._list(length, "length", dev, _I64, n)
        pools, n_pools = self._describe_pools(dev)
        ws = scratch(nb, self.refs.device, stream)
        _check("v4a_pages_fork", library().v4a_pages_fork(
            byref(desc), pools, n_pools, n, a, b, c, None if ws is None else ws.data_ptr(), nb,
            *self._end(dev, dev_err, stream)))

    def copy(self, src, dst, dev_err=None, stream=None):
        """Copy whole pages src[i] -> dst[i] (int32 [n]) in every pool. No page that is written may
        be in another pair."""
        dev, desc, _ = self._describe()
        n = src.shape[0] if isinstance(src, torch.Tensor) and src.dim() else 0
        a, b = self._list(src, "src", dev, _I32, n), self._list(dst, "dst", dev, _I32, n)
        pools, n_pools = self._describe_pools(dev)
        _check("v4a_pages_copy", library().v4a_pages_copy(
            byref(desc), pools, n_pools, n, a, b, *self._end(dev, dev_err, stream)))

    def compact(self, moved=None, dev_err=None, stream=None):
        """Move the used pages to the pools' front; the table and the counts follow. Returns how
        many there are (int32 [1] on the device). moved: int32 [n_pages] to receive every page's
        new number (-1: was free), for holders of pages besides the table."""
        dev, desc, nb = self._describe()
        m = None if moved is None else self._list(moved, "moved", dev, _I32, self.refs.shape[0])
        pools, n_pools = self._describe_pools(dev)
        used = _new((1,), _I32, self.refs.device, stream)
        ws = scratch(nb, self.refs.device, stream)
        _check("v4a_pages_compact", library().v4a_pages_compact(
            byref(desc), pools, n_pools, used.data_ptr(), m,
            None if ws is None else ws.data_ptr(), nb, *self._end(dev, dev_err, stream)))
        return used
