"""CPU: what the host side of the page table and of the windowed calls does around a library call,
with stand-ins for the GPU, the allocator and the library."""
import pytest
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300 import latent, pages
from compressed_sparse_long_gb300.layer import PagedPool
from test_latent_host import BF, I32, I64, _World

U8 = torch.uint8


class _Pages:
    """Stands in for libv4a: every page call notes its arguments; a call wants `nbytes` of workspace."""
    nbytes = 512

    def __init__(self):
        self.seen = []

    def v4a_pages_workspace_size(self, table):
        return self.nbytes

    def __getattr__(self, name):
        if not name.startswith("v4a_"):
            raise AttributeError(name)
        if name.endswith("workspace_size"):
            return lambda *a: self.nbytes
        return lambda *a: (self.seen.append((name, a)), 0)[1]


@pytest.fixture
def world(monkeypatch):
    w = _World(monkeypatch)
    w.lib = _Pages()
    monkeypatch.setattr(pages, "library", lambda: w.lib)
    monkeypatch.setattr(pages, "_current_raw", lambda dev: 0)
    return w


def table(world, n_seq=3, blocks=4, n=6):
    z = world.zeros
    bt = z(n_seq, blocks, dtype=I32)
    pools = [PagedPool(z(n * 256, 576), None, bt, 256),
             PagedPool(z(n * 64, 128, dtype=U8), z(n * 64, dtype=torch.float32), bt, 64)]
    return pages.PageTable(pools, bt, z(n, dtype=I32))


def test_calls_describe_table_and_pools_as_they_are(world):
    t, z = table(world), world.zeros
    t.fork(z(2, dtype=I32), z(2, dtype=I32), z(2, dtype=I64))
    name, a = world.lib.seen.pop()
    desc, pools = a[0]._obj, a[1]
    assert name == "v4a_pages_fork" and a[2:4] == (2, 2)
    assert (desc.n_seq, desc.max_blocks, desc.n_pages) == (3, 4, 6)
    assert [(p.row_bytes, p.rows_per_block) for p in pools] == [(1152, 256), (128, 64)]
    assert pools[0].scale is None and pools[1].scale == t.pools[1].scale.data_ptr()
    # a pool that another replaces, and one that changes in place, are looked at again
    other = z(6 * 256, 64)
    t.pools[0] = PagedPool(other, None, t.block_table, 256)
    t.compact()
    name, a = world.lib.seen.pop()
    assert name == "v4a_pages_compact" and a[1][0].data == other.data_ptr() and a[1][0].row_bytes == 128
    other.resize_(6 * 256, 32)
    t.copy(z(1, dtype=I32), z(1, dtype=I32))
    assert world.lib.seen.pop()[1][1][0].row_bytes == 64
    other.resize_(5 * 256, 32)
    with pytest.raises(ValueError):
        t.compact()


def test_a_table_keeps_no_workspace_and_refuses_other_cards(world):
    t, z = table(world), world.zeros
    t.grow(z(3, dtype=I32), z(3, dtype=I32))
    t.fork(z(1, dtype=I32), z(1, dtype=I32), z(1, dtype=I64))
    t.compact()
    assert len(world.scratch) == 3 and all(r() is None for r in world.scratch)
    world.card = 1
    with pytest.raises(ValueError):
        t.free(z(3, dtype=I32), z(3, dtype=I32))
    world.card = 0
    with pytest.raises(ValueError):
        pages.PageTable([PagedPool(z(512, 576), None, z(1, 2, dtype=I32), 256)], z(1, 2, dtype=I32),
                        z(2, dtype=I32)).compact()


@pytest.mark.parametrize("fp4", [False, True])
def test_windowed_calls_go_to_their_entry_point(world, fp4):
    z = world.zeros
    cfg = v4a.latent_cfg(v4a.BF16, 4, 512, v4a.rope_cfg(64),
                         cache_format=v4a.LATENT_FP4 if fp4 else v4a.LATENT_PLAIN)
    bt = z(1, 2, dtype=I32)
    pool = (PagedPool(z(512, 416, dtype=U8), z(512, dtype=torch.float32), bt, 256) if fp4
            else PagedPool(z(512, 576), None, bt, 256))
    lay = latent.LatentLayer(cfg, pool)
    cu, start, q = z(2, dtype=I32), z(1, dtype=I64), z(3, 4, 576)
    lay.attention(cu, start, 400, q, window=100, sinks=7)
    name, a = world.lib.seen.pop()
    assert name == "v4a_latent_attn_window" and a[5:8] == (400, 100, 7)
    assert a[9]._obj.scale == (pool.scale.data_ptr() if fp4 else None) and a[9]._obj.row_width == 576
    lay.attention(cu, start, 400, q)
    assert world.lib.seen.pop()[0] == "v4a_latent_attn"
    assert all(r() is None for r in world.scratch)
    assert q.dtype is BF
