"""CPU: what the latent layer's host side does around a library call, with stand-ins for the
GPUs (CPU tensors that name a card), the allocator and the library."""
import threading
import weakref

import pytest
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300 import latent
from compressed_sparse_long_gb300.layer import PagedPool

BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64


class _Card0(torch.Tensor):
    card = 0
    is_cuda = True

    def get_device(self):
        return self.card

    @property
    def device(self):
        return torch.device("cuda", self.card)


class _Card1(_Card0):
    card = 1


CARDS = (_Card0, _Card1)


class _Library:
    """Stands in for libv4a: both attention forms want `nbytes` of workspace, and `during` is
    called with the workspace's address while such a call runs."""
    nbytes = 4096

    def __init__(self):
        self.during = lambda ws: None

    def v4a_latent_attn_workspace_size(self, *a):
        return self.nbytes

    v4a_latent_attn_expanded_workspace_size = v4a_latent_attn_workspace_size

    def v4a_latent_attn(self, *a):
        self.during(a[-4])
        return 0

    v4a_latent_attn_expanded = v4a_latent_attn


class _World:
    def __init__(self, monkeypatch):
        self.card, self.owner, self.scratch, self.lib = 0, {}, [], _Library()
        real = torch.empty

        def empty(*shape, dtype=None, device=None, **kw):
            card = self.card if device is None else torch.device(device).index
            shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
            t = real(shape, dtype=dtype).as_subclass(CARDS[card])
            if dtype is torch.uint8:
                self.owner[t.data_ptr()] = card
                self.scratch.append(weakref.ref(t))
            return t
        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
        monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.card)
        # the default stream has the same handle on every card
        monkeypatch.setattr(latent, "_current_raw", lambda dev: 0)
        monkeypatch.setattr(latent, "library", lambda: self.lib)

    def zeros(self, *shape, dtype=BF):
        return torch.zeros(*shape, dtype=dtype).as_subclass(CARDS[self.card])

    def call(self, lay, form):
        z, h = self.zeros, lay.cfg.n_heads
        cu = z(2, dtype=I32)
        if form == "absorbed":
            return lay.attention(cu, z(1, dtype=I64), 5000, z(3, h, 576))
        return lay.attention_expanded(cu, cu, z(3, h, 192), z(5, h, 128), z(5, 64), z(5, h, 128))

    def layer(self, form):
        cfg = v4a.latent_cfg(v4a.BF16, 4, 512, v4a.rope_cfg(64))
        if form == "expanded":
            return latent.LatentLayer(cfg, None)
        return latent.LatentLayer(cfg, PagedPool(self.zeros(512, 576), None,
                                                 self.zeros(1, 2, dtype=I32), 256))


@pytest.fixture
def world(monkeypatch):
    return _World(monkeypatch)


def test_workspace_lies_on_the_card_of_the_call(world):
    """One layer for the expanded form used on two cards, whose default streams' handles are
    alike: each call gets memory of its own card."""
    lay, seen = world.layer("expanded"), []
    world.lib.during = lambda ws: seen.append((world.card, world.owner[ws]))
    for card in (0, 1, 0, 1):
        world.card = card
        world.call(lay, "expanded")
    assert seen == [(0, 0), (1, 1), (0, 0), (1, 1)]


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_calls_of_two_threads_have_workspaces_of_their_own(world, form):
    """A call enqueues several kernels that meet in its workspace, and the library runs without
    the interpreter's lock: a second thread's call on the same layer and stream may come in
    between."""
    lay, seen = world.layer(form), []

    def during(ws):
        seen.append(ws)
        if len(seen) == 1:
            t = threading.Thread(target=world.call, args=(lay, form))
            t.start()
            t.join(20)
            assert not t.is_alive()
    world.lib.during = during
    world.call(lay, form)
    assert len(seen) == 2 and seen[0] != seen[1]


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_a_layer_keeps_no_workspace(world, form):
    lay = world.layer(form)
    world.call(lay, form)
    assert world.scratch and all(r() is None for r in world.scratch)


def test_a_pool_changed_in_place_is_described_as_it_is(world):
    """Tables and pools that change under the same tensors, and tensors that replace others."""
    lay, seen = world.layer("absorbed"), []
    lay.pool.block_table = world.zeros(3, 8, dtype=I32)

    def call(n_seq):
        z = world.zeros
        lay.attention(z(n_seq + 1, dtype=I32), z(n_seq, dtype=I64), 5000, z(3, 4, 576))
        return seen.pop()
    world.lib.during = lambda ws: None
    take, lib = world.lib.v4a_latent_attn, world.lib
    lib.v4a_latent_attn = lambda *a: (seen.append(a[7]._obj), take(*a))[1]
    first = call(3)
    assert (first.max_blocks, first.n_pages) == (8, 2)
    lay.pool.block_table.resize_(3, 5)             # same tensor, same address
    lay.pool.data.resize_(256, 576)
    assert lay.pool.block_table.data_ptr() == first.block_table
    cache = call(3)
    assert (cache.max_blocks, cache.n_pages) == (5, 1)
    lay.pool.block_table.resize_(2, 5)
    with pytest.raises(ValueError):
        call(3)
    for bad in (dict(data=world.zeros(512, 575)), dict(data=world.zeros(512, 576, dtype=torch.float32)),
                dict(data=torch.zeros(512, 576, dtype=BF)), dict(block_table=world.zeros(8, dtype=I32)),
                dict(block_table=world.zeros(3, 8, dtype=I64)), dict(block_table=world.zeros(8, 3, dtype=I32).t())):
        kept = lay.pool
        lay.pool = PagedPool(**dict(dict(data=kept.data, scale=None, block_table=kept.block_table,
                                         rows_per_block=256), **bad))
        with pytest.raises(ValueError):
            call(1)
        lay.pool = kept
    lay.gamma = torch.ones(512)                    # on the host
    with pytest.raises(ValueError):
        lay.insert(world.zeros(2, dtype=I32), world.zeros(1, dtype=I64), world.zeros(1, 512), world.zeros(1, 64))


def test_long_sequences_beside_many_short_units_can_be_split():
    """A 606-token chunk on a short context and one decode token on 100,000 cached ones, 64 heads:
    more units than whole ones need, and one as long as 780 tiles. Splitting it needs a workspace."""
    cfg = v4a.latent_cfg(v4a.BF16, 64, 512, v4a.rope_cfg(64))
    for n_tokens in (600, 607, 5000):
        assert v4a.v4a_latent_attn_workspace_size(cfg, 2, n_tokens, 99999) > 0
    small = v4a.latent_cfg(v4a.FP32, 8, 128, v4a.rope_cfg(32))
    assert v4a.v4a_latent_attn_workspace_size(small, 2, 5000, 99999) > 0
    # steps past what the device counts in: whole units, as the host alone can have them
    assert v4a.v4a_latent_attn_workspace_size(cfg, 2, 10000, (1 << 36) - 1) == 0
