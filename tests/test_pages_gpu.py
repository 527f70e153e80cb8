"""GPU: the page table's calls against their plain forms, and a serving run of them together with
the latent layers' calls."""
import numpy as np
import pytest
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300.latent import LatentLayer
from compressed_sparse_long_gb300.layer import PagedPool
from compressed_sparse_long_gb300.pages import PageTable
from latent_helpers import BF, F32, err_word, ints
from oracle import pages_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


I32, I64 = torch.int32, torch.int64
KINDS = {"bf16": (256, 8, BF, False), "fp4": (256, 416, torch.uint8, True), "two": (2, 64, torch.uint8, True),
         "entries": (64, 4, F32, False), "odd": (3, 12, F32, True)}


class Case:
    """A table, counts and pools on the device and on the host."""

    def __init__(self, rng, n_seq, blocks, pages, kinds=(), fill=0.6, shared=0.2):
        self.refs = np.zeros(pages, np.int32)
        self.bt = np.full((n_seq, blocks), -1, np.int32)
        free = list(rng.permutation(pages))
        for b in range(n_seq):
            for k in range(blocks):
                if rng.random() < fill and free:
                    used = np.nonzero(self.refs)[0]
                    page = rng.choice(used) if len(used) and rng.random() < shared else free.pop()
                    self.bt[b, k] = page
                    self.refs[page] += 1
        self.d_bt = ints(self.bt, I32)
        self.pools, self.host = [], []
        for kind in kinds:
            R, width, dtype, scaled = KINDS[kind]
            data = (torch.from_numpy(rng.integers(0, 256, (pages * R, width))).to("cuda", dtype))
            scale = torch.from_numpy(rng.random(pages * R)).to("cuda", F32) if scaled else None
            self.pools.append(PagedPool(data, scale, self.d_bt, R))
            self.host.append((data.float().cpu().numpy(), R))
            if scaled:
                self.host.append((scale.cpu().numpy(), R))
        self.table = PageTable(self.pools, self.d_bt, ints(self.refs, I32))

    def check(self):
        assert self.d_bt.cpu().numpy().tolist() == self.bt.tolist()
        assert self.table.refs.cpu().numpy().tolist() == self.refs.tolist()
        got = []
        for p in self.pools:
            got.append(p.data.float().cpu().numpy())
            if p.scale is not None:
                got.append(p.scale.cpu().numpy())
        for g, (want, _) in zip(got, self.host):
            assert np.array_equal(g, want)


@pytest.mark.parametrize("n_seq,blocks,pages", [(1, 1, 1), (3, 7, 40), (5, 300, 1100), (64, 130, 9001),
                                                (1024, 3, 4096), (2, 1000, 12289)])
def test_grow_and_free(n_seq, blocks, pages):
    rng = np.random.default_rng(n_seq + blocks)
    c, e = Case(rng, n_seq, blocks, pages, fill=0.4), err_word()
    for step in range(4):
        first = rng.integers(-2, blocks + 1, n_seq)
        last = first + rng.integers(-3, blocks + 3, n_seq)
        if step % 2:
            c.table.free(ints(first, I32), ints(last, I32), dev_err=e)
            O.free(c.bt, c.refs, first, last)
            assert v4a.v4a_get_error(e) == 0
        else:
            c.table.grow(ints(first, I32), ints(last, I32), dev_err=e)
            there = O.grow(c.bt, c.refs, first, last)
            assert v4a.v4a_get_error(e) == (0 if there else v4a.DEV_NO_PAGE)
        c.check()


def test_grow_when_pages_run_out():
    c, e = Case(np.random.default_rng(0), 4, 6, 10, fill=0.0), err_word()
    c.table.grow(ints([0, 1, 0, 0], I32), ints([3, 1, 6, 6], I32), dev_err=e)
    assert v4a.v4a_get_error(e) == v4a.DEV_NO_PAGE
    assert not O.grow(c.bt, c.refs, [0, 1, 0, 0], [3, 1, 6, 6])
    c.check()
    assert (c.refs == 1).all()
    c.table.free(ints([0] * 4, I32), ints([6] * 4, I32), dev_err=e)
    assert v4a.v4a_get_error(e) == 0 and (c.table.refs == 0).all() and (c.d_bt == -1).all()
    # a pool without a page, and one of exactly what is needed
    none = PageTable([], ints(np.full((2, 3), -1), I32), torch.zeros(0, dtype=I32, device="cuda"))
    none.grow(ints([0, 0], I32), ints([0, 1], I32), dev_err=e)
    assert v4a.v4a_get_error(e) == v4a.DEV_NO_PAGE and (none.block_table == -1).all()
    assert int(none.compact()) == 0


def test_bad_entries_of_a_table():
    bt = np.array([[0, 77, -5, 1], [1, 0, 2, -1]], np.int32)
    e = err_word()
    t = PageTable([], ints(bt, I32), ints([1, 2, 0, 0], I32))
    t.free(ints([1, 2], I32), ints([3, 3], I32), dev_err=e)      # 77, -5, and page 2, whose count is 0
    assert v4a.v4a_get_error(e) == v4a.DEV_BAD_PAGE
    assert t.block_table.tolist() == [[0, -1, -1, 1], [1, 0, -1, -1]] and t.refs.tolist() == [1, 2, 0, 0]
    t = PageTable([], ints(bt, I32), ints([2, 2, 1, 0], I32))
    t.grow(ints([0, 0], I32), ints([4, 0], I32), dev_err=e)      # bad entries are blocks without a page
    assert v4a.v4a_get_error(e) == v4a.DEV_BAD_PAGE | v4a.DEV_NO_PAGE
    assert t.block_table.tolist() == [[0, 3, -5, 1], [1, 0, 2, -1]]
    t = PageTable([], ints(bt, I32), ints([2, 2, 1, -3], I32))   # a count below 0 is a free page
    assert int(t.compact(dev_err=e)) == 3
    assert v4a.v4a_get_error(e) == v4a.DEV_BAD_PAGE


@pytest.mark.parametrize("kinds", [(), ("bf16",), ("fp4", "two", "entries", "odd", "bf16")])
def test_fork(kinds):
    rng = np.random.default_rng(len(kinds))
    for n_seq, blocks, pages, n in ((2, 1, 3, 1), (9, 5, 60, 6), (70, 9, 5000, 40)):
        c, e = Case(rng, n_seq, blocks, pages, kinds, fill=0.7), err_word()
        parents = n_seq - n
        dst = parents + rng.permutation(n)
        full = [0] * parents + [blocks] * n
        c.table.free(ints([0] * n_seq, I32), ints(full, I32), dev_err=e)
        O.free(c.bt, c.refs, [0] * n_seq, full)
        src = rng.integers(0, parents, n)
        length = rng.integers(0, blocks * 256 + 1, n)
        length[0] = blocks * 256
        if n > 4:
            length[1:5] = 0, 1, 255, 256
        c.table.fork(ints(src, I32), ints(dst, I32), ints(length, I64), dev_err=e)
        there = O.fork(c.bt, c.refs, c.host, src, dst, length)
        assert v4a.v4a_get_error(e) == (0 if there else v4a.DEV_NO_PAGE)
        c.check()


def test_fork_leaves_bad_entries_out():
    rng = np.random.default_rng(3)
    c, e = Case(rng, 12, 3, 40, ("bf16",), fill=1.0, shared=0.0), err_word()
    empty = [0] * 4 + [3] * 8
    c.table.free(ints([0] * 12, I32), ints(empty, I32))
    O.free(c.bt, c.refs, [0] * 12, empty)
    src = [0, 1, 2, 3, 0, 12, -1, 1, 2, 5]
    dst = [4, 5, 5, 3, 1, 6, 7, 12, 8, 9]        # 5 twice (and a source), itself, a parent, outside
    length = [300, 10, 10, 10, 10, 10, 10, 10, 3 * 256 + 1, 0]
    c.table.fork(ints(src, I32), ints(dst, I32), ints(length, I64), dev_err=e)
    assert v4a.v4a_get_error(e) == v4a.DEV_BAD_INDEX
    before = c.refs.copy()
    assert O.fork(c.bt, c.refs, c.host, src, dst, length)
    c.check()
    assert c.refs.sum() - before.sum() == 2      # entry 0: one block shared, one copied
    # no page left: the cut block stays without, the others are shared
    full = Case(rng, 3, 2, 2, (), fill=0.0)
    for x in (full.table.grow, lambda a, b: O.grow(full.bt, full.refs, a.tolist(), b.tolist())):
        x(ints([0, 0, 0], I32), ints([2, 0, 0], I32))
    full.table.fork(ints([0, 0], I32), ints([1, 2], I32), ints([257, 256], I64), dev_err=e)
    assert v4a.v4a_get_error(e) == v4a.DEV_NO_PAGE
    assert not O.fork(full.bt, full.refs, [], [0, 0], [1, 2], [257, 256])
    full.check()


@pytest.mark.parametrize("kinds", [("bf16",), ("fp4", "two", "entries", "odd")])
def test_copy_and_compact(kinds):
    rng = np.random.default_rng(11)
    for n_seq, blocks, pages, fill in ((1, 1, 1, 1.0), (4, 6, 50, 0.5), (30, 20, 4097, 0.5), (9, 30, 300, 0.0),
                                       (8, 40, 260, 1.0)):
        c, e = Case(rng, n_seq, blocks, pages, kinds, fill=fill), err_word()
        at = rng.permutation(pages)
        n = min(7, pages // 2)
        src, dst = at[:n], at[n:2 * n]
        c.table.copy(ints(src, I32), ints(dst, I32), dev_err=e)
        for data, R in c.host:
            for a, b in zip(src, dst):
                data[b * R:(b + 1) * R] = data[a * R:(a + 1) * R]
        c.check()
        moved = ints(np.full(pages, 99), I32)
        used = c.table.compact(moved=moved, dev_err=e)
        want_used, want = O.compact(c.bt, c.refs, c.host)
        assert v4a.v4a_get_error(e) == 0
        assert int(used) == want_used and moved.tolist() == want.tolist()
        c.check()
        assert int(c.table.compact()) == want_used                # nothing is left to move
        c.check()
    c.table.copy(ints([0, 1, 2], I32), ints([1 << 20, -1, 2], I32), dev_err=e)
    assert v4a.v4a_get_error(e) == v4a.DEV_BAD_PAGE
    c.check()


def test_counts_made_from_the_table_and_refusals():
    rng = np.random.default_rng(5)
    c = Case(rng, 6, 5, 30, ("bf16", "fp4"))
    t = PageTable(c.pools, c.d_bt)
    assert t.refs.tolist() == c.refs.tolist()
    other = ints(c.bt, I32)
    for bad in ([PagedPool(c.pools[0].data, None, other, 256)],
                [PagedPool(c.pools[0].data[:256], None, c.d_bt, 256)],
                [PagedPool(c.pools[1].data, c.pools[1].scale[:-1], c.d_bt, 256)],
                [PagedPool(c.pools[0].data.t(), None, c.d_bt, 256)],
                [PagedPool(torch.zeros(30 * 256, 3, device="cuda"), None, c.d_bt, 256)]):
        with pytest.raises(ValueError):
            PageTable(bad, c.d_bt, t.refs).compact()
    for call in (lambda: t.free(ints([0] * 5, I32), ints([1] * 6, I32)),
                 lambda: t.grow(ints([0] * 6, I64), ints([1] * 6, I32)),
                 lambda: t.fork(ints([0], I32), ints([1], I32), ints([1], I32)),
                 lambda: t.copy(ints([0], I32), ints([1, 2], I32)),
                 lambda: t.compact(moved=ints([0], I32)),
                 lambda: t.free(torch.zeros(6, dtype=I32), ints([1] * 6, I32))):
        with pytest.raises(ValueError):
            call()
    c.check()


def test_captured_and_on_a_stream_of_its_own():
    """A step of free, grow, fork and compact captured once and replayed on other tables."""
    rng = np.random.default_rng(8)
    c = Case(rng, 10, 6, 64, ("bf16", "two"), fill=0.5, shared=0.0)
    first, last = ints([0] * 10, I32), ints([0] * 8 + [6, 6], I32)
    src, dst, length = ints([0, 1], I32), ints([8, 9], I32), ints([700, 300], I64)
    g0, g1 = ints([2] * 10, I32), ints([4] * 8 + [0, 0], I32)
    used = []

    def step(stream=None):
        c.table.free(first, last, stream=stream)
        c.table.grow(g0, g1, stream=stream)
        c.table.fork(src, dst, length, stream=stream)
        used[:] = [c.table.compact(stream=stream)]

    def plain():
        a, b = [0] * 10, [0] * 8 + [6, 6]
        O.free(c.bt, c.refs, a, b)
        O.grow(c.bt, c.refs, g0.tolist(), g1.tolist())
        O.fork(c.bt, c.refs, c.host, [0, 1], [8, 9], [700, 300])
        return O.compact(c.bt, c.refs, c.host)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert plain() == int(used[0])
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        c.table.free(ints([1] * 10, I32), ints([3] * 10, I32))
        O.free(c.bt, c.refs, [1] * 10, [3] * 10)
        graph.replay()
        assert plain() == int(used[0])
        c.check()


@pytest.mark.parametrize("fmt", ["plain", "fp4"])
def test_serving_run_of_all_calls_together(fmt):
    """A prompt is inserted, forked into samples that decode on, the window's older blocks are given
    back, the pool is drawn together; every sample's attention equals that of a run in which each
    sequence had pages of its own all along."""
    rng = np.random.default_rng(21)
    H, L, W, S, steps = 16, 1200, 300, 5, 3
    cfg = v4a.latent_cfg(v4a.BF16, H, 512, v4a.rope_cfg(64),
                         cache_format=v4a.LATENT_FP4 if fmt == "fp4" else v4a.LATENT_PLAIN)

    def make(pages, n_seq):
        bt = ints(np.full((n_seq, 5), -1), I32)
        if fmt == "fp4":
            data = torch.randint(0, 256, (pages * 256, 416), dtype=torch.uint8, device="cuda")
            pool = PagedPool(data, torch.full((pages * 256,), float("nan"), device="cuda"), bt, 256)
        else:
            pool = PagedPool(torch.full((pages * 256, 576), float("nan"), dtype=BF, device="cuda"), None, bt, 256)
        return LatentLayer(cfg, pool), PageTable([pool], bt)
    prompt = torch.from_numpy(rng.standard_normal((L, 576))).to("cuda", BF)
    steps_x = torch.from_numpy(rng.standard_normal((steps, 3, 576))).to("cuda", BF)
    steps_q = torch.from_numpy(rng.standard_normal((steps, 3, H, 576))).to("cuda", BF)
    e = err_word()

    def ins(lay, rows, starts, x):
        n = [0] * lay.pool.block_table.shape[0]
        start = [0] * len(n)
        for r, s, k in zip(rows, starts, x):
            n[r], start[r] = len(k), s
        cu = np.concatenate([[0], np.cumsum(n)])
        packed = torch.cat([k for _, k in sorted(zip(rows, x), key=lambda v: v[0])])
        lay.insert(ints(cu, I32), ints(start, I64), packed[:, :512], packed[:, 512:], dev_err=e)
        return ints(cu, I32), ints(start, I64)
    # the run with shared pages: row 0 the prompt, rows 1 .. 3 its samples
    lay, table = make(24, 4)
    table.grow(ints([0] * 4, I32), ints([5, 0, 0, 0], I32), dev_err=e)
    ins(lay, [0], [0], [prompt])
    lengths = [L, 512, 130]
    table.fork(ints([0, 0, 0], I32), ints([1, 2, 3], I32), ints(lengths, I64), dev_err=e)
    table.free(ints([0] * 4, I32), ints([5, 0, 0, 0], I32), dev_err=e)
    # the run without
    own, own_table = make(24, 3)
    own_table.grow(ints([0] * 3, I32), ints([5] * 3, I32), dev_err=e)
    ins(own, [0, 1, 2], [0, 0, 0], [prompt[:n] for n in lengths])
    for i in range(steps):
        at = [n + i for n in lengths]
        table.grow(ints([0] + [a // 256 for a in at], I32), ints([0] + [a // 256 + 1 for a in at], I32), dev_err=e)
        x = [steps_x[i, k:k + 1] for k in range(3)]
        cu, start = ins(lay, [1, 2, 3], at, x)
        cu0, start0 = ins(own, [0, 1, 2], at, x)
        # blocks behind the window and the sinks
        gone = [max(0, (a + 1 - W) // 256) for a in at]
        table.free(ints([1] * 4, I32), ints([0] + gone, I32), dev_err=e)
        used = int(table.compact(dev_err=e))
        assert used == int((table.refs > 0).sum()) and (table.refs[:used] > 0).all()
        got = lay.attention(cu, start, max(at), steps_q[i], window=W, sinks=S, dev_err=e)
        want = own.attention(cu0, start0, max(at), steps_q[i], window=W, sinks=S, dev_err=e)
        assert v4a.v4a_get_error(e) == 0
        assert torch.isfinite(got).all() and (got != 0).any()
        # another number of sequences may cut the keys elsewhere, so weights are taken against other
        # references: each side rounds weights (half a step of bf16, on values up to the largest) and
        # the result (half a step)
        tol = 2 ** -7 * (prompt.float().abs().max() + want.float().abs().max())
        assert (got.float() - want.float()).abs().max() <= tol
    assert table.block_table[1].tolist()[1:3] == [-1, -1]   # 1200 positions: behind the window
