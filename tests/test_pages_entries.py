"""A page table over compressed layers, whose entry caches are still written by tokens behind a
block's end: parent and children that go on after a fork hold what they would hold on pages of their
own. On the CPU with the plain forms, on the GPU with Layer and PageTable."""
from dataclasses import replace
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import compressed_sparse_long_gb300 as v4a
import workloads as wl
from compressed_sparse_long_gb300.layer import Layer, PagedPool
from compressed_sparse_long_gb300.pages import PageTable
from oracle import pages_oracle as P
from oracle import v4a_oracle as O
from test_pages_host import world  # noqa: F401  (fixture)

I32, I64 = torch.int32, torch.int64
FORKS = [255, 256, 257, 259, 260, 512]       # a c4a block is complete 4 tokens behind its end
END, MORE, BLOCKS = 520, 8, 4
ROWS = 1 + 2 * len(FORKS)                    # the parent, children at once, children afterwards
LENGTHS = [END] + 2 * FORKS


def late_of(spec):
    return max(0, spec.W - spec.S + spec.win_off)


def tokens(rng, spec):
    """The prompt's inputs, and those of every row's own tokens."""
    def draw(n):
        b = wl.make_batch(rng, replace(spec, kind="c4a"), [0], [n])    # (with an indexer's)
        return [b.kv, b.s, b.ik, b.is_]
    return draw(END), [draw(MORE) for _ in range(ROWS)]


def scenario(run, prompt, own):
    """Parent and children on shared pages: forks as the parent passes their lengths, then again when
    it is behind all of them; then every row goes on."""
    at, n = 0, len(FORKS)
    for to in FORKS + [END]:
        run.grow([at // 256] + [0] * (ROWS - 1), [-(-to // 256)] + [0] * (ROWS - 1))
        run.insert([0], [at], [[x[at:to] for x in prompt]])
        if to in FORKS:
            run.fork([0], [1 + FORKS.index(to)], [to])
        at = to
    run.fork([0] * n, [1 + n + i for i in range(n)], FORKS)
    go_on(run, own)


def apart(run, prompt, own):
    """The same tokens in the same calls, every row on pages of its own."""
    run.grow([0] * ROWS, [BLOCKS] * ROWS)
    at = 0
    for to in FORKS + [END]:
        rows = [r for r in range(ROWS) if LENGTHS[r] >= to]
        run.insert(rows, [at] * len(rows), [[x[at:to] for x in prompt]] * len(rows))
        at = to
    go_on(run, own)


def go_on(run, own):
    for i in range(0, MORE, 4):
        run.grow([(n + i) // 256 for n in LENGTHS], [-(-(n + i + 4) // 256) for n in LENGTHS])
        run.insert(range(ROWS), [n + i for n in LENGTHS], [[x[i:i + 4] for x in t] for t in own])


def packed(rows, starts, xs):
    """(cu, start, inputs) of a batch in which `rows` have new tokens."""
    count, start = [0] * ROWS, [0] * ROWS
    for r, s, x in zip(rows, starts, xs):
        count[r], start[r] = len(x[0]), s
    cu = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    order = [x for _, x in sorted(zip(rows, xs), key=lambda v: v[0])]
    return cu, np.asarray(start, np.int64), [np.concatenate([x[k] for x in order]) for k in range(4)]


def logical_rows(spec, end):
    """(pool, rows) that hold something of a sequence of `end` tokens."""
    last = end - 1 - (spec.win_off + spec.W - 1)
    n = 0 if last < 0 else last // spec.S + 1
    yield "attn", np.arange(n)
    if spec.has_indexer:
        yield "idx", np.arange(n)
    yield "swa", np.arange(end)
    yield "state", np.arange(max(0, end - spec.W), end)


# ----------------------------------------------------------------------------------- CPU
class Plain:
    def __init__(self, rng, spec, pages, late):
        self.spec, self.late = spec, late
        self.bt = np.full((ROWS, BLOCKS), -1, np.int32)
        self.refs = np.zeros(pages, np.int32)
        R = spec.rows_per_block

        def pool(width, rows):
            return wl.Paged(rng.standard_normal((pages * rows, width)), None, self.bt, rows)
        self.pools = O.Pools(spec, pool(spec.D, R), pool(spec.d_I, R) if spec.has_indexer else None,
                             pool(spec.D, 256), pool(spec.state_width, 256))
        self.all = [p for p in (self.pools.attn, self.pools.idx, self.pools.swa, self.pools.state) if p]
        for p in self.all:
            p.bt = self.bt
        g = np.random.default_rng(1)
        self.params = wl.layer_params(g, spec)

    def grow(self, first, last):
        assert P.grow(self.bt, self.refs, first, last)

    def insert(self, rows, starts, xs):
        cu, start, x = packed(rows, starts, xs)
        O.compress_insert(self.spec, *self.params, self.pools, cu, start, *x)

    def fork(self, src, dst, length):
        assert P.fork(self.bt, self.refs, [(p.data, p.R) for p in self.all], src, dst, length, self.late)


def wrong_rows(spec, a, b):
    """(sequence, pool, row) of what differs between two runs."""
    bad = []
    for r in range(ROWS):
        for name, rows in logical_rows(spec, LENGTHS[r] + MORE):
            x, y = (getattr(p, name).data[getattr(p, name).slots(r, rows)] for p in (a.pools, b.pools))
            bad += [(r, name, int(k)) for k in rows[(x != y).any(1)]]
    return bad


SMALL = dict(D=16, d_r=8, H=1, H_I=1, d_I=8, swa=32)


@pytest.mark.parametrize("kind,win_off", [("c4a", 0), ("c4a", -2), ("c4a", -4), ("c4a", -7), ("c128a", 0),
                                          ("c128a", -64)])
def test_rows_go_on_apart_after_a_fork(kind, win_off):
    rng = np.random.default_rng(4)
    spec = wl.LayerSpec(kind, False, win_off=win_off, **SMALL)
    prompt, own = tokens(rng, spec)
    late = late_of(spec)
    assert late == (4 + win_off if kind == "c4a" and win_off > -4 else 0)
    alone = Plain(rng, spec, ROWS * BLOCKS, 0)
    apart(alone, prompt, own)
    shared = Plain(rng, spec, ROWS * BLOCKS, late)
    scenario(shared, prompt, own)
    assert wrong_rows(spec, shared, alone) == []
    assert (shared.refs == np.bincount(shared.bt[shared.bt >= 0], minlength=len(shared.refs))).all()
    assert shared.refs.sum() > (shared.refs > 0).sum()                 # blocks are shared all the same
    if late:
        # sharing every whole block is not enough, nor is a token less than the layer says
        for less in (0, late - 1):
            wrong = Plain(rng, spec, ROWS * BLOCKS, less)
            scenario(wrong, prompt, own)
            assert wrong_rows(spec, wrong, alone) != []


def test_fork_with_late_rows_by_hand():
    bt = np.array([[2, 0, -1], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1]], np.int32)
    refs = np.array([1, 0, 1, 0, 0, 0, 0], np.int32)
    data = np.arange(7 * 64)
    # 256 + 3 positions: entry 63 of the first block is not complete; 256 + 4: it is
    assert P.fork(bt, refs, [(data, 64)], [0, 0, 0], [1, 2, 3], [259, 260, 512], late=4)
    assert bt.tolist() == [[2, 0, -1], [1, 3, -1], [2, 4, -1], [2, 5, -1]]
    assert refs.tolist() == [1, 1, 3, 1, 1, 1, 0]
    assert data[64:128].tolist() == list(range(128, 192)) and data[192] == 0 and data[193] == 193
    assert data[5 * 64:6 * 64].tolist() == list(range(64))


def test_layers_say_how_late_their_entries_are():
    def pool():
        return PagedPool(torch.zeros(1, 1), None, torch.zeros(1, 1, dtype=I32), 64)
    for kind, w, s, off, want in ((v4a.C4A, 8, 4, 0, 4), (v4a.C4A, 8, 4, -4, 0), (v4a.C4A, 8, 4, -6, 0),
                                  (v4a.C128A, 128, 128, 0, 0)):
        cfg = v4a.layer_cfg(kind, v4a.FP32, 128, 32, 8, 4, 32, w, s, off, 128, 1e4, 1e-6, 0.1)
        lay = Layer(cfg, None, None, None, pool(), pool(), pool(), pool())
        assert [p.late for p in (lay.attn, lay.idx, lay.swa, lay.state)] == [want, want, 0, 0]
        assert lay.attn.clone().late == want


@pytest.mark.parametrize("late,want", [(-1, v4a.ERR_ARG), (256, v4a.ERR_ARG)])
def test_late_outside_a_block_is_refused(late, want):
    lib = v4a.library()
    t = v4a.PageTableDesc(block_table=256, refs=4096, n_seq=4, max_blocks=8, n_pages=100)
    one = (v4a.Pool * 1)(v4a.Pool(4096, None, 1152, 256, late, 0))
    assert lib.v4a_pages_fork(t, one, 1, 2, 64, 64, 64, 4096, 1 << 20, None, None) == want
    assert lib.v4a_pages_copy(t, one, 1, 2, 64, 64, None, None) == want
    assert lib.v4a_pages_compact(t, one, 1, 64, None, 4096, 1 << 20, None, None) == want


def test_the_table_hands_late_on(world):  # noqa: F811
    z = world.zeros
    bt = z(3, 4, dtype=I32)
    pool = PagedPool(z(6 * 64, 128, dtype=torch.uint8), z(6 * 64, dtype=torch.float32), bt, 64)
    t = PageTable([pool, PagedPool(z(6 * 256, 576), None, bt, 256)], bt, z(6, dtype=I32))
    for late in (0, 4, 255):
        pool.late = late                                # a pool that changes is looked at again
        t.fork(z(1, dtype=I32), z(1, dtype=I32), z(1, dtype=I64))
        assert [(p.late, p.reserved) for p in world.lib.seen.pop()[1][1]] == [(late, 0), (0, 0)]
    for late in (-1, 256, 1 << 16):
        pool.late = late
        with pytest.raises(ValueError):
            t.fork(z(1, dtype=I32), z(1, dtype=I32), z(1, dtype=I64))


# ----------------------------------------------------------------------------------- GPU
def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)


class Device:
    """Layers whose pools share one table."""

    def __init__(self, rng, specs, pages):
        self.specs, self.err = specs, torch.zeros(1, dtype=I32, device="cuda")
        self.bt = torch.full((ROWS, BLOCKS), -1, dtype=I32, device="cuda")
        self.layers, g = [], np.random.default_rng(1)
        for spec in specs:
            R = spec.rows_per_block
            host = SimpleNamespace(spec=spec, **dict(zip(("bias", "gamma", "ibias"), wl.layer_params(g, spec))))
            none = np.zeros((1, 1), np.int32)

            def pool(width, rows, coded):
                n = pages * rows
                if not coded:
                    return wl.Paged(wl._round(rng.standard_normal((n, width)), True), None, none, rows)
                return wl.Paged(rng.integers(0, 120, (n, width)).astype(np.uint8),
                                rng.random(n).astype(np.float32), none, rows)
            host.attn = pool(spec.D, R, spec.fp8)
            host.idx = None
            if spec.has_indexer:
                host.idx = pool(spec.d_I // 2 if spec.idx_fp4 else spec.d_I, R, spec.fp8)
            host.swa, host.state = pool(spec.D, 256, spec.fp8), pool(spec.state_width, 256, False)
            lay = Layer.from_host(host)
            for p in (lay.attn, lay.idx, lay.swa, lay.state):
                if p is not None:
                    p.block_table = self.bt
            self.layers.append(lay)
        pools = [p for lay in self.layers for p in (lay.attn, lay.idx, lay.swa, lay.state) if p is not None]
        self.table = PageTable(pools, self.bt)

    def grow(self, first, last):
        self.table.grow(dev(np.asarray(first), I32), dev(np.asarray(last), I32), dev_err=self.err)

    def fork(self, src, dst, length):
        self.table.fork(dev(np.asarray(src), I32), dev(np.asarray(dst), I32), dev(np.asarray(length), I64),
                        dev_err=self.err)

    def insert(self, rows, starts, xs):
        cu, start, x = packed(rows, starts, xs)
        cu, start = dev(cu, I32), dev(start, I64)
        for spec, lay in zip(self.specs, self.layers):
            kv, s, ik, is_ = (dev(v, lay.in_dtype) for v in x)
            lay.compress_insert(cu, start, kv, s, *((ik, is_) if spec.has_indexer else ()), dev_err=self.err)

    def attend(self, rng):
        """Every layer's output for a query behind each row's last token."""
        n = ROWS
        seq, pos = dev(np.arange(n), I32), dev(np.asarray(LENGTHS) + MORE - 1, I64)
        outs = []
        for spec, lay in zip(self.specs, self.layers):
            q = wl.make_queries(rng, spec, np.arange(n), np.arange(n), w_uniform=False)
            top = None
            if spec.has_indexer:
                top = lay.index_topk(seq, pos, END + MORE, dev(q.q_idx, lay.in_dtype), dev(q.w, torch.float32),
                                     dev_err=self.err)
                outs.append(top)
            outs.append(lay.attention(seq, pos, END + MORE, dev(q.q, lay.in_dtype), top, dev_err=self.err))
        return outs


def held(pool, row, rows):
    """Bytes (and scales) of logical rows of a sequence."""
    bt, R = pool.block_table.cpu().numpy(), pool.rows_per_block
    s = torch.from_numpy(bt[row, rows // R].astype(np.int64) * R + rows % R).cuda()
    assert (s >= 0).all()
    return pool.data[s], None if pool.scale is None else pool.scale[s]


@pytest.mark.gpu
@pytest.mark.parametrize("specs", [
    [wl.LayerSpec("c4a", True), wl.LayerSpec("c128a", True)],
    [wl.LayerSpec("c4a", True, idx_fp4=True, win_off=-2)],
    [wl.LayerSpec("c4a", False, D=128, d_r=32, H=8, H_I=4, d_I=32, top_k=64)]],
    ids=["c4a+c128a", "fp4 index, offset -2", "fp32"])
def test_layers_go_on_apart_after_a_fork(specs):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    rng = np.random.default_rng(9)
    prompt, own = tokens(rng, specs[0])
    shared, alone = Device(rng, specs, 40), Device(rng, specs, ROWS * BLOCKS)
    scenario(shared, prompt, own)
    apart(alone, prompt, own)
    for run in (shared, alone):
        assert v4a.v4a_get_error(run.err) == 0
    bt, refs = shared.bt.cpu().numpy(), shared.table.refs.cpu().numpy()
    assert (refs == np.bincount(bt[bt >= 0], minlength=len(refs))).all() and refs.max() > 1
    for spec, a, b in zip(specs, shared.layers, alone.layers):
        for r in range(ROWS):
            for name, rows in logical_rows(spec, LENGTHS[r] + MORE):
                (x, xs), (y, ys) = held(getattr(a, name), r, rows), held(getattr(b, name), r, rows)
                assert torch.equal(x, y), (spec.kind, r, name, rows[(x != y).any(1).cpu().numpy()])
                assert xs is None or torch.equal(xs, ys), (spec.kind, r, name)
    for x, y in zip(shared.attend(np.random.default_rng(2)), alone.attend(np.random.default_rng(2))):
        assert torch.equal(x, y) and torch.isfinite(x.float()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("late", [4, 100, 255])
def test_fork_equals_the_plain_form(late):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from test_pages_gpu import Case
    rng = np.random.default_rng(late)
    e = torch.zeros(1, dtype=I32, device="cuda")
    for n_seq, blocks, pages, n, fill in ((2, 1, 3, 1, 0.7), (9, 5, 60, 6, 0.7), (9, 5, 26, 6, 1.0),
                                          (70, 9, 9000, 40, 0.7)):
        c = Case(rng, n_seq, blocks, pages, ("bf16", "entries", "two", "fp4", "odd"), fill=fill)
        c.pools[1].late, c.pools[2].late = late, late // 2
        parents = n_seq - n
        full = [0] * parents + [blocks] * n
        c.table.free(dev(np.zeros(n_seq), I32), dev(np.asarray(full), I32), dev_err=e)
        P.free(c.bt, c.refs, [0] * n_seq, full)
        src, dst = rng.integers(0, parents, n), parents + rng.permutation(n)
        length = rng.integers(0, blocks * 256 + 1, n)
        length[0] = blocks * 256
        if n > 4:
            length[1:5] = 256, 255 + late, 256 + late, 0
        c.table.fork(dev(src, I32), dev(dst, I32), dev(length, I64), dev_err=e)
        there = P.fork(c.bt, c.refs, c.host, src, dst, length, late)
        assert v4a.v4a_get_error(e) == (0 if there else v4a.DEV_NO_PAGE)
        c.check()


@pytest.mark.gpu
def test_a_captured_fork_follows_lengths_and_tables():
    """One capture, on a stream of its own, replayed with other lengths and sources."""
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from test_pages_gpu import Case
    rng = np.random.default_rng(17)
    c, e = Case(rng, 9, 5, 60, ("entries", "bf16"), fill=0.8), torch.zeros(1, dtype=I32, device="cuda")
    c.pools[0].late = 4
    full = np.array([0] * 5 + [5] * 4)
    zero, last = dev(np.zeros(9), I32), dev(full, I32)
    src, dst, length = dev(np.zeros(4), I32), dev(np.arange(5, 9), I32), dev(np.zeros(4), I64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        c.table.free(zero, last, dev_err=e)
        c.table.fork(src, dst, length, dev_err=e)
    for lengths in ([256, 257, 259, 260], [1280, 1024, 515, 3], [0, 512, 768, 771]):
        parents = rng.integers(0, 5, 4)
        src.copy_(dev(parents, I32))
        length.copy_(dev(np.asarray(lengths), I64))
        graph.replay()
        P.free(c.bt, c.refs, [0] * 9, full)
        there = P.fork(c.bt, c.refs, c.host, parents, list(range(5, 9)), lengths, 4)
        assert v4a.v4a_get_error(e) == (0 if there else v4a.DEV_NO_PAGE)
        c.check()
