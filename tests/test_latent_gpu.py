"""GPU: rotary positions, the latent cache and both forms of latent attention against their
64-bit definitions. Tolerances are derived in latent_helpers and beside each check."""
import numpy as np
import pytest
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300.latent import LatentLayer, rope
from latent_helpers import (BF, F32, attn_tolerance, batch, check, err_word, f64, half_step, ints,
                            layer, logit_bound, rand)
from oracle import latent_oracle as O

pytestmark = pytest.mark.gpu

SCALED = dict(base=10000.0, factor=8.0, orig_max_pos=4096.0, low=1.0, high=32.0)
KINDS = {"none": v4a.ROPE_SCALE_NONE, "linear": v4a.ROPE_SCALE_LINEAR,
         "parts": v4a.ROPE_SCALE_BY_PARTS, "yarn": v4a.ROPE_SCALE_YARN}


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------- rope
def _rope_case(dim, layout, scaling, amp=1.0):
    kw = {} if scaling == "none" else dict(SCALED)
    cfg = v4a.rope_cfg(dim, v4a.ROPE_HALF if layout == "half" else v4a.ROPE_INTERLEAVED,
                       scaling=KINDS[scaling], amplitude=amp, **kw)
    rate = O.rates(dim, 10000.0, scaling, 8.0, 4096.0, 1.0, 32.0)
    return cfg, rate


def _rope_tol(x, ref, dtype, layout, amp):
    """fp32: the angle's constants are fp32 numbers in cfg (exact here); cosine, sine, two
    products and a sum each round within 2^-23 of the pair's size; then one rounding."""
    d = x.shape[-1]
    a, b = (x[..., :d // 2], x[..., d // 2:]) if layout == "half" else (x[..., ::2], x[..., 1::2])
    size = amp * (np.abs(a) + np.abs(b))
    size = (np.concatenate([size, size], -1) if layout == "half"
            else np.repeat(size, 2, -1))
    return 4 * 2.0 ** -23 * size + half_step(dtype) * np.abs(ref) + 1e-30


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["pairs", "half"])
@pytest.mark.parametrize("scaling", ["none", "linear", "parts", "yarn"])
def test_rope_matches_its_definition(dtype, layout, scaling):
    rng = np.random.default_rng(5)
    for dim, n, h, amp in ((64, 37, 5, 1.0), (32, 3, 64, 1.25), (2, 7, 3, 1.0), (10, 5, 1, 0.5),
                           (256, 4, 2, 1.0)):
        cfg, rate = _rope_case(dim, layout, scaling, amp)
        x = rand(rng, dtype, n, h, dim)
        pos = rng.integers(0, 1 << 21, n)
        pos[0], pos[-1] = 0, (1 << 36) - 1
        for inverse in (False, True):
            e = err_word()
            y = rope(cfg, x, ints(pos, torch.int64), inverse=inverse, dev_err=e)
            assert v4a.v4a_get_error(e) == 0
            # the largest position times a 64-bit rate is only known to 2^36 2^-53 radians
            ref = O.rope(f64(x), pos, rate, layout, amp, inverse)
            tol = _rope_tol(f64(x), ref, dtype, layout, amp)
            tol[-1] += 2.0 ** -14 * amp * np.abs(f64(x[-1])).max()
            check(y, ref, tol)


def test_rope_inverse_undoes_it_and_is_its_gradient():
    rng = np.random.default_rng(6)
    cfg, rate = _rope_case(64, "half", "yarn", 1.1)
    x, g = rand(rng, F32, 9, 4, 64), rand(rng, F32, 9, 4, 64)
    pos = ints(rng.integers(0, 100000, 9), torch.int64)
    y, gx = rope(cfg, x, pos), rope(cfg, g, pos, inverse=True)
    back = rope(cfg, y, pos, inverse=True)
    # two passes, each within 4 2^-23 of the pair's size (at most 2 max |x| amp^2)
    assert (back - 1.1 ** 2 * x).abs().max() <= 8 * 2.0 ** -23 * 4 * 1.21 * x.abs().max()
    # <g, J dx> = <J^T g, dx>, and J by differences of the 64-bit form
    dx = rng.standard_normal(tuple(x.shape))
    step = 1e-6
    p = pos.cpu().numpy()
    dy = (O.rope(f64(x) + step * dx, p, rate, "half", 1.1) -
          O.rope(f64(x) - step * dx, p, rate, "half", 1.1)) / (2 * step)
    lhs, rhs = float((f64(g) * dy).sum()), float((f64(gx) * dx).sum())
    assert abs(lhs - rhs) <= 1e-5 * float((np.abs(f64(g)) * np.abs(dy)).sum())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["pairs", "half"])
def test_rope_part_of_wider_heads_in_place_and_unaligned(dtype, layout):
    rng = np.random.default_rng(7)
    cfg, rate = _rope_case(64, layout, "none")
    pos = rng.integers(0, 5000, 11)
    for off, width in ((512, 576), (3, 77), (0, 64)):
        q = rand(rng, dtype, 11, 6, width)
        before = q.clone()
        part = q[..., off:off + 64]
        assert rope(cfg, part, ints(pos, torch.int64), out=part) is part
        ref = O.rope(f64(before[..., off:off + 64]), pos, rate, layout)
        check(q[..., off:off + 64], ref,
              _rope_tol(f64(before[..., off:off + 64]), ref, dtype, layout, 1.0))
        assert torch.equal(q[..., :off], before[..., :off])
        assert torch.equal(q[..., off + 64:], before[..., off + 64:])
    # rows shared by every head (stride 0) and a transposed batch
    x = rand(rng, dtype, 11, 1, 64).expand(11, 6, 64)
    y = rope(cfg, x, ints(pos, torch.int64))
    assert all(torch.equal(y[:, 0], y[:, h]) for h in range(6))
    z = rand(rng, dtype, 6, 11, 64)
    assert torch.equal(rope(cfg, z.transpose(0, 1), ints(pos, torch.int64)),
                       rope(cfg, z.transpose(0, 1).contiguous(), ints(pos, torch.int64)))


def test_rope_bad_positions_are_left_unwritten():
    rng = np.random.default_rng(8)
    cfg, _ = _rope_case(64, "pairs", "none")
    x, e = rand(rng, BF, 4, 2, 64), err_word()
    out = torch.full_like(x, 7.0)
    rope(cfg, x, ints([3, -1, 1 << 36, 9], torch.int64), out=out, dev_err=e)
    assert v4a.v4a_get_error(e) == v4a.DEV_BAD_POS
    assert (out[1:3] == 7).all() and (out[0] != 7).any()
    # 2-D rows, no rows
    assert torch.equal(rope(cfg, x[:, 0], ints([0, 1, 2, 3], torch.int64)),
                       rope(cfg, x, ints([0, 1, 2, 3], torch.int64))[:, 0])
    assert rope(cfg, x[:0], ints([], torch.int64)).shape == (0, 2, 64)


# ---------------------------------------------------------------------- insert, gather
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("latent,dim,layout,norm", [(512, 64, "pairs", True), (512, 64, "half", False),
                                                    (8, 8, "half", True), (1024, 128, "pairs", True),
                                                    (136, 24, "half", True)])
def test_insert_then_gather(dtype, latent, dim, layout, norm):
    rng = np.random.default_rng(9)
    total, new = [1, 700, 40, 513, 0, 256], [1, 300, 40, 2, 0, 1]
    kw = dict(layout=v4a.ROPE_HALF if layout == "half" else v4a.ROPE_INTERLEAVED,
              scaling=v4a.ROPE_SCALE_YARN, amplitude=1.1, **SCALED)
    lay, bt = layer(rng, dtype, 4, total, latent, dim, gamma=norm, rope_kw=kw)
    cu, start = batch(total, new)
    n, pad = int(cu[-1]), 3                        # three rows behind the last sequence
    x = rand(rng, dtype, n + pad, latent + dim + 8)
    x[n:] = float("nan")
    before, e = lay.pool.data.clone(), err_word()
    lay.insert(ints(cu, torch.int32), ints(start, torch.int64), x[:, :latent],
               x[:, latent:latent + dim], dev_err=e)
    assert v4a.v4a_get_error(e) == 0
    ref = f64(before)
    g = f64(lay.gamma) if norm else None
    rate = O.rates(dim, 10000.0, "yarn", 8.0, 4096.0, 1.0, 32.0)
    wrote = O.insert(ref, bt, cu, start, f64(x[:, :latent]), f64(x[:, latent:latent + dim]), g,
                     1e-6, rate, layout, 1.1)
    assert sorted(set(wrote)) == sorted(wrote) and len(wrote) == n
    keep = np.setdiff1d(np.arange(len(ref)), wrote)
    assert torch.equal(lay.pool.data[keep], before[keep])
    # the mean square is a sum of `latent` fp32 products, then a root, a division, two
    # products: (latent + 8) 2^-24 of the value; the rotation as in the rope tests
    tol = np.zeros((n, latent + dim))
    xs = f64(x[:n])
    tol[:, :latent] = (latent + 8) * 2.0 ** -24 * np.abs(ref[wrote][:, :latent])
    tol[:, latent:] = _rope_tol(xs[:, latent:latent + dim], ref[wrote][:, latent:], F32, layout, 1.1)
    check(lay.pool.data[wrote], ref[wrote], tol + half_step(dtype) * np.abs(ref[wrote]) + 1e-30)

    # gather every position of every sequence, into a longer result
    cuk = np.concatenate([[0], np.cumsum(total)])
    out = torch.full((int(cuk[-1]) + 2, latent + dim), 5.0, dtype=dtype, device="cuda")
    zero = torch.zeros(len(total), dtype=torch.int64, device="cuda")
    assert lay.gather(ints(cuk, torch.int32), zero, len(out), out=out, dev_err=e) is out
    assert v4a.v4a_get_error(e) == 0
    rows = [O.slot(bt, b, p) for b, t in enumerate(total) for p in range(t)]
    assert torch.equal(out[:len(rows)], lay.pool.data[rows]) and (out[len(rows):] == 5).all()
    # a middle range
    part = lay.gather(ints([0, 0, 100, 100, 110, 110, 110], torch.int32),
                      ints([0, 250, 0, 500, 0, 0], torch.int64), 110)
    rows = [O.slot(bt, 1, p) for p in range(250, 350)] + [O.slot(bt, 3, p) for p in range(500, 510)]
    assert torch.equal(part, lay.pool.data[rows])


def test_insert_and_gather_with_missing_and_bad_pages():
    rng = np.random.default_rng(10)
    lay, bt = layer(rng, BF, 4, [600, 300], hole=(0, 1))
    lay.pool.block_table[1, 1] = 10 ** 6
    cu, start = batch([600, 300], [400, 300])
    x, before, e = rand(rng, BF, 700, 576), lay.pool.data.clone(), err_word()
    lay.insert(ints(cu, torch.int32), ints(start, torch.int64), x[:, :512], x[:, 512:], dev_err=e)
    assert v4a.v4a_get_error(e) == v4a.DEV_MISSING_PAGE | v4a.DEV_BAD_PAGE
    same = (lay.pool.data == before).all(1).cpu().numpy()
    hit = sorted([O.slot(bt, 0, p) for p in list(range(200, 256)) + list(range(512, 600))] +
                 [O.slot(bt, 1, p) for p in range(256)])
    assert np.flatnonzero(~same).tolist() == hit
    out = lay.gather(ints([0, 600, 900], torch.int32), ints([0, 0], torch.int64), 900, dev_err=e)
    assert v4a.v4a_get_error(e) == v4a.DEV_MISSING_PAGE | v4a.DEV_BAD_PAGE
    assert (out[256:512] == 0).all() and (out[600 + 256:] == 0).all()
    assert torch.equal(out[512:600], lay.pool.data[[O.slot(bt, 0, p) for p in range(512, 600)]])
    # positions outside the table, and negative ones
    lay.insert(ints([0, 1, 2], torch.int32), ints([-1, 256 * bt.shape[1]], torch.int64), x[:2, :512],
               x[:2, 512:], dev_err=e)
    assert v4a.v4a_get_error(e) == v4a.DEV_BAD_POS | v4a.DEV_MISSING_PAGE
    out = lay.gather(ints([0, 2, 2], torch.int32), ints([-1, 0], torch.int64), 2, dev_err=e)
    assert v4a.v4a_get_error(e) == v4a.DEV_MISSING_PAGE
    assert (out[0] == 0).all() and torch.equal(out[1], lay.pool.data[O.slot(bt, 0, 0)])


# ------------------------------------------------------------------- absorbed attention
def _attn(lay, bt, total, new, q, max_pos=None, start=None, out=None):
    cu, st = batch(total, new)
    start = st if start is None else np.asarray(start)
    e = err_word()
    mp = max(max(total) - 1, 0) if max_pos is None else max_pos
    got = lay.attention(ints(cu, torch.int32), ints(start, torch.int64), mp, q, dev_err=e, out=out)
    flags = v4a.v4a_get_error(e)
    pool = np.nan_to_num(f64(lay.pool.data))       # rows that no query sees may hold anything
    c, s = lay.cfg.latent_dim, lay.cfg.softmax_scale
    ref, mag = O.attention(pool, bt, cu, start, f64(q)[:cu[-1]], s, c, mp)
    tol = attn_tolerance(lay.dtype, ref, mag, lay.width, max(total),
                         logit_bound(f64(q)[:cu[-1]], pool, s))
    return got, ref, tol, flags


SHAPES = [
    # dtype, heads, latent, rope, total, new
    (F32, 8, 128, 32, [1, 5, 300], [1, 1, 1]),
    (F32, 3, 96, 8, [130, 40], [7, 40]),
    (F32, 2, 1024, 128, [70], [2]),
    (BF, 5, 256, 32, [33, 1000], [4, 1]),
    (BF, 64, 512, 64, [1], [1]),
    (BF, 64, 512, 64, [127, 128, 129, 1, 700], [1, 1, 1, 1, 1]),
    (BF, 128, 512, 64, [1500, 31], [1, 1]),
    (BF, 128, 512, 64, [300, 260], [3, 1]),
    (BF, 1, 512, 64, [257, 900], [1, 1]),
    (BF, 16, 512, 64, [500, 7, 0, 1300], [30, 7, 0, 1]),
    (BF, 5, 512, 64, [200, 400], [77, 13]),
    (BF, 96, 512, 64, [130], [130]),
    (BF, 64, 512, 64, [5000], [2]),
    (BF, 64, 512, 64, [700, 40, 2], [650, 40, 1]),       # many units: whole ones in turn
    (BF, 128, 512, 64, [300, 290], [290, 1]),
    (BF, 40, 512, 64, [256, 255], [2, 255]),
    (F32, 16, 64, 16, [1300], [1300]),
    (BF, 300, 512, 64, [200, 3], [1, 2]),
]


@pytest.mark.parametrize("dtype,heads,latent,dim,total,new", SHAPES)
def test_attention_matches_its_definition(dtype, heads, latent, dim, total, new):
    rng = np.random.default_rng(11)
    lay, bt = layer(rng, dtype, heads, total, latent, dim, fill=float("nan"))
    q = rand(rng, dtype, sum(new), heads, latent + dim)
    got, ref, tol, flags = _attn(lay, bt, total, new, q)
    assert flags == 0
    check(got, ref, tol)


@pytest.mark.parametrize("gain", [0.01, 6.0])
def test_attention_flat_and_peaked(gain):
    """Nearly uniform weights, and logits in the hundreds (running maxima that keep rising)."""
    rng = np.random.default_rng(12)
    total, new = [2500, 900], [1, 2]
    lay, bt = layer(rng, BF, 64, total)
    for b in range(2):                             # later keys longer: the maximum moves
        for blk in range(bt.shape[1]):
            if bt[b, blk] >= 0:
                lay.pool.data[bt[b, blk] * 256:(bt[b, blk] + 1) * 256] *= 0.2 + 0.2 * blk
    q = gain * rand(rng, BF, 3, 64, 576)
    got, ref, tol, flags = _attn(lay, bt, total, new, q)
    assert flags == 0
    check(got, ref, tol)


def test_attention_rows_behind_the_last_sequence_are_left_alone():
    rng = np.random.default_rng(13)
    for heads in (64, 16):
        lay, bt = layer(rng, BF, heads, [400, 90])
        q = rand(rng, BF, 7, heads, 576)
        q[5:] = float("nan")
        out = torch.full((7, heads, 512), 3.0, dtype=BF, device="cuda")
        got, ref, tol, flags = _attn(lay, bt, [400, 90], [4, 1], q, out=out)
        assert flags == 0 and got is out and (out[5:] == 3).all()
        check(got[:5], ref, tol)


@pytest.mark.parametrize("dtype,heads", [(BF, 64), (BF, 16), (F32, 4)])
def test_attention_missing_pages_and_positions(dtype, heads):
    rng = np.random.default_rng(14)
    total, new = [1000, 200, 300], [2, 1, 1]
    lay, bt = layer(rng, dtype, heads, total, hole=(0, 1))
    bt[1, 0] = -1                                  # a sequence without any key
    lay.pool.block_table[1, 0] = -1
    q = rand(rng, dtype, 4, heads, 576)
    got, ref, tol, flags = _attn(lay, bt, total, new, q)
    assert flags == v4a.DEV_MISSING_PAGE
    assert (got[2] == 0).all()
    check(got, ref, tol)
    # positions past max_pos see the keys up to it; negative ones none
    got, ref, tol, flags = _attn(lay, bt, total, new, q, max_pos=250, start=[-1, -5, 100])
    assert flags == v4a.DEV_BAD_POS
    got, ref, tol, flags = _attn(lay, bt, total, new, q, max_pos=250, start=[-1, -5, 299])
    assert flags == v4a.DEV_BAD_POS
    assert (got[0] == 0).all() and (got[2] == 0).all()
    check(got, ref, tol)
    # a page outside the pool is not read
    lay.pool.block_table[2, 1] = 1 << 30
    bt[2, 1] = -1
    got, ref, tol, flags = _attn(lay, bt, total, new, q)
    assert flags == v4a.DEV_MISSING_PAGE | v4a.DEV_BAD_PAGE
    check(got, ref, tol)


def test_attention_not_finite_keys():
    """A NaN that a query sees reaches its output, and no other sequence's."""
    rng = np.random.default_rng(15)
    lay, bt = layer(rng, BF, 64, [300, 300])
    lay.pool.data[O.slot(bt, 0, 150), 3] = float("nan")
    q = rand(rng, BF, 2, 64, 576)
    got = lay.attention(ints([0, 1, 2], torch.int32), ints([299, 299], torch.int64), 299, q)
    assert got[0].isnan().all() and got[1].isfinite().all()


def test_attention_is_repeatable_and_independent_of_the_batch():
    rng = np.random.default_rng(16)
    total = [3000, 10, 777, 1]
    lay, bt = layer(rng, BF, 64, total)
    q = rand(rng, BF, 4, 64, 576)
    cu, st = ints([0, 1, 2, 3, 4], torch.int32), ints(np.array(total) - 1, torch.int64)
    a = lay.attention(cu, st, 2999, q)
    assert all(torch.equal(a, lay.attention(cu, st, 2999, q)) for _ in range(5))


def test_attention_two_streams_and_graph():
    """Calls on two streams at once, and two captured graphs replayed together, each with a
    workspace of its own."""
    rng = np.random.default_rng(17)
    total = [6000, 2500]
    lay, bt = layer(rng, BF, 64, total)
    cu, st = ints([0, 1, 2], torch.int32), ints(np.array(total) - 1, torch.int64)
    qs = [rand(rng, BF, 2, 64, 576) for _ in range(2)]
    ref = [lay.attention(cu, st, 5999, q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            outs[i].append(lay.attention(cu, st, 5999, qs[i], stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref[i]) for i in range(2) for o in outs[i])
    graphs, gout = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gout.append(lay.attention(cu, st, 5999, qs[i]))
        graphs.append(g)
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(gout[i], ref[i]) for i in range(2))
    # the lengths are read on the device: a captured call follows them
    st.copy_(ints([99, 1700], torch.int64))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(gout[0], lay.attention(cu, st, 5999, qs[0]))


def test_attention_many_sequences():
    rng = np.random.default_rng(18)
    total = [int(x) for x in rng.integers(0, 60, 1024)]
    new = [min(t, int(x)) for t, x in zip(total, rng.integers(0, 3, 1024))]
    lay, bt = layer(rng, BF, 8, total)
    q = rand(rng, BF, sum(new), 8, 576)
    got, ref, tol, flags = _attn(lay, bt, total, new, q)
    assert flags == 0
    check(got, ref, tol)


# ------------------------------------------------------------------- expanded attention
EXPANDED = [
    # dtype, heads, nope, rope, v, keys, queries
    (F32, 3, 32, 8, 40, [1, 50, 100], [1, 50, 3]),
    (F32, 2, 256, 128, 256, [60], [33]),
    (BF, 4, 64, 32, 64, [200], [130]),
    (BF, 2, 128, 64, 128, [1], [1]),
    (BF, 3, 128, 64, 128, [127, 128, 129, 0, 255], [127, 128, 129, 0, 255]),
    (BF, 2, 128, 64, 128, [700, 300], [257, 1]),
    (BF, 1, 128, 64, 128, [500, 9, 1025], [500, 9, 400]),
    (BF, 5, 128, 64, 128, [384], [256]),
    (BF, 2, 128, 64, 128, [90, 0, 513], [200, 6, 513]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,heads,nope,dim,vd,nk,nq", EXPANDED)
def test_expanded_matches_its_definition(dtype, heads, nope, dim, vd, nk, nq, causal):
    """Ragged lengths (more queries than keys among them: rows without a key), keys and
    values as slices of one projection, and NaN in the rows behind the last sequence."""
    rng = np.random.default_rng(19)
    rc = v4a.rope_cfg(dim)
    cfg = v4a.latent_cfg(v4a.BF16 if dtype == BF else v4a.FP32, heads, 512, rc, nope, vd)
    lay = LatentLayer(cfg, None)
    cuq, cuk = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    q = rand(rng, dtype, int(cuq[-1]) + 2, heads, nope + dim)
    kv = rand(rng, dtype, int(cuk[-1]) + 3, heads, nope + vd)
    pe = rand(rng, dtype, int(cuk[-1]) + 3, 512 + dim)[:, 512:]
    for t, n in ((q, cuq[-1]), (kv, cuk[-1]), (pe, cuk[-1])):
        t[int(n):] = float("nan")
    out = torch.full((len(q), heads, vd), 3.0, dtype=dtype, device="cuda")
    lay.attention_expanded(ints(cuq, torch.int32), ints(cuk, torch.int32), q, kv[..., :nope], pe,
                           kv[..., nope:], causal=causal, out=out)
    n = int(cuk[-1])
    qh, kh, ph, vh = f64(q)[:cuq[-1]], f64(kv)[:n, :, :nope], f64(pe)[:n], f64(kv)[:n, :, nope:]
    ref, mag = O.attention_expanded(cuq, cuk, qh, kh, ph, vh, cfg.softmax_scale, causal)
    lm = max(logit_bound(qh[:, h], np.concatenate([kh[:, h], ph], 1), cfg.softmax_scale)
             for h in range(heads))
    check(out[:cuq[-1]], ref, attn_tolerance(dtype, ref, mag, nope + dim, max(nk), lm))
    assert (out[int(cuq[-1]):] == 3).all()


def test_expanded_peaked_and_two_streams():
    rng = np.random.default_rng(20)
    cfg = v4a.latent_cfg(v4a.BF16, 4, 512, v4a.rope_cfg(64))
    lay = LatentLayer(cfg, None)
    q, kv, pe = 5 * rand(rng, BF, 600, 4, 192), rand(rng, BF, 600, 4, 256), rand(rng, BF, 600, 64)
    kv[:, :, :128] *= torch.linspace(0.2, 2, 600, device="cuda", dtype=BF)[:, None, None]
    cu = ints([0, 600], torch.int32)
    ref, mag = O.attention_expanded([0, 600], [0, 600], f64(q), f64(kv)[..., :128], f64(pe),
                                    f64(kv)[..., 128:], cfg.softmax_scale, True)
    lm = max(logit_bound(f64(q)[:, h], np.concatenate([f64(kv)[:, h, :128], f64(pe)], 1),
                         cfg.softmax_scale) for h in range(4))
    a = lay.attention_expanded(cu, cu, q, kv[..., :128], pe, kv[..., 128:])
    check(a, ref, attn_tolerance(BF, ref, mag, 192, 600, lm))
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for s in (torch.cuda.Stream(), torch.cuda.Stream()):
            outs.append(lay.attention_expanded(cu, cu, q, kv[..., :128], pe, kv[..., 128:],
                                               stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) for o in outs)


def _expanded(cfg, cuq, cuk, q, k, pe, v, causal=True, **kw):
    lay = LatentLayer(cfg, None)
    got = lay.attention_expanded(ints(cuq, torch.int32), ints(cuk, torch.int32), q, k, pe, v,
                                 causal=causal, **kw)
    ref, mag = O.attention_expanded(cuq, cuk, f64(q), f64(k), f64(pe), f64(v), cfg.softmax_scale,
                                    causal)
    lm = max(logit_bound(f64(q)[:, h], np.concatenate([f64(k)[:, h], f64(pe)], 1), cfg.softmax_scale)
             for h in range(q.shape[1]))
    return got, ref, attn_tolerance(BF, ref, mag, 192, len(k), lm)


def test_expanded_heads_outermost_and_captured():
    """Keys and values stored [H, n, d] (the token stride below the head stride), a call captured
    into a graph and replayed on new inputs."""
    rng = np.random.default_rng(23)
    cfg = v4a.latent_cfg(v4a.BF16, 3, 512, v4a.rope_cfg(64))
    k, v = rand(rng, BF, 3, 1500, 128).transpose(0, 1), rand(rng, BF, 3, 1500, 136).transpose(0, 1)[..., 8:]
    q, pe = rand(rng, BF, 40, 3, 192), rand(rng, BF, 1500, 64)
    got, ref, tol = _expanded(cfg, [0, 40], [0, 1500], q, k, pe, v)
    check(got, ref, tol)
    lay, cu, ck = LatentLayer(cfg, None), ints([0, 40], torch.int32), ints([0, 1500], torch.int32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = lay.attention_expanded(cu, ck, q, k, pe, v)
    q.copy_(rand(rng, BF, 40, 3, 192))
    g.replay()
    torch.cuda.synchronize()
    got, ref, tol = _expanded(cfg, [0, 40], [0, 1500], q, k, pe, v)
    check(got, ref, tol)
    assert torch.equal(out, got)


def test_expanded_many_sequences_and_rows_of_none():
    rng = np.random.default_rng(24)
    nq = rng.integers(0, 4, 1024)
    nk = nq + rng.integers(0, 150, 1024)
    cuq, cuk = np.concatenate([[2], 2 + np.cumsum(nq)]), np.concatenate([[1], 1 + np.cumsum(nk)])
    cfg = v4a.latent_cfg(v4a.BF16, 2, 512, v4a.rope_cfg(64))
    q, kv, pe = (rand(rng, BF, int(cuq[-1]), 2, 192), rand(rng, BF, int(cuk[-1]), 2, 256),
                 rand(rng, BF, int(cuk[-1]), 64))
    out = torch.full((len(q), 2, 128), 3.0, dtype=BF, device="cuda")
    got, ref, tol = _expanded(cfg, cuq, cuk, q, kv[..., :128], pe, kv[..., 128:], out=out)
    assert (got[:2] == 3).all()                    # rows before the first sequence
    check(got[2:], ref[2:], tol[2:])


def test_large_values_and_rising_logits():
    """Values near the type's limits under logits that jump from tile to tile: neither sums nor
    weights overflow on the way."""
    rng = np.random.default_rng(25)
    cfg = v4a.latent_cfg(v4a.BF16, 2, 512, v4a.rope_cfg(64))
    n = 700
    rise = torch.linspace(0, 3, n, device="cuda")[:, None, None]
    q, pe = rand(rng, BF, 150, 2, 192).abs(), rand(rng, BF, n, 64)
    k, v = (rand(rng, F32, n, 2, 128) * 0.3 + rise).to(BF), 1e30 * rand(rng, BF, n, 2, 128)
    got, ref, tol = _expanded(cfg, [0, 150], [0, n], q, k, pe, v)
    check(got, ref, tol)
    lay, bt = layer(rng, BF, 16, [n])
    rows = [O.slot(bt, 0, x) for x in range(n)]
    big = 1e15 * rand(rng, BF, n, 576)             # latents are keys too: 1e15 x 1e-15 logits
    big[:, 512:] = (rise[:, :, 0] * 4 + 0.1 * rand(rng, F32, n, 64)).to(BF)
    lay.pool.data[rows] = big
    qa = rand(rng, BF, 3, 16, 576)
    qa[..., :512] *= 1e-16
    qa[..., 512:] = qa[..., 512:].abs()
    got, ref, tol, flags = _attn(lay, bt, [n], [3], qa)
    assert flags == 0
    check(got, ref, tol)


def test_raw_stream_handles():
    rng = np.random.default_rng(26)
    lay, bt = layer(rng, BF, 16, [3000])
    cu, st, q = ints([0, 1], torch.int32), ints([2999], torch.int64), rand(rng, BF, 1, 16, 576)
    ref = lay.attention(cu, st, 2999, q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [lay.attention(cu, st, 2999, q, stream=h) for h in (s, s.cuda_stream, 0)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, ref) for g in got)


def test_python_refusals():
    """Types, shapes, strides and hosts that the layer does not take: refused before any launch."""
    rng = np.random.default_rng(28)
    lay, bt = layer(rng, BF, 16, [300, 20])
    cu, st = ints([0, 1, 2], torch.int32), ints([299, 19], torch.int64)
    q = rand(rng, BF, 2, 16, 576)
    good = dict(cu=cu, start=st, max_pos=299, q=q)
    assert lay.attention(**good).shape == (2, 16, 512)
    for bad in (dict(q=q.float()), dict(q=q[..., :512]), dict(q=q[:, :8]), dict(q=q.cpu()),
                dict(q=rand(rng, BF, 2, 16, 600)[..., :576]), dict(cu=cu.long()), dict(cu=cu[:0]),
                dict(cu=ints([0, 1, 2, 2], torch.int32)), dict(start=st.int()), dict(start=st[:1]),
                dict(start=[299, 19]), dict(cu=cu[None]), dict(out=torch.empty_like(q)),
                dict(dev_err=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            lay.attention(**dict(good, **bad))
    x = rand(rng, BF, 2, 576)
    for c, pe in ((x[:, :512].float(), x[:, 512:]), (x[:, :500], x[:, 512:]), (x[:1, :512], x[:, 512:]),
                  (rand(rng, BF, 512, 2).t(), x[:, 512:]), (x[:, :512], None)):
        with pytest.raises(ValueError):
            lay.insert(cu, st, c, pe)
    with pytest.raises(v4a.V4AError):              # rows that do not start on 16 bytes
        lay.insert(cu, st, rand(rng, BF, 2, 579)[:, 3:515], x[:, 512:])
    with pytest.raises(ValueError):
        lay.gather(cu, st, 2, out=torch.empty(2, 512, dtype=BF, device="cuda"))
    kv, pe = rand(rng, BF, 4, 16, 256), rand(rng, BF, 4, 64)
    qe, ce = rand(rng, BF, 2, 16, 192), ints([0, 2], torch.int32)
    ok = dict(cu_q=ce, cu_k=ints([0, 4], torch.int32), q=qe, k=kv[..., :128], k_pe=pe, v=kv[..., 128:])
    assert lay.attention_expanded(**ok).shape == (2, 16, 128)
    for bad in (dict(k_pe=pe[:3]), dict(v=kv[:3, :, 128:]), dict(k=kv[..., :120]), dict(q=qe.float()),
                dict(cu_k=ce[:1]), dict(v=None), dict(q=qe[..., ::2])):
        with pytest.raises(ValueError):
            lay.attention_expanded(**dict(ok, **bad))
    with pytest.raises(v4a.V4AError):              # one key head for all: its stride is 0
        lay.attention_expanded(**dict(ok, k=kv[:, :1, :128].expand(4, 16, 128)))
    with pytest.raises(ValueError):
        rope(lay.cfg.rope, q, ints([0, 1], torch.int64))
    with pytest.raises(v4a.V4AError):              # rows of the result on top of each other
        rope(lay.cfg.rope, rand(rng, BF, 2, 3, 64), ints([0, 1], torch.int64),
             out=torch.empty(2, 1, 64, dtype=BF, device="cuda").expand(2, 3, 64))


# -------------------------------------------------------------------------- together
def test_a_prompt_and_a_decode_step_on_tensor_cores():
    """bf16, as a model would run them: a prompt through the expanded form on gathered rows, then
    a decode step through the cache; each call against its definition on what it was given."""
    rng = np.random.default_rng(27)
    heads, dt = 16, BF
    lay, bt = layer(rng, dt, heads, [520, 300], gamma=True, rope_kw=dict(layout=v4a.ROPE_HALF))
    wkv = rand(rng, F32, 512, heads * 256) / 512 ** 0.5
    rate, done = O.rates(64), [0, 0]
    for new in ([519, 299], [1, 1]):
        cu, _ = batch(new, new)
        start, n = np.array(done), int(cu[-1])
        pos = np.concatenate([start[b] + np.arange(new[b]) for b in range(2)])
        cud, std, posd = ints(cu, torch.int32), ints(start, torch.int64), ints(pos, torch.int64)
        x = rand(rng, dt, n, 576)
        total = [d + m for d, m in zip(done, new)]
        if new[0] > 1:
            lay.insert(cud, std, x[:, :512], x[:, 512:])
            cuk = np.array([0, total[0], sum(total)])
            rows = lay.gather(ints(cuk, torch.int32), torch.zeros(2, dtype=torch.int64, device="cuda"),
                              sum(total))
            kv = (rows[:, :512].float() @ wkv).to(dt).view(-1, heads, 256)
            q = rand(rng, dt, n, heads, 192)
            rope(lay.cfg.rope, q[..., 128:], posd, out=q[..., 128:])
            got, ref, tol = _expanded(lay.cfg, cu, cuk, q, kv[..., :128], rows[:, 512:], kv[..., 128:])
        else:
            q = rand(rng, dt, n, heads, 576)
            before = f64(q[..., 512:])
            got = lay.step(cud, std, max(total) - 1, posd, x[:, :512], x[:, 512:], q)
            turned = O.rope(before, pos, rate, "half")
            check(q[..., 512:], turned, _rope_tol(before, turned, dt, "half", 1.0))
            ref, mag = O.attention(f64(lay.pool.data), bt, cu, start, f64(q), lay.cfg.softmax_scale, 512)
            tol = attn_tolerance(dt, ref, mag, 576, max(total),
                                 logit_bound(f64(q), f64(lay.pool.data), lay.cfg.softmax_scale))
        check(got, ref, tol)
        done = total


def test_absorbed_and_expanded_forms_agree_through_the_cache():
    """A prompt in two chunks and a decode step: rows inserted, queries absorbed and attended
    over the pages, against the expanded form on the gathered rows' projections. In fp32, so
    that both are exact to the projections' rounding."""
    rng = np.random.default_rng(21)
    heads, latent, dim, nope, vd = 4, 128, 32, 64, 48
    lay, bt = layer(rng, F32, heads, [333, 150], latent, dim, nope, vd, gamma=True)
    wk = rand(rng, F32, heads, nope, latent) / latent ** 0.5
    wv = rand(rng, F32, heads, vd, latent) / latent ** 0.5
    done = [0, 0]
    for new in ([200, 149], [132, 0], [1, 1]):
        cu, _ = batch(new, new)
        start = np.array(done)
        n = int(cu[-1])
        pos = np.concatenate([start[b] + np.arange(new[b]) for b in range(2)])
        x, q = rand(rng, F32, n, latent + dim), rand(rng, F32, n, heads, nope + dim)
        cud, std, posd = ints(cu, torch.int32), ints(start, torch.int64), ints(pos, torch.int64)
        qa = torch.empty(n, heads, latent + dim, device="cuda")
        qa[..., :latent] = torch.einsum("nhd,hdc->nhc", q[..., :nope].double(), wk.double())
        qa[..., latent:] = q[..., nope:]
        total = [d + m for d, m in zip(done, new)]
        o = lay.step(cud, std, max(total) - 1, posd, x[:, :latent], x[:, latent:], qa)
        absorbed = torch.einsum("nhc,hdc->nhd", o.double(), wv.double())
        cuk = ints([0, total[0], total[0] + total[1]], torch.int32)
        rows = lay.gather(cuk, torch.zeros(2, dtype=torch.int64, device="cuda"), sum(total))
        c = rows[:, :latent].double()
        kv = torch.cat([torch.einsum("nc,hdc->nhd", c, wk.double()),
                        torch.einsum("nc,hdc->nhd", c, wv.double())], -1).float()
        rope(lay.cfg.rope, q[..., nope:], posd, out=q[..., nope:])
        e = lay.attention_expanded(cud, cuk, q, kv[..., :nope], rows[:, latent:], kv[..., nope:])
        # fp32 sums of at most 160 products and 333 weights on either side, values of order 1
        assert (absorbed - e.double()).abs().max() <= 1e-4
        done = total


def test_expanded_offsets_pass_31_bits():
    """Keys and values of more than 2^31 elements: the last heads of the last tokens."""
    g = torch.Generator(device="cuda").manual_seed(29)
    n, heads, nq = 140000, 64, 3
    kv = torch.randn(n, heads, 256, generator=g, device="cuda", dtype=BF)
    assert kv.numel() > 1 << 31
    pe = torch.randn(n, 64, generator=g, device="cuda", dtype=BF)
    q = torch.randn(nq, heads, 192, generator=g, device="cuda", dtype=BF)
    lay = LatentLayer(v4a.latent_cfg(v4a.BF16, heads, 512, v4a.rope_cfg(64)), None)
    got = lay.attention_expanded(ints([0, nq], torch.int32), ints([0, n], torch.int32), q,
                                 kv[..., :128], pe, kv[..., 128:])
    for h in (0, 63):
        k = np.concatenate([f64(kv[:, h, :128]), f64(pe)], 1)
        v = f64(kv[:, h, 128:])
        for i in range(nq):
            m = n - nq + i + 1
            ref, mag = O.attend(f64(q)[i, h][None], k[:m], v[:m], lay.cfg.softmax_scale)
            check(got[i, h][None], ref,
                  attn_tolerance(BF, ref, mag, 192, n, logit_bound(f64(q)[i, h][None], k, lay.cfg.softmax_scale)))


def test_long_cache_offsets_pass_31_bits():
    """A pool of more than 2^31 elements: the last pages are read and written where they are."""
    rng = np.random.default_rng(22)
    pages = (1 << 31) // (256 * 576) + 40
    data = torch.zeros((pages * 256, 576), dtype=BF, device="cuda")
    bt = np.array([[pages - 1, 3, pages - 2]], np.int32)
    from compressed_sparse_long_gb300.layer import PagedPool
    lay = LatentLayer(v4a.latent_cfg(v4a.BF16, 64, 512, v4a.rope_cfg(64)),
                      PagedPool(data, None, ints(bt, torch.int32), 256))
    x = rand(rng, BF, 700, 576)
    cu, st = ints([0, 700], torch.int32), ints([0], torch.int64)
    lay.insert(cu, st, x[:, :512], x[:, 512:])
    got = lay.gather(cu, st, 700)
    assert torch.equal(got[:, :512], x[:, :512])
    q = rand(rng, BF, 1, 64, 576)
    o = lay.attention(ints([0, 1], torch.int32), ints([699], torch.int64), 699, q)
    rows = f64(got)
    ref, mag = O.attend(f64(q)[0], rows, rows[:, :512], lay.cfg.softmax_scale)
    check(o[0], ref, attn_tolerance(BF, ref, mag, 576, 700, logit_bound(f64(q), rows, lay.cfg.softmax_scale)))
