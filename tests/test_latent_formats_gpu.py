"""GPU: the 4-bit latent cache and windowed latent attention against their definitions. Tolerances
are derived in latent_helpers and beside each check."""
import numpy as np
import pytest
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300.latent import LatentLayer
from compressed_sparse_long_gb300.layer import PagedPool
from latent_helpers import (BF, F32, attn_tolerance, batch, check, err_word, f64, half_step, ints,
                            layer, logit_bound, rand)
from oracle import latent_oracle as O

pytestmark = pytest.mark.gpu
I32, I64 = torch.int32, torch.int64


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


def fp4_layer(rng, dtype, heads, total, latent=512, rope=64, gamma=False, hole=None, rope_kw=None,
              junk=False, spread=1.0, keep=None):
    """A layer on a 4-bit pool: rows of random codes, block scales 2^-3 .. 2^3 of their middle, rotary
    parts N(0, 1) and row scales `spread` apart, each standing for values of about N(0, 1) at
    spread 1. junk: every byte of rows behind the sequences' ends is 255 and their scales NaN.
    keep(b, block): whether the block has a page."""
    plain, bt = layer(rng, dtype, heads, total, 32, 8, gamma=False, hole=hole)
    pages = plain.pool.data.shape[0] // 256
    rows = pages * 256
    width = -(-(latent // 2 + 2 * rope + latent // 16) // 16) * 16
    raw = np.zeros((rows, width), np.uint8)
    raw[:, :latent // 2] = rng.integers(0, 256, (rows, latent // 2))
    raw[:, latent // 2:latent // 2 + 2 * rope] = (
        rng.standard_normal((rows, rope)) * 1024).astype(np.float16).view(np.uint8)
    raw[:, latent // 2 + 2 * rope:latent // 2 + 2 * rope + latent // 16] = rng.integers(
        (7 + 4) << 3, (7 + 8) << 3, (rows, latent // 16))
    scale = (2.0 ** -10 * spread ** rng.uniform(-1, 1, rows)).astype(np.float32)
    if junk:
        used = np.zeros(rows, bool)
        for b, t in enumerate(total):
            for blk in range(-(-t // 256)):
                s = bt[b, blk] * 256
                if s >= 0:
                    used[s:s + min(256, t - blk * 256)] = True
        raw[~used], scale[~used] = 255, np.nan
    if keep is not None:
        for b in range(len(bt)):
            for k in range(bt.shape[1]):
                if not keep(b, k) and bt[b, k] >= 0:
                    raw[bt[b, k] * 256:bt[b, k] * 256 + 256] = 255
                    scale[bt[b, k] * 256:bt[b, k] * 256 + 256] = np.nan
                    bt[b, k] = -1
    cfg = v4a.latent_cfg(v4a.BF16 if dtype == BF else v4a.FP32, heads, latent,
                         v4a.rope_cfg(rope, **(rope_kw or {})), cache_format=v4a.LATENT_FP4)
    g = torch.from_numpy(1 + 0.1 * rng.standard_normal(latent)).to("cuda", F32) if gamma else None
    pool = PagedPool(torch.from_numpy(raw).cuda(), torch.from_numpy(scale).cuda(), ints(bt, I32), 256)
    return LatentLayer(cfg, pool, g), bt


def values(lay):
    c = lay.cfg
    return O.fp4_values(lay.pool.data.cpu().numpy(), lay.pool.scale.cpu().numpy(), c.latent_dim, c.rope.dim)


# ----------------------------------------------------------------------------- insert
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("latent,dim,layout,norm", [(512, 64, "pairs", True), (512, 64, "half", False),
                                                    (32, 8, "half", True), (1024, 128, "pairs", True),
                                                    (544, 24, "half", True)])
def test_insert_writes_the_stated_rows(dtype, latent, dim, layout, norm):
    rng = np.random.default_rng(9)
    total, new = [1, 700, 40, 513, 0, 256], [1, 300, 40, 2, 0, 1]
    kw = dict(layout=v4a.ROPE_HALF if layout == "half" else v4a.ROPE_INTERLEAVED)
    lay, bt = fp4_layer(rng, dtype, 4, total, latent, dim, gamma=norm, rope_kw=kw)
    cu, start = batch(total, new)
    n = int(cu[-1])
    x = rand(rng, dtype, n + 3, latent + dim + 8)
    x *= torch.from_numpy(10.0 ** rng.uniform(-3, 3, (n + 3, 1))).to("cuda", dtype)
    if n > 60:                                     # outliers in a block, a block of zeros, a zero row
        x[7, 5] *= 200
        x[8, 16:32] = 0
        x[9] = 0
        x[10, :latent] *= 1e-4                     # the rotary part sets the scale
    x[n:] = float("nan")
    raw, scale, e = lay.pool.data.clone(), lay.pool.scale.clone(), err_word()
    lay.insert(ints(cu, I32), ints(start, I64), x[:, :latent], x[:, latent:latent + dim], dev_err=e)
    assert v4a.v4a_get_error(e) == 0
    got, got_s = lay.pool.data.cpu().numpy(), lay.pool.scale.cpu().numpy()
    rate = O.rates(dim)
    c = x[:n, :latent].float().cpu().numpy()
    z = c * lay.gamma.cpu().numpy() if norm else c
    written, seq = [], np.repeat(np.arange(len(total)), new)
    a, h_at = latent // 2, latent // 2 + 2 * dim
    for i in range(n):
        pos = int(start[seq[i]]) + i - int(cu[seq[i]])
        slot = O.slot(bt, seq[i], pos)
        written.append(slot)
        row, v = got[slot], O.fp4_values(got[slot:slot + 1], np.ones(1), latent, dim)[0]
        r = 1 / np.sqrt((c[i].astype(np.float64) ** 2).mean() + float(np.float32(1e-6))) if norm else 1.0
        k = O.rope(f64(x[i:i + 1, latent:latent + dim]), [pos], rate, layout)[0]
        code, block, half, s = O.fp4_row(z[i], k, r)
        # the mean square is a sum of `latent` products, then a root and a division; the rotary part's
        # largest value is off by 4 2^-23 of its pair
        assert abs(got_s[slot] - s) <= ((latent + 16) * 2.0 ** -24) * s
        by_rope = np.abs(k).max() / 32768 > r * float(np.abs(z[i]).max()) / 2688 * (1 - 1e-5)
        gb = row[h_at:h_at + latent // 16].copy()
        gv = v[:latent]
        if not by_rope:
            want_b = torch.from_numpy(block.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            assert np.array_equal(gb, want_b)
            assert np.array_equal(gv, code * np.repeat(block, 16))
        else:
            # the scale's own error may move a value over a rounding border: a step at most
            b = np.repeat(torch.from_numpy(gb).view(torch.float8_e4m3fn).double().numpy(), 16)
            t = np.abs(z[i].astype(np.float64)) * r / float(got_s[slot])
            assert (np.abs(np.abs(gv) - t) <= np.maximum(b, 2.0 ** -10 * 6) * (1 + 2.0 ** -18)).all()
        pair = 8 * 2.0 ** -23 * np.abs(x[i, latent:latent + dim].float().cpu().numpy()).max()
        tol = 2.0 ** -11 * np.abs(k) + 2.0 ** -25 * s + pair + (latent + 16) * 2.0 ** -23 * np.abs(k)
        assert (np.abs(v[latent:] * float(got_s[slot]) - k) <= tol).all()
        assert np.array_equal(row[h_at + latent // 16:], raw[slot, h_at + latent // 16:].cpu().numpy())
    assert a and sorted(set(written)) == sorted(written)
    rest = np.setdiff1d(np.arange(len(got)), written)
    assert np.array_equal(got[rest], raw.cpu().numpy()[rest])
    assert np.array_equal(got_s[rest], scale.cpu().numpy()[rest])


def test_insert_of_rows_that_are_not_finite_and_missing_pages():
    rng = np.random.default_rng(10)
    lay, bt = fp4_layer(rng, BF, 4, [300, 20], hole=(0, 1))
    x = rand(rng, BF, 6, 576)
    x[0, 3], x[1, 500], x[2, 570] = float("nan"), float("inf"), float("nan")
    x[3, 515] = float("-inf")
    cu, start, e = [0, 5, 6], [252, 1 << 36], err_word()
    lay.insert(ints(cu, I32), ints(start, I64), x[:, :512], x[:, 512:], dev_err=e)
    # position 256 of the first sequence has no page, the second one's position is out of range
    assert v4a.v4a_get_error(e) == v4a.DEV_MISSING_PAGE | v4a.DEV_BAD_POS
    rows = lay.gather(ints([0, 4], I32), ints([252], I64), 4)
    assert not torch.isfinite(rows).all(1).any()
    lay.insert(ints([0, 4], I32), ints([252], I64), x[4:5, :512].expand(4, -1).contiguous(),
               x[4:5, 512:].expand(4, -1).contiguous())
    assert torch.isfinite(lay.gather(ints([0, 4], I32), ints([252], I64), 4)).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("latent,dim", [(512, 64), (32, 8), (1024, 128), (96, 24)])
def test_gather_returns_what_rows_stand_for(dtype, latent, dim):
    rng = np.random.default_rng(12)
    total = [1, 0, 300, 513, 70]
    lay, bt = fp4_layer(rng, dtype, 4, total, latent, dim, spread=1000.0, hole=(3, 1))
    n, start = [1, 0, 200, 513, 7], [0, 5, 100, 0, 63]
    cu = np.concatenate([[0], np.cumsum(n)])
    out, e = torch.full((int(cu[-1]) + 2, latent + dim), 7.0, dtype=dtype, device="cuda"), err_word()
    lay.gather(ints(cu, I32), ints(start, I64), int(cu[-1]) + 2, out=out, dev_err=e)
    assert v4a.v4a_get_error(e) == v4a.DEV_MISSING_PAGE
    # one product in 32 bits of exact factors, rounded once
    exact = O.fp4_values(lay.pool.data.cpu().numpy(), np.ones(len(lay.pool.scale)), latent, dim)
    val = exact.astype(np.float32) * lay.pool.scale.cpu().numpy()[:, None]
    want = np.zeros((int(cu[-1]), latent + dim), np.float32)
    for b in range(5):
        for i in range(n[b]):
            s = O.slot(bt, b, start[b] + i)
            if s >= 0:
                want[cu[b] + i] = val[s]
    assert torch.equal(out[:-2].cpu(), torch.from_numpy(want).to(dtype)) and (out[-2:] == 7).all()


# -------------------------------------------------------------------------- attention
def run_attention(lay, bt, total, new, q, window=None, sinks=0, e=None, max_pos=None, spread=1.0):
    cu, start = batch(total, new)
    rows = values(lay) if lay._fp4 else f64(lay.pool.data)
    mp = max(total) - 1 if max_pos is None else max_pos
    got = lay.attention(ints(cu, I32), ints(start, I64), mp, q, dev_err=e, window=window, sinks=sinks)
    c = lay.cfg
    ref, mag = O.attention(rows, bt, cu, start, f64(q), c.softmax_scale, c.latent_dim, max_pos, window, sinks)
    seen = np.zeros(len(rows), bool)
    for b, t in enumerate(total):
        for x in range(t):
            s = O.slot(bt, b, x)
            if s >= 0:
                seen[s] = True
    keys = rows[seen & np.isfinite(rows).all(1)]
    tol = attn_tolerance(lay.dtype, ref, mag, lay.width, max(total), logit_bound(f64(q), keys, c.softmax_scale))
    if lay._fp4 and lay.dtype == BF and len(keys):
        # weight times row scale is held in f16 down to 2^-24 of a number that is at most 2^26 times
        # smaller than the head's largest such product; times the largest value over the scale, 2688
        tol = tol + 2.0 ** -20 * np.abs(keys[:, :c.latent_dim]).max()
    return got, ref, tol


WINDOWS = [(None, 0), (1, 0), (7, 3), (128, 0), (130, 129), (513, 4), (100000, 0)]
SHAPES = [(BF, 512, 64, 16), (BF, 512, 64, 5), (BF, 512, 64, 128), (BF, 128, 32, 3), (F32, 128, 32, 8),
          (F32, 1024, 8, 2)]


def make(rng, fmt, dtype, heads, total, latent, dim, **kw):
    if fmt == "fp4":
        return fp4_layer(rng, dtype, heads, total, latent, dim, junk=True, **kw)
    kw.pop("spread", None)
    return layer(rng, dtype, heads, total, latent, dim, fill=float("nan"), **kw)


@pytest.mark.parametrize("fmt", ["plain", "fp4"])
@pytest.mark.parametrize("dtype,latent,dim,heads", SHAPES)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_attention_matches_its_definition(fmt, dtype, latent, dim, heads, window, sinks):
    """Decode and chunks of ragged batches: lengths 0 and 1, odd ones, pages that end inside a tile;
    rows behind every sequence's end hold NaN."""
    if fmt == "plain" and window is None:
        pytest.skip("the plain form's own tests")
    rng = np.random.default_rng(latent + heads + (window or 0))
    for total, new in (([1, 700, 129, 256, 0, 1025], [1, 1, 1, 1, 0, 1]),
                       ([3, 600, 257, 128], [3, 40, 1, 128])):
        lay, bt = make(rng, fmt, dtype, heads, total, latent, dim)
        q, e = rand(rng, dtype, sum(new), heads, latent + dim), err_word()
        got, ref, tol = run_attention(lay, bt, total, new, q, window, sinks, e)
        assert v4a.v4a_get_error(e) == 0
        check(got, ref, tol)


@pytest.mark.parametrize("fmt", ["plain", "fp4"])
@pytest.mark.parametrize("dtype,latent,dim,heads", [(BF, 512, 64, 64), (F32, 128, 32, 8)])
def test_longer_contexts_and_prompts(fmt, dtype, latent, dim, heads):
    rng = np.random.default_rng(77)
    for total, new, window, sinks in (([5000, 3001], [1, 1], None, 0), ([5000, 3001], [1, 1], 2000, 7),
                                      ([900], [900], None, 0), ([900], [900], 200, 4), ([2500, 40], [130, 33], 77, 0)):
        if fmt == "plain" and window is None:
            continue
        lay, bt = make(rng, fmt, dtype, heads, total, latent, dim)
        sub = 3 if sum(new) > 200 else 1           # the oracle takes some heads of a prompt
        q = rand(rng, dtype, sum(new), heads, latent + dim)
        cu, start = batch(total, new)
        got = lay.attention(ints(cu, I32), ints(start, I64), max(total) - 1, q, window=window, sinks=sinks)
        pick = list(range(heads)) if sub == 1 else [0, heads // 2, heads - 1]
        rows = values(lay) if fmt == "fp4" else f64(lay.pool.data)
        at = np.arange(sum(new)) if sub == 1 else np.unique(np.linspace(0, sum(new) - 1, 61).astype(int))
        c = lay.cfg
        live = rows[np.isfinite(rows).all(1)]
        bound = logit_bound(f64(q[at][:, pick]), live, c.softmax_scale)
        for i in at:
            b = int(np.searchsorted(cu, i, "right") - 1)
            pos = int(start[b] + i - cu[b])
            ref, mag = O.attention(rows, bt[b:b + 1], [0, 1], [pos], f64(q[i:i + 1])[:, pick], c.softmax_scale,
                                   latent, None, window, sinks)
            tol = attn_tolerance(dtype, ref, mag, lay.width, pos + 1, bound)
            if fmt == "fp4" and dtype == BF:
                tol = tol + 2.0 ** -20 * np.abs(live[:, :latent]).max()   # as in run_attention
            check(got[i:i + 1][:, pick], ref, tol)


@pytest.mark.parametrize("fmt", ["plain", "fp4"])
@pytest.mark.parametrize("dtype,latent,dim,heads", [(BF, 512, 64, 8), (F32, 128, 32, 4)])
def test_blocks_outside_the_windows_need_no_page(fmt, dtype, latent, dim, heads):
    rng = np.random.default_rng(31)
    total, new, window, sinks = [2000, 700, 90], [3, 1, 2], 300, 130
    if fmt == "fp4":
        lay, bt = fp4_layer(rng, dtype, heads, total, latent, dim,
                            keep=lambda b, k: k == 0 or k * 256 + 255 > total[b] - new[b] - window)
    else:
        lay, bt = layer(rng, dtype, heads, total, latent, dim)
        for b in range(3):
            for k in range(1, bt.shape[1]):
                if k * 256 + 255 <= total[b] - new[b] - window and bt[b, k] >= 0:
                    lay.pool.data[bt[b, k] * 256:bt[b, k] * 256 + 256] = float("nan")
                    bt[b, k] = -1
        lay.pool.block_table = ints(bt, I32)
    assert (bt[0] == -1).sum() >= 4
    q, e = rand(rng, dtype, sum(new), heads, latent + dim), err_word()
    got, ref, tol = run_attention(lay, bt, total, new, q, window, sinks, e)
    assert v4a.v4a_get_error(e) == 0
    check(got, ref, tol)
    # without a window the same table has holes: they are reported and left out
    got, ref, tol = run_attention(lay, bt, total, new, q, None, 0, e)
    assert v4a.v4a_get_error(e) == v4a.DEV_MISSING_PAGE
    check(got, ref, tol)


@pytest.mark.parametrize("fmt", ["plain", "fp4"])
def test_missing_and_bad_pages_and_positions(fmt):
    rng = np.random.default_rng(32)
    for dtype, latent, dim in ((BF, 512, 64), (F32, 64, 16)):
        lay, bt = make(rng, fmt, dtype, 6, [600, 10, 300], latent, dim, hole=(0, 1))
        bt[1, 0] = 10 ** 6
        lay.pool.block_table = ints(bt, I32)
        q, e = rand(rng, dtype, 3, 6, latent + dim), err_word()
        holes = bt.copy()
        holes[1, 0] = -1
        for window, sinks in ((None, 0), (200, 3)):
            got, ref, tol = run_attention(lay, holes, [600, 10, 300], [1, 1, 1], q, window, sinks, e)
            assert v4a.v4a_get_error(e) == v4a.DEV_MISSING_PAGE | v4a.DEV_BAD_PAGE
            check(got, ref, tol)
            assert (got[1] == 0).all()             # no key at all
        # a token past max_pos sees the keys up to it, of its own window
        got, ref, tol = run_attention(lay, holes, [600, 10, 300], [1, 1, 1], q, 250, 130, e, max_pos=255)
        assert v4a.v4a_get_error(e) & v4a.DEV_BAD_POS
        check(got, ref, tol)


@pytest.mark.parametrize("fmt", ["plain", "fp4"])
@pytest.mark.parametrize("dtype,latent,dim", [(BF, 512, 64), (F32, 64, 16)])
def test_keys_that_are_not_finite_outside_the_window(fmt, dtype, latent, dim):
    """Between the sinks and a decode token's window, in the same tile and page as seen keys."""
    rng = np.random.default_rng(33)
    lay, bt = make(rng, fmt, dtype, 4, [500, 300], latent, dim)
    window, sinks = 150, 5
    for b, t in ((0, 500), (1, 300)):
        for x in range(sinks, t - window):
            s = O.slot(bt, b, x)
            if fmt == "fp4":
                lay.pool.scale[s] = float("inf") if x % 2 else float("nan")
            else:
                lay.pool.data[s] = float("inf") if x % 2 else float("nan")
    q, e = rand(rng, dtype, 2, 4, latent + dim), err_word()
    got, ref, tol = run_attention(lay, bt, [500, 300], [1, 1], q, window, sinks, e)
    check(got, ref, tol)
    seen = lay.attention(ints([0, 1, 2], I32), ints([499, 299], I64), 499, q)
    assert not torch.isfinite(seen).any()


@pytest.mark.parametrize("heads", [1, 64])
def test_fp4_rows_of_very_different_scales(heads):
    """Row scales from 2^-40 to 1 beside one another, rows of zeros, logits that rise along the
    keys and a first tile that holds nothing to see."""
    rng = np.random.default_rng(34)
    total, new = [1300, 140], [1, 2]
    lay, bt = fp4_layer(rng, BF, heads, total)
    for b in range(2):
        for x in range(total[b]):
            lay.pool.scale[O.slot(bt, b, x)] = 2.0 ** (-10 + 10 * (x / 1300) - (30 if x % 3 else 0))
    lay.pool.data[O.slot(bt, 0, 5)] = 0
    lay.pool.scale[O.slot(bt, 0, 5)] = 2.0 ** -100
    q = rand(rng, BF, 3, heads, 576) * 2.0 ** -10
    for window, sinks in ((None, 0), (400, 2)):
        got, ref, tol = run_attention(lay, bt, total, new, q, window, sinks)
        check(got, ref, tol)
    # queries of very different sizes in one call
    q = rand(rng, BF, 3, heads, 576)
    q[0] *= 2.0 ** -60
    q[1] *= 2.0 ** -14
    q[2] *= 2.0 ** -20
    got, ref, tol = run_attention(lay, bt, total, new, q)
    check(got, ref, tol)


def test_fp4_results_repeat_and_ignore_other_calls():
    """Two streams, a captured call replayed with other lengths, a call of no tokens."""
    rng = np.random.default_rng(35)
    total, new = [4000, 900, 33], [1, 1, 1]
    lay, bt = fp4_layer(rng, BF, 32, total)
    q = rand(rng, BF, 3, 32, 576)
    cu, start = ints([0, 1, 2, 3], I32), ints([3999, 899, 32], I64)
    want = lay.attention(cu, start, 3999, q)
    wide = lay.attention(cu, start, 3999, q, window=500, sinks=2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            outs.append((lay.attention(cu, start, 3999, q), lay.attention(cu, start, 3999, q, window=500, sinks=2)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, wide) for a, b in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lay.attention(cu, start, 3999, q, window=500, sinks=2)
    for s in ([3999, 899, 32], [10, 700, 0], [2500, 1, 31]):
        start.copy_(ints(s, I64))
        graph.replay()
        assert torch.equal(out, lay.attention(cu, start, 3999, q, window=500, sinks=2))
    assert lay.attention(ints([0, 0, 0, 0], I32), start, 3999, q[:0]).shape == (0, 32, 512)


def test_step_on_a_4_bit_cache_with_a_window():
    """insert, rotation and attention in one call equal the three calls; a prompt's rows read back
    feed the expanded form."""
    rng = np.random.default_rng(36)
    total, new = [400, 260], [1, 5]
    lay, bt = fp4_layer(rng, BF, 8, total, gamma=True)
    cu, start = batch(total, new)
    n = int(cu[-1])
    x, q = rand(rng, BF, n, 576), rand(rng, BF, n, 8, 576)
    pos = np.concatenate([np.arange(s, t) for s, t in zip(start, total)])
    dcu, dst, dpos = ints(cu, I32), ints(start, I64), ints(pos, I64)
    q1 = q.clone()
    o = lay.step(dcu, dst, 399, dpos, x[:, :512], x[:, 512:], q1, window=100, sinks=3)
    turned = q.clone()
    v4a.v4a_rope(lay.cfg.rope, v4a.BF16, n, 8, dpos, turned[..., 512:], 8 * 576, 576, turned[..., 512:], 8 * 576, 576)
    assert torch.equal(q1, turned)
    assert torch.equal(o, lay.attention(dcu, dst, 399, turned, window=100, sinks=3))
    rows = lay.gather(ints([0, 400, 660], I32), ints([0, 0], I64), 660)
    got = rows[[399] + list(range(655, 660))].float()
    ref = x[:, :512].float() * lay.gamma / torch.sqrt(x[:, :512].float().square().mean(1, keepdim=True) + 1e-6)
    # a value is off by less than its block's scale (half a step of e2m1 is at most 1, the largest is 6)
    step = ref.view(n, 32, 16).abs().amax(2, keepdim=True) / 6 * (1 + 2 ** -4)
    assert ((got[:, :512] - ref).view(n, 32, 16).abs() <= step * 1.01).all()
    with pytest.raises(ValueError):
        lay.attention(dcu, dst, 399, q, sinks=3)
    for bad in (dict(scale=None), dict(scale=lay.pool.scale.half()), dict(scale=lay.pool.scale[:-1]),
                dict(data=lay.pool.data.view(torch.int8)), dict(data=lay.pool.data[:, :400].contiguous())):
        kept = lay.pool
        lay.pool = PagedPool(**dict(dict(data=kept.data, scale=kept.scale, block_table=kept.block_table,
                                         rows_per_block=256), **bad))
        with pytest.raises(ValueError):
            lay.attention(dcu, dst, 399, q)
        lay.pool = kept
    assert half_step(BF) == 2 ** -8


def test_fp4_offsets_pass_31_bits():
    """A pool of more than 2^31 bytes: rows at its far end."""
    pages = (1 << 31) // (256 * 416) + 40
    data = torch.zeros(pages * 256, 416, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(pages * 256, device="cuda")
    bt = ints([[pages - 1, pages - 7, 3]], I32)
    cfg = v4a.latent_cfg(v4a.BF16, 16, 512, v4a.rope_cfg(64), cache_format=v4a.LATENT_FP4)
    lay = LatentLayer(cfg, PagedPool(data, scale, bt, 256))
    rng = np.random.default_rng(37)
    x, q = rand(rng, BF, 600, 576), rand(rng, BF, 1, 16, 576)
    lay.insert(ints([0, 600], I32), ints([0], I64), x[:, :512], x[:, 512:])
    small = LatentLayer(cfg, PagedPool(data[:3 * 256].clone(), scale[:3 * 256].clone(), ints([[0, 2, 1]], I32), 256))
    small.insert(ints([0, 600], I32), ints([0], I64), x[:, :512], x[:, 512:])
    a, b = ints([0, 600], I32), ints([0], I64)
    assert torch.equal(lay.gather(a, b, 600), small.gather(a, b, 600))
    for kw in ({}, dict(window=100, sinks=2)):
        assert torch.equal(lay.attention(ints([0, 1], I32), ints([599], I64), 599, q, **kw),
                           small.attention(ints([0, 1], I32), ints([599], I64), 599, q, **kw))


@pytest.mark.parametrize("window", [None, 200])
def test_fp4_queries_that_are_not_finite_stay_their_own(window):
    """Heads of one token share a unit of the tensor-core kernel, and one factor that brings its queries
    into f16: an infinite or missing number in one head reaches no other; nor do queries of 2^120."""
    rng = np.random.default_rng(38)
    lay, bt = fp4_layer(rng, BF, 20, [700, 300])
    q = rand(rng, BF, 2, 20, 576)
    q[1] *= 2.0 ** -40
    bad = q.clone()
    bad[0, 3, 7], bad[0, 11, 570], bad[1, 0, 0] = float("inf"), float("nan"), float("-inf")
    kw = dict(window=window, sinks=3) if window else {}
    a, b = ints([0, 1, 2], I32), ints([699, 299], I64)
    got, want = lay.attention(a, b, 699, bad, **kw), lay.attention(a, b, 699, q, **kw)
    hit = torch.zeros(2, 20, dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[0, 11] = hit[1, 0] = True
    assert not torch.isfinite(got[hit]).any() and torch.equal(got[~hit], want[~hit])
    # one head far larger than the others: its weights are one key's, the others keep their bits
    big = rand(rng, BF, 2, 20, 576)
    big[0, 5] *= 2.0 ** 20
    got, ref, tol = run_attention(lay, bt, [700, 300], [1, 1], big, window, 3 if window else 0)
    keep = [h for h in range(20) if h != 5]
    c = lay.cfg
    live = values(lay)
    bound = logit_bound(f64(big[:, keep]), live, c.softmax_scale)
    _, mag = O.attention(live, bt, [0, 1, 2], [699, 299], f64(big), c.softmax_scale, 512, None, window, 3 if window else 0)
    tol = attn_tolerance(BF, ref, mag, 576, 700, bound) + 2.0 ** -20 * np.abs(live[:, :512]).max()
    check(got[:, keep], ref[:, keep], tol[:, keep])


@pytest.mark.parametrize("heads,window", [(64, None), (16, None), (128, 3)])
def test_fp4_many_pieces_of_one_tile(heads, window):
    """Several pieces a CTA, of one tile each, whose queries' sizes are far apart: what brings one piece's
    queries into f16 reaches no other."""
    rng = np.random.default_rng(39)
    total = [1 + 41 * i % 128 for i in range(620)]
    lay, bt = fp4_layer(rng, BF, heads, total, junk=True)
    size = torch.from_numpy(2.0 ** rng.integers(-24, 1, 620)).to("cuda", BF)
    q, e = rand(rng, BF, 620, heads, 576) * size[:, None, None], err_word()
    got, ref, tol = run_attention(lay, bt, total, [1] * 620, q, window, 1 if window else 0, e)
    assert v4a.v4a_get_error(e) == 0
    check(got, ref, tol)


@pytest.mark.parametrize("dtype,latent,dim,heads", [(BF, 512, 64, 16), (F32, 128, 32, 3)])
def test_rows_behind_the_last_sequence_stay(dtype, latent, dim, heads):
    """A batch padded to more rows than its sequences have: the rows behind them are neither read nor
    written, by any of the calls."""
    rng = np.random.default_rng(40)
    total, new = [300, 0, 700], [2, 0, 3]
    cu, start = ints([0, 2, 2, 5], I32), ints([298, 0, 697], I64)
    a, bt = fp4_layer(rng, dtype, heads, total, latent, dim)
    b = LatentLayer(a.cfg, PagedPool(a.pool.data.clone(), a.pool.scale.clone(), a.pool.block_table, 256))
    x = rand(rng, dtype, 9, latent + dim)
    x[5:] = float("nan")
    a.insert(cu, start, x[:5, :latent], x[:5, latent:])
    b.insert(cu, start, x[:, :latent], x[:, latent:])
    assert torch.equal(a.pool.data, b.pool.data) and torch.equal(a.pool.scale, b.pool.scale)
    rows = torch.full((9, latent + dim), 7.0, dtype=dtype, device="cuda")
    b.gather(cu, start, 9, out=rows)
    assert torch.equal(rows[:5], a.gather(cu, start, 5)) and (rows[5:] == 7).all()
    q = rand(rng, dtype, 9, heads, latent + dim)
    q[5:] = float("nan")
    for window, sinks in ((None, 0), (200, 3)):
        e = err_word()
        out = torch.full((9, heads, latent), 7.0, dtype=dtype, device="cuda")
        b.attention(cu, start, 699, q, out=out, dev_err=e, window=window, sinks=sinks)
        got, ref, tol = run_attention(a, bt, total, new, q[:5], window, sinks)
        assert v4a.v4a_get_error(e) == 0 and (out[5:] == 7).all()
        check(out[:5], ref, tol)
        check(got, ref, tol)
