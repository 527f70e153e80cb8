"""GPU: the rotation's gradients and far positions, and latent attention at the ends of its ranges:
large and small values, lengths that differ widely, positions past the block table. Tolerances as
in latent_helpers."""
import decimal
import math

import numpy as np
import pytest
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300.latent import LatentLayer, rope
from latent_helpers import (BF, F32, attn_tolerance, batch, check, err_word, f64, half_step, ints,
                            layer, logit_bound, rand)
from oracle import latent_oracle as O
from test_latent_gpu import _attn, _expanded, _rope_case, _rope_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


# ----------------------------------------------------------------------- far positions
PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def _turn(dim, scaling, pos):
    """Angles below one turn of exact positions, from rates in 60 digits."""
    with decimal.localcontext(decimal.Context(prec=60)):
        out = []
        for i in range(dim // 2):
            keep = decimal.Decimal(1)
            if scaling == "yarn":
                def pair(t):
                    return dim * math.log(4096 / (t * 2 * math.pi)) / (2 * math.log(10000))
                a, b = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), dim - 1)
                keep -= min(decimal.Decimal(1), max(decimal.Decimal(0), decimal.Decimal(i - a) / (b - a)))
            theta = decimal.Decimal(10000) ** (decimal.Decimal(-2 * i) / dim)
            theta *= keep + (1 - keep) / 8
            out.append([float(p * theta % (2 * PI)) for p in pos])
    return np.array(out).T


@pytest.mark.parametrize("layout", ["pairs", "half"])
@pytest.mark.parametrize("scaling", ["none", "yarn"])
def test_rope_far_positions(layout, scaling):
    """The rates are 64-bit numbers of a few roundings (two powers, a product, the scaling, the
    division by 2 pi: at most 12 2^-53 in all, and no rate is above 1), so an angle is off by up to
    12 2^-53 of its position, beside the 4 2^-23 of near ones."""
    rng = np.random.default_rng(48)
    dim, far = 64, [2 ** 21 + 1, 2 ** 24 - 1, 2 ** 24 + 12345, 2 ** 28 + 77, 2 ** 30 - 3, 2 ** 32 + 999, 2 ** 36 - 1]
    cfg, _ = _rope_case(dim, layout, scaling)
    x = rand(rng, F32, len(far), 2, dim)
    got, ang, xs = rope(cfg, x, ints(far, torch.int64)), _turn(dim, scaling, far), f64(x)
    a, b = (xs[..., :32], xs[..., 32:]) if layout == "half" else (xs[..., ::2], xs[..., 1::2])
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    r0, r1, size = a * c - b * s, a * s + b * c, np.abs(a) + np.abs(b)
    if layout == "half":
        ref, size = np.concatenate([r0, r1], -1), np.concatenate([size, size], -1)
    else:
        ref, size = np.stack([r0, r1], -1).reshape(xs.shape), np.repeat(size, 2, -1)
    off = 4 * 2.0 ** -23 + 12 * 2.0 ** -53 * np.array(far, np.float64)[:, None, None]
    check(got, ref, off * size)


# --------------------------------------------------------------------------- gradients
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["pairs", "half"])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_records_its_gradient(dtype, layout, inverse):
    """An x that requires grad gets the formula's gradient, J^T g with J the rotation, through a
    slice of wider heads; a plain call's bytes are the same."""
    rng = np.random.default_rng(44)
    cfg, rate = _rope_case(64, layout, "yarn", 1.1)
    q = rand(rng, dtype, 9, 4, 80).requires_grad_()
    p = rng.integers(0, 100000, 9)
    pos, g = ints(p, torch.int64), rand(rng, dtype, 9, 4, 64)
    y = rope(cfg, q[..., 8:72], pos, inverse=inverse)
    assert y.requires_grad
    with torch.no_grad():
        plain = rope(cfg, q[..., 8:72], pos, inverse=inverse)
    assert not plain.requires_grad and torch.equal(plain, y)
    (y * g).sum().backward()
    ref = O.rope(f64(g), p, rate, layout, 1.1, not inverse)
    check(q.grad[..., 8:72], ref, _rope_tol(f64(g), ref, dtype, layout, 1.1))
    assert (q.grad[..., :8] == 0).all() and (q.grad[..., 72:] == 0).all()
    # by differences of the 64-bit form, along one direction
    dx, step = rng.standard_normal((9, 4, 64)), 1e-6
    x = f64(q)[..., 8:72]
    dy = (O.rope(x + step * dx, p, rate, layout, 1.1, inverse) -
          O.rope(x - step * dx, p, rate, layout, 1.1, inverse)) / (2 * step)
    lhs, rhs = float((f64(g) * dy).sum()), float((f64(q.grad)[..., 8:72] * dx).sum())
    size = float(((np.abs(f64(q.grad))[..., 8:72] + 4) * np.abs(dx)).sum())
    assert abs(lhs - rhs) <= (1e-5 + half_step(dtype)) * size


def test_rope_gradient_of_a_gradient_shared_heads_and_sums():
    rng = np.random.default_rng(45)
    cfg, _ = _rope_case(32, "half", "none")
    pos = ints(rng.integers(0, 9000, 5), torch.int64)
    x = rand(rng, F32, 5, 1, 32).requires_grad_()
    y = rope(cfg, x.expand(5, 3, 32), pos)         # one row for three heads: their gradients add
    (gx,) = torch.autograd.grad(y.sum(), x, create_graph=True)   # of a sum: an expanded scalar
    one = rope(cfg, torch.ones(5, 1, 32, device="cuda"), pos, inverse=True)
    # each rotated 1 is a sum of two products of cosine and sine, all three alike
    assert (gx - 3 * one).abs().max() <= 3 * 4 * 2.0 ** -23 * 2
    w = rand(rng, F32, 5, 3, 32).requires_grad_()
    (gx,) = torch.autograd.grad((rope(cfg, x.expand(5, 3, 32), pos) * w).sum(), x, create_graph=True)
    (gw,) = torch.autograd.grad(gx.sum(), w)       # d/dw of 1 . J^T w is J 1
    assert torch.equal(gw, rope(cfg, torch.ones(5, 3, 32, device="cuda"), pos))


def test_rope_recorded_calls_of_bad_positions_configurations_and_graphs():
    rng = np.random.default_rng(46)
    cfg, _ = _rope_case(64, "pairs", "none")
    x, pos = rand(rng, F32, 4, 2, 64).requires_grad_(), ints([3, -1, 1 << 36, 9], torch.int64)
    y = rope(cfg, x, pos)
    cfg.base = 500.0                               # the call's configuration was taken with it
    y.sum().backward()
    assert (y[1:3] == 0).all() and (x.grad[1:3] == 0).all()
    cfg.base = 10000.0
    assert torch.equal(x.grad[0], rope(cfg, torch.ones(4, 2, 64, device="cuda"), pos, inverse=True)[0])
    # writing a given tensor is not recorded: refused where a gradient is asked for
    with pytest.raises(ValueError):
        rope(cfg, x, pos, out=torch.empty_like(x))
    with torch.no_grad():
        rope(cfg, x, pos, out=torch.empty_like(x))
    # forward and backward captured and replayed on other values
    leaf, pos = rand(rng, BF, 6, 3, 64).requires_grad_(), ints([0, 5, 70, 800, 9000, 7], torch.int64)
    w = rand(rng, BF, 6, 3, 64)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.autograd.grad((rope(cfg, leaf, pos) * w).sum(), leaf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (grad,) = torch.autograd.grad((rope(cfg, leaf, pos) * w).sum(), leaf)
    w.copy_(rand(rng, BF, 6, 3, 64))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(grad, rope(cfg, w, pos, inverse=True))


def test_a_step_on_queries_that_require_grad_runs_as_it_is():
    """Inference without no_grad on a model's own outputs: the layer is forward only."""
    rng = np.random.default_rng(47)
    lay, bt = layer(rng, BF, 16, [300])
    q, x = rand(rng, BF, 1, 16, 576), rand(rng, BF, 1, 576)
    args = (ints([0, 1], torch.int32), ints([299], torch.int64), 299, ints([299], torch.int64), x[:, :512], x[:, 512:])
    ref = lay.step(*args, q.clone())
    q.requires_grad_()
    out = lay.step(*args, q * 1)
    assert torch.equal(out, ref) and not out.requires_grad


# ------------------------------------------------------------------------------ ranges
# Values of 1e35 under 700 keys: the weighted sum in 32 bits, with weights of at most 1, reaches
# 7e37 at most, so the softmax's definition is computable and its result is of order 1e35. The
# keys behind the first tile weigh up to 2^15 of those in it: no weight may count for more than 1.
@pytest.mark.parametrize("size", [1e35, 1e-28])
def test_expanded_values_near_the_ends_of_the_type(size):
    rng = np.random.default_rng(40)
    heads, n, nq = 64, 700, 3                      # a pair of CTAs walks several tiles of an item
    cfg = v4a.latent_cfg(v4a.BF16, heads, 512, v4a.rope_cfg(64))
    q, pe = torch.ones(nq, heads, 192, device="cuda", dtype=BF), torch.zeros(n, 64, device="cuda", dtype=BF)
    k = torch.zeros(n, heads, 128, device="cuda", dtype=BF)
    k[128:] = 0.6377                               # 8.5 in log2 units above the first tile
    v = (size * rand(rng, torch.float32, n, heads, 128).abs()).to(BF)
    cu = [0, nq], [0, n]
    got = LatentLayer(cfg, None).attention_expanded(ints(cu[0], torch.int32), ints(cu[1], torch.int32),
                                                    q, k, pe, v)
    vs = f64(v) / size                             # the tolerance's absolute part is for values of order 1
    ref, mag = O.attention_expanded(*cu, f64(q), f64(k), f64(pe), vs, cfg.softmax_scale, True)
    lm = logit_bound(f64(q)[:, 0], np.concatenate([f64(k)[:, 0], f64(pe)], 1), cfg.softmax_scale)
    check(got.double() / size, ref, attn_tolerance(BF, ref, mag, 192, n, lm))


@pytest.mark.parametrize("size", [1e35, 1e-28])
def test_absorbed_values_near_the_ends_of_the_type(size):
    """1024 heads, so that a CTA walks several tiles of a sequence from the first on."""
    rng = np.random.default_rng(41)
    heads, total = 1024, [700] * 4
    lay, bt = layer(rng, BF, heads, total)
    for b in range(4):
        rows = [O.slot(bt, b, x) for x in range(700)]
        lay.pool.data[rows, :512] = (size * rand(rng, torch.float32, 700, 512).abs()).to(BF)
        lay.pool.data[rows, 512:] = 0
        lay.pool.data[rows[128:], 512:] = 2.25     # 15 in log2 units above the first tile
    q = torch.zeros(4, heads, 576, device="cuda", dtype=BF)
    q[..., 512:] = 1
    cu, start = [0, 1, 2, 3, 4], [699] * 4
    got = lay.attention(ints(cu, torch.int32), ints(start, torch.int64), 699, q)
    # every head's query is the same
    pool, q1 = f64(lay.pool.data), f64(q)[:, :1]
    pool[:, :512] /= size
    ref, mag = O.attention(pool, bt, cu, start, q1, lay.cfg.softmax_scale, 512)
    used = pool[[O.slot(bt, b, x) for b in range(4) for x in range(700)]]
    tol = attn_tolerance(BF, ref, mag, 576, 700, logit_bound(q1, used, lay.cfg.softmax_scale))
    assert all(torch.equal(got[:, :1], got[:, h:h + 1]) for h in range(1, heads))
    check(got[:, :1].double() / size, ref, tol)


# -------------------------------------------------------------------- uneven batches
@pytest.mark.parametrize("dtype,heads,latent,dim,total,new", [
    (BF, 64, 512, 64, [606, 20000], [606, 1]),           # split: one decode token is a third of all
    (BF, 64, 512, 64, [9000, 700, 300], [1, 700, 2]),
    (BF, 64, 512, 64, [900], [900]),                     # whole units
    (BF, 64, 512, 64, [5000], [620]),                    # split: the units are alike
    (BF, 128, 512, 64, [40, 5000, 0, 500], [40, 1, 0, 330]),
    (F32, 16, 64, 16, [3000, 1400], [2, 1400]),
    (F32, 16, 64, 16, [9000, 1300], [1, 1300]),
])
def test_many_units_beside_long_ones(dtype, heads, latent, dim, total, new):
    """More units than the GPU needs whole, with one sequence much longer than the others and
    without; captured once and replayed on the lengths of the other kind."""
    rng = np.random.default_rng(42)
    lay, bt = layer(rng, dtype, heads, total, latent, dim, fill=float("nan"))
    q = rand(rng, dtype, sum(new), heads, latent + dim)
    got, ref, tol, flags = _attn(lay, bt, total, new, q)
    assert flags == 0
    check(got, ref, tol)
    cu, start = (ints(x, t) for x, t in zip(batch(total, new), (torch.int32, torch.int64)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = lay.attention(cu, start, max(total) - 1, q)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, got)
    long = int(np.argmax(total))
    if new[long] < 3 and len(total) > 1:                 # the long sequence's first keys alone
        start[long] = 40
        g.replay()
        torch.cuda.synchronize()
        few = list(total)
        few[long] = 40 + new[long]
        got, ref, tol, flags = _attn(lay, bt, few, new, q, max_pos=max(total) - 1)
        assert flags == 0 and torch.equal(out, got)
        check(got, ref, tol)


def test_expanded_items_over_many_pairs_of_ctas():
    """One head and 5,000 keys: an item's 40 key tiles fall to more pairs than a warp has lanes."""
    rng = np.random.default_rng(50)
    cfg = v4a.latent_cfg(v4a.BF16, 1, 512, v4a.rope_cfg(64))
    for nq in (1, 300, 513):
        q, kv, pe = rand(rng, BF, nq, 1, 192), rand(rng, BF, 5000, 1, 256), rand(rng, BF, 5000, 64)
        got, ref, tol = _expanded(cfg, [0, nq], [0, 5000], q, kv[..., :128], pe, kv[..., 128:])
        check(got, ref, tol)


def test_a_sequence_alone_and_in_a_batch():
    """The others in a batch move the cuts along the keys, and with them the order of sums, but
    nothing else: each sequence alone is within the definition's bounds of itself in the batch."""
    rng = np.random.default_rng(43)
    total, new = [3000, 10, 777, 1, 5000], [1, 1, 3, 1, 2]
    lay, bt = layer(rng, BF, 64, total)
    q = rand(rng, BF, sum(new), 64, 576)
    got, ref, tol, _ = _attn(lay, bt, total, new, q)
    check(got, ref, tol)
    cu, start = batch(total, new)
    pages = lay.pool.block_table
    for b in range(len(total)):
        part = slice(int(cu[b]), int(cu[b + 1]))
        lay.pool.block_table = pages[b:b + 1].contiguous()
        one = lay.attention(ints([0, new[b]], torch.int32), ints(start[b:b + 1], torch.int64),
                            total[b] - 1, q[part].contiguous())
        check(one, f64(got)[part], 2 * tol[part])        # either is within tol of the definition


@pytest.mark.parametrize("dtype,heads", [(BF, 64), (BF, 16), (F32, 4)])
def test_positions_past_the_block_table(dtype, heads):
    """Keys that the table does not reach are left out like any block without a page, and not
    walked: a call whose positions run into the billions takes no longer than its table."""
    rng = np.random.default_rng(49)
    total, new = [500, 700], [1, 2]
    lay, bt = layer(rng, dtype, heads, total)
    q = rand(rng, dtype, 3, heads, 576)
    got, ref, tol, flags = _attn(lay, bt, total, new, q, start=[4000, 699], max_pos=4500)
    assert flags == v4a.DEV_MISSING_PAGE
    check(got, ref, tol)
    cu = ints([0, 1, 3], torch.int32)
    for start, max_pos, want in (([1 << 31, (1 << 31) - 7], 1 << 32, v4a.DEV_MISSING_PAGE),
                                 ([(1 << 63) - 9, 1 << 31], 1 << 32, v4a.DEV_MISSING_PAGE | v4a.DEV_BAD_POS)):
        e = err_word()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        far = lay.attention(cu, ints(start, torch.int64), max_pos, q, dev_err=e)
        b.record()
        assert v4a.v4a_get_error(e) == want
        near, ref, tol, _ = _attn(lay, bt, total, new, q, start=[767, 767], max_pos=767)
        check(far, ref, tol)                         # every key of either table
        assert a.elapsed_time(b) < 1000              # (tiles of 2^31 keys would take half a minute)
