"""What the 4-bit latent cache's documentation promises beyond the tolerances of its other tests: the
published code values, weights of 11 bits, row scales that do not depend on how sums are formed."""
import json
import os

import numpy as np
import pytest
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300.latent import LatentLayer
from compressed_sparse_long_gb300.layer import PagedPool
from latent_helpers import BF, F32, check, half_step
from oracle import latent_oracle as O

GOLDEN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "golden", "e2m1_format.json")


# ------------------------------------------------------------------------------ codes
def test_codes_are_the_published_ones():
    table = json.load(open(GOLDEN))
    level = np.array(table["magnitudes"])
    x = np.linspace(-9, 9, 7201)
    got = O.e2m1(x)
    # every value of the table is its own code, everything else goes to a nearest one
    assert O.e2m1(level).tolist() == level.tolist() and O.e2m1(-level).tolist() == (-level).tolist()
    assert set(np.abs(got)) == set(level.tolist()) and (np.sign(got) * np.sign(x) >= 0).all()
    cut = np.minimum(np.abs(x), table["max_normal"])
    assert np.allclose(np.abs(np.abs(got) - cut), np.abs(cut[:, None] - level).min(1), atol=1e-12)
    assert O.e2m1(1e9) == table["max_normal"] and O.e2m1(-1e9) == -table["max_normal"]
    assert level[level > 0].min() == table["max_subnormal"] and level[level > 0.5].min() == table["min_normal"]
    # a row of all sixteen codes, block scales of 1
    raw = np.zeros((1, 48), np.uint8)
    raw[0, :8] = np.arange(0, 16, 2) | np.arange(1, 16, 2) << 4
    raw[0, 16 + 16:16 + 16 + 2] = 7 << 3
    row = O.fp4_values(raw, np.ones(1), 32, 8)[0]
    assert row[:16].tolist() == level.tolist() + (-level).tolist()


# ----------------------------------------------------------------------------- weights
C, R, H = 512, 64, 64
LENGTHS = [2, 2, 4, 10, 64, 300, 700]


def opposite_pairs(rng):
    """Rows in pairs of opposite values and equal scales, without rotary parts; queries of one element,
    so that a logit is one product and at most 1. (raw rows, row scales, queries by sequence)"""
    n = sum(LENGTHS)
    raw = np.zeros((n, 416), np.uint8)
    raw[0::2, :C // 2] = rng.integers(0, 256, (n // 2, C // 2))
    raw[1::2, :C // 2] = raw[0::2, :C // 2] ^ 0x88
    raw[0::2, C // 2 + 2 * R:C // 2 + 2 * R + C // 16] = rng.integers((7 + 4) << 3, (7 + 8) << 3, (n // 2, C // 16))
    raw[1::2, C // 2 + 2 * R:] = raw[0::2, C // 2 + 2 * R:]
    scale = np.repeat(2.0 ** rng.uniform(-13, -7, n // 2), 2).astype(np.float32)
    rows = O.fp4_values(raw, scale, C, R)
    q, at = np.zeros((len(LENGTHS), H, C + R)), 0
    for b, t in enumerate(LENGTHS):
        for h in range(H):
            d = rng.integers(0, C)
            most = np.abs(rows[at:at + t, d]).max()
            q[b, h, d] = rng.uniform(0.02, 1) / max(most, 2.0 ** -10) * (C + R) ** 0.5
        at += t
    q = torch.from_numpy(q).to(BF)
    return raw, scale, rows, q


SCALE = (C + R) ** -0.5


def expected(rows, q, window=None):
    """(result, tolerance). Opposite values cancel, so the result's own rounding (half a step of it) is
    small beside what rounding the weights does: half a step of f16 on each, 2^-11. Besides: a logit is
    one exact product, scaled in 32 bits with the row's scale, log2 e and the query's power of two (four
    roundings), the scale's logarithm is added (2 ulp, of a number below 16) and the reference subtracted:
    numbers below 32 in all, off by at most 8 2^-20, times ln 2; the exponential adds 2^-22, the sums of
    n weights n 2^-23, the products' f16 terms nothing."""
    ref, tol, at = np.zeros((len(LENGTHS), H, C)), np.zeros((len(LENGTHS), H, C)), 0
    for b, t in enumerate(LENGTHS):
        k = rows[at:at + t]
        k = k if window is None else k[-window:]
        for h in range(H):
            o, mag = O.attend(q[b:b + 1, h], k, k[:, :C], SCALE)
            rel = 2.0 ** -11 + 8 * 2.0 ** -20 + 2.0 ** -22 + len(k) * 2.0 ** -23
            ref[b, h], tol[b, h] = o[0], rel * mag[0] + half_step(BF) * np.abs(o[0]) + 1e-30
        at += t
    return ref, tol


def rounded(rows, scale, q, dtype):
    """The result with weights times row scales held in `dtype`, all else in 64 bits."""
    out, at = np.zeros((len(LENGTHS), H, C)), 0
    for b, t in enumerate(LENGTHS):
        k, s = rows[at:at + t], scale[at:at + t].astype(np.float64)
        x = (q[b] @ k.T) * SCALE * np.log2(np.e) + np.log2(s)
        w = 2.0 ** (x - x.max(1, keepdims=True) + 6)
        held = torch.from_numpy(w).to(dtype).double().numpy()
        out[b] = (held @ (k[:, :C] / s[:, None])) / (w / s).sum(1, keepdims=True)
        at += t
    return torch.from_numpy(out).to(BF)


def test_the_tolerance_tells_eleven_bits_from_eight():
    rng = np.random.default_rng(5)
    _, scale, rows, q = opposite_pairs(rng)
    ref, tol = expected(rows, q.double().numpy())
    check(rounded(rows, scale, q.double().numpy(), torch.float16), ref, tol)
    with pytest.raises(AssertionError):
        check(rounded(rows, scale, q.double().numpy(), BF), ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [None, 2, 64])
def test_weights_keep_eleven_bits(window):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    rng = np.random.default_rng(5)
    raw, scale, rows, q = opposite_pairs(rng)
    blocks = [-(-t // 256) for t in LENGTHS]
    pages, at, page = sum(blocks), 0, 0
    bt = np.full((len(LENGTHS), max(blocks)), -1, np.int32)
    data = np.zeros((pages * 256, 416), np.uint8)
    s = np.zeros(pages * 256, np.float32)
    for b, t in enumerate(LENGTHS):
        data[page * 256:page * 256 + t], s[page * 256:page * 256 + t] = raw[at:at + t], scale[at:at + t]
        bt[b, :blocks[b]] = np.arange(page, page + blocks[b])
        at, page = at + t, page + blocks[b]
    cfg = v4a.latent_cfg(v4a.BF16, H, C, v4a.rope_cfg(R), softmax_scale=SCALE, cache_format=v4a.LATENT_FP4)
    lay = LatentLayer(cfg, PagedPool(torch.from_numpy(data).cuda(), torch.from_numpy(s).cuda(),
                                     torch.from_numpy(bt).cuda(), 256))
    cu = torch.arange(len(LENGTHS) + 1, dtype=torch.int32, device="cuda")
    start = torch.tensor(LENGTHS, dtype=torch.int64, device="cuda") - 1
    got = lay.attention(cu, start, max(LENGTHS) - 1, q.cuda(), window=window)
    check(got, *expected(rows, q.double().numpy(), window))


# ------------------------------------------------------------------------- row scales
@pytest.mark.gpu
@pytest.mark.parametrize("latent,dim", [(512, 64), (1024, 128), (32, 8), (544, 24)])
def test_row_scales_of_fp32_layers_are_the_formulas(latent, dim):
    """s = r u with r the formula's in 64 bits, rounded to 32: the kernel forms the mean square and the
    root to about 2^-44, so it rounds to another number in one row of some hundred thousand. A sum in 32
    bits gives a neighbour in about a quarter of all rows."""
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    rng, n, f = np.random.default_rng(latent), 2000, np.float32
    c = rng.standard_normal((n, latent)) * 10.0 ** rng.uniform(-3, 3, (n, 1))
    c[n // 2:] *= 10.0 ** rng.uniform(-2, 2, (n - n // 2, latent))       # and far apart within a row
    c, k = c.astype(f), (0.1 * rng.standard_normal((n, dim))).astype(f)
    gamma = (1 + 0.1 * rng.standard_normal(latent)).astype(f)
    r = (1 / np.sqrt((c.astype(np.float64) ** 2).mean(1) + float(f(1e-6)))).astype(f)
    u = np.abs(c * gamma).max(1) * (f(1) / f(2688))
    want = r * u
    assert want.dtype == f and (want > 2 * np.abs(k).max(1) * 2 / 32768).all()   # the rotary part does not decide
    cfg = v4a.latent_cfg(v4a.FP32, 4, latent, v4a.rope_cfg(dim), cache_format=v4a.LATENT_FP4)
    pages = -(-n // 256)
    pool = PagedPool(torch.zeros(pages * 256, v4a.latent_row_bytes(cfg), dtype=torch.uint8, device="cuda"),
                     torch.zeros(pages * 256, device="cuda"),
                     torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1), 256)
    lay = LatentLayer(cfg, pool, torch.from_numpy(gamma).cuda())
    x = torch.from_numpy(np.concatenate([c, k], 1)).to("cuda", F32)
    lay.insert(torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"),
               x[:, :latent], x[:, latent:])
    assert np.array_equal(pool.scale.cpu().numpy()[:n], want)
