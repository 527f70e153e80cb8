"""Plain 64-bit numpy forms of the latent-attention operators, written from their definitions
(one token, one row, one pair at a time where that is cheap enough)."""
from __future__ import annotations

import math

import numpy as np


def rates(dim, base=10000.0, scaling="none", factor=1.0, orig=0.0, low=0.0, high=0.0):
    """Radians per position of each pair."""
    out = []
    for i in range(dim // 2):
        theta = base ** (-2.0 * i / dim)
        turns = orig * theta / (2 * math.pi)
        if scaling == "none":
            keep = 1.0
        elif scaling == "linear":
            keep = 0.0
        elif scaling == "parts":
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
        else:
            def pair(t):
                return dim * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(base))
            a = max(math.floor(pair(high)), 0)
            b = min(math.ceil(pair(low)), dim - 1)
            keep = 1.0 - min(1.0, max(0.0, (i - a) / max(b - a, 1e-3)))
        out.append(theta if scaling == "none" else theta * (keep + (1 - keep) / factor))
    return np.array(out)


def rope(x, pos, rate, layout="pairs", amplitude=1.0, inverse=False):
    """x [n, ..., d] rotated at integer positions pos [n]."""
    x = np.asarray(x, np.float64)
    n, d = x.shape[0], x.shape[-1]
    y = np.empty_like(x)
    for t in range(n):
        ang = float(pos[t]) * rate
        c, s = amplitude * np.cos(ang), amplitude * np.sin(ang)
        if inverse:
            s = -s
        if layout == "half":
            a, b = slice(0, d // 2), slice(d // 2, d)
        else:
            a, b = slice(0, d, 2), slice(1, d, 2)
        y[t][..., a] = x[t][..., a] * c - x[t][..., b] * s
        y[t][..., b] = x[t][..., a] * s + x[t][..., b] * c
    return y


def slot(bt, seq, pos, rows=256):
    blk = pos // rows
    if pos < 0 or blk >= bt.shape[1] or bt[seq, blk] < 0:
        return -1
    return int(bt[seq, blk]) * rows + pos % rows


def insert(pool, bt, cu, start, c, k_pe, gamma, eps, rate, layout="pairs", amplitude=1.0):
    """pool (float64, updated in place) and the list of written slots."""
    written = []
    for b in range(len(cu) - 1):
        for i in range(cu[b], cu[b + 1]):
            p = int(start[b]) + i - cu[b]
            s = slot(bt, b, p)
            if s < 0:
                continue
            row = np.asarray(c[i], np.float64)
            if gamma is not None:
                row = np.asarray(gamma, np.float64) * row / math.sqrt(np.mean(row * row) + eps)
            pe = rope(np.asarray(k_pe[i])[None], [p], rate, layout, amplitude)[0]
            pool[s] = np.concatenate([row, pe])
            written.append(s)
    return written


def attend(q, keys, values, scale):
    """Softmax-weighted sums of q [h, d] over keys [n, d], values [n, v], and the same sums of
    |values| (the yardstick of a tolerance); zeros when there is no key."""
    if len(keys) == 0:
        z = np.zeros((len(q), values.shape[1]))
        return z, z
    s = scale * (q @ keys.T)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    return p @ values, p @ np.abs(values)


def attention(pool, bt, cu, start, q, scale, latent, max_pos=None, window=None, sinks=0):
    """Absorbed form: q [n, H, w], keys without a page left out; (out, sums of |values|). With a
    window a token at p sees the keys above p - window and the first `sinks` of those up to its own."""
    out = np.zeros(q.shape[:2] + (latent,))
    mag = np.zeros_like(out)
    for b in range(len(cu) - 1):
        for i in range(cu[b], cu[b + 1]):
            p = int(start[b]) + i - cu[b]
            last = p if max_pos is None else min(p, max_pos)
            rows = [slot(bt, b, x) for x in range(last + 1)
                    if window is None or x > p - window or x < sinks]
            k = pool[[r for r in rows if r >= 0]]
            out[i], mag[i] = attend(q[i], k, k[:, :latent], scale)
    return out, mag


def e4m3(x):
    """Nearest e4m3 number (ties to even, saturating) of x >= 0."""
    x = np.minimum(np.asarray(x, np.float64), 448.0)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(x, 2.0 ** -20))), -6) - 3)
    return np.minimum(np.rint(x / step) * step, 448.0)


def e2m1(x):
    """Nearest e2m1 number (ties to the even code, saturating)."""
    a = np.minimum(np.abs(np.asarray(x, np.float64)), 6.0)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    return np.copysign(np.rint(a / step) * step, x)


def fp4_row(z, k, r):
    """A 4-bit row of values r z and rotary part k: (codes as values, block scales, rotary part,
    row scale). Products are taken in 32 bits, as the format states them; z is fp32."""
    f = np.float32
    z, k, r = np.asarray(z, f), np.asarray(k, np.float64), float(r)
    u = np.abs(z).max() * f(1 / 2688)
    s = f(r * float(u))
    least = max(f(np.abs(k).max() * (1 / 32768)), f(2.0 ** -100))
    if s < least:
        s = least
        u = f(float(least) / r)
    t = (z * (f(1) / u)).reshape(-1, 16)
    assert t.dtype == f
    block = e4m3(np.abs(t).max(1) * f(1 / 6))
    inv = np.where(block > 0, f(1) / np.maximum(block, 1e-30).astype(f), f(0)).astype(f)
    code = e2m1(t * inv[:, None])
    return code.ravel(), block, np.float16(k / float(s)).astype(np.float64), float(s)


def fp4_values(raw, scale, latent, rope):
    """Values that 4-bit rows stand for: raw uint8 [n, row bytes], scale [n]; 64 bits, exact but for
    the products with the row scale."""
    raw, n = np.asarray(raw), len(raw)
    level = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    code = np.empty((n, latent), np.int64)
    code[:, 0::2], code[:, 1::2] = raw[:, :latent // 2] & 15, raw[:, :latent // 2] >> 4
    value = level[code & 7] * np.where(code & 8, -1, 1)
    h = raw[:, latent // 2:latent // 2 + 2 * rope].copy().view(np.float16).astype(np.float64)
    b = raw[:, latent // 2 + 2 * rope:latent // 2 + 2 * rope + latent // 16].astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    block = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7.0), m * 2.0 ** -9)
    lat = value.reshape(n, -1, 16) * block[..., None]
    return np.concatenate([lat.reshape(n, latent), h], 1) * np.asarray(scale, np.float64)[:, None]


def attention_expanded(cu_q, cu_k, q, k, k_pe, v, scale, causal):
    """Expanded form; (out, sums of |values|)."""
    out = np.zeros(q.shape[:2] + (v.shape[2],))
    mag = np.zeros_like(out)
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        ks = slice(cu_k[b], cu_k[b + 1])
        for h in range(q.shape[1]):
            keys = np.concatenate([k[ks, h], k_pe[ks]], 1)
            for i in range(nq):
                n = max(0, nk - nq + i + 1) if causal else nk
                o, m = attend(q[cu_q[b] + i, h][None], keys[:n], v[ks, h][:n], scale)
                out[cu_q[b] + i, h], mag[cu_q[b] + i, h] = o[0], m[0]
    return out, mag
