"""Inputs and tolerances of the latent-attention tests."""
import numpy as np
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300.latent import LatentLayer
from compressed_sparse_long_gb300.layer import PagedPool
from oracle import latent_oracle as O

BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().double().numpy()


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def ints(x, dtype):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def layer(rng, dtype, heads, total, latent=512, rope=64, nope=128, v=128, rope_kw=None,
          gamma=False, hole=None, spare=1, fill=None):
    """A layer whose sequences hold total[b] cached positions on shuffled pages (`spare` more
    pages in the pool than needed; `hole` = (sequence, block) to leave without a page). Rows
    behind a sequence's last position hold `fill` when given."""
    rc = v4a.rope_cfg(rope, **(rope_kw or {}))
    cfg = v4a.latent_cfg(v4a.BF16 if dtype == BF else v4a.FP32, heads, latent, rc, nope_dim=nope,
                         v_dim=v)
    blocks = [max(0, -(-t // 256)) for t in total]
    pages = sum(blocks) + spare
    bt = np.full((len(total), max(blocks + [1])), -1, np.int32)
    perm = rng.permutation(pages)
    at = 0
    for b, n in enumerate(blocks):
        bt[b, :n] = perm[at:at + n]
        at += n
    data = torch.from_numpy(rng.standard_normal((pages * 256, latent + rope))).to("cuda", dtype)
    if fill is not None:
        used = np.zeros(pages * 256, bool)
        for b, t in enumerate(total):
            for blk in range(blocks[b]):
                s = bt[b, blk] * 256
                used[s:s + min(256, t - blk * 256)] = True
        data[torch.from_numpy(~used).cuda()] = fill
    if hole is not None:
        bt[hole] = -1
    g = None
    if gamma:
        g = torch.from_numpy(1 + 0.1 * rng.standard_normal(latent)).to("cuda", F32)
    return LatentLayer(cfg, PagedPool(data, None, ints(bt, torch.int32), 256), g), bt


def rand(rng, dtype, *shape):
    return torch.from_numpy(rng.standard_normal(shape)).to("cuda", dtype)


def batch(total, new):
    """(cu, start) of the last new[b] of total[b] positions."""
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    return cu, np.asarray(total, np.int64) - np.asarray(new, np.int64)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def attn_tolerance(dtype, ref, mag, width, n_keys, logit_mag):
    """What rounding may do to a softmax-weighted sum.

    mag = sum p |v|. The logits are fp32 sums of `width` products whose magnitudes sum to at
    most logit_mag: off by at most width 2^-24 logit_mag, which changes every weight by twice
    that, relatively; exponentials and sums over n_keys add (2^-21 + n_keys 2^-24). A bf16
    layer also rounds each weight once (half a step) before it multiplies the values, and the
    result is rounded once to the output type."""
    rel = 2 * width * 2.0 ** -24 * logit_mag + 2.0 ** -20 + n_keys * 2.0 ** -23
    if dtype == BF:
        rel += half_step(BF)
    return rel * mag + half_step(dtype) * np.abs(ref) + 1e-30


def logit_bound(q, keys, scale):
    return float(scale * (np.abs(q).reshape(-1, q.shape[-1]) @ np.abs(keys).T).max()) if len(keys) else 0.0


def check(got, ref, tol):
    got = f64(got)
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(got - ref) / tol)),
                           np.argwhere(bad)[:3].tolist())
