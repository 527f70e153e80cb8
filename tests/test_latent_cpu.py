"""CPU: the latent-attention entry points' refusals and struct layouts, and the 64-bit
definitions pinned by closed forms. Nothing here touches a GPU."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300 import latent
from oracle import latent_oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, UNS, OK = v4a.ERR_ARG, v4a.ERR_UNSUPPORTED, v4a.OK
B = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(v4a.LIB_PATH):
        from compressed_sparse_long_gb300 import build
        build.build()
    return v4a.library()


def test_struct_layouts_match_c(tmp_path):
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "v4a.h"\n'
                    'int main(void){printf("%zu %zu %zu %zu %zu %d %d\\n", sizeof(v4a_rope_cfg),'
                    ' offsetof(v4a_rope_cfg, amplitude), sizeof(v4a_latent_cfg),'
                    ' offsetof(v4a_latent_cfg, softmax_scale), offsetof(v4a_latent_cfg, rope),'
                    ' V4A_MAX_SEQ, V4A_BF16); return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(prog), "-o",
                    str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [ctypes.sizeof(v4a.RopeCfg), v4a.RopeCfg.amplitude.offset,
                   ctypes.sizeof(v4a.LatentCfg), v4a.LatentCfg.softmax_scale.offset,
                   v4a.LatentCfg.rope.offset, v4a.MAX_SEQ, v4a.BF16]


def _rope(**kw):
    base = dict(dim=64)
    base.update(kw)
    return v4a.rope_cfg(**base)


BAD_ROPES = [(dict(dim=0), UNS), (dict(dim=3), UNS), (dict(dim=258), UNS), (dict(layout=2), UNS),
             (dict(scaling=4), UNS), (dict(scaling=-1), UNS), (dict(base=0.0), ARG),
             (dict(base=float("inf")), ARG), (dict(amplitude=0.0), ARG),
             (dict(scaling=1, factor=0.0), ARG), (dict(scaling=2, factor=2.0), ARG),
             (dict(scaling=2, factor=2.0, orig_max_pos=4096.0, low=4.0, high=4.0), ARG),
             (dict(scaling=3, factor=2.0, orig_max_pos=4096.0, low=1.0, high=4.0, base=1.0), ARG),
             (dict(amplitude=float("nan")), ARG)]


@pytest.mark.parametrize("kw,want", BAD_ROPES)
def test_bad_rotations_are_refused(lib, kw, want):
    r = _rope(**kw)
    assert lib.v4a_rope(B(r), v4a.BF16, 0, 0, None, None, 0, 0, None, 0, 0, 0, None, None) == want
    c = v4a.latent_cfg(v4a.BF16, 64, 512, r, softmax_scale=0.1)
    assert lib.v4a_latent_insert(B(c), 0, 0, None, None, None, 0, None, 0, None, None, None,
                                 None) == want


def test_rope_arguments(lib):
    r = _rope()

    def call(dtype=v4a.BF16, n=2, h=2, pos=256, x=256, xt=128, xh=64, y=512, yt=128, yh=64, cfg=r):
        return lib.v4a_rope(None if cfg is None else B(cfg), dtype, n, h, pos, x, xt, xh, y, yt,
                            yh, 0, None, None)
    assert call(n=0) == OK and call(h=0) == OK and call(n=0, pos=None, x=None, y=None) == OK
    for kw in (dict(cfg=None), dict(n=-1), dict(h=-1), dict(pos=None), dict(x=None), dict(y=None),
               dict(x=257), dict(y=513), dict(xt=-1), dict(yh=63), dict(yt=63), dict(yt=-128),
               dict(x=512, xt=256), dict(x=512, xh=32)):
        assert call(**kw) == ARG, kw
    assert call(dtype=v4a.BF16_FP8) == UNS


def _cfg(**kw):
    base = dict(dtype=v4a.BF16, n_heads=64, latent_dim=512, rope=_rope())
    base.update(kw)
    return v4a.latent_cfg(**base)


CACHE = dict(data=4096, scale=None, block_table=256, max_blocks=4, rows_per_block=256,
             n_pages=10, row_width=576, reserved=0)
BAD_CFGS = [(dict(dtype=v4a.BF16_FP8), UNS), (dict(dtype=7), UNS), (dict(n_heads=0), ARG),
            (dict(n_heads=1025), ARG), (dict(latent_dim=0), UNS), (dict(latent_dim=508), UNS),
            (dict(latent_dim=1032), UNS), (dict(nope_dim=4), UNS), (dict(nope_dim=264), UNS),
            (dict(v_dim=0), UNS), (dict(v_dim=264), UNS), (dict(rope=_rope(dim=36)), UNS),
            (dict(rope=_rope(dim=136)), UNS), (dict(rms_eps=-1.0), ARG),
            (dict(rms_eps=float("nan")), ARG), (dict(softmax_scale=-1.0), ARG),
            (dict(softmax_scale=float("inf")), ARG)]


def _calls(lib, cfg, cache, **kw):
    """The four cache calls and the expanded one on the same arguments."""
    a = dict(n_seq=2, n=4, cu=64, start=64, q=4096, ws=None, wb=0, max_pos=100)
    a.update(kw)
    c, k = None if cfg is None else B(cfg), None if cache is None else B(cache)
    return dict(
        insert=lib.v4a_latent_insert(c, a["n_seq"], a["n"], a["cu"], a["start"], a["q"], 576, a["q"],
                                     576, None, k, None, None),
        gather=lib.v4a_latent_gather(c, a["n_seq"], a["n"], a["cu"], a["start"], k, a["q"], None,
                                     None),
        attn=lib.v4a_latent_attn(c, a["n_seq"], a["n"], a["cu"], a["start"], a["max_pos"], a["q"], k,
                                 a["q"], a["ws"], a["wb"], None, None))


@pytest.mark.parametrize("kw,want", BAD_CFGS)
def test_bad_layers_are_refused(lib, kw, want):
    got = _calls(lib, _cfg(**kw), v4a.Cache(**CACHE))
    assert set(got.values()) == {want}, got
    e = lib.v4a_latent_attn_expanded(B(_cfg(**kw)), 1, 1, 64, 1, 64, 4096, 4096, 128, 128, 4096, 64,
                                     4096, 128, 128, 1, 4096, None, 0, None, None)
    assert e == want
    assert v4a.v4a_latent_attn_workspace_size(_cfg(**kw), 1, 1, 100000) == 0


def test_bad_batches_and_caches_are_refused(lib):
    good = v4a.Cache(**CACHE)
    for kw in (dict(n_seq=-1), dict(n=-1), dict(cu=None), dict(start=None), dict(q=None),
               dict(q=4104)):
        got = _calls(lib, _cfg(), good, **kw)
        assert set(got.values()) == {ARG}, (kw, got)
    assert set(_calls(lib, _cfg(), good, n_seq=v4a.MAX_SEQ + 1).values()) == {UNS}
    assert set(_calls(lib, None, good).values()) == {ARG}
    assert set(_calls(lib, _cfg(), None).values()) == {ARG}
    # nothing to do: nothing is looked at
    for kw in (dict(n=0), dict(n_seq=0)):
        assert set(_calls(lib, _cfg(), None, cu=None, start=None, q=None, **kw).values()) == {OK}
    for kw, want in ((dict(data=None), ARG), (dict(data=4104), ARG), (dict(block_table=None), ARG),
                     (dict(rows_per_block=64), ARG), (dict(row_width=512), ARG),
                     (dict(max_blocks=0), ARG), (dict(reserved=1), ARG), (dict(n_pages=-1), ARG),
                     (dict(n_pages=1 << 23), UNS)):
        got = _calls(lib, _cfg(), v4a.Cache(**dict(CACHE, **kw)))
        assert set(got.values()) == {want}, (kw, got)


def test_insert_and_attention_arguments(lib):
    c, k = _cfg(), v4a.Cache(**CACHE)

    def ins(c_=4096, cs=576, pe=4096, ks=576, g=None):
        return lib.v4a_latent_insert(B(c), 1, 1, 64, 64, c_, cs, pe, ks, g, B(k), None, None)
    for kw in (dict(c_=4098), dict(pe=4098), dict(cs=577), dict(ks=4), dict(cs=-576), dict(g=4100),
               dict(c_=None), dict(pe=None)):
        assert ins(**kw) == ARG, kw
    # positions: none, negative, past the limit
    for mp in (-1, 1 << 36):
        assert _calls(lib, c, k, max_pos=mp)["attn"] == ARG
        assert v4a.v4a_latent_attn_workspace_size(c, 2, 4, mp) == 0
    # the workspace: missing, misaligned, too small
    need = v4a.v4a_latent_attn_workspace_size(c, 2, 4, 100000)
    assert need > 0
    for kw in (dict(ws=None, wb=need), dict(ws=4100, wb=need), dict(ws=4096, wb=need - 1)):
        assert _calls(lib, c, k, max_pos=100000, **kw)["attn"] == ARG
    # one key tile a sequence at most: nothing is split
    assert v4a.v4a_latent_attn_workspace_size(c, 2, 4, 20) == 0
    # more (token, head) rows than the plan counts
    assert _calls(lib, _cfg(n_heads=1024), k, n=1 << 21)["attn"] == UNS


def test_expanded_arguments(lib):
    def call(cfg=_cfg(), n_seq=1, n_q=2, cu_q=64, n_k=2, cu_k=64, q=4096, k=4096, kt=128, kh=128,
             pe=4096, ps=64, v=4096, vt=128, vh=128, out=4096, ws=None, wb=0):
        return lib.v4a_latent_attn_expanded(B(cfg), n_seq, n_q, cu_q, n_k, cu_k, q, k, kt, kh, pe,
                                            ps, v, vt, vh, 1, out, ws, wb, None, None)
    for kw in (dict(n_seq=-1), dict(n_q=-1), dict(n_k=-1), dict(cu_q=None), dict(cu_k=None),
               dict(q=None), dict(out=None), dict(q=4104), dict(out=4104), dict(k=None),
               dict(k=4104), dict(pe=None), dict(v=None), dict(kt=100), dict(kh=0), dict(ps=-64),
               dict(vt=1), dict(vh=12), dict(pe=4100), dict(v=4098)):
        assert call(**kw) == ARG, kw
    assert call(cfg=_cfg(nope_dim=0, softmax_scale=1.0)) == UNS
    assert call(n_seq=v4a.MAX_SEQ + 1) == UNS
    need = v4a.v4a_latent_attn_expanded_workspace_size(_cfg(), 1, 2, 5000)
    assert need > 0 and v4a.v4a_latent_attn_expanded_workspace_size(_cfg(), 1, 2, 128) == 0
    assert v4a.v4a_latent_attn_expanded_workspace_size(_cfg(nope_dim=64), 1, 2, 5000) == 0
    for kw in (dict(ws=None, wb=need), dict(ws=4100, wb=need), dict(ws=4096, wb=need - 1)):
        assert call(n_k=5000, **kw) == ARG, kw
    # more (item, key tile) steps than the plan counts
    assert call(n_q=1 << 24, n_k=1 << 24) == UNS
    assert call(n_q=0, q=None, out=None, cu_q=None) == OK and call(n_seq=0) == OK


def test_python_layer_refuses_host_tensors():
    with pytest.raises(ValueError):
        latent.rope(_rope(), torch.zeros(2, 3, 64), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        latent.rope(_rope(), torch.zeros(2, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        latent.LatentLayer(_cfg(dtype=v4a.BF16_FP8), None)
    lay = latent.LatentLayer(_cfg(), None)
    with pytest.raises(ValueError):
        lay.insert(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int64),
                   torch.zeros(1, 512), torch.zeros(1, 64))


# ------------------------------------------------------------------------ the definitions
def test_rates_of_the_scalings():
    plain = O.rates(64)
    assert plain[0] == 1.0 and math.isclose(plain[16], 0.01) and len(plain) == 32
    assert np.allclose(O.rates(64, scaling="linear", factor=4.0), plain / 4)
    kw = dict(factor=8.0, orig=4096.0, low=1.0, high=32.0)
    for kind in ("parts", "yarn"):
        r = O.rates(64, scaling=kind, **kw)
        turns = 4096 * plain / (2 * math.pi)
        assert np.allclose(r[turns > 40], plain[turns > 40])          # fast pairs keep their rate
        assert np.allclose(r[turns < 0.7], plain[turns < 0.7] / 8)    # slow ones are interpolated
        assert (r <= plain).all() and (r >= plain / 8 * (1 - 1e-12)).all()
    # halfway up the ramp in turns: t = 1/2, so the rate is (1 + 1/8) / 2 of the plain one
    half = 2 * math.pi * 16.5 / 4096
    r = O.rates(2, base=10.0, scaling="parts", factor=8.0, orig=16.5 * 2 * math.pi, low=1.0, high=32.0)
    assert math.isclose(r[0], (1 + 1 / 8) / 2) and half > 0


def test_rope_closed_forms():
    rng = np.random.default_rng(1)
    rate = O.rates(8)
    x = rng.standard_normal((5, 3, 8))
    pos = np.array([0, 1, 7, 100, 12345])
    for layout in ("pairs", "half"):
        y = O.rope(x, pos, rate, layout)
        assert np.allclose(y[0], x[0]) and np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.allclose(O.rope(y, pos, rate, layout, inverse=True), x)
        # a product of two rotated vectors depends on the distance of their positions alone
        a, b = rng.standard_normal((1, 8)), rng.standard_normal((1, 8))
        dot = [float((O.rope(a, [p], rate, layout) * O.rope(b, [p + 9], rate, layout)).sum())
               for p in (0, 50)]
        assert math.isclose(*dot, rel_tol=1e-9, abs_tol=1e-12)
    perm = np.array([0, 4, 1, 5, 2, 6, 3, 7])
    assert np.allclose(O.rope(x[..., perm], pos, rate, "pairs"), O.rope(x, pos, rate, "half")[..., perm])


def test_attention_definitions_agree():
    """The absorbed form over [latent | rotary] rows equals the expanded form with the
    projections applied to keys and values; torch's softmax is the third opinion."""
    rng = np.random.default_rng(2)
    C, R, N, V, H, L = 24, 8, 16, 12, 3, 70
    rows = rng.standard_normal((256, C + R))
    bt = np.array([[0]], np.int32)
    wk, wv = rng.standard_normal((H, N, C)), rng.standard_normal((H, V, C))
    q = rng.standard_normal((4, H, N + R))
    qa = np.concatenate([np.einsum("nhd,hdc->nhc", q[..., :N], wk), q[..., N:]], -1)
    o, mag = O.attention(rows, bt, [0, 4], [L - 4], qa, 0.05, C)
    absorbed = np.einsum("nhc,hvc->nhv", o, wv)
    k, v = np.einsum("xc,hdc->xhd", rows[:L, :C], wk), np.einsum("xc,hvc->xhv", rows[:L, :C], wv)
    e, _ = O.attention_expanded([0, 4], [0, L], q, k, rows[:L, C:], v, 0.05, True)
    assert np.allclose(absorbed, e) and (mag >= np.abs(o) - 1e-12).all()
    t = torch.from_numpy
    keys = np.concatenate([k, np.repeat(rows[:L, None, C:], H, 1)], -1)
    s = 0.05 * torch.einsum("nhd,xhd->hnx", t(q), t(keys))
    mask = torch.arange(L)[None] <= torch.arange(L - 4, L)[:, None]
    ref = torch.einsum("hnx,xhv->nhv", torch.softmax(s.masked_fill(~mask, -math.inf), -1), t(v))
    assert np.allclose(e, ref.numpy())
    z, _ = O.attention_expanded([0, 3], [0, 2], q[:3], k[:2], rows[:2, C:], v[:2], 0.05, True)
    assert (z[0] == 0).all() and np.allclose(z[1], v[0])
