"""CPU: refusals of the 4-bit latent cache and of windowed latent attention, and their definitions
pinned by tables and brute force."""
import ctypes
import json
import os
import subprocess

import numpy as np
import pytest
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300 import latent
from compressed_sparse_long_gb300.layer import PagedPool
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


def _cfg(fp4=True, latent_dim=512, rope=64, **kw):
    base = dict(dtype=v4a.BF16, n_heads=64, latent_dim=latent_dim, rope=v4a.rope_cfg(rope),
                cache_format=v4a.LATENT_FP4 if fp4 else v4a.LATENT_PLAIN)
    base.update(kw)
    return v4a.latent_cfg(**base)


CACHE = dict(data=4096, scale=8192, block_table=256, max_blocks=4, rows_per_block=256, n_pages=10,
             row_width=576, reserved=0)


def _calls(lib, cfg, cache, window=10, sinks=2, ws=None, wb=0, max_pos=100, n=4, n_seq=2, q=4096):
    c, k = B(cfg), B(cache)
    return dict(
        insert=lib.v4a_latent_insert(c, n_seq, n, 64, 64, q, 576, q, 576, None, k, None, None),
        gather=lib.v4a_latent_gather(c, n_seq, n, 64, 64, k, q, None, None),
        attn=lib.v4a_latent_attn(c, n_seq, n, 64, 64, max_pos, q, k, q, ws, wb, None, None),
        window=lib.v4a_latent_attn_window(c, n_seq, n, 64, 64, max_pos, window, sinks, q, k, q, ws, wb,
                                          None, None))


@pytest.mark.parametrize("kw,want", [(dict(cache_format=2), UNS), (dict(cache_format=-1), UNS),
                                     (dict(latent_dim=136), UNS), (dict(latent_dim=16), UNS),
                                     (dict(n_heads=0), ARG), (dict(rope=36), UNS)])
def test_bad_layers_are_refused(lib, kw, want):
    got = _calls(lib, _cfg(**kw), v4a.Cache(**CACHE))
    assert set(got.values()) == {want}, got
    assert v4a.v4a_latent_attn_window_workspace_size(_cfg(**kw), 1, 1, 100000, 5000, 0) == 0


def test_bad_caches_are_refused(lib):
    for kw in (dict(scale=None), dict(scale=8196), dict(data=None), dict(data=4104), dict(row_width=416),
               dict(rows_per_block=64), dict(reserved=1)):
        got = _calls(lib, _cfg(), v4a.Cache(**dict(CACHE, **kw)))
        assert set(got.values()) == {ARG}, (kw, got)


@pytest.mark.parametrize("fp4", [False, True])
def test_window_arguments(lib, fp4):
    cfg, cache = _cfg(fp4), v4a.Cache(**dict(CACHE, scale=8192 if fp4 else None))
    for kw in (dict(window=0), dict(window=-5), dict(sinks=-1), dict(max_pos=-1), dict(max_pos=1 << 36),
               dict(q=None), dict(q=4104), dict(n=-1), dict(n_seq=-1)):
        assert _calls(lib, cfg, cache, **kw)["window"] == ARG, kw
    size = v4a.v4a_latent_attn_window_workspace_size
    for window, sinks in ((0, 0), (-1, 0), (5, -1)):
        assert size(cfg, 2, 4, 100000, window, sinks) == 0
    need = size(cfg, 2, 4, 100000, 5000, 3)
    assert need > 0
    for kw in (dict(ws=None, wb=need), dict(ws=4100, wb=need), dict(ws=4096, wb=need - 1)):
        assert _calls(lib, cfg, cache, max_pos=100000, window=5000, sinks=3, **kw)["window"] == ARG
    assert _calls(lib, cfg, cache, n=0)["window"] == OK and _calls(lib, cfg, cache, n_seq=0)["window"] == OK
    # the work counts the window, not the context: a context of 2^34 positions is no more than one of 2^17
    assert size(cfg, 900, 900, (1 << 34) - 1, 4096, 4) == size(cfg, 900, 900, (1 << 17) - 1, 4096, 4) > 0
    assert size(cfg, 8, 8, 100, 200, 0) == v4a.v4a_latent_attn_workspace_size(cfg, 8, 8, 100)


def test_python_layer_checks_its_pool():
    lay = latent.LatentLayer(_cfg(), None)
    assert v4a.latent_row_bytes(lay.cfg) == 416 and v4a.latent_row_bytes(_cfg(False)) == 1152
    assert v4a.latent_row_bytes(_cfg(False, dtype=v4a.FP32)) == 2304
    for data, scale in ((torch.zeros(256, 576), None), (torch.zeros(256, 416, dtype=torch.uint8), None)):
        with pytest.raises(ValueError):
            latent.LatentLayer(_cfg(), PagedPool(data, scale, torch.zeros(1, 1, dtype=torch.int32), 256))


# ------------------------------------------------------------------------ the definitions
def test_e2m1_and_e4m3_of_the_definition():
    """Against the published value table and torch's e4m3 cast, ties and saturation included."""
    table = json.load(open(os.path.join(ROOT, "tests", "golden", "e2m1_format.json")))
    level = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    assert str([0.5, 1, 1.5, 2, 3, 4, 6]) and "6" in json.dumps(table)
    x = np.concatenate([np.linspace(-8, 8, 4001), (level[1:] + level[:-1]) / 2, -level])
    got = O.e2m1(x)
    dist = np.abs(np.abs(np.minimum(np.abs(x), 6))[:, None] - level)
    assert np.allclose(np.abs(np.abs(got) - np.minimum(np.abs(x), 6)), dist.min(1))
    assert O.e2m1([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]).tolist() == [0, 1, 1, 2, 2, 4, 4]
    y = np.concatenate([2.0 ** np.linspace(-12, 8.8, 5000), [0, 2 ** -10, 2 ** -9, 17, 447.9, 448]])
    y = np.minimum(y, 448).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3(y), want)


def test_fp4_rows_by_hand_and_their_error():
    z = np.zeros(32, np.float32)
    z[:4] = 6, 3, -1.5, 0.4
    z[16:18] = 0.75, -0.5
    code, block, half, s = O.fp4_row(z, np.array([1.0, -2.0]), 2.0)
    # u = 6 / 2688, so z / u = 448 z: the first block's scale is 448, the second's nearest to 56
    assert np.isclose(s, 12 / 2688) and block.tolist() == [448, 56]
    assert code[:4].tolist() == [6, 3, -1.5, 0.5] and code[16:18].tolist() == [6, -4]
    assert np.allclose(half * s, [1, -2], rtol=2 ** -11)
    rng = np.random.default_rng(0)
    for scale in (1e-20, 1e-3, 1.0, 1e15):
        z = (rng.standard_normal(512) * scale).astype(np.float32)
        code, block, half, s = O.fp4_row(z, rng.standard_normal(64) * scale, 1.0)
        b = np.repeat(block, 16) * s
        # half a step of e2m1 is at most 1; a block scale that rounded down cuts its largest value
        # (up to 6 / (1 - 1/16)) by less
        assert (np.abs(z - code * b) <= b * (1 + 2.0 ** -20)).all()
    # a rotary part that dwarfs the latent one, rows of zeros
    code, block, half, s = O.fp4_row(z * 1e-18, np.full(8, 1e6), 0.5)
    assert np.isclose(s, 1e6 / 32768) and np.allclose(half * s, 1e6, rtol=2 ** -11)
    code, block, half, s = O.fp4_row(np.zeros(32), np.zeros(8), 1.0)
    assert s == 2.0 ** -100 and not code.any() and not half.any()


def test_windowed_attention_by_brute_force():
    rng = np.random.default_rng(4)
    bt = np.array([[1, 0, -1]], np.int32)
    pool, q = rng.standard_normal((512, 12)), rng.standard_normal((3, 2, 12))
    for window, sinks in ((1, 0), (7, 3), (300, 0), (10 ** 9, 0), (5, 400)):
        o, _ = O.attention(pool, bt, [0, 3], [297], q, 0.3, 8, window=window, sinks=sinks)
        for i, p in enumerate((297, 298, 299)):
            keys = [x for x in range(p + 1) if p - x < window or x < sinks]
            rows = np.array([pool[bt[0, x // 256] * 256 + x % 256] for x in keys])
            for h in range(2):
                w = np.exp(0.3 * rows @ q[i, h])
                assert np.allclose(o[i, h], w @ rows[:, :8] / w.sum())


def test_the_format_field_by_its_name_before(lib, tmp_path):
    """The field was called `reserved` and had to be 0: programs that say so go on, and another value
    is not taken for 0."""
    rope = v4a.rope_cfg(64)
    kw = dict(dtype=v4a.BF16, n_heads=4, latent_dim=512, nope_dim=128, v_dim=128, rms_eps=1e-6,
              softmax_scale=0.1, rope=rope)
    for value, ok in ((0, True), (v4a.LATENT_FP4, True), (7, False)):
        cfg = v4a.LatentCfg(reserved=value, **kw)
        assert cfg.cache_format == cfg.reserved == value
        assert (lib.v4a_latent_attn_workspace_size(B(cfg), 2, 2, 1000) > 0) == ok
    cfg = v4a.LatentCfg(**kw)
    assert cfg.reserved == 0
    prog = tmp_path / "names.c"
    prog.write_text('#include "v4a.h"\n'
                    'int main(void){ v4a_latent_cfg a = {.dtype = V4A_BF16, .v_dim = 128, .reserved = 0},'
                    ' b = {.dtype = V4A_BF16, .cache_format = V4A_LATENT_FP4};'
                    ' v4a_latent_cfg c = {V4A_BF16, 4, 512, 128, 128, 0, 1e-6f, 0.1f, a.rope};'
                    ' b.reserved -= 1; return a.cache_format + b.cache_format + c.reserved; }\n')
    exe = tmp_path / "names"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Wno-missing-field-initializers",
                    "-Wno-missing-braces", "-Werror",
                    "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
