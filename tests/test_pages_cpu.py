"""CPU: the page calls' refusals, struct layouts and Python checks, and their plain forms pinned on
cases worked by hand."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300.pages import PageTable
from oracle import pages_oracle as O

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
                    'int main(void){printf("%zu %zu %zu %zu %zu %zu %d %u %d %d\\n",'
                    ' sizeof(v4a_page_table), offsetof(v4a_page_table, n_pages),'
                    ' sizeof(v4a_pool), offsetof(v4a_pool, row_bytes),'
                    ' offsetof(v4a_pool, rows_per_block), offsetof(v4a_latent_cfg, cache_format),'
                    ' V4A_MAX_POOLS, V4A_DEV_NO_PAGE, V4A_LATENT_FP4,'
                    ' V4A_LATENT_FP4_ROW_BYTES(128, 32)); return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(prog), "-o",
                    str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    small = v4a.latent_cfg(v4a.BF16, 4, 128, v4a.rope_cfg(32), cache_format=v4a.LATENT_FP4)
    assert got == [ctypes.sizeof(v4a.PageTableDesc), v4a.PageTableDesc.n_pages.offset,
                   ctypes.sizeof(v4a.Pool), v4a.Pool.row_bytes.offset,
                   v4a.Pool.rows_per_block.offset, v4a.LatentCfg.cache_format.offset,
                   v4a.MAX_POOLS, v4a.DEV_NO_PAGE, v4a.LATENT_FP4, v4a.latent_row_bytes(small)]
    assert got[-1] == 144


TABLE = dict(block_table=256, refs=4096, n_seq=4, max_blocks=8, n_pages=100)
POOL = dict(data=4096, scale=None, row_bytes=1152, rows_per_block=256, reserved=0)


def _calls(lib, table=TABLE, pools=(POOL,), ws=4096, wb=1 << 20, first=64, last=64, src=64, dst=64,
           length=64, n=2, used=64, n_pools=None):
    t = None if table is None else B(v4a.PageTableDesc(**table))
    ps = (v4a.Pool * max(1, len(pools)))(*[v4a.Pool(**p) for p in pools]) if pools is not None else None
    k = n_pools if n_pools is not None else len(pools)
    return dict(free=lib.v4a_pages_free(t, first, last, None, None),
                grow=lib.v4a_pages_grow(t, first, last, ws, wb, None, None),
                fork=lib.v4a_pages_fork(t, ps, k, n, src, dst, length, ws, wb, None, None),
                copy=lib.v4a_pages_copy(t, ps, k, n, src, dst, None, None),
                compact=lib.v4a_pages_compact(t, ps, k, used, None, ws, wb, None, None))


@pytest.mark.parametrize("kw,want", [
    (None, ARG), (dict(n_seq=-1), ARG), (dict(max_blocks=-1), ARG), (dict(n_pages=-1), ARG),
    (dict(block_table=None), ARG), (dict(refs=None), ARG), (dict(refs=4104), ARG),
    (dict(block_table=258), ARG), (dict(n_seq=v4a.MAX_SEQ + 1), UNS),
    (dict(n_pages=(1 << 23) + 1), UNS), (dict(max_blocks=(1 << 20) + 1), UNS)])
def test_bad_tables_are_refused(lib, kw, want):
    table = None if kw is None else dict(TABLE, **kw)
    got = _calls(lib, table=table)
    assert set(got.values()) == {want}, got
    if table is not None:
        assert v4a.v4a_pages_workspace_size(v4a.PageTableDesc(**table)) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(data=None), ARG), (dict(data=4104), ARG), (dict(scale=4098), ARG), (dict(row_bytes=0), ARG),
    (dict(row_bytes=-16), ARG), (dict(row_bytes=100), ARG), (dict(rows_per_block=0), ARG),
    (dict(rows_per_block=257), ARG), (dict(reserved=1), ARG), (dict(row_bytes=(1 << 20) + 16), UNS)])
def test_bad_pools_are_refused(lib, kw, want):
    got = _calls(lib, pools=(POOL, dict(POOL, **kw)))
    assert {got[k] for k in ("fork", "copy", "compact")} == {want}, got


def test_bad_lists_and_workspaces_are_refused(lib):
    for kw, who in ((dict(first=None), ("free", "grow")), (dict(last=None), ("free", "grow")),
                    (dict(src=None), ("fork", "copy")), (dict(dst=None), ("fork", "copy")),
                    (dict(length=None), ("fork",)), (dict(n=-1), ("fork", "copy")),
                    (dict(used=None), ("compact",)), (dict(ws=None), ("grow", "fork", "compact")),
                    (dict(ws=4100), ("grow", "fork", "compact")),
                    (dict(wb=100), ("grow", "fork", "compact")),
                    (dict(n_pools=-1), ("fork", "copy", "compact"))):
        # (an invalid list alone decides: nothing is enqueued)
        t = B(v4a.PageTableDesc(**TABLE))
        a = dict(ws=4096, wb=1 << 20, first=64, last=64, src=64, dst=64, length=64, n=2, used=64, n_pools=1)
        a.update(kw)
        ps = (v4a.Pool * 1)(v4a.Pool(**POOL))
        call = dict(
            free=lambda: lib.v4a_pages_free(t, a["first"], a["last"], None, None),
            grow=lambda: lib.v4a_pages_grow(t, a["first"], a["last"], a["ws"], a["wb"], None, None),
            fork=lambda: lib.v4a_pages_fork(t, ps, a["n_pools"], a["n"], a["src"], a["dst"], a["length"],
                                            a["ws"], a["wb"], None, None),
            copy=lambda: lib.v4a_pages_copy(t, ps, a["n_pools"], a["n"], a["src"], a["dst"], None, None),
            compact=lambda: lib.v4a_pages_compact(t, ps, a["n_pools"], a["used"], None, a["ws"], a["wb"],
                                                  None, None))
        for name in who:
            assert call[name]() == ARG, (kw, name)
    many = (v4a.Pool * (v4a.MAX_POOLS + 1))(*[v4a.Pool(**POOL)] * (v4a.MAX_POOLS + 1))
    t = B(v4a.PageTableDesc(**TABLE))
    assert lib.v4a_pages_copy(t, many, v4a.MAX_POOLS + 1, 2, 64, 64, None, None) == UNS
    assert lib.v4a_pages_fork(t, many, 1, v4a.MAX_SEQ + 1, 64, 64, 64, 4096, 1 << 20, None, None) == UNS
    assert lib.v4a_pages_copy(t, many, 1, (1 << 20) + 1, 64, 64, None, None) == UNS
    # nothing to do
    empty = B(v4a.PageTableDesc(**dict(TABLE, n_seq=0, block_table=None)))
    assert lib.v4a_pages_free(empty, None, None, None, None) == OK
    assert lib.v4a_pages_grow(empty, None, None, None, 0, None, None) == OK
    assert lib.v4a_pages_fork(t, None, 0, 0, None, None, None, None, 0, None, None) == OK
    assert lib.v4a_pages_copy(t, None, 0, 3, None, None, None, None) == OK


def test_python_table_refuses_what_does_not_fit():
    with pytest.raises(ValueError):
        PageTable([], torch.zeros(2, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))


# ------------------------------------------------------------------------ the definitions
def test_grow_and_free_by_hand():
    bt = np.array([[3, -1, -1], [-1, 0, -1]], np.int32)
    refs = np.array([1, 0, 0, 1, 0], np.int32)
    assert O.grow(bt, refs, [0, 0], [2, 2])
    assert bt.tolist() == [[3, 1, -1], [2, 0, -1]] and refs.tolist() == [1, 1, 1, 1, 0]
    assert not O.grow(bt, refs, [0, 2], [3, 3])             # one page left for two blocks
    assert bt.tolist() == [[3, 1, 4], [2, 0, -1]] and refs.tolist() == [1] * 5
    O.free(bt, refs, [1, 0], [9, 0])
    assert bt.tolist() == [[3, -1, -1], [2, 0, -1]] and refs.tolist() == [1, 0, 1, 1, 0]


def test_fork_by_hand():
    bt = np.array([[2, 0, -1], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1]], np.int32)
    refs = np.array([1, 0, 1, 0], np.int32)
    data = np.arange(4 * 256)
    # 256 + 3 positions: the first block is shared, three rows of the second are copied
    assert O.fork(bt, refs, [(data, 256)], [0, 0, 0], [1, 2, 2], [259, 256, 5])
    assert bt.tolist() == [[2, 0, -1], [2, 1, -1], [-1, -1, -1], [-1, -1, -1]]   # 2 is named twice
    assert refs.tolist() == [1, 1, 2, 0]
    assert data[256:259].tolist() == [0, 1, 2] and data[259] == 259


def test_compact_by_hand():
    bt = np.array([[5, 1], [4, 1]], np.int32)
    refs = np.array([0, 2, 0, 0, 1, 1], np.int32)
    data = np.arange(6)
    used, moved = O.compact(bt, refs, [(data, 1)])
    assert used == 3 and moved.tolist() == [-1, 1, -1, -1, 0, 2]
    assert bt.tolist() == [[2, 1], [0, 1]] and refs.tolist() == [1, 2, 1, 0, 0, 0]
    assert data.tolist() == [4, 1, 5, 3, 4, 5]
