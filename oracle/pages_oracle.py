"""Plain forms of the page table's calls, one block and one page at a time, from their definitions.
bt [n_seq, max_blocks] and refs [n_pages] are changed in place; pools are (data, R) pairs, data
[n_pages * R, ..]."""
from __future__ import annotations

import numpy as np

BLOCK = 256


def free(bt, refs, first, last):
    for b in range(len(bt)):
        for k in range(max(0, first[b]), min(bt.shape[1], last[b])):
            if bt[b, k] >= 0:
                refs[bt[b, k]] -= 1
                bt[b, k] = -1


def take(refs):
    """The lowest free page, or -1."""
    at = np.nonzero(refs <= 0)[0]
    if len(at) == 0:
        return -1
    refs[at[0]] = 1
    return int(at[0])


def grow(bt, refs, first, last):
    """True when every block got a page."""
    all_there = True
    for b in range(len(bt)):
        for k in range(max(0, first[b]), min(bt.shape[1], last[b])):
            if bt[b, k] < 0:
                bt[b, k] = take(refs)
                all_there &= bt[b, k] >= 0
    return all_there


def fork_ok(bt, src, dst, length, i):
    n_seq, s, d = len(bt), src[i], dst[i]
    if not (0 <= s < n_seq and 0 <= d < n_seq and s != d and 0 <= length[i] <= bt.shape[1] * BLOCK):
        return False
    others = [j for j in range(len(src)) if j != i]
    return not any(dst[j] == d or src[j] == d for j in others) and (bt[d] < 0).all()


def fork(bt, refs, pools, src, dst, length, late=0):
    """True when every block that needs a page got one. late: how many tokens behind a block's end
    still write into its rows, the most of the pools'."""
    good = [i for i in range(len(src)) if fork_ok(bt, src, dst, length, i)]
    new = {}
    for i in good:
        n = int(length[i])
        for k in range(-(-n // BLOCK)):
            # the block's last rows are written by the token at (k + 1) * BLOCK + late - 1
            if bt[src[i], k] >= 0 and n < (k + 1) * BLOCK + late:
                new[i, k] = take(refs)
    for i in good:
        n = int(length[i])
        for k in range(-(-n // BLOCK)):
            page = bt[src[i], k]
            if (i, k) not in new:
                bt[dst[i], k] = page
                if page >= 0:
                    refs[page] += 1
            elif new[i, k] >= 0:
                bt[dst[i], k] = new[i, k]
                for data, R in pools:
                    rows = -(-R * min(BLOCK, n - k * BLOCK) // BLOCK)
                    a, b = page * R, new[i, k] * R
                    data[b:b + rows] = data[a:a + rows]
    return all(p >= 0 for p in new.values())


def compact(bt, refs, pools):
    """(used pages, new number of every page)."""
    used = int((refs > 0).sum())
    moved = np.where(refs > 0, np.arange(len(refs)), -1)
    high = [p for p in range(used, len(refs)) if refs[p] > 0]
    low = [p for p in range(used) if refs[p] <= 0]
    for a, b in zip(high, low):
        for data, R in pools:
            data[b * R:(b + 1) * R] = data[a * R:(a + 1) * R]
        bt[bt == a] = b
        refs[b], refs[a] = refs[a], 0
        moved[a] = b
    return used, moved
