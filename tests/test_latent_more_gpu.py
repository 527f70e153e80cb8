"""GPU: latent attention and rotary positions at the ends of their ranges: lengths
that differ widely. Tolerances as in latent_helpers."""
import numpy as np
import pytest
import torch

from latent_helpers import BF, F32, batch, check, f64, ints, layer, rand
from test_latent_gpu import _attn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


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
