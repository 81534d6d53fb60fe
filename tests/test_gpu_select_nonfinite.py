"""kivi_block_select with NaN and infinities in the query or the statistics:
the documented products and maxima, through which a NaN is carried."""
import numpy as np
import pytest
import torch

from _attend import f16, make_cache, quantized, scores_ref
from test_gpu_select import run_select

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def choose(scores, nb, keep):
    """The `keep` largest of scores[:nb], NaN lowest, ties to the lower index."""
    order = sorted(range(nb), key=lambda i: (bool(np.isnan(scores[i])), 0.0 if np.isnan(scores[i]) else -scores[i], i))
    order = order[:keep]
    return sorted(order) + [-1] * (keep - len(order))


def check(cache, lens, q, keep):
    blocks, scores = run_select(cache, q, keep)
    with np.errstate(invalid="ignore"):
        want = scores_ref(cache, q).max(axis=2)  # numpy's maxima carry NaN
    for b, n in enumerate(lens):
        nb = quantized(n, cache.G, cache.R) // cache.G
        for h in range(cache.H):
            assert np.array_equal(scores[b, h, :nb], want[b, h, :nb], equal_nan=True), f"b={b} h={h}"
            assert blocks[b, h].tolist() == choose(want[b, h], nb, keep), f"b={b} h={h}"
    return want


@pytest.mark.parametrize("D,gq", [(64, 1), (128, 4), (256, 16), (64, 7)])
def test_nan_in_a_query(cuda, D, gq):
    """One head's NaN channel: every score of its KV head is NaN, and the lowest
    indices are kept; the other KV heads do not notice."""
    lens = [900, 40, 1300]
    cache = make_cache(cuda, 3, 2, D, 2, 2, 32, 0, lens, seed=160)
    q = f16(torch.Generator().manual_seed(161), 3, 2 * gq, D)
    q[0, gq // 2, D - 1] = NAN
    q[2, 2 * gq - 1, 0] = NAN
    want = check(cache, lens, q, 5)
    assert np.isnan(want[0, 0, :28]).all() and not np.isnan(want[0, 1, :28]).any() and np.isnan(want[2, 1, :40]).all()


@pytest.mark.parametrize("D,gq,rows", [(64, 1, 2), (128, 4, 2), (128, 1, 700)])
def test_nan_and_infinite_statistics(cuda, D, gq, rows):
    """A NaN scale counts whatever the query's sign; an infinite scale beside a
    negative query leaves the other product, beside zero it is NaN."""
    cache = make_cache(cuda, 1, rows, D, 4, 4, 32, 0, [640], seed=162)
    q = f16(torch.Generator().manual_seed(163), 1, rows * gq, D)
    q[..., 4] = -q[..., 4].abs() - 0.5
    q[..., 5] = q[..., 5].abs() + 0.5
    q[..., 6] = 0.0
    cache.kscale[0, :, 3, 4] = NAN
    cache.kscale[0, :, 7, 5] = NAN
    cache.kzero[0, :, 8, 9] = NAN
    cache.kscale[0, :, 11, 4] = INF
    cache.kscale[0, :, 12, 5] = INF
    cache.kscale[0, :, 13, 6] = INF
    cache.kzero[0, 0, 15, 4] = -INF
    want = check(cache, [640], q, 17)[0]
    for g, kind in ((3, np.isnan), (7, np.isnan), (8, np.isnan), (11, np.isfinite), (12, np.isposinf), (13, np.isnan)):
        assert kind(want[:, g]).all(), g


@pytest.mark.parametrize("value", [INF, -INF])
def test_infinite_query(cuda, value):
    lens = [700]
    cache = make_cache(cuda, 1, 2, 128, 2, 2, 32, 32, lens, seed=164)
    q = f16(torch.Generator().manual_seed(165), 1, 4, 128)
    q[0, 1, 77] = value
    check(cache, lens, q, 6)
