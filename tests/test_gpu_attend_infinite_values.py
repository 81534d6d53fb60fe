"""A drafted token's infinite values reach exactly the rows that attend it,
wherever the token and the rows lie in the split of the work."""
import math

import pytest
import torch

from _attend import make_cache, mask_words
from test_gpu_attend import run_tree, tree_inputs

pytestmark = pytest.mark.gpu

INF = float("inf")


def expected_infinite(v, mask):
    """Per channel the sum of the attended drafts' values that are not finite (0: none)."""
    js = [j for j in range(v.shape[0]) if mask >> j & 1]
    x = v[js].double()
    return torch.where(torch.isfinite(x), 0.0, x).sum(0)


@pytest.mark.parametrize("D,N,n", [(128, 16, 56), (64, 16, 56), (256, 8, 60), (128, 32, 120), (64, 60, 100),
                                   (256, 32, 120), (128, 100, 100)])
def test_infinite_values_on_both_sides_of_a_cut(cuda, D, N, n):
    """A chain of drafts whose tokens lie in two pieces of their row, infinite
    values in each: a row that attends those of the first piece only (so that it
    attends no token of the second) is infinite, not NaN."""
    lens = [n]
    cache = make_cache(cuda, 1, 2, D, 2, 2, 32, 32, lens, seed=150)
    q, k, v, _, _ = tree_inputs((1, 2, 2, D, 2, 2, 32, 32, lens, N, None), seed=151)
    rows = [(2 << i) - 1 for i in range(N)]
    v[0, :, 2, 4], v[0, :, 2, D - 3] = INF, -INF
    v[0, :, N - 3, 4], v[0, :, N - 3, 9] = INF, INF
    v[0, :, N - 2, D - 3] = INF                       # beside -inf: NaN
    out = run_tree(cache, q, k, v, mask_words(rows, N)[None])
    for h in range(2):
        for i in range(N):
            want = expected_infinite(v[0, h], rows[i])
            got = out[0, h, i].double()
            assert torch.equal(torch.isnan(got), torch.isnan(want)), (h, i)
            assert torch.equal(torch.isinf(got), torch.isinf(want)), (h, i)
            assert torch.equal(got[torch.isinf(got)], want[torch.isinf(want)]), (h, i)


@pytest.mark.parametrize("D,N", [(128, 6), (64, 12), (128, 20)])
def test_infinite_values_in_many_rows(cuda, D, N):
    """Ranges that hold the end of one row and the beginning of the next: the
    next one's first piece lies among cached tokens only."""
    B, H = 120, 4
    lens = [200 + 13 * (i % 40) for i in range(B)]
    cache = make_cache(cuda, B, H, D, 2, 2, 32, 32, lens, seed=152)
    q, k, v, _, _ = tree_inputs((B, H, H, D, 2, 2, 32, 32, lens, N, None), seed=153)
    rows = [(2 << i) - 1 for i in range(N)]
    v[:, :, 1, 11] = INF
    v[:, :, N - 1, 12] = -INF
    out = run_tree(cache, q, k, v, torch.stack([mask_words(rows, N)] * B))
    want = torch.zeros((N, D))
    want[1:, 11] = INF
    want[N - 1, 12] = -INF
    inf = torch.isinf(want).expand(out.shape)
    assert torch.equal(torch.isinf(out), inf)
    assert torch.equal(out[inf], want.expand(out.shape)[inf])
    assert torch.isfinite(out[~inf]).all()


@pytest.mark.parametrize("n", [10, 3000], ids=["uncut", "cut"])
@pytest.mark.parametrize("D,N", [(128, 6), (64, 20), (256, 6), (128, 60)])
def test_an_infinite_value_of_no_weight(cuda, D, N, n):
    """The softmax of finite logits is positive, so a draft's infinite value
    makes its rows infinite however far its logit lies behind (here some 2000,
    past what fp32 can hold of its weight)."""
    lens = [n]
    cache = make_cache(cuda, 1, 1, D, 2, 2, 32, 32, lens, seed=154)
    q, k, v, _, _ = tree_inputs((1, 1, 1, D, 2, 2, 32, 32, lens, N, None), seed=155)
    rows = [1 | 1 << i for i in range(N)]
    k[0, 0, 0] = 0.0
    q[0, 0, :, 0] = 200.0
    k[0, 0, 0, 0] = -200.0
    v[0, 0, 0, 5] = INF
    out = run_tree(cache, q, k, v, mask_words(rows, N)[None], sm=0.05)
    assert math.isclose(0.05 * 200 * 200, 2000.0)
    assert (out[0, 0, :, 5] == INF).all()
    rest = [d for d in range(D) if d != 5]
    assert torch.isfinite(out[0, 0, :, rest]).all()
