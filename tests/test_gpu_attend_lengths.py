"""Lengths outside [0, Tmax], which selection and the attentions take as the
nearest one inside: the same bits as with that length, and nothing is read
outside the cache's arrays."""
import pytest
import torch

from _attend import f16, make_cache
from test_gpu_attend import run_sparse, run_tree, tree_inputs
from test_gpu_select import run_select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,gq,N", [(64, 1, 5), (128, 2, 8), (128, 4, 9), (256, 1, 20)])
def test_lengths_outside_the_cache(cuda, D, gq, N):
    B, H = 4, 2
    cache = make_cache(cuda, B, H, D, 2, 4, 32, 32, [512] * B, seed=190)
    assert cache.Tmax == 544
    q, k, v, _, mask = tree_inputs((B, H, H * gq, D, 2, 4, 32, 32, [512] * B, N, None), seed=191)
    q1 = f16(torch.Generator().manual_seed(192), B, H * gq, D)
    blocks = torch.randint(-1, 18, (B, H, 9), generator=torch.Generator().manual_seed(193), dtype=torch.int32)
    res = []
    for lens in ([0, 544, 544, 0], [-1, 545, 2 ** 31 - 1, -2 ** 31]):
        cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        res.append((*run_select(cache, q1, 7), run_sparse(cache, q1, blocks), run_tree(cache, q, k, v, mask)))
    for a, b in zip(*res):
        a, b = torch.as_tensor(a), torch.as_tensor(b)
        assert torch.equal(a.nan_to_num(7.0) if a.is_floating_point() else a,
                           b.nan_to_num(7.0) if b.is_floating_point() else b)
    assert (res[0][2][[0, 3]] == 0).all()
