"""Two copies of the library in one process, as two packages that bring one
each, or a default and a bounds-checked build: neither may take the other's
record of what it has set up for its own kernels."""
import shutil

import pytest
import torch

from _attend import f16, make_cache
from kivi_bit_kv_gb300 import abi
from test_gpu_attend import run_sparse, run_tree, tree_inputs
from test_gpu_select import run_select

pytestmark = pytest.mark.gpu


def test_a_second_copy_of_the_library(cuda, tmp_path, monkeypatch):
    first = abi.load()
    second = abi.load(shutil.copy(abi.LIB_PATH, tmp_path / "libkivi_copy.so"))
    assert second is not first
    lens = [700, 90]
    for D, N in ((128, 4), (64, 14), (256, 5), (128, 20), (64, 40), (128, 100), (256, 20)):
        cache = make_cache(cuda, 2, 2, D, 2, 2, 32, 32, lens, seed=180)
        q, k, v, rows, mask = tree_inputs((2, 2, 2, D, 2, 2, 32, 32, lens, N, None), seed=181)
        q1 = f16(torch.Generator().manual_seed(182), 2, 2, D)
        res = []
        for lib in (first, second):
            monkeypatch.setattr(abi, "_LIB", lib)
            blocks, scores = run_select(cache, q1, 5)
            dec = torch.zeros((2, 2, D), device=cuda)
            abi.kivi_decode_attention(cache, q1.to(cuda), dec, cache.workspace(2))
            res.append((blocks, run_sparse(cache, q1, blocks), run_tree(cache, q, k, v, mask)))
        assert all(torch.equal(a, b) for a, b in zip(*res)), (D, N)
