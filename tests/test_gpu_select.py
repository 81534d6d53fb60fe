"""kivi_block_select against the documented fp32 arithmetic: scores bit for
bit, the choice exactly (ties to the lower index), unwritten entries left
alone; and the chain select -> sparse attention -> append as a decode step."""
import numpy as np
import pytest
import torch

from _attend import choose_ref, f16, make_cache, quantized, scores_ref
from _parity import new_cache
from kivi_bit_kv_gb300 import abi

pytestmark = pytest.mark.gpu


def run_select(cache, q, keep, stream=None):
    dev = cache.device
    blocks = torch.full((cache.B, cache.H, keep), -7, dtype=torch.int32, device=dev)
    scores = torch.full((cache.B, cache.H, cache.Tmax // cache.G), float("nan"), device=dev)
    abi.kivi_block_select(cache, q.to(dev), blocks, scores, stream=stream)
    torch.cuda.synchronize(dev)
    return blocks.cpu(), scores.cpu().numpy()


def check_select(cache, lens, q, keep, blocks, scores):
    want = scores_ref(cache, q).max(axis=2)
    for b, n in enumerate(lens):
        nb = quantized(n, cache.G, cache.R) // cache.G
        for h in range(cache.H):
            got = scores[b, h]
            assert np.array_equal(got[:nb], want[b, h, :nb]), f"b={b} h={h}"
            assert np.isnan(got[nb:]).all(), "entries past the quantized groups were written"
            assert blocks[b, h].tolist() == choose_ref(want[b, h], nb, keep), f"b={b} h={h}"


# (B, H, Hq, D, bits_k, bits_v, G, R, lengths, n_keep)
CASES = {
    "mha_int2": (2, 3, 3, 128, 2, 2, 32, 128, [700, 4100], 9),
    "gqa4": (1, 2, 8, 128, 2, 2, 32, 128, [9001], 64),
    "gqa7_d64": (2, 1, 7, 64, 4, 8, 32, 32, [1333, 64], 5),
    "gqa16_d256": (1, 2, 32, 256, 8, 4, 64, 0, [3000], 6),
    "g128": (2, 2, 4, 128, 8, 8, 128, 128, [1999, 640], 3),
    "short": (5, 2, 2, 128, 4, 2, 32, 32, [0, 1, 63, 64, 96], 3),
    "keep_one": (1, 1, 1, 64, 2, 2, 64, 0, [8192], 1),
    "keep_most": (1, 2, 2, 64, 2, 2, 32, 0, [2080], 64),
    "keep_all": (1, 2, 2, 64, 2, 2, 32, 0, [2080], 65),
    "long": (1, 1, 2, 64, 2, 2, 32, 0, [70000], 100),
    "many_rows": (40, 5, 5, 64, 2, 2, 32, 32, [100 + 31 * i for i in range(40)], 4),
}


@pytest.mark.parametrize("name", CASES)
def test_select_matches_documented_arithmetic(cuda, name):
    B, H, Hq, D, bk, bv, G, R, lens, keep = CASES[name]
    cache = make_cache(cuda, B, H, D, bk, bv, G, R, lens, seed=31)
    q = f16(torch.Generator().manual_seed(32), B, Hq, D)
    check_select(cache, lens, q, keep, *run_select(cache, q, keep))


def test_scores_bound_every_key(cuda):
    """score >= q . K_hat for every token of a group, to the rounding of the fp32 sums."""
    from _attend import materialized
    lens = [900]
    cache = make_cache(cuda, 1, 2, 128, 2, 2, 32, 32, lens, seed=33)
    q = f16(torch.Generator().manual_seed(34), 1, 6, 128)
    _, scores = run_select(cache, q, 4)
    K = materialized(cache, 0)
    nb = quantized(900, 32, 32) // 32
    for h in range(2):
        s = (q[0, 3 * h:3 * h + 3].double() @ K[0, h, :nb * 32].T).view(3, nb, 32).amax((0, 2))
        # x_hat is rounded to fp16 (2^-11 relative per key) after the bound's fp32 values
        slack = (q[0, 3 * h:3 * h + 3].double().abs() @ K[0, h, :nb * 32].abs().T).amax() * 2.0 ** -10
        assert (torch.from_numpy(scores[0, h, :nb]).double() >= s - slack).all()


@pytest.mark.parametrize("keep", [1, 5, 13, 31])
def test_ties_go_to_the_lowest_index(cuda, keep):
    """Groups with the same statistics score the same bits; negative and zero
    scores, -0 against +0 included."""
    cache = new_cache(1, 3, 64, 2, 2, 32, 0, 32 * 32, cuda)
    cache.lens.fill_(32 * 32)
    g = torch.Generator().manual_seed(35)
    kinds = torch.randint(0, 4, (32,), generator=g)
    for i, kd in enumerate(kinds.tolist()):
        cache.kzero[0, 0, i] = [-3.0, -1.0, 0.0, 2.0][kd]      # negative scores among them
        cache.kscale[0, 0, i] = [1.0, 0.5, 0.0, 0.0][kd]
    cache.kzero[0, 1] = -1.0                                     # all equal
    cache.kzero[0, 2] = 0.0                                      # all zero: +0 and -0 products
    q = f16(g, 1, 3, 64)
    blocks, scores = run_select(cache, q, keep)
    check_select(cache, [32 * 32], q, keep, blocks, scores)
    assert blocks[0, 1].tolist() == list(range(keep)) and blocks[0, 2].tolist() == list(range(keep))


def test_nan_scores_rank_last(cuda):
    lens = [640]
    cache = make_cache(cuda, 1, 1, 64, 2, 2, 32, 0, lens, seed=36)
    cache.kscale[0, 0, 3] = float("nan")
    q = f16(torch.Generator().manual_seed(37), 1, 1, 64)
    blocks, scores = run_select(cache, q, 19)
    assert blocks[0, 0].tolist() == [i for i in range(20) if i != 3]


def test_stream_graph_and_repeats(cuda):
    lens = [5000, 801]
    cache = make_cache(cuda, 2, 2, 128, 2, 2, 32, 32, lens, seed=38)
    q = f16(torch.Generator().manual_seed(39), 2, 4, 128)
    want = run_select(cache, q, 17)
    got = run_select(cache, q, 17, stream=torch.cuda.Stream())
    assert torch.equal(got[0], want[0]) and np.array_equal(got[1], want[1], equal_nan=True)
    qd = q.to(cuda)
    blocks = torch.zeros((2, 2, 17), dtype=torch.int32, device=cuda)
    scores = torch.zeros((2, 2, cache.Tmax // 32), device=cuda)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.kivi_block_select(cache, qd, blocks, scores)
    for qq in (q, q.flip(0).contiguous()):
        qd.copy_(qq)
        blocks.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(blocks.cpu(), run_select(cache, qq, 17)[0])


def test_decode_loop_with_drafts(cuda):
    """The operators as a decode loop uses them, with a flush on the way:
    sparse decode steps with a fresh selection, a tree verified over the
    cache, its path appended; each output against float64 over the
    materialized cache of that moment."""
    from test_gpu_attend import check_sparse, check_tree, run_sparse, run_tree, tree_inputs
    lens = [420, 130]
    cache = make_cache(cuda, 2, 2, 64, 2, 4, 32, 32, lens, seed=40, room=96)
    g = torch.Generator().manual_seed(41)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    for step in range(4):
        q = f16(g, 2, 4, 64)
        blocks, scores = run_select(cache, q, 3)
        check_select(cache, lens, q, 3, blocks, scores)
        check_sparse(cache, lens, q, blocks, run_sparse(cache, q, blocks))
        case = (2, 2, 4, 64, 2, 4, 32, 32, lens, 14, None)
        tq, tk, tv, rows, mask = tree_inputs(case, seed=50 + step)
        check_tree(cache, lens, tq, tk, tv, rows, None, run_tree(cache, tq, tk, tv, mask))
        counts = [3 + 5 * (step % 3), 14 - step]
        path = torch.stack([torch.randperm(14, generator=g).int() for _ in range(2)]).to(cuda)
        abi.kivi_append_path(cache, tk.to(cuda), tv.to(cuda), path,
                             torch.tensor(counts, dtype=torch.int32, device=cuda), status)
        torch.cuda.synchronize()
        lens = [n + c for n, c in zip(lens, counts)]
        assert cache.lens.tolist() == lens and int(status.item()) == 0
