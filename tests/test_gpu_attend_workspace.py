"""Sparse and tree attention with a workspace that holds other things: what a
call of another shape left there, or small integers.  The header says that its
contents need not be initialized, and its size depends on neither B nor H, so
one workspace serves several caches in turn."""
import pytest
import torch

from _attend import f16, make_cache
from kivi_bit_kv_gb300 import abi
from test_gpu_attend import check_tree, run_sparse, run_tree, tree_inputs

pytestmark = pytest.mark.gpu


def ints(ws):
    return ws.view(torch.int32)


def same(a, b):
    """Equal bits; rows that were not written are NaN in both."""
    return torch.equal(a.view(torch.int32), b.view(torch.int32))


def setup(cuda, B, H, gq, D, lens, N, seed):
    cache = make_cache(cuda, B, H, D, 2, 2, 32, 32, lens, seed=seed)
    return cache, tree_inputs((B, H, H * gq, D, 2, 2, 32, 32, lens, N, None), seed=seed + 1)


@pytest.mark.parametrize("n_draft", [[0, 8, 8, 8], [8, 0, -3, 8], [0, 0, 0, 5], [0, 0, 0, 0]])
def test_a_row_without_drafts_merges_nothing(cuda, n_draft):
    """Records that name rows in range, one for every row of the call, whatever
    part of them the call writes itself."""
    B, H, N = 4, 8, 8
    lens = [1000, 4000, 2500, 3000]
    cache, (q, k, v, rows, mask) = setup(cuda, B, H, 1, 128, lens, N, 100)
    want = run_tree(cache, q, k, v, mask, n_draft, ws=cache.attend_workspace(H, N).zero_())
    check_tree(cache, lens, q, k, v, rows, n_draft, want, heads=[0, H - 1])
    for shift in (0, 1, H, 2 * H + 3):
        for pieces in (1, 3, 9):
            ws = cache.attend_workspace(H, N).zero_()
            for r in range(B * H):
                at = (r + shift) % (B * H)
                ints(ws)[4 + 4 * r:8 + 4 * r] = torch.tensor([r + pieces, r, at // H, at % H], dtype=torch.int32)
            assert same(run_tree(cache, q, k, v, mask, n_draft, ws=ws), want), (shift, pieces)


def test_a_workspace_after_calls_of_other_shapes(cuda):
    """One workspace, in turn: more rows (the other kernel, whose records lie at
    the same place), another number of heads, one range a record, a list."""
    lens = [4096] * 4
    small, (q, k, v, rows, mask) = setup(cuda, 4, 2, 1, 64, lens, 6, 110)
    n_draft = [6, 6, 0, 6]
    clean = run_tree(small, q, k, v, mask, n_draft, ws=small.attend_workspace(2, 6).zero_())
    check_tree(small, lens, q, k, v, rows, n_draft, clean)
    big, (q2, k2, v2, _, m2) = setup(cuda, 2, 4, 1, 64, [6000, 5000], 6, 112)
    many, (q3, k3, v3, _, m3) = setup(cuda, 20, 20, 1, 64, [64 + 9 * i for i in range(20)], 6, 114)
    wide, (q4, k4, v4, _, m4) = setup(cuda, 4, 8, 1, 64, lens, 32, 116)
    blocks = torch.arange(60, dtype=torch.int32).expand(2, 4, 60).contiguous()
    ws = max((c.attend_workspace(c.H, n) for c, n in ((small, 6), (big, 6), (many, 6), (wide, 32))),
             key=lambda t: t.numel())
    before = {"more heads": lambda: run_tree(big, q2, k2, v2, m2, ws=ws),
              "many rows": lambda: run_tree(many, q3, k3, v3, m3, ws=ws),
              "more drafts": lambda: run_tree(wide, q4, k4, v4, m4, ws=ws),
              "a list": lambda: run_sparse(big, q2[:, :, 0].contiguous(), blocks, ws=ws),
              "small integers": lambda: ints(ws).copy_(torch.arange(ws.numel(), dtype=torch.int32) // 3 % 7)}
    for name, call in before.items():
        call()
        assert same(run_tree(small, q, k, v, mask, n_draft, ws=ws), clean), name


def test_graphs_of_several_shapes_share_a_workspace(cuda):
    """Captured calls of two caches replayed in turn on one workspace, with a
    number of drafts that becomes zero between replays."""
    lens = [3000, 700, 4096]
    one, (q, k, v, _, mask) = setup(cuda, 3, 4, 2, 128, lens, 8, 120)
    two, (q2, k2, v2, _, mask2) = setup(cuda, 2, 3, 1, 128, [2000, 5000], 8, 122)
    ws = one.attend_workspace(8, 8)
    assert ws.numel() >= two.attend_workspace(3, 8).numel()
    d = [t.to(cuda) for t in (q, k, v, mask)]
    d2 = [t.to(cuda) for t in (q2, k2, v2, mask2)]
    nd = torch.tensor([8, 8, 8], dtype=torch.int32, device=cuda)
    out, out2 = torch.zeros(q.shape, device=cuda), torch.zeros(q2.shape, device=cuda)
    torch.cuda.synchronize()
    graphs = []
    for call in (lambda: abi.kivi_tree_attention(one, *d, out, ws, n_draft=nd),
                 lambda: abi.kivi_tree_attention(two, *d2, out2, ws)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    want2 = run_tree(two, q2, k2, v2, mask2)
    for n in ([8, 8, 8], [0, 8, 3], [8, 0, 0], [1, 8, 0]):
        nd.copy_(torch.tensor(n, dtype=torch.int32))
        for g in (graphs[1], graphs[0], graphs[1], graphs[0]):
            out.fill_(float("nan")), out2.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            if g is graphs[0]:
                assert same(out.cpu(), run_tree(one, q, k, v, mask, n, ws=one.attend_workspace(8, 8).zero_())), n
            else:
                assert same(out2.cpu(), want2), n


def test_sparse_rows_in_a_used_workspace(cuda):
    """Sparse attention writes a record for every row, sequences without tokens included."""
    cache = make_cache(cuda, 3, 5, 64, 4, 4, 32, 32, [0, 900, 3000], seed=130)
    q = f16(torch.Generator().manual_seed(131), 3, 5, 64)
    blocks = torch.arange(80, dtype=torch.int32).expand(3, 5, 80).contiguous()
    want = run_sparse(cache, q, blocks, ws=cache.attend_workspace(5).zero_())
    assert (want[0] == 0).all()
    ws = cache.attend_workspace(5)
    ints(ws).copy_(torch.arange(ws.numel(), dtype=torch.int32) // 2 % 9)
    assert same(run_sparse(cache, q, blocks, ws=ws), want)
