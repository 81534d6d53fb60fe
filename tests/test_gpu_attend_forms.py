"""Block selection, sparse and tree attention in every form the library picks
by size: a warp's or a CTA's choice, one or several chunks of a row, the warp
kernel with 8 and 16 rows, the tcgen05 kernel with 32, 64 and 128, every code
width and mixed ones, rows cut into many pieces, logits far outside fp16, more
rows than a grid's second dimension holds, captured graphs."""
import numpy as np
import pytest
import torch

from _attend import attend_ref, check_rows, f16, make_cache, mask_words, materialized, pairwise, quantized
from _parity import new_cache
from kivi_bit_kv_gb300 import abi
from test_gpu_attend import check_sparse, check_tree, run_sparse, run_tree, tree_inputs
from test_gpu_select import check_select, run_select

NAN = float("nan")
pytestmark = pytest.mark.gpu

WIDTHS = [(2, 2), (4, 4), (8, 8), (8, 2), (2, 4)]
FORMS = [(D, M, WIDTHS[(i + j) % 5]) for j, D in enumerate((64, 128))
         for i, M in enumerate((1, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129))]
FORMS += [(256, M, WIDTHS[i % 5]) for i, M in enumerate((1, 8, 9, 32, 33))]
FORMS += [(128, M, w) for M in (8, 16, 32, 64, 128) for w in WIDTHS]


@pytest.mark.parametrize("D,M,widths", sorted(set(FORMS)))
def test_tree_rows_of_every_form(cuda, D, M, widths):
    """M query rows as M drafts of one head, or half as many of two heads."""
    gq = 2 if M % 2 == 0 else 1
    lens = [0, 70, 345]
    case = (3, 1, gq, D, *widths, 32, 32, lens, M // gq, None)
    cache = make_cache(cuda, 3, 1, D, *widths, 32, 32, lens, seed=50 + M)
    q, k, v, rows, mask = tree_inputs(case, seed=51 + M)
    nd = [M // gq, max(M // gq - 3, 0), (M // gq + 1) // 2]
    out = run_tree(cache, q, k, v, mask, nd)
    check_tree(cache, lens, q, k, v, rows, nd, out)


@pytest.mark.parametrize("D,G,N", [(64, 64, 16), (128, 32, 12), (128, 128, 24), (128, 32, 60), (64, 32, 100),
                                   (256, 64, 7), (256, 128, 12)])
def test_tree_row_in_many_pieces(cuda, D, G, N):
    """One long sequence: its row tile is cut into as many pieces as there are CTAs or warps."""
    lens = [20011]
    case = (1, 1, 1, D, 2, 4, G, G, lens, N, None)
    cache = make_cache(cuda, 1, 1, D, 2, 4, G, G, lens, seed=60)
    q, k, v, rows, mask = tree_inputs(case, seed=61)
    check_tree(cache, lens, q, k, v, rows, None, run_tree(cache, q, k, v, mask))


@pytest.mark.parametrize("N", [3, 14, 20])
def test_logits_far_outside_fp16(cuda, N):
    """Logits of some 10^7: the softmax is the token with the largest one where
    the runner-up is further behind than fp32 sums can tell."""
    n, D = 500, 128
    cache = make_cache(cuda, 1, 1, D, 2, 2, 32, 32, [n], seed=62)
    case = (1, 1, 1, D, 2, 2, 32, 32, [n], N, None)
    q, k, v, rows, mask = tree_inputs(case, seed=63)
    q = (q.float() * 20000).clamp(-60000, 60000).half()
    out = run_tree(cache, q, k, v, mask, sm=8.0)
    assert torch.isfinite(out).all()
    K, V = materialized(cache, 0)[0, 0, :n], materialized(cache, 1)[0, 0, :n]
    checked = 0
    for i in range(N):
        js = [j for j in range(N) if rows[0][i] >> j & 1]
        ks, vs = torch.cat([K, k[0, 0, js].double()]), torch.cat([V, v[0, 0, js].double()])
        x = q[0, 0, i].double()
        s = ks @ x * 8.0
        # an fp32 sum of D terms and two roundings of the scaled logit, for both tokens
        slack = 2 * 8.0 * (D + 2) * 2.0 ** -23 * float((ks.abs() @ x.abs()).max())
        top = torch.topk(s, 2)
        if float(top.values[0] - top.values[1]) > slack + 40:  # the rest weighs less than n e^-40
            checked += 1
            # one weight of 1 as two fp16 terms, and its quotient by itself
            want = vs[top.indices[0]]
            check_rows(out[0, 0, i], want, 2.0 ** -20 * want.abs() + 1e-12, f"row {i}")
    assert checked >= N // 2


@pytest.mark.parametrize("D,gq", [(256, 16), (256, 9), (256, 8), (128, 16), (64, 9)])
def test_sparse_skips_bad_entries_in_every_form(cuda, D, gq):
    """Whole tiles and units of skipped entries, the first ones too."""
    lens = [1500, 700, 90]
    cache = make_cache(cuda, 3, 1, D, 4, 2, 32, 32, lens, seed=90)
    q = f16(torch.Generator().manual_seed(91), 3, gq, D)
    blocks = torch.full((3, 1, 20), -1, dtype=torch.int32)
    blocks[0, 0, 9:] = torch.tensor([45, 3, 46, -2 ** 31, 3, 0, 2 ** 31 - 1, 1, 2, 44, 7])
    blocks[1, 0, ::3] = torch.tensor([20, 21, 0, 5, 5, 5, 19])
    check_sparse(cache, lens, q, blocks, run_sparse(cache, q, blocks))


def test_long_sparse_batch_keeps_its_precision(cuda):
    """Rows whose whole list one warp walks: the error does not grow with the
    length (an accumulation that truncates would lose 2^-23 of the output per
    token run, always in the same direction)."""
    B, H, n = 64, 40, 2100
    cache = make_cache(cuda, B, H, 64, 4, 4, 32, 32, [n] * B, seed=64, outliers=False)
    cache.vzero.abs_()  # one sign: nothing cancels
    cache.kzero.mul_(0.1)
    cache.kscale.mul_(0.1)
    q = f16(torch.Generator().manual_seed(65), B, H, 64)
    nb = quantized(n, 32, 32) // 32
    blocks = torch.arange(nb, dtype=torch.int32).expand(B, H, nb).contiguous()
    out = run_sparse(cache, q, blocks)
    K, V = materialized(cache, 0)[0, :, :n], materialized(cache, 1)[0, :, :n]
    s = torch.einsum("hnd,hd->hn", K, q[0].double()) * 64 ** -0.5
    want = torch.einsum("hn,hnd->hd", torch.softmax(s, 1), V)
    rel = float((out[0].double() - want).norm() / want.norm())
    # 66 additions a channel rounded to nearest (2^-24 each), 66 truncated units
    # of 8 products (2^-23 each of a 66th of the sum), weights to 2^-21
    assert rel < 66 * 2.0 ** -24 + 8 * 2.0 ** -23 + 2.0 ** -21, rel


@pytest.mark.parametrize("D,gq,N", [(64, 1, 6), (128, 2, 5), (128, 1, 14), (128, 1, 20), (64, 2, 30), (128, 1, 60),
                                    (128, 2, 50), (256, 1, 7), (256, 1, 21)])
def test_values_that_are_not_finite_reach_only_their_rows(cuda, D, gq, N):
    """A drafted token whose key or values are NaN or infinite, attended by some
    rows: the others match the formula without it."""
    lens = [300, 33]
    case = (2, 2, 2 * gq, D, 2, 2, 32, 32, lens, N, None)
    cache = make_cache(cuda, 2, 2, D, 2, 2, 32, 32, lens, seed=80)
    q, k, v, _, _ = tree_inputs(case, seed=81)
    rng = np.random.default_rng(82)
    rows = [[int.from_bytes(rng.bytes(8), "little") & ((1 << N) - 1) for _ in range(N)] for _ in range(2)]
    jv, jk = N // 3, N - 1
    v[:, :, jv, 5], v[:, :, jv, D - 1], v[:, :, jv, 20] = NAN, float("inf"), -float("inf")
    k[:, :, jk, 9] = float("inf")
    out = run_tree(cache, q, k, v, torch.stack([mask_words(x, N) for x in rows]))
    K, V = materialized(cache, 0), materialized(cache, 1)
    seen = 0
    for b in range(2):
        for i in range(N):
            if rows[b][i] >> jk & 1:
                continue  # an infinite (or NaN) logit: the row is 0 of it, or NaN
            js = [j for j in range(N) if rows[b][i] >> j & 1 and j != jv]
            o = out[b, :, i]
            if not rows[b][i] >> jv & 1:
                for hq in range(2 * gq):
                    h = hq // gq
                    want, bound = attend_ref(q[b, hq, i].double(), torch.cat([K[b, h, :lens[b]], k[b, h, js].double()]),
                                             torch.cat([V[b, h, :lens[b]], v[b, h, js].double()]), D ** -0.5)
                    check_rows(o[hq], want, bound, f"b={b} hq={hq} i={i}")
                continue
            seen += 1
            assert torch.isnan(o[:, 5]).all() and (o[:, D - 1] == float("inf")).all()
            assert (o[:, 20] == -float("inf")).all()
            rest = [d for d in range(D) if d not in (5, 20, D - 1)]
            assert torch.isfinite(o[:, rest]).all(), f"b={b} i={i}"
    assert seen > 0


SELECT = {
    "warp_choice": (80, 8, 8, 64, 2, 2, 32, 32, [64 + 23 * i for i in range(80)], 5),
    "warp_choice_most": (90, 7, 14, 128, 4, 4, 32, 0, [900] * 90, 27),
    "several_steps_a_warp": (41, 8, 8, 256, 2, 2, 32, 32, [40 + 47 * i for i in range(41)], 7),
    "several_steps_a_warp_d128": (40, 8, 16, 128, 2, 2, 32, 64, [4000 - 90 * i for i in range(40)], 33),
}


@pytest.mark.parametrize("name", SELECT)
def test_select_forms(cuda, name):
    B, H, Hq, D, bk, bv, G, R, lens, keep = SELECT[name]
    cache = make_cache(cuda, B, H, D, bk, bv, G, R, lens, seed=70)
    q = f16(torch.Generator().manual_seed(71), B, Hq, D)
    check_select(cache, lens, q, keep, *run_select(cache, q, keep))


@pytest.mark.parametrize("keep", [1, 5, 13, 31])
def test_ties_with_a_warp_a_row(cuda, keep):
    H = 700
    cache = new_cache(1, H, 64, 2, 2, 32, 0, 32 * 32, cuda)
    cache.lens.fill_(32 * 32)
    g = torch.Generator().manual_seed(72)
    kinds = torch.randint(0, 4, (32,), generator=g)
    lo = torch.tensor([-2.0, 0.0, -0.0, 1.0])[kinds]
    cache.kzero.copy_(lo[None, None, :, None].expand_as(cache.kzero).to(cuda))
    cache.kscale.zero_()
    q = torch.ones((1, H, 64)).half()
    check_select(cache, [32 * 32], q, keep, *run_select(cache, q, keep))


def test_select_more_rows_than_a_grid_dimension(cuda):
    """70000 KV heads: rows go to the grid's first dimension."""
    H = 70000
    cache = new_cache(1, H, 64, 2, 2, 32, 0, 96, cuda)
    cache.lens.fill_(96)
    g = torch.Generator().manual_seed(73)
    cache.kzero.copy_(torch.randn(cache.kzero.shape, generator=g))
    cache.kscale.copy_(torch.rand(cache.kscale.shape, generator=g))
    q = f16(g, 1, H, 64)
    blocks, scores = run_select(cache, q, 2)
    lo = cache.kzero.cpu().numpy()
    hi = (lo + (cache.kscale.cpu().numpy() * np.float32(3)).astype(np.float32)).astype(np.float32)
    x = q.float().numpy()[:, :, None]
    want = pairwise(np.maximum((x * lo).astype(np.float32), (x * hi).astype(np.float32)))
    assert np.array_equal(scores, want)
    kept = np.sort(np.argsort(-want, axis=-1, kind="stable")[..., :2], axis=-1)
    assert np.array_equal(blocks.numpy(), kept)


def test_more_rows_than_a_grid_dimension(cuda):
    """Sparse and tree attention over 70000 KV heads (checked at some)."""
    H, n = 70000, 65
    cache = make_cache(cuda, 1, H, 64, 2, 2, 32, 0, [n], seed=74, outliers=False)
    g = torch.Generator().manual_seed(75)
    heads = [0, 1, 32767, 65535, 65536, H - 1]
    kv = []
    for which in (0, 1):
        x = torch.zeros((1, H, cache.Tmax, 64), dtype=torch.float16, device=cuda)
        abi.kivi_dequant(cache, which, x)
        kv.append({h: x[0, h].cpu().double() for h in heads})
    K, V = kv
    q = f16(g, 1, H, 64)
    blocks = torch.randint(0, 2, (1, H, 1), generator=g, dtype=torch.int32)
    out = run_sparse(cache, q, blocks)
    assert torch.isfinite(out).all()
    for h in heads:
        e = int(blocks[0, h, 0])
        tok = list(range(32 * e, 32 * e + 32)) + [64]
        want, bound = attend_ref(q[0, h].double(), K[h][tok], V[h][tok], 64 ** -0.5)
        check_rows(out[0, h], want, bound, f"h={h}")
    q, k, v = f16(g, 1, H, 2, 64), f16(g, 1, H, 2, 64), f16(g, 1, H, 2, 64)
    rows = [[1, 3]]
    out = run_tree(cache, q, k, v, mask_words(rows[0], 2)[None])
    assert torch.isfinite(out).all()
    for h in heads:
        for i in range(2):
            want, bound = attend_ref(q[0, h, i].double(), torch.cat([K[h][:n], k[0, h, :i + 1].double()]),
                                     torch.cat([V[h][:n], v[0, h, :i + 1].double()]), 64 ** -0.5)
            check_rows(out[0, h, i], want, bound, f"h={h} i={i}")


def test_several_captured_graphs_share_a_workspace(cuda):
    """Two graphs with one workspace, replayed one after the other on a stream,
    and two with a workspace each, replayed at once, give what eager calls give."""
    lens = [900, 333]
    cache = make_cache(cuda, 2, 2, 128, 2, 2, 32, 32, lens, seed=76)
    case = (2, 2, 4, 128, 2, 2, 32, 32, lens, 20, None)
    q, k, v, rows, mask = tree_inputs(case, seed=77)
    q1, k, v, mask = q[:, :, 0].contiguous().to(cuda), k.to(cuda), v.to(cuda), mask.to(cuda)
    q = q.to(cuda)
    blocks = torch.tensor([[[0, 3, 7]] * 2] * 2, dtype=torch.int32, device=cuda)
    ws = [cache.attend_workspace(4, 20) for _ in range(2)]
    outs = [torch.zeros((2, 4, 20, 128), device=cuda), torch.zeros((2, 4, 128), device=cuda)]

    def tree(s, w):
        abi.kivi_tree_attention(cache, q, k, v, mask, outs[0], w, stream=s)

    def sparse(s, w):
        abi.kivi_sparse_attention(cache, q1, blocks, outs[1], w, stream=s)

    def graph(call, w):
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            call(s, w)
        return g

    tree(None, ws[0])
    sparse(None, ws[0])
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    shared = [graph(tree, ws[0]), graph(sparse, ws[0])]
    own = [graph(tree, ws[0]), graph(sparse, ws[1])]
    for graphs, streams, used in ((shared, None, ws[:1]), (own, [torch.cuda.Stream(), torch.cuda.Stream()], ws)):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            for i, g in enumerate(graphs):
                if streams is None:
                    g.replay()
                else:
                    with torch.cuda.stream(streams[i]):
                        g.replay()
        torch.cuda.synchronize()
        for w in used:
            assert int(w[:1].view(torch.int32).item()) == abi.KIVI_OK
        for o, x in zip(outs, want):
            assert torch.equal(o, x)
