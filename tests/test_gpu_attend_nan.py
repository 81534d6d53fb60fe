"""Sparse and tree attention with logits that are NaN or infinite: a row whose
softmax is NaN is NaN wherever it lies in the split of the work."""
import numpy as np
import pytest
import torch

from _attend import attend_ref, check_rows, f16, make_cache, mask_words, materialized, quantized
from test_gpu_attend import run_sparse, run_tree, tree_inputs

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")

# (D, query heads a KV head, drafts): the warp kernel with 8 and 16 rows, the
# tcgen05 kernel with 32, 64 and 128
FORMS = [(64, 1, 6), (128, 2, 8), (256, 1, 7), (64, 2, 9), (128, 1, 20), (256, 2, 11), (64, 1, 40), (128, 2, 50)]


def dense_rows(N, seed):
    """Masks of about half of the drafts and the token itself."""
    rng = np.random.default_rng(seed)
    return [int.from_bytes(rng.bytes(8), "little") & ((1 << N) - 1) | 1 << i for i in range(N)]


def check_row(cache, lens, b, hq, i, q, k, v, mask, out, skip=()):
    """Row i of head hq against float64 attention without the drafts in skip."""
    h = hq // (q.shape[1] // cache.H)
    K, V = materialized(cache, 0), materialized(cache, 1)
    js = [j for j in range(q.shape[2]) if mask >> j & 1 and j not in skip]
    want, bound = attend_ref(q[b, hq, i].double(), torch.cat([K[b, h, :lens[b]], k[b, h, js].double()]),
                             torch.cat([V[b, h, :lens[b]], v[b, h, js].double()]), cache.D ** -0.5)
    check_rows(out[b, hq, i], want, bound, f"b={b} hq={hq} i={i}")


@pytest.mark.parametrize("n", [10, 3000], ids=["uncut", "cut"])
@pytest.mark.parametrize("D,gq,N", FORMS)
def test_nan_logits_make_their_row_nan(cuda, D, gq, N, n):
    """A NaN in a query or in an attended draft's key."""
    lens = [n]
    cache = make_cache(cuda, 1, 1, D, 2, 2, 32, 32, lens, seed=140)
    q, k, v, _, _ = tree_inputs((1, 1, gq, D, 2, 2, 32, 32, lens, N, None), seed=141)
    rows = dense_rows(N, 142)
    iq, jk = N // 2, N - 2
    rows[iq] &= ~(1 << jk)
    rows[0] &= ~(1 << jk)
    q[0, gq - 1, iq, 3] = NAN
    k[0, 0, jk, D - 2] = NAN
    out = run_tree(cache, q, k, v, mask_words(rows, N)[None])
    good = 0
    for hq in range(gq):
        for i in range(N):
            if rows[i] >> jk & 1 or (hq == gq - 1 and i == iq):
                assert torch.isnan(out[0, hq, i]).all(), f"hq={hq} i={i}"
            else:
                good += 1
                check_row(cache, lens, 0, hq, i, q, k, v, rows[i], out)
    assert good > 0


@pytest.mark.parametrize("n", [10, 3000], ids=["uncut", "cut"])
@pytest.mark.parametrize("D,gq,N", FORMS)
def test_infinite_logits(cuda, D, gq, N, n):
    """An attended draft with an infinite key: logit +inf makes the row NaN
    (inf - inf), -inf weighs nothing."""
    lens = [n]
    cache = make_cache(cuda, 1, 1, D, 4, 4, 32, 32, lens, seed=143)
    q, k, v, _, _ = tree_inputs((1, 1, gq, D, 4, 4, 32, 32, lens, N, None), seed=144)
    rows = dense_rows(N, 145)
    jk = N // 3
    k[0, 0, jk, 7] = INF
    q[0, :, ::2, 7], q[0, :, 1::2, 7] = 1.0, -1.0
    rows[0], rows[1] = rows[0] | 1 << jk, rows[1] | 1 << jk
    out = run_tree(cache, q, k, v, mask_words(rows, N)[None])
    for hq in range(gq):
        for i in range(N):
            attends, up = bool(rows[i] >> jk & 1), float(q[0, hq, i, 7]) > 0
            if attends and up:
                assert torch.isnan(out[0, hq, i]).all(), f"hq={hq} i={i}"
            else:
                check_row(cache, lens, 0, hq, i, q, k, v, rows[i], out, skip=(jk,))


@pytest.mark.parametrize("n", [10, 3000], ids=["uncut", "cut"])
@pytest.mark.parametrize("D,gq,N", FORMS)
def test_logits_that_overflow(cuda, D, gq, N, n):
    """sm_scale 1e38: any product past 3 becomes an infinite logit."""
    lens = [n]
    cache = make_cache(cuda, 1, 1, D, 8, 8, 32, 32, lens, seed=146)
    q, k, v, rows, mask = tree_inputs((1, 1, gq, D, 8, 8, 32, 32, lens, N, None), seed=147)
    s = torch.einsum("hid,td->hit", q[0].double(), materialized(cache, 0)[0, 0, :n])
    assert (s.amax(-1) > 3).any()
    out = run_tree(cache, q, k, v, mask, sm=1e38)
    assert torch.isnan(out[0][s.amax(-1) > 3]).all()


@pytest.mark.parametrize("n", [30, 3000], ids=["uncut", "cut"])
@pytest.mark.parametrize("D,gq", [(128, 4), (64, 12), (256, 16)])
def test_sparse_nan_query(cuda, D, gq, n):
    cache = make_cache(cuda, 1, 2, D, 2, 2, 32, 32, [n], seed=148)
    q = f16(torch.Generator().manual_seed(149), 1, 2 * gq, D)
    q[0, gq + 1, 5] = NAN
    nb = max(quantized(n, 32, 32) // 32, 1)
    blocks = torch.arange(nb, dtype=torch.int32).expand(1, 2, nb).contiguous()
    out = run_sparse(cache, q, blocks)
    bad = torch.isnan(out[0]).all(-1)
    assert bad.tolist() == [i == gq + 1 for i in range(2 * gq)]
    assert torch.isfinite(out[0][~bad]).all()
