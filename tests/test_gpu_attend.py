"""kivi_sparse_attention and kivi_tree_attention against float64 attention over
the materialized cache, with error bounds derived from the kernel's arithmetic
(tests/_attend.py): head layouts, widths, group sizes, lengths of zero and one,
lists with skipped and repeated entries, masks that leave a row nothing, rows
and sequences that must keep their contents, streams, graphs and repeatability."""
import numpy as np
import pytest
import torch

from _attend import (attend_ref, check_rows, f16, make_cache, mask_words, materialized, quantized, random_tree)
from kivi_bit_kv_gb300 import KiviCache, KiviError, abi

pytestmark = pytest.mark.gpu

NAN = float("nan")


def run_sparse(cache, q, blocks, sm=None, stream=None, ws=None):
    out = torch.full((cache.B, q.shape[1], cache.D), NAN, device=cache.device)
    ws = cache.attend_workspace(q.shape[1]) if ws is None else ws
    abi.kivi_sparse_attention(cache, q.to(cache.device), blocks.to(cache.device), out, ws, sm_scale=sm, stream=stream)
    torch.cuda.synchronize(cache.device)
    assert int(ws[:1].view(torch.int32).item()) == abi.KIVI_OK
    return out.cpu()


def check_sparse(cache, lens, q, blocks, out, sm=None):
    sm = cache.D ** -0.5 if sm is None else sm
    K, V = materialized(cache, 0), materialized(cache, 1)
    G, R, gq = cache.G, cache.R, q.shape[1] // cache.H
    for b, n in enumerate(lens):
        Tq = quantized(n, G, R)
        for h in range(cache.H):
            tok = []
            for e in blocks[b, h, :min(blocks.shape[2], Tq // G)].tolist():
                if 0 <= e < Tq // G:
                    tok += range(e * G, e * G + G)
            tok += range(Tq, n)
            for i in range(gq):
                hq = h * gq + i
                want, bound = attend_ref(q[b, hq].double(), K[b, h, tok], V[b, h, tok], sm)
                check_rows(out[b, hq], want, bound, f"b={b} hq={hq}")


# (B, H, Hq, D, bits_k, bits_v, G, R, lengths, n_keep)
SPARSE = {
    "mha_int2": (2, 2, 2, 128, 2, 2, 32, 128, [700, 1500], 9),
    "gqa4_int2": (1, 2, 8, 128, 2, 2, 32, 128, [3001], 40),
    "gqa7_d64": (2, 1, 7, 64, 4, 8, 32, 32, [333, 64], 5),
    "gqa16_d256": (1, 1, 16, 256, 8, 4, 64, 0, [1000], 6),
    "int8_g128": (2, 2, 4, 128, 8, 8, 128, 128, [1999, 640], 3),
    "d256_g128": (1, 2, 2, 256, 2, 2, 128, 256, [1700], 4),
    "k4v2_short": (4, 2, 2, 128, 4, 2, 32, 32, [0, 1, 63, 64], 3),
    "all_groups": (1, 2, 4, 128, 2, 4, 32, 64, [1111], 64),
    "one_of_many": (1, 1, 1, 64, 2, 2, 64, 0, [8192], 1),
    "no_residual": (1, 1, 2, 64, 4, 4, 32, 0, [256], 8),
    "many_rows": (24, 8, 8, 64, 2, 2, 32, 32, [64 + 7 * i for i in range(24)], 2),
}


@pytest.mark.parametrize("name", SPARSE)
def test_sparse_matches_float64(cuda, name):
    B, H, Hq, D, bk, bv, G, R, lens, keep = SPARSE[name]
    cache = make_cache(cuda, B, H, D, bk, bv, G, R, lens, seed=1)
    g = torch.Generator().manual_seed(2)
    q = f16(g, B, Hq, D)
    rng = np.random.default_rng(3)
    blocks = torch.full((B, H, keep), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        nb = quantized(n, G, R) // G
        for h in range(H):
            m = min(keep, nb)
            blocks[b, h, :m] = torch.from_numpy(np.sort(rng.permutation(nb)[:m]).astype(np.int32))
    out = run_sparse(cache, q, blocks)
    check_sparse(cache, lens, q, blocks, out)
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all()


def test_sparse_skips_bad_entries_and_counts_repeats(cuda):
    lens = [600, 420]
    cache = make_cache(cuda, 2, 2, 128, 2, 2, 32, 64, lens, seed=5)
    g = torch.Generator().manual_seed(6)
    q = f16(g, 2, 4, 128)
    nb = [quantized(n, 32, 64) // 32 for n in lens]
    blocks = torch.tensor([[[3, 3, 0, -1, nb[0], 2, 2 ** 31 - 1, 5], [nb[0] - 1, 1, 0, 7, -5, -2 ** 31, 1, 1]],
                           [[-1] * 8, [8, 7, 6, 5, 4, 3, 2, 1]]], dtype=torch.int32)
    out = run_sparse(cache, q, blocks)
    check_sparse(cache, lens, q, blocks, out)


def test_sparse_list_longer_than_the_cache(cuda):
    """Only the first Tq/G entries of a list are read."""
    lens = [200]
    cache = make_cache(cuda, 1, 1, 64, 4, 4, 32, 32, lens, seed=7)
    g = torch.Generator().manual_seed(8)
    q = f16(g, 1, 1, 64)
    blocks = torch.arange(12, dtype=torch.int32).flip(0).view(1, 1, 12)
    check_sparse(cache, lens, q, blocks, run_sparse(cache, q, blocks))


def test_sparse_all_groups_agrees_with_decode(cuda):
    """With every group listed it is decode attention over x_hat: equal to
    kivi_decode_attention but for the fp16 rounding of x_hat."""
    lens = [1500, 900]
    cache = make_cache(cuda, 2, 2, 128, 4, 4, 32, 128, lens, seed=9)
    g = torch.Generator().manual_seed(10)
    q = f16(g, 2, 8, 128)
    nb = max(quantized(n, 32, 128) // 32 for n in lens)
    blocks = torch.arange(nb, dtype=torch.int32).expand(2, 2, nb).contiguous()
    out = run_sparse(cache, q, blocks)
    dec = torch.empty((2, 8, 128), device=cuda)
    abi.kivi_decode_attention(cache, q.to(cuda), dec, cache.workspace(8))
    torch.cuda.synchronize()
    err = (out - dec.cpu()).abs().amax(-1) / dec.cpu().abs().amax(-1)
    assert float(err.max()) < 2e-3


@pytest.mark.parametrize("sm", [0.0, -0.3, 1.0])
def test_sparse_scale(cuda, sm):
    lens = [500]
    cache = make_cache(cuda, 1, 2, 64, 2, 2, 32, 32, lens, seed=11)
    g = torch.Generator().manual_seed(12)
    q = f16(g, 1, 4, 64)
    blocks = torch.tensor([[[0, 3, 9, 10], [1, 2, 4, 13]]], dtype=torch.int32)
    check_sparse(cache, lens, q, blocks, run_sparse(cache, q, blocks, sm=sm), sm)


# ------------------------------------------------------------------- tree ---

def run_tree(cache, q, k, v, mask, n_draft=None, sm=None, stream=None, ws=None, out=None):
    dev = cache.device
    B, Hq, N, D = q.shape
    out = torch.full((B, Hq, N, D), NAN, device=dev) if out is None else out
    ws = cache.attend_workspace(Hq, N) if ws is None else ws
    nd = None if n_draft is None else torch.tensor(n_draft, dtype=torch.int32, device=dev)
    abi.kivi_tree_attention(cache, q.to(dev), k.to(dev), v.to(dev), mask.to(dev), out, ws, n_draft=nd, sm_scale=sm,
                            stream=stream)
    torch.cuda.synchronize(dev)
    assert int(ws[:1].view(torch.int32).item()) == abi.KIVI_OK
    return out.cpu()


def check_tree(cache, lens, q, k, v, rows, n_draft, out, sm=None, heads=None):
    """rows[b][i]: Python-int mask of token i of sequence b."""
    sm = cache.D ** -0.5 if sm is None else sm
    K, V = materialized(cache, 0), materialized(cache, 1)
    B, Hq, N, D = q.shape
    gq = Hq // cache.H
    for b, n in enumerate(lens):
        nd = N if n_draft is None else min(max(n_draft[b], 0), N)
        for hq in range(Hq) if heads is None else heads:
            h = hq // gq
            assert torch.isnan(out[b, hq, nd:]).all(), "rows past n_draft were written"
            for i in range(nd):
                js = [j for j in range(nd) if rows[b][i] >> j & 1]
                want, bound = attend_ref(q[b, hq, i].double(), torch.cat([K[b, h, :n], k[b, h, js].double()]),
                                         torch.cat([V[b, h, :n], v[b, h, js].double()]), sm)
                check_rows(out[b, hq, i], want, bound, f"b={b} hq={hq} i={i}")


# (B, H, Hq, D, bits_k, bits_v, G, R, lengths, N, n_draft)
TREE = {
    "one_token": (2, 2, 2, 128, 2, 2, 32, 128, [700, 1500], 1, None),
    "chain8": (2, 2, 2, 128, 2, 2, 32, 128, [300, 999], 8, None),
    "gqa4_n32": (1, 2, 8, 128, 2, 2, 32, 128, [1300], 32, None),
    "gqa7_odd": (2, 1, 7, 64, 4, 8, 32, 32, [333, 64], 13, [13, 5]),
    "gqa16_n33": (1, 1, 16, 128, 8, 4, 32, 0, [515], 33, None),
    "d256": (1, 2, 4, 256, 8, 8, 64, 64, [700], 11, None),
    "d256_g128_k2": (1, 1, 1, 256, 2, 2, 128, 128, [1001], 20, None),
    "g128_int8": (2, 2, 2, 128, 8, 8, 128, 128, [1999, 640], 17, [17, 1]),
    "empty_and_short": (5, 2, 2, 128, 4, 2, 32, 32, [0, 1, 63, 64, 65], 6, [6, 6, 0, 3, 6]),
    "words2": (1, 1, 2, 64, 2, 4, 32, 32, [130], 65, None),
    "n256": (1, 1, 1, 128, 4, 4, 32, 32, [200], 256, [250]),
    "long": (1, 1, 1, 64, 2, 2, 64, 0, [30000], 3, None),
    "many_rows": (16, 4, 8, 64, 2, 2, 32, 32, [40 + 9 * i for i in range(16)], 5, None),
}


def tree_inputs(case, seed=21):
    B, H, Hq, D, bk, bv, G, R, lens, N, nd = case
    g = torch.Generator().manual_seed(seed)
    q, k, v = f16(g, B, Hq, N, D), f16(g, B, H, N, D), f16(g, B, H, N, D)
    rng = np.random.default_rng(seed)
    rows = [random_tree(rng, N) for _ in range(B)]
    return q, k, v, rows, torch.stack([mask_words(r, N) for r in rows])


@pytest.mark.parametrize("name", TREE)
def test_tree_matches_float64(cuda, name):
    case = TREE[name]
    B, H, Hq, D, bk, bv, G, R, lens, N, nd = case
    cache = make_cache(cuda, B, H, D, bk, bv, G, R, lens, seed=20)
    q, k, v, rows, mask = tree_inputs(case)
    out = run_tree(cache, q, k, v, mask, nd)
    check_tree(cache, lens, q, k, v, rows, nd, out)


def test_tree_rows_that_attend_nothing(cuda):
    """An empty sequence with a mask row of zeros: out = 0; a row without a
    draft on a full sequence attends the cache alone; bits past n_draft and
    past N are not read."""
    case = (2, 1, 2, 64, 2, 2, 32, 32, [0, 100], 4, [4, 3])
    cache = make_cache(cuda, *case[:2], *case[3:8], case[8], seed=22)
    q, k, v, _, _ = tree_inputs(case)
    rows = [[0, 0b0010, 0, 0b1010], [0, 0b111, 0b1000, 0]]
    mask = torch.stack([mask_words(r, 4) for r in rows]) | (-1 << 4)
    k[1, :, 3] = NAN
    v[1, :, 3] = NAN
    out = run_tree(cache, q, k, v, mask, case[10])
    assert (out[0, :, 0] == 0).all() and (out[0, :, 2] == 0).all()
    check_tree(cache, case[8], q, k, v, rows, case[10], out)


def test_tree_unattended_draft_may_hold_anything(cuda):
    """A draft no row attends (a hole in the tree) is not read: NaN there
    changes nothing."""
    case = (1, 2, 4, 128, 2, 2, 32, 32, [777], 12, None)
    cache = make_cache(cuda, 1, 2, 128, 2, 2, 32, 32, [777], seed=23)
    q, k, v, rows, _ = tree_inputs(case)
    rows = [[m & ~((1 << 5) | (1 << 11)) for m in rows[0]]]
    k[:, :, [5, 11]], v[:, :, [5, 11]] = NAN, float("inf")
    out = run_tree(cache, q, k, v, torch.stack([mask_words(rows[0], 12)]))
    check_tree(cache, [777], q, k, v, rows, None, out)


def test_tree_of_one_is_decode_of_the_next_token(cuda):
    """One draft attending itself equals decode attention after appending it
    (to the rounding of x_hat, which the decode path does not round)."""
    cache = make_cache(cuda, 2, 2, 128, 8, 8, 32, 64, [500, 93], seed=24, room=64)
    g = torch.Generator().manual_seed(25)
    q, k, v = f16(g, 2, 4, 1, 128), f16(g, 2, 2, 1, 128), f16(g, 2, 2, 1, 128)
    out = run_tree(cache, q, k, v, torch.ones((2, 1, 1), dtype=torch.int64))
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    path = torch.zeros((2, 1), dtype=torch.int32, device=cuda)
    abi.kivi_append_path(cache, k.to(cuda), v.to(cuda), path, torch.ones(2, dtype=torch.int32, device=cuda), status)
    dec = torch.empty((2, 4, 128), device=cuda)
    abi.kivi_decode_attention(cache, q.to(cuda), dec, cache.workspace(4))
    torch.cuda.synchronize()
    assert cache.lens.tolist() == [501, 94] and int(status.item()) == 0
    err = (out[:, :, 0] - dec.cpu()).abs().amax(-1) / dec.cpu().abs().amax(-1)
    assert float(err.max()) < 2e-3


def test_streams_graphs_and_repeats(cuda):
    """The same bits on another stream, from a replayed graph after the inputs
    changed in place, from two graphs replayed in turn, and with a workspace
    full of NaN; the cache is unchanged."""
    case = (3, 2, 8, 128, 2, 4, 32, 64, [900, 0, 333], 9, [9, 4, 7])
    B, H, Hq, D = case[:4]
    cache = make_cache(cuda, B, H, D, *case[4:8], case[8], seed=26)
    before = {n: getattr(cache, n).clone() for n in ("kq", "vq", "kres", "lens")}
    q, k, v, rows, mask = tree_inputs(case)
    qs = q[:, :, 0].contiguous()
    blocks = torch.randint(0, 20, (B, H, 6), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    want_t, want_s = run_tree(cache, q, k, v, mask, case[10]), run_sparse(cache, qs, blocks)
    side = torch.cuda.Stream()
    wst, wss = cache.attend_workspace(Hq, 9).fill_(NAN), cache.attend_workspace(Hq).fill_(NAN)
    torch.cuda.synchronize()
    got_t = run_tree(cache, q, k, v, mask, case[10], stream=side, ws=wst)
    got_s = run_sparse(cache, qs, blocks, stream=side, ws=wss)
    assert torch.equal(got_t.nan_to_num(7.0), want_t.nan_to_num(7.0)) and torch.equal(got_s, want_s)

    d = {n: t.to(cuda) for n, t in dict(q=q, k=k, v=v, mask=mask, qs=qs, blocks=blocks,
                                        nd=torch.tensor(case[10], dtype=torch.int32)).items()}
    ot, os_ = torch.full((B, Hq, 9, D), NAN, device=cuda), torch.full((B, Hq, D), NAN, device=cuda)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        abi.kivi_tree_attention(cache, d["q"], d["k"], d["v"], d["mask"], ot, wst, n_draft=d["nd"])
    with torch.cuda.graph(g2):
        abi.kivi_sparse_attention(cache, d["qs"], d["blocks"], os_, wss)
    for _ in range(3):
        ot.fill_(NAN), os_.fill_(NAN)
        g1.replay(), g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(ot.cpu().nan_to_num(7.0), want_t.nan_to_num(7.0)) and torch.equal(os_.cpu(), want_s)
    q2 = q.flip(0).contiguous()
    d["q"].copy_(q2)
    ot.fill_(NAN)
    g1.replay()
    torch.cuda.synchronize()
    got = ot.cpu()
    assert torch.equal(got.nan_to_num(7.0), run_tree(cache, q2, k, v, mask, case[10]).nan_to_num(7.0))
    for n, t in before.items():
        assert torch.equal(getattr(cache, n), t), n


def test_two_calls_at_once(cuda):
    """Two attentions on two streams with a workspace each."""
    case = (2, 4, 8, 128, 2, 2, 32, 128, [4000, 3500], 16, None)
    cache = make_cache(cuda, *case[:2], *case[3:8], case[8], seed=27)
    q, k, v, rows, mask = tree_inputs(case)
    want = run_tree(cache, q, k, v, mask)
    d = [t.to(cuda) for t in (q, k, v, mask)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [cache.attend_workspace(8, 16) for _ in streams]
    outs = [torch.zeros((2, 8, 16, 128), device=cuda) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, w, o in zip(streams, ws, outs):
            abi.kivi_tree_attention(cache, *d, o, w, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.cpu(), want)


def test_offsets_past_32_bits(cuda):
    """The last slices of a cache whose code buffers pass 2^31 words."""
    B, H, D, G, R, Tmax = 3, 8, 256, 32, 32, 1 << 21
    cache = KiviCache(B, H, D, 8, 8, G, R, Tmax, device=cuda)
    assert cache.vq.numel() > 2 ** 31 and cache.kq.numel() > 2 ** 31
    g = torch.Generator().manual_seed(28)
    n = 400
    K, V = f16(g, B, H, n, D).to(cuda), f16(g, B, H, n, D).to(cuda)
    lens = torch.tensor([0, 5, n], dtype=torch.int32, device=cuda)
    abi.kivi_quant_keys(cache, K, lens)
    abi.kivi_quant_values(cache, V, lens)
    small = KiviCache(B, H, D, 8, 8, G, R, 512, device=cuda)
    abi.kivi_quant_keys(small, K, lens)
    abi.kivi_quant_values(small, V, lens)
    q, k, v = f16(g, B, H, 3, D), f16(g, B, H, 3, D), f16(g, B, H, 3, D)
    mask = torch.stack([mask_words([1, 3, 5], 3)] * B)
    assert torch.equal(run_tree(cache, q, k, v, mask), run_tree(small, q, k, v, mask))
    blocks = torch.tensor([0, 4, 9, 10], dtype=torch.int32).expand(B, H, 4).contiguous()
    q1 = q[:, :, 0].contiguous()
    assert torch.equal(run_sparse(cache, q1, blocks), run_sparse(small, q1, blocks))
    sc, bl = [torch.zeros((B, H, c.Tmax // G), device=cuda) for c in (cache, small)], []
    for c, s in zip((cache, small), sc):
        bl.append(torch.zeros((B, H, 4), dtype=torch.int32, device=cuda))
        abi.kivi_block_select(c, q1.to(cuda), bl[-1], s)
    torch.cuda.synchronize()
    assert torch.equal(bl[0], bl[1]) and torch.equal(sc[0][..., :16], sc[1])


def test_refusals_need_no_launch(cuda):
    cache = make_cache(cuda, 1, 2, 64, 2, 2, 32, 32, [100], seed=29)
    q = torch.zeros((1, 2, 64), dtype=torch.float16, device=cuda)
    out = torch.zeros((1, 2, 64), device=cuda)
    blocks = torch.zeros((1, 2, 3), dtype=torch.int32, device=cuda)
    ws = cache.attend_workspace(2)
    with pytest.raises(KiviError) as e:
        abi.kivi_sparse_attention(cache, q, blocks, out, ws[:3])
    assert e.value.status == abi.KIVI_EWORKSPACE
    with pytest.raises(ValueError):
        abi.kivi_sparse_attention(cache, q, blocks[:, :, ::2], out, ws)
    with pytest.raises(ValueError):
        abi.kivi_sparse_attention(cache, q.cpu(), blocks, out, ws)
    with pytest.raises(TypeError):
        abi.kivi_sparse_attention(cache, q, blocks.long(), out, ws)
    with pytest.raises(ValueError):
        abi.kivi_sparse_attention(cache, q, blocks, out[:, :1], ws)
