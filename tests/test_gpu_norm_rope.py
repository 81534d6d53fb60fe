"""kivi_norm_rope against its formula in 64 bits: types, head counts, pairings,
rotated shares, axes, positions, strides, ragged tokens, single tokens.

Error of an output y of a pair of magnitude h (fp32 path, one rounding to fp16):
half a step of fp16 (2^-11 |y|, 2^-25 for subnormals) and, from fp32,
    norm      sum of squares: 16 chained and 4 paired additions, half of which
              reaches the root: 10 units of 2^-24; mean and eps 1; rsqrtf 2 ulp: 4;
              two products: 2
    angle     the sum of its terms below 2 half turns: 3 units, times pi: 10 (t < 2^24)
    rotation  sine and cosine 2 ulp: 4; two products and a sum: 3
35 units on |a| + |c| <= sqrt(2) h: below 64 units, 2^-18 h.  Beyond t = 2^24 the
angle's second term has a relative error of 2^-49 and roundings of 2^-24: for
t / pi < 2^30 below 2^-18 half turns, 2^-16 h."""
import pytest
import torch

from _step import norm_rope64
from kivi_bit_kv_gb300 import KiviCache, abi

pytestmark = pytest.mark.gpu


def freqs(rot, theta=10000.0):
    return (theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()


def small_cache(dev, B, H, D):
    return KiviCache(B, H, D, 2, 2, 32, 32, 32, device=dev)


def check(got, want, pair, extra=2.0 ** -18):
    err = (got.double().cpu() - want).abs()
    bound = 2.0 ** -11 * want.abs() + 2.0 ** -25 + extra * pair
    assert bool((err <= bound).all()), f"error {float((err - bound).max()):.3g} over its bound"


def magnitudes(x, weight, eps, half, interleaved):
    """|(a, c)| of every channel's pair, [B, heads, N, D]."""
    y = norm_rope64(x, weight, eps, None, None, None, False)
    h = y.abs().clone()
    for j in range(half):
        a, c = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        m = torch.sqrt(y[..., a] ** 2 + y[..., c] ** 2)
        h[..., a] = m
        h[..., c] = m
    return h


# (B, N, H, gq, D, dtype, rot, interleaved, axes, norm, base, ragged)
CASES = {
    "token": (1, 1, 4, 1, 64, "fp16", 64, False, 1, True, True, False),
    "odd_heads": (3, 7, 5, 3, 128, "bf16", 128, False, 1, True, True, True),
    "one_head": (2, 3, 1, 1, 256, "fp32", 256, False, 1, True, False, False),
    "d64_interleaved": (2, 9, 3, 2, 64, "bf16", 64, True, 1, True, True, True),
    "partial_half": (2, 5, 2, 4, 128, "fp16", 32, False, 1, True, True, False),
    "partial_inter": (2, 5, 2, 4, 256, "fp16", 48, True, 1, False, True, False),
    "rot16": (1, 33, 7, 1, 128, "fp32", 16, False, 1, True, False, False),
    "no_rotation": (2, 4, 3, 1, 128, "bf16", 0, False, 1, True, False, False),
    "no_norm": (2, 4, 3, 2, 64, "fp16", 64, False, 1, False, True, False),
    "axes3": (2, 50, 2, 2, 128, "bf16", 128, False, 3, True, True, True),
    "axes8": (1, 19, 2, 1, 256, "fp16", 128, True, 8, True, False, False),
    "many": (4, 700, 3, 2, 128, "bf16", 96, False, 1, True, True, True),
    "long": (1, 5003, 4, 1, 64, "fp16", 64, True, 1, True, False, False),
}
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def inputs(dev, name, seed, fused=True):
    B, N, H, gq, D, dtype, rot, inter, axes, norm, base, ragged = CASES[name]
    g = torch.Generator().manual_seed(seed)
    Hq, dt = H * gq, TYPES[dtype]
    if fused:
        x = (torch.randn((B, N, Hq + 2 * H, D), generator=g) * 1.5).to(dt).to(dev)
        xs = [x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:]]
    else:
        xs = [(torch.randn((B, N, h, D), generator=g) * 1.5).to(dt).to(dev) for h in (Hq, H, H)]
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dev) for _ in range(2)] if norm else [None, None]
    f = freqs(rot).to(dev) if rot else None
    pos = axis = None
    if axes > 1:
        pos = torch.randint(0, 9000, (axes, B, N), generator=g, dtype=torch.int32).to(dev)
        axis = torch.randint(-1, axes + 1, (rot // 2,), generator=g, dtype=torch.int32).to(dev)
    b = torch.randint(0, 1 << 20, (B,), generator=g, dtype=torch.int32).to(dev) if base else None
    n = torch.tensor([N - (i * 3) % (N + 1) for i in range(B)], dtype=torch.int32).to(dev) if ragged else None
    return xs, w, f, pos, axis, b, n


def positions(N, B, pos, base):
    p = torch.arange(N).view(1, 1, N).expand(1, B, N) if pos is None else pos.cpu().long().view(-1, B, N)
    return p + (0 if base is None else base.cpu().long().view(1, B, 1))


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("name", CASES)
def test_against_the_formula(cuda, name, fused):
    B, N, H, gq, D, dtype, rot, inter, axes, norm, base, ragged = CASES[name]
    xs, w, f, pos, axis, b, n = inputs(cuda, name, 5, fused)
    outs = [torch.full((B, h, N, D), 7.0, dtype=torch.float16, device=cuda) for h in (H * gq, H, H)]
    abi.kivi_norm_rope(small_cache(cuda, B, H, D), *xs, *outs, f, pos=pos, base=b, axis=axis, interleaved=inter,
                       q_weight=w[0], k_weight=w[1], eps=1e-5, n_tok=n)
    torch.cuda.synchronize()
    p = positions(N, B, pos, b)
    here = torch.ones(B, 1, N, 1, dtype=torch.bool) if n is None else (torch.arange(N) < n.cpu().view(B, 1)).view(B, 1, N, 1)
    for x, y, wt, turned in zip(xs, outs, (w[0], w[1], None), (True, True, False)):
        want = norm_rope64(x, wt, 1e-5, None if f is None else f.cpu(), p, None if axis is None else axis.cpu(), inter, turned)
        h = magnitudes(x, wt, 1e-5, rot // 2 if turned else 0, inter)
        here_all = here.expand(want.shape)
        check(y.cpu()[here_all], want[here_all], h[here_all], 2.0 ** -18 if turned else 0.0)
        assert bool((y.cpu()[~here_all] == 7.0).all())         # rows past a sequence's tokens


def test_views_with_any_strides(cuda):
    """Heads of q, k and v interleaved in memory, padded tokens, a broadcast batch."""
    B, N, H, D = 2, 6, 3, 128
    g = torch.Generator().manual_seed(9)
    x = torch.randn((N, H, 3, D + 8), generator=g).half().to(cuda)
    xs = [x[None, :, :, i, :D].expand(B, N, H, D) for i in range(3)]
    assert xs[0].stride(0) == 0 and xs[0].stride(2) == 3 * (D + 8)
    f, w = freqs(D).to(cuda), torch.ones(D, device=cuda)
    cache, outs = small_cache(cuda, B, H, D), [torch.zeros((B, H, N, D), dtype=torch.float16, device=cuda) for _ in range(3)]
    abi.kivi_norm_rope(cache, *xs, *outs, f, q_weight=w, k_weight=w)
    again = [torch.zeros_like(o) for o in outs]
    abi.kivi_norm_rope(cache, *(t.contiguous() for t in xs), *again, f, q_weight=w, k_weight=w)
    for a, b in zip(outs, again):
        assert torch.equal(a, b)
    with pytest.raises(abi.KiviError):                          # a token stride of 8 bytes more than a multiple of 16
        bad = torch.zeros((B, N, H * D + 4), dtype=torch.float16, device=cuda)[..., :H * D].unflatten(-1, (H, D))
        abi.kivi_norm_rope(cache, bad, None, None, outs[0], None, None, f)


def test_groups_left_out(cuda):
    B, N, H, D = 2, 11, 2, 64
    xs, w, f, *_ = inputs(cuda, "d64_interleaved", 11)
    B, N, H, gq, D = CASES["d64_interleaved"][:5]
    cache = small_cache(cuda, B, H, D)
    full = [torch.zeros((B, h, N, D), dtype=torch.float16, device=cuda) for h in (H * gq, H, H)]
    abi.kivi_norm_rope(cache, *xs, *full, f, q_weight=w[0], k_weight=w[1])
    for keep in range(1, 7):
        part = [torch.zeros_like(t) if keep >> i & 1 else None for i, t in enumerate(full)]
        abi.kivi_norm_rope(cache, *(x if p is not None else None for x, p in zip(xs, part)), *part, f, q_weight=w[0],
                           k_weight=w[1])
        for a, b in zip(part, full):
            assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("far,extra", [([0, 1, 4096, (1 << 24) - 1], 2.0 ** -18),
                                       ([(1 << 31) - 1, -(1 << 31), (1 << 30) + 12345, -77], 2.0 ** -16)])
def test_far_positions(cuda, far, extra):
    B, N, H, D = 1, len(far), 2, 128
    g = torch.Generator().manual_seed(12)
    x = torch.randn((B, N, H, D), generator=g).half().to(cuda)
    f = freqs(D)
    f[0] = 1.0
    out = torch.zeros((B, H, N, D), dtype=torch.float16, device=cuda)
    pos = torch.tensor([far], dtype=torch.int32, device=cuda)
    abi.kivi_norm_rope(small_cache(cuda, B, H, D), None, x, None, None, out, None, f.to(cuda), pos=pos)
    want = norm_rope64(x, None, 0.0, f, pos.cpu().long().view(1, 1, N), None, False)
    check(out, want, magnitudes(x, None, 0.0, D // 2, False), extra)


def test_rows_of_zeros_infinities_and_nan_keep_to_themselves(cuda):
    """A head that is all zero gives zeros, one with a NaN gives NaN, and the
    heads and tokens beside them keep their results."""
    B, N, H, D = 2, 5, 4, 128
    xs, w, f, *_ = inputs(cuda, "odd_heads", 13)
    x = xs[1][:2, :5, :4].contiguous()
    cache = small_cache(cuda, B, H, D)
    clean, out = (torch.zeros((B, H, N, D), dtype=torch.float16, device=cuda) for _ in range(2))
    abi.kivi_norm_rope(cache, None, x, None, None, clean, None, f, k_weight=w[1])
    y = x.clone()
    y[0, 1, 2] = 0
    y[1, 3, 0, 17] = float("nan")
    y[1, 4, 1, 100] = float("inf")
    abi.kivi_norm_rope(cache, None, y, None, None, out, None, f, k_weight=w[1])
    touched = torch.zeros((B, H, N), dtype=torch.bool, device=cuda)
    touched[0, 2, 1] = touched[1, 0, 3] = touched[1, 1, 4] = True
    assert torch.equal(out[~touched], clean[~touched])
    assert bool((out[0, 2, 1] == 0).all()) and bool(out[1, 0, 3].isnan().all())
    assert bool(out[1, 1, 4, 100].isnan())                      # infinity times a reciprocal root of 0


def test_values_are_rounded_once(cuda):
    """bf16 and fp32 values to fp16: nearest, ties to even, infinity beyond it."""
    v = torch.tensor([0.0, -0.0, 1.0, 65504.0, 65520.0, -70000.0, 2.0 ** -24, 2.0 ** -25, 3 * 2.0 ** -25, 1 + 2.0 ** -11,
                      1 + 3 * 2.0 ** -11, float("inf"), float("nan")]).repeat(5)[:64]
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        x = v.to(dtype).view(1, 1, 1, 64).to(cuda)
        out = torch.zeros((1, 1, 1, 64), dtype=torch.float16, device=cuda)
        abi.kivi_norm_rope(small_cache(cuda, 1, 1, 64), None, None, x, None, None, out, None)
        torch.testing.assert_close(out.flatten(), x.flatten().half(), rtol=0, atol=0, equal_nan=True)


def test_other_stream_and_graph(cuda):
    """On a side stream, and captured: a replay works on the inputs of its time."""
    B, N, H, gq, D, dtype, rot, inter, axes, norm, base, ragged = CASES["many"]
    xs, w, f, pos, axis, b, n = inputs(cuda, "many", 14)
    cache = small_cache(cuda, B, H, D)

    def outs():
        return [torch.zeros((B, h, N, D), dtype=torch.float16, device=cuda) for h in (H * gq, H, H)]

    def call(o, stream=None):
        abi.kivi_norm_rope(cache, *xs, *o, f, base=b, n_tok=n, q_weight=w[0], k_weight=w[1], stream=stream)

    want, got, held = outs(), outs(), outs()
    call(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(got, side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(held)
    graph.replay()
    for x, y, z in zip(want, got, held):
        assert torch.equal(x, y) and torch.equal(x, z)
    b.add_(17)
    n.clamp_(max=650)
    for o in (*want, *held):
        o.zero_()
    graph.replay()
    call(want)
    for x, z in zip(want, held):
        assert torch.equal(x, z)


def test_offsets_past_32_bits(cuda):
    """2.3e9 outputs: the last heads lie past 2^31 elements, 2^32 bytes."""
    N, H, D = 70001, 128, 256
    x = torch.randn((1, 1, H, D), device=cuda).half()
    out = torch.zeros((1, H, N, D), dtype=torch.float16, device=cuda)
    abi.kivi_norm_rope(small_cache(cuda, 1, H, D), None, None, x.expand(1, N, H, D), None, None, out, None)
    assert torch.equal(out, x.transpose(1, 2).expand(1, H, N, D))


def test_refusals_name_the_argument(cuda):
    B, N, H, D = 2, 3, 2, 64
    c = small_cache(cuda, B, H, D)
    x = torch.zeros((B, N, H, D), dtype=torch.float16, device=cuda)
    y = torch.zeros((B, H, N, D), dtype=torch.float16, device=cuda)
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=cuda)  # noqa: E731
    f = freqs(D).to(cuda)
    good = dict(q_in=x, k_in=x, v_in=x, q=y, k=y.clone(), v=y.clone(), inv_freq=f)
    abi.kivi_norm_rope(c, **good)
    for bad, kind, needle in (
            (dict(q=y[:, :1]), ValueError, "q shape"), (dict(k_in=x[:, :2]), ValueError, "k_in shape"),
            (dict(v=None), ValueError, "v_in and v"), (dict(q=y.float()), TypeError, "q must be"),
            (dict(k_in=x.float()), TypeError, "k_in must be"), (dict(q=y.transpose(2, 3).contiguous().transpose(2, 3)), ValueError, "q must be contiguous"),
            (dict(inv_freq=f.double()), TypeError, "inv_freq must be"), (dict(inv_freq=f[:20]), abi.KiviError, "rot=40"),
            (dict(pos=i(B, 2)), ValueError, "pos shape"), (dict(pos=i(9, B, N)), abi.KiviError, "n_axes=9"),
            (dict(pos=i(B, N).long()), TypeError, "pos must be"), (dict(axis=i(5)), ValueError, "axis shape"),
            (dict(base=i(3)), ValueError, "base shape"), (dict(n_tok=i(1)), ValueError, "n_tok shape"),
            (dict(q_weight=f), ValueError, "q_weight shape"), (dict(eps=-1.0), abi.KiviError, "eps"),
            (dict(q_in=torch.zeros((B, N, 3, D), dtype=torch.float16, device=cuda),
                  q=torch.zeros((B, 3, N, D), dtype=torch.float16, device=cuda)), abi.KiviError, "multiple of H"),
            (dict(k=x.view(B, H, N, D)), abi.KiviError, "k overlaps"),
            (dict(q_in=x.cpu()), ValueError, "q_in must be a CUDA tensor")):
        with pytest.raises(kind, match=needle):
            abi.kivi_norm_rope(c, **(good | bad))
