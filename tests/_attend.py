"""Inputs and 64-bit references for the tests of block selection, sparse and
tree attention and path appends."""
from __future__ import annotations

import numpy as np
import torch

from _parity import gpu_encode, new_cache, roundup
from kivi_bit_kv_gb300 import abi


def make_cache(dev, B, H, D, bk, bv, G, R, lens, seed=0, room=0, outliers=True):
    """An encoded cache of sequences of `lens` tokens with room for more."""
    g = torch.Generator().manual_seed(seed)
    T = max(max(lens), 1)
    K = torch.randn((B, H, T, D), generator=g)
    if outliers:
        K[..., 3] *= 8.0
        K[..., D // 2 + 1] *= 5.0
    V = torch.randn((B, H, T, D), generator=g)
    cache = new_cache(B, H, D, bk, bv, G, R, roundup(T + room + G, G), dev)
    gpu_encode(cache, K.half(), V.half(), list(lens))
    return cache


def f16(g, *shape):
    return torch.randn(shape, generator=g).half()


def materialized(cache, which):
    """Keys or values of the whole cache as kivi_dequant gives them, float64
    on the CPU ([B, H, Tmax, D]; zero past a sequence's end)."""
    out = torch.zeros((cache.B, cache.H, cache.Tmax, cache.D), dtype=torch.float16, device=cache.device)
    abi.kivi_dequant(cache, which, out)
    torch.cuda.synchronize(cache.device)
    return out.cpu().double()


def quantized(n, G, R):
    return max(0, (n - R) // G * G)


def attend_ref(q, K, V, sm):
    """Softmax attention of one query row in float64 and the largest error the
    kernel may make on each output.

    q [D], K, V [n, D], all float64.  The kernel forms s = q . K in fp32 from
    exact fp16 products: at most D 2^-23 sum_d |q_d k_d| off (an fp32 sum of D
    terms, each addition rounded or truncated to 24 bits), and scales it into
    the exponent's argument, two more roundings of a number of size |s| + 16.
    So each weight is off by a factor of at most 1 + e, e = 2 ds + 2^-21 (the
    exponential and the two-term split of the weight are 2^-22 each), which
    acts on the sum of weights and on the weighted sum.  The weighted sum adds
    256 products per 128 tokens and one term per 128 tokens, the sum of the
    weights n/128 + 64 terms, each addition at most 2^-23 of the partial sum
    of magnitudes.  (Up to 16 rows: 64 products and one rounded addition, 2^-24,
    per 32 tokens; a sum of weights adds four per 32 tokens of one warp's range,
    32 of which are 128 additions of 2^-24.)"""
    n = K.shape[0]
    if n == 0:
        z = torch.zeros_like(q)
        return z, z
    s = K @ q * sm
    ds = abs(sm) * q.shape[0] * 2.0 ** -23 * float((K.abs() @ q.abs()).max()) + (float(s.abs().max()) * 1.5 + 16) * 2.0 ** -22
    p = torch.softmax(s, 0)
    mag = p @ V.abs()
    return p @ V, (4 * ds + 2.0 ** -20 + (512 + n / 64) * 2.0 ** -23) * mag


def check_rows(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = err > bound + 1e-30
    if bool(bad.any()):
        i = int(torch.argmax(err - bound))
        raise AssertionError(f"{what}: channel {i}: got {float(got.flatten()[i])}, want {float(want.flatten()[i])}, "
                             f"error {float(err.flatten()[i]):.3g} over {float(bound.flatten()[i]):.3g}")


def pairwise(x):
    """fp32 sums over the last axis (a power of two long), neighbours first."""
    while x.shape[-1] > 1:
        x = (x[..., 0::2] + x[..., 1::2]).astype(np.float32)
    return x[..., 0]


def scores_ref(cache, q):
    """Scores of every group in the documented fp32 order (numpy)."""
    lo = cache.kzero.cpu().numpy()[:, :, None]
    hi = (lo + (cache.kscale.cpu().numpy()[:, :, None] * np.float32((1 << cache.bits_k) - 1)).astype(np.float32)).astype(np.float32)
    x = q.cpu().float().numpy().reshape(cache.B, cache.H, -1, 1, cache.D)
    with np.errstate(invalid="ignore"):
        t = np.maximum((x * lo).astype(np.float32), (x * hi).astype(np.float32))
        return pairwise(t)  # [B, H, gq, groups]


def choose_ref(scores, nb, keep):
    """Indices of the `keep` largest of scores[:nb], ties to the lower index,
    ascending, padded with -1."""
    order = sorted(range(nb), key=lambda i: (-scores[i], i))[:keep]
    return sorted(order) + [-1] * (keep - min(keep, nb))


def random_tree(rng, N, back=5):
    """Masks (Python ints) of a random token tree: each token attends itself and its ancestors."""
    rows = []
    for i in range(N):
        parent = int(rng.integers(max(-1, i - back), i)) if i else -1
        rows.append((1 << i) | (rows[parent] if parent >= 0 else 0))
    return rows


def mask_words(rows, N):
    """int64 [N, ceil(N/64)] of the Python-int masks."""
    W = (N + 63) // 64
    u = np.array([[(m >> (64 * w)) & (2 ** 64 - 1) for w in range(W)] for m in rows], dtype=np.uint64)
    return torch.from_numpy(u.view(np.int64).copy())
