"""kivi_append_path against the same tokens appended one at a time by
kivi_append_token: every byte of the cache, with ragged counts, several flushes
in one call, repeated nodes, and sequences that must stay as they were."""
import numpy as np
import pytest
import torch

from _attend import f16, make_cache, quantized
from kivi_bit_kv_gb300 import KiviCache, abi

pytestmark = pytest.mark.gpu

BUFS = ("kq", "kscale", "kzero", "vq", "vscale", "vzero", "kres", "vres", "lens")


def clone_row(cache, b):
    one = KiviCache(1, cache.H, cache.D, cache.bits_k, cache.bits_v, cache.G, cache.R, cache.Tmax, device=cache.device)
    for n in BUFS:
        getattr(one, n).copy_(getattr(cache, n)[b:b + 1])
    return one


# (B, H, D, bits_k, bits_v, G, R, lengths, N, counts)
CASES = {
    "ragged_int2": (4, 3, 128, 2, 2, 32, 128, [700, 158, 0, 159], 16, [5, 3, 16, 1]),
    "flush_now": (3, 2, 64, 4, 8, 32, 32, [63, 127, 95], 8, [1, 8, 0]),
    "several_flushes": (2, 2, 128, 8, 4, 32, 0, [31, 500], 100, [100, 97]),
    "r0_g64": (2, 2, 64, 2, 2, 64, 0, [63, 0], 130, [130, 64]),
    "g128": (2, 1, 128, 4, 4, 128, 128, [255, 300], 40, [40, 0]),
    "d256": (1, 2, 256, 8, 8, 64, 64, [127], 70, [70]),
}


@pytest.mark.parametrize("name", CASES)
def test_path_equals_single_appends(cuda, name):
    B, H, D, bk, bv, G, R, lens, N, counts = CASES[name]
    cache = make_cache(cuda, B, H, D, bk, bv, G, R, lens, seed=61, room=max(counts))
    g = torch.Generator().manual_seed(62)
    k, v = f16(g, B, H, N, D).to(cuda), f16(g, B, H, N, D).to(cuda)
    P = max(max(counts), 1)
    path = torch.randint(0, N, (B, P), generator=g, dtype=torch.int32)   # repeats allowed
    status = torch.full((1,), 99, dtype=torch.int32, device=cuda)
    rows = [clone_row(cache, b) for b in range(B)]
    abi.kivi_append_path(cache, k, v, path.to(cuda), torch.tensor(counts, dtype=torch.int32, device=cuda), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 99
    assert cache.lens.tolist() == [n + c for n, c in zip(lens, counts)]
    st1 = torch.zeros(1, dtype=torch.int32, device=cuda)
    for b, one in enumerate(rows):
        for i in range(counts[b]):
            t = int(path[b, i])
            abi.kivi_append_token(one, k[b:b + 1, :, t].contiguous(), v[b:b + 1, :, t].contiguous(), st1)
        torch.cuda.synchronize()
        for n in BUFS:
            got, want = getattr(cache, n)[b:b + 1], getattr(one, n)
            same = torch.equal(got.view(torch.int16) if got.dtype == torch.float16 else got,
                               want.view(torch.int16) if want.dtype == torch.float16 else want)
            assert same, f"{n} of sequence {b}"


def test_refused_sequences_stay_as_they_were(cuda):
    lens = [100, 90, 120, 60, 30, 95]
    cache = make_cache(cuda, 6, 2, 64, 2, 2, 32, 32, lens, seed=63)      # Tmax 160
    before = {n: getattr(cache, n).clone() for n in BUFS}
    g = torch.Generator().manual_seed(64)
    N, P = 70, 65
    k, v = f16(g, 6, 2, N, 64).to(cuda), f16(g, 6, 2, N, 64).to(cuda)
    path = torch.zeros((6, P), dtype=torch.int32)
    path[1, 1] = N                      # bad node in use
    path[2, 0] = -1
    path[3, 5] = 2 ** 31 - 1            # bad node past the count: not used
    counts = torch.tensor([P + 1, 2, 1, 4, -1, 0], dtype=torch.int32, device=cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    abi.kivi_append_path(cache, k, v, path.to(cuda), counts, status)
    torch.cuda.synchronize()
    assert int(status.item()) == abi.KIVI_EINVAL
    assert cache.lens.tolist() == [100, 90, 120, 64, 30, 95]
    for n in BUFS:
        for b in (0, 1, 2, 4, 5):
            assert torch.equal(getattr(cache, n)[b], before[n][b]), (n, b)
    # capacity: exactly full is fine, one more is refused
    status.zero_()
    counts = torch.tensor([60, 61, 41, 65, 1, 65], dtype=torch.int32, device=cuda)
    counts[1] = 65
    counts[3], counts[5] = 0, 65
    path.zero_()
    lens0 = cache.lens.clone()
    abi.kivi_append_path(cache, k, v, path.to(cuda), counts, status)
    torch.cuda.synchronize()
    want = [int(n) + int(c) if int(n) + int(c) <= cache.Tmax else int(n) for n, c in zip(lens0, counts)]
    assert cache.lens.tolist() == want and 160 in want
    assert int(status.item()) == (abi.KIVI_ECAPACITY if any(int(n) + int(c) > 160 for n, c in zip(lens0, counts)) else 0)


def test_append_path_in_a_graph(cuda):
    cache = make_cache(cuda, 2, 2, 64, 2, 2, 32, 32, [50, 61], seed=65, room=64)
    g = torch.Generator().manual_seed(66)
    k, v = f16(g, 2, 2, 8, 64).to(cuda), f16(g, 2, 2, 8, 64).to(cuda)
    path = torch.tensor([[0, 2, 5], [1, 3, 7]], dtype=torch.int32, device=cuda)
    counts = torch.tensor([2, 3], dtype=torch.int32, device=cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    twin = KiviCache(2, 2, 64, 2, 2, 32, 32, cache.Tmax, device=cuda)
    for n in BUFS:
        getattr(twin, n).copy_(getattr(cache, n))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.kivi_append_path(cache, k, v, path, counts, status)
    for _ in range(4):
        graph.replay()
        abi.kivi_append_path(twin, k, v, path, counts, status)
    torch.cuda.synchronize()
    assert cache.lens.tolist() == [58, 73] and int(status.item()) == 0
    for n in BUFS:
        assert torch.equal(getattr(cache, n), getattr(twin, n)), n
