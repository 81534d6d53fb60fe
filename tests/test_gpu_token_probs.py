"""kivi_token_probs against its formula in 64 bits.

Error of a probability p of a logit x below the largest, x over T in natural
units: the difference, the reciprocal temperature (a quotient of a rounded
constant) and their product are each half a unit of 2^-24 off, 4 |x|/T units of
2^-24 at most on p; the power of two 2 ulp, 4 units; the quotient 2; the sum of
the weights carries the same errors, averaged (below 4 * 14 units: the mean of
|x|/T over the weights is at most ln V), and one unit for each addition of a
chain, at most V / 512 + 32.  Weights below 2^-126 may be flushed."""
import numpy as np
import pytest
import torch

from _step import probs64
from kivi_bit_kv_gb300 import abi

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def check(got, logits, T):
    want = probs64(logits, T)
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    l = logits.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        x = np.where(np.isneginf(l), 0.0, (np.nanmax(l) - l) / T if T > 0 else 0.0)
        bound = want * (4 * np.abs(x) + 62 + len(l) / 512 + 32) * 2.0 ** -24 + 2.0 ** -125
        bad = np.abs(got - want) > bound
    assert not bad.any(), (np.abs(got - want)[bad].max(), want[bad][:4], got[bad][:4])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 4096, 32000, 50001, 131072, 262207, 1 << 20])
def test_against_the_formula(cuda, V, dtype):
    B, N = 2, 3
    g = torch.Generator(device=cuda).manual_seed(V)
    x = (2.5 * torch.randn((B, N, V), generator=g, device=cuda)).to(TYPES[dtype])
    temp = torch.tensor([0.7, 1.3], device=cuda)
    out = torch.full((B, N, V), 9.0, device=cuda)
    abi.kivi_token_probs(x, out, temperature=temp)
    one = torch.full((B, N, V), 9.0, device=cuda)
    abi.kivi_token_probs(x, one)
    for b in range(B):
        for i in range(N):
            check(out[b, i], x[b, i], float(temp[b]))
            check(one[b, i], x[b, i], 1.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,pad,skip", [(1000, 24, 0), (1000, 1, 0), (50001, 3, 1), (32000, 0, 3), (999, 5, 2)])
def test_rows_at_any_element(cuda, V, pad, skip, dtype):
    B, N = 3, 4
    g = torch.Generator(device=cuda).manual_seed(V + pad)
    buf = (2 * torch.randn((B, N + 1, V + pad + skip), generator=g, device=cuda)).to(TYPES[dtype])
    x = buf[:, 1:, skip:skip + V]
    out, want = (torch.zeros((B, N, V), device=cuda) for _ in range(2))
    abi.kivi_token_probs(x, out)
    abi.kivi_token_probs(x.contiguous(), want)
    check(out[1, 2], x[1, 2], 1.0)
    assert bool(((out - want).abs() <= 2.0 ** -18 * want).all())    # other vectors, another order of the sum
    t = x.transpose(0, 1)                                           # sequences and rows the other way round
    out2 = torch.zeros((N, B, V), device=cuda)
    abi.kivi_token_probs(t, out2)
    assert torch.equal(out2.transpose(0, 1), out)


def test_in_place_is_refused(cuda):
    x = torch.zeros((2, 3, 1000), device=cuda)
    with pytest.raises(abi.KiviError, match="overlaps"):
        abi.kivi_token_probs(x, x)
    both = torch.zeros(12000, device=cuda)
    abi.kivi_token_probs(both[:6000].view(2, 3, 1000), both[6000:].view(2, 3, 1000))    # side by side


def test_one_row_for_all_by_broadcast(cuda):
    x = torch.randn(4096, device=cuda).half()
    out = torch.zeros((5, 2, 4096), device=cuda)
    abi.kivi_token_probs(x.expand(5, 2, 4096), out)
    check(out[4, 1], x, 1.0)
    assert bool((out == out[0, 0]).all())


@pytest.mark.parametrize("V", [5, 1000, 40001, 131072])
def test_temperatures(cuda, V):
    """0 and below: the first of the largest; infinite: equal weights of what is not
    -infinity; tiny: those of the largest alone; NaN: NaN."""
    g = torch.Generator(device=cuda).manual_seed(3)
    temps = [0.0, -1.0, float("-inf"), float("inf"), 1e-42, 1e-30, float("nan"), 1e30, 0.02]
    B = len(temps)
    x = (torch.randn((B, 1, V), generator=g, device=cuda) * 2).bfloat16()
    x[:, 0, 1] = float("-inf")
    top = x[:, 0].float().amax(-1)
    x[:, 0, V // 2] = x[:, 0, V - 1] = top.bfloat16()           # ties
    out = torch.zeros((B, 1, V), device=cuda)
    abi.kivi_token_probs(x, out, temperature=torch.tensor(temps, device=cuda))
    for b, T in enumerate(temps):
        check(out[b, 0], x[b, 0], T)


@pytest.mark.parametrize("T", [0.0, 1.0])
@pytest.mark.parametrize("V", [7, 4096, 50001, 200000])
def test_masked_and_nonfinite_rows(cuda, V, T):
    B, N = 1, 7
    g = torch.Generator(device=cuda).manual_seed(4)
    x = torch.randn((B, N, V), generator=g, device=cuda).half()
    x[0, 0] = float("-inf")
    x[0, 1, :-1] = float("-inf")
    x[0, 2, V // 3] = float("nan")
    x[0, 3, V // 2] = float("inf")
    x[0, 4] = torch.finfo(torch.float16).min                     # a mask of the type's lowest value: equal weights
    x[0, 5] = float("-inf")
    x[0, 5, 3] = float("nan")
    out = torch.zeros((B, N, V), device=cuda)
    abi.kivi_token_probs(x, out, temperature=torch.full((1,), T, device=cuda))
    for i in range(N):
        check(out[0, i], x[0, i], T)


@pytest.mark.parametrize("V", [999, 32000])
def test_rows_past_the_end_are_left(cuda, V):
    B, N = 5, 6
    x = torch.randn((B, N, V), device=cuda).half()
    n = torch.tensor([6, 0, 3, -2, 99], dtype=torch.int32, device=cuda)
    out = torch.full((B, N, V), 5.0, device=cuda)
    full = torch.zeros_like(out)
    abi.kivi_token_probs(x, out, n_rows=n)
    abi.kivi_token_probs(x, full)
    for b, m in enumerate([6, 0, 3, 0, 6]):
        assert torch.equal(out[b, :m], full[b, :m]) and bool((out[b, m:] == 5.0).all())


def test_many_rows_offsets_past_32_bits(cuda):
    """2.3e9 outputs: the last rows lie past 2^31 elements, 2^33 bytes."""
    B, N, V = 9, 2000, 131072
    x = torch.randn((1, 1, V), device=cuda).half()
    out = torch.zeros((B, N, V), device=cuda)
    abi.kivi_token_probs(x.expand(B, N, V), out)
    check(out[B - 1, N - 1], x[0, 0], 1.0)
    assert torch.equal(out[B - 1, N - 1], out[0, 0]) and torch.equal(out[B - 1, 77], out[0, 0])


def test_other_stream_and_graph(cuda):
    B, N, V = 4, 3, 50001
    x = torch.randn((B, N, V), device=cuda).bfloat16()
    temp = torch.tensor([1.0, 0.0, 0.5, 2.0], device=cuda)
    want, got, held = (torch.zeros((B, N, V), device=cuda) for _ in range(3))
    abi.kivi_token_probs(x, want, temperature=temp)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    abi.kivi_token_probs(x, got, temperature=temp, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.kivi_token_probs(x, held, temperature=temp)
    graph.replay()
    assert torch.equal(want, got) and torch.equal(want, held)
    x.copy_(torch.randn((B, N, V), device=cuda))
    temp.fill_(0.9)
    graph.replay()
    abi.kivi_token_probs(x, want, temperature=temp)
    assert torch.equal(want, held)
