"""How near kivi_token_probs comes to its formula, part by part, in units of 2^-24
relative to the value.

A quotient is 2^(d log2(e) / T) / S with d = l - max.  Its errors: the difference d rounds
to half a step, |x| units (x = |d| / T); the two-term reciprocal temperature and the
exponent's rounding, made good to first order, leave below 0.1; the power of two 2 ulp: 4;
the product with the sum's inverse and the correction 1 each; the inverse's rounding is
made good.  So |x| + 6.2 beside the sum's own error."""
import numpy as np
import pytest
import torch

from _step import probs64
from kivi_bit_kv_gb300 import abi

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -24
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def far_below(k, V, dtype, T=1.0):
    """k logits of 0 among V - k between -80 T and -40 T: distances are exact, and the
    sum is k, of which what the others add is far below a unit."""
    g = torch.Generator().manual_seed(V)
    x = (-T * (40 + 39.9 * torch.rand(V, generator=g, dtype=torch.float64))).to(dtype)
    top = (torch.arange(k) * 29 + 5) % V
    assert len(set(top.tolist())) == k
    x[top] = 0.0
    return x, top


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1.0, 1.0009765625, 1.25, 0.75])
@pytest.mark.parametrize("V", [1000, 4099, 50003])
def test_exponents_far_from_zero(cuda, V, T, dtype):
    """Values down to 2^-116: an exponent's rounding alone is up to 44 units off at
    |x| = 80, a reciprocal temperature in one term up to 160."""
    x, _ = far_below(1, V, TYPES[dtype], T)
    out = torch.zeros((1, 1, V), device=cuda)
    abi.kivi_token_probs(x.view(1, 1, V).to(cuda), out, temperature=torch.tensor([T], device=cuda))
    want = np.exp(x.double().numpy() / T)
    want /= want.sum()
    err = np.abs(out[0, 0].double().cpu().numpy() - want) / want / UNIT
    assert err.max() <= 6.2, err.max()


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
def test_rounding_of_the_sums_inverse(cuda, dtype):
    """Rows whose sum is 1 and k over the same small logits.  Uncorrected, all values of the
    second share the rounding of 1/k; corrected, the two rows differ by three roundings
    of each value, each at most a unit in any direction: for a thousand distinct
    values and more their mean has a standard deviation below 0.04."""
    V = 4096
    one, _ = far_below(1, V, TYPES[dtype])
    ks = [k for k in range(3, 96, 2) if abs(float(np.float32(1 / k)) * k - 1) / UNIT > 0.6]
    assert len(ks) > 3
    for k in ks[:6]:
        x, top = far_below(k, V, TYPES[dtype])
        small = np.setdiff1d(np.arange(V), top.numpy())
        assert torch.equal(one[small], x[small]) and len(set(x[small].tolist())) > 900
        out = torch.zeros((1, 2, V), device=cuda)
        abi.kivi_token_probs(torch.stack([one, x]).view(1, 2, V).to(cuda), out)
        a, b = out[0].double().cpu().numpy()[:, small]
        mean = float(np.mean(b * k / a - 1)) / UNIT
        assert abs(mean) <= 0.25, (k, mean)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1000, 32000, 50001, 131072, 262207, 1 << 20])
def test_ordinary_rows(cuda, V, dtype):
    """With the sum: a term is off by 4 units (the power of two) and 3 |x| (the difference and two
    roundings of the exponent; where maxima are replaced on the way, the |x| of the steps
    add up to it), 3 ln V in the weighted mean, as the mean of |x| is at most the entropy.
    A thread takes sixteen values at a time, V / 16384 + 1 times: eight roundings of the sum
    and 8 of a rescaled one each; then 11 additions over lanes and warps, and three
    weights of 7 each."""
    g = torch.Generator(device=cuda).manual_seed(V)
    x = (2.5 * torch.randn((1, 2, V), generator=g, device=cuda)).to(TYPES[dtype])
    temp = torch.tensor([0.7])
    out = torch.zeros((1, 2, V), device=cuda)
    abi.kivi_token_probs(x, out, temperature=temp.to(cuda))
    for i in range(2):
        l = x[0, i].double().cpu().numpy()
        want = probs64(x[0, i], float(temp[0]))
        far = np.abs(l - l.max()) / float(temp[0])
        bound = want * (far + 6.2 + 3 * np.log(V) + 4 + 16 * (V // 16384 + 1) + 11 + 21) * UNIT + 2.0 ** -125
        err = np.abs(out[0, i].double().cpu().numpy() - want)
        assert (err <= bound).all(), (err / np.maximum(bound, 1e-300)).max()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [999, 1000, 4099, 50001, 131071, 600001])
def test_where_a_row_lies_does_not_show(cuda, V, dtype):
    """The same logits at any element and behind any neighbours: the same bits."""
    g = torch.Generator(device=cuda).manual_seed(V)
    x = (2 * torch.randn((3, 2, V), generator=g, device=cuda)).to(TYPES[dtype])
    want = torch.zeros((3, 2, V), device=cuda)
    abi.kivi_token_probs(x, want)
    for skip in range(1, 5):
        for pad in (0, 1, 6):
            buf = torch.zeros((3, 2, V + skip + pad), dtype=TYPES[dtype], device=cuda)
            buf[..., skip:skip + V] = x
            out = torch.zeros((3, 2, V), device=cuda)
            abi.kivi_token_probs(buf[..., skip:skip + V], out)
            assert torch.equal(out, want)
