"""kivi_token_probs at temperatures and logits from both ends of fp32, against its
formula in 64 bits.

A distance from the largest logit, the reciprocal temperature, the power of two and the
sum have the errors that test_gpu_token_probs.py counts: powers of two between them, as
which far temperatures come in, are exact."""
import pytest
import torch

from test_gpu_token_probs import check
from kivi_bit_kv_gb300 import abi

pytestmark = pytest.mark.gpu

LARGE = [float("inf"), 3.4e38, 3e38, 1.5e38, 1e38, 3e37, 2.0 ** 100, 2.0 ** 100 * (1 - 2.0 ** -24), 1e30, 1e20]
TINY = [2.0 ** -149, 1e-42, 1e-39, 2.0 ** -126, 1e-35, 2.0 ** -100, 2.0 ** -100 * (1 - 2.0 ** -24), 1e-25]
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def run_rows(cuda, x, temps):
    """Every row of x [N, V] at every temperature."""
    t = torch.tensor(temps, dtype=torch.float32, device=cuda)
    B, (N, V) = len(temps), x.shape
    x = x.to(cuda)
    out = torch.full((B, N, V), 9.0, device=cuda)
    abi.kivi_token_probs(x.expand(B, N, V), out, temperature=t)
    for b in range(B):
        for i in range(N):
            check(out[b, i], x[i], float(t[b]))
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [5, 1003, 40001, 131072])
def test_masks_of_the_lowest_value(cuda, V, dtype):
    """Masked by the type's lowest value, the largest at either end of the range: up to
    an infinite temperature, where masked tokens weigh as much as the others."""
    g = torch.Generator().manual_seed(V)
    info = torch.finfo(TYPES[dtype])
    x = torch.randn((5, V), generator=g)
    masked = torch.rand((5, V), generator=g) < 0.3
    masked[:, 1], masked[:, 2] = True, False
    x[masked] = info.min
    x[1, 3], x[2, V - 1], x[3] = info.max, info.max / 2, info.min
    x[4] = torch.where(masked[4], float("-inf"), info.max * (torch.rand(V, generator=g) - 0.5))
    out = run_rows(cuda, x.to(TYPES[dtype]), LARGE)
    assert bool((out[0, :4] == out[0, :4, :1]).all())           # equal weights
    assert bool((out[0, 4] == 0).cpu().eq(masked[4]).all())     # but for -infinity


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [7, 1003, 40001])
def test_small_logits_over_small_temperatures(cuda, V, dtype):
    """Logits some temperatures apart, ever so small, beside ordinary and lowest ones;
    and rows whose largest is far from 0."""
    g = torch.Generator().manual_seed(V + 1)
    info = torch.finfo(TYPES[dtype])
    for T in TINY:
        near = (-8 * T * torch.rand((4, V), generator=g).double()).float()
        other = torch.rand((4, V), generator=g) < 0.2
        other[:, 0] = False
        near[other] = torch.randn((4, V), generator=g)[other].abs() * -1
        near[1][other[1]] = info.min
        near[2] += 1.5                                           # one step apart is far at these temperatures
        near[3] -= 2.0 ** 70
        run_rows(cuda, near.to(TYPES[dtype]), [T])
