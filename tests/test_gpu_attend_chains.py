"""Logits as exact as their sums of products allow.

The tensor core truncates the running sum of a chain of 16-channel products: by
up to one unit of 2^-23 of it a step, (n + 1) / 2 units of 2^-23 of the whole
after n steps of equal size, always downwards.  The warp kernel's chains have 4
steps, and are added with rounding.

One token's keys lie in its first 16 channels only, so that its chain is exact
after one step; the others' products are positive and spread over all channels.
All logits are near 100.  What the chains lose shows in the first token's share
of the softmax: delta logit(p) = their common loss."""
import pytest
import torch

from _attend import materialized
from kivi_bit_kv_gb300 import KiviCache, abi

pytestmark = pytest.mark.gpu

STEPS = 4


@pytest.mark.parametrize("R", [0, 32], ids=["codes", "residual"])
@pytest.mark.parametrize("D,gq", [(64, 1), (64, 16), (128, 1), (128, 8), (128, 16), (256, 1), (256, 8)])
def test_chains_of_products_lose_little(cuda, D, gq, R):
    H, T, size = 64, 32, 100.0
    g = torch.Generator().manual_seed(200)
    K = torch.rand((1, H, T, D), generator=g) + 0.5
    K[:, :, 0] = 0.0
    K[:, :, 0, :16] = (torch.rand((1, H, 16), generator=g) + 0.5) * (D / 16)
    V = torch.zeros((1, H, T, D))
    V[:, :, 0, 0] = 1.0                       # out[0] = the first token's share
    cache = KiviCache(1, H, D, 8, 8, 32, R, 64, device=cuda)
    abi.kivi_quant_keys(cache, K.half().to(cuda))
    abi.kivi_quant_values(cache, V.half().to(cuda))
    assert torch.equal(materialized(cache, 1)[0, :, :T], V[0].double())
    q = (torch.rand((1, H * gq, D), generator=g) + 0.5).half()
    S = torch.einsum("hgd,htd->hgt", q[0].double().view(H, gq, D), materialized(cache, 0)[0, :, :T])
    sm = float(torch.tensor(size / float(S.mean()), dtype=torch.float32))
    p = torch.softmax(S * sm, -1)[..., 0]
    out = torch.zeros((1, H * gq, D), device=cuda)
    blocks = torch.zeros((1, H, 1), dtype=torch.int32, device=cuda)
    abi.kivi_sparse_attention(cache, q.to(cuda), blocks, out, cache.attend_workspace(H * gq), sm_scale=sm)
    torch.cuda.synchronize()
    got = out.cpu().double()[0, :, 0].view(H, gq)
    # where both the share and the rest are well above the rounding of the output
    ok = (p > 1e-3) & (p < 0.9)
    assert int(ok.sum()) > 10
    loss = (torch.logit(got) - torch.logit(p))[ok] / size * 2.0 ** 23
    # the chain, and half a unit for the roundings of the scaled logits (a size of
    # 144 in base 2: 2^-17 each, 0.44 units) and the exponentials (0.02)
    assert -0.5 < float(loss.mean()) < (STEPS + 1) / 2 + 0.5, float(loss.mean())
