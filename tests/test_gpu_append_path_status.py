"""The status of a kivi_append_path call that refuses several sequences for
different reasons."""
import pytest
import torch

from _attend import make_cache
from kivi_bit_kv_gb300 import abi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [[0], [599], [0, 1, 300], list(range(0, 600, 7))])
@pytest.mark.parametrize("before", [0, 99, abi.KIVI_EINVAL, abi.KIVI_ECAPACITY])
def test_a_bad_entry_outranks_a_full_sequence(cuda, bad, before):
    """The same status whatever order the sequences are looked at in."""
    B, H, D, P = 600, 2, 64, 3
    cache = make_cache(cuda, B, H, D, 2, 2, 32, 32, [60] * B, seed=170)
    cache.lens.fill_(cache.Tmax - 1)
    lens = cache.lens.clone()
    k = torch.zeros((B, H, 4, D), dtype=torch.float16, device=cuda)
    path = torch.zeros((B, P), dtype=torch.int32, device=cuda)
    counts = torch.full((B,), 2, dtype=torch.int32, device=cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)

    def call():
        status.fill_(before)
        for _ in range(3):
            abi.kivi_append_path(cache, k, k, path, counts, status)
        torch.cuda.synchronize()
        assert torch.equal(cache.lens, lens)
        return int(status.item())

    assert call() == abi.KIVI_ECAPACITY
    for i, b in enumerate(bad):
        if i % 2:
            counts[b] = -1
        else:
            path[b, 1] = 4
    assert call() == abi.KIVI_EINVAL
    counts.fill_(0)
    assert call() == before
