"""Which descriptors and head counts kivi_norm_rope takes."""
import ctypes as C

import pytest
import torch

from test_abi import _desc, _with_ptrs
from test_step_host import heads


def message(kivi_lib, d, args):
    """The refusal of a call that has no inv_freq, which is looked at after the heads."""
    from kivi_bit_kv_gb300 import abi
    assert kivi_lib.kivi_norm_rope(C.byref(d), args, None) == abi.KIVI_EINVAL
    return abi.kivi_last_error()


@pytest.mark.parametrize("Hq", [0, -1, 6, 4 * 17, 2 ** 31 - 1])
def test_the_number_of_query_heads_matters_with_queries_only(kivi_lib, Hq):
    d = _with_ptrs(_desc())
    far = 2 ** 62                                                # strides of a group left out are not read
    assert "inv_freq is NULL" in message(kivi_lib, d, heads(Hq=Hq, q_in=0, q=0, qs=(far, -far, far), inv_freq=0))
    assert "multiple of H" in message(kivi_lib, d, heads(Hq=Hq, inv_freq=0))


def test_a_capacity_that_split_decode_has_no_grid_for(kivi_lib):
    """B H chunks of 2^31 and more: refused where chunks are launched, not here."""
    from kivi_bit_kv_gb300 import abi
    d = _with_ptrs(_desc(B=1 << 20, H=64, Tmax=1 << 24))
    assert kivi_lib.kivi_decode_qk(C.byref(d), 0x10000, 64, 1.0, 0x20000, 1 << 24, None) == abi.KIVI_EINVAL
    assert "decode CTAs" in abi.kivi_last_error()
    far = 1 << 44
    args = heads(Hq=64, N=1, inv_freq=0, q=far, k=2 * far, v=3 * far)
    assert "inv_freq is NULL" in message(kivi_lib, d, args)


@pytest.mark.gpu
def test_keys_alone_without_a_number_of_query_heads(cuda):
    from kivi_bit_kv_gb300 import KiviCache, abi
    B, N, H, D = 2, 5, 3, 64
    cache = KiviCache(B, H, D, 2, 2, 32, 32, 32, device=cuda)
    x = torch.randn((B, N, H, D), device=cuda).half()
    f = (10000.0 ** (-torch.arange(0, D, 2, device=cuda) / D)).float()
    out, want = (torch.zeros((B, H, N, D), dtype=torch.float16, device=cuda) for _ in range(2))
    s = x.stride()[:3]
    args = abi._HEADS.pack(0, N, abi.KIVI_F16, D, 0, 1, 1e-6, 0, 0, x.data_ptr(), 0, 0, 0, 0, *s, 0, 0, 0, 0, 0, f.data_ptr(),
                           0, 0, 0, 0, 0, out.data_ptr(), 0)
    assert abi.load().kivi_norm_rope(C.byref(cache.desc), args, C.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    abi.kivi_norm_rope(cache, None, x, None, None, want, None, f)
    assert torch.equal(out, want)
