"""Sizes of the workspaces of sparse and tree attention: one that is large
enough for N drafted tokens serves any smaller number and sparse attention.
No call here reaches a launch (its addresses belong to no device)."""
import ctypes as C

import pytest

from test_abi import _desc, _with_ptrs

DIMS = [(64, 32), (64, 64), (128, 32), (128, 128), (256, 64)]


@pytest.mark.parametrize("D,G", DIMS)
@pytest.mark.parametrize("gq", [1, 2, 3, 7, 16])
def test_bytes_do_not_fall_with_the_drafts(kivi_lib, D, G, gq):
    from kivi_bit_kv_gb300 import abi
    cache = type("c", (), {"desc": _desc(D=D, G=G, R=G)})()
    sizes = [abi.kivi_attend_workspace_bytes(cache, gq * cache.desc.H, n) for n in range(1, abi.KIVI_MAX_DRAFT + 1)]
    assert sizes[0] > 0
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("D,G", DIMS)
def test_a_workspace_for_many_drafts_is_taken_for_fewer(kivi_lib, D, G):
    from kivi_bit_kv_gb300 import abi
    desc = _with_ptrs(_desc(D=D, G=G, R=G))
    cache, ref = type("c", (), {"desc": desc})(), C.byref(desc)
    Hq = 2 * desc.H
    Q, K, V, M, OUT, WS, BLK = (0x20000 + 0x10000 * i for i in range(7))
    one = C.c_float(1.0)
    for most in (1, 4, 8, 17, 33, 256):
        room = abi.kivi_attend_workspace_bytes(cache, Hq, most)
        st = kivi_lib.kivi_sparse_attention(ref, Q, Hq, one, BLK, 4, OUT, WS, room, None)
        assert st not in (abi.KIVI_OK, abi.KIVI_EWORKSPACE)
        for n in range(1, most + 1):
            st = kivi_lib.kivi_tree_attention(ref, Q, Hq, n, K, V, M, None, one, OUT, WS, room, None)
            assert st not in (abi.KIVI_OK, abi.KIVI_EWORKSPACE), (most, n)
