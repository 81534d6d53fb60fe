"""Host-side checks of the speculative and sparse decode entry points that need
no GPU: argument errors and workspace sizes.  No call here reaches a launch."""
import ctypes as C

import pytest
import torch

from test_abi import _desc, _with_ptrs

Q, OUT, WS, BLK, SC = 0x20000, 0x30000, 0x40000, 0x50000, 0x60000
ONE = C.c_float(1.0)


def test_block_select_refusals(kivi_lib):
    from kivi_bit_kv_gb300 import abi
    d = _with_ptrs(_desc())
    f, ref = kivi_lib.kivi_block_select, C.byref(d)
    for args, needle in (((Q, 6, BLK, 4, SC), "multiple of H"), ((None, 4, BLK, 4, SC), "q is NULL"),
                         ((Q, 4, BLK, 0, SC), "n_keep=0"), ((Q, 4, None, 4, SC), "blocks is NULL"),
                         ((Q, 4, BLK + 4, 4, SC), "blocks is not"), ((Q, 4, BLK, 4, None), "scores is NULL"),
                         ((Q + 2, 4, BLK, 4, SC), "q is not"), ((Q, 4 * 17, BLK, 4, SC), "<= 16")):
        assert f(ref, *args, None) == abi.KIVI_EINVAL
        assert needle in abi.kivi_last_error(), abi.kivi_last_error()
    assert f(None, Q, 4, BLK, 4, SC, None) == abi.KIVI_EINVAL
    bad = _with_ptrs(_desc(D=96))
    assert f(C.byref(bad), Q, 4, BLK, 4, SC, None) == abi.KIVI_EINVAL


def test_attention_refusals(kivi_lib):
    from kivi_bit_kv_gb300 import abi
    d = _with_ptrs(_desc())
    ref = C.byref(d)
    big = 1 << 40
    sp = kivi_lib.kivi_sparse_attention
    for args, st in (((Q, 6, ONE, BLK, 4, OUT, WS, big), abi.KIVI_EINVAL),
                     ((None, 4, ONE, BLK, 4, OUT, WS, big), abi.KIVI_EINVAL),
                     ((Q, 4, ONE, BLK, 0, OUT, WS, big), abi.KIVI_EINVAL),
                     ((Q, 4, ONE, None, 4, OUT, WS, big), abi.KIVI_EINVAL),
                     ((Q, 4, ONE, BLK, 4, None, WS, big), abi.KIVI_EINVAL),
                     ((Q, 4, ONE, BLK, 4, OUT, None, big), abi.KIVI_EINVAL),
                     ((Q, 4, ONE, BLK, 4, OUT, WS, 8), abi.KIVI_EWORKSPACE)):
        assert sp(ref, *args, None) == st, args
    tr = kivi_lib.kivi_tree_attention
    K, V, M, ND = 0x70000, 0x80000, 0x90000, 0xA0000
    for args, st in (((Q, 4, 0, K, V, M, ND, ONE, OUT, WS, big), abi.KIVI_EINVAL),
                     ((Q, 4, 257, K, V, M, ND, ONE, OUT, WS, big), abi.KIVI_EINVAL),
                     ((Q, 5, 8, K, V, M, ND, ONE, OUT, WS, big), abi.KIVI_EINVAL),
                     ((Q, 4, 8, None, V, M, ND, ONE, OUT, WS, big), abi.KIVI_EINVAL),
                     ((Q, 4, 8, K, V + 8, M, ND, ONE, OUT, WS, big), abi.KIVI_EINVAL),
                     ((Q, 4, 8, K, V, None, ND, ONE, OUT, WS, big), abi.KIVI_EINVAL),
                     ((Q, 4, 8, K, V, M, ND + 2, ONE, OUT, WS, big), abi.KIVI_EINVAL),
                     ((Q, 4, 8, K, V, M, ND, ONE, OUT, WS, 8), abi.KIVI_EWORKSPACE),
                     ((Q, 4, 8, K, V, M, None, ONE, OUT, WS, 8), abi.KIVI_EWORKSPACE)):
        assert tr(ref, *args, None) == st, args


def test_append_path_refusals(kivi_lib):
    from kivi_bit_kv_gb300 import abi
    d = _with_ptrs(_desc())
    f, ref = kivi_lib.kivi_append_path, C.byref(d)
    K, V, P, N, S = 0x70000, 0x80000, 0x90000, 0xA0000, 0xB0000
    for args in ((None, V, 8, P, 4, N, S), (K, V, 0, P, 4, N, S), (K, V, 8, P, 0, N, S), (K, V, 8, None, 4, N, S),
                 (K, V, 8, P, 4, None, S), (K, V, 8, P, 4, N, None), (K + 8, V, 8, P, 4, N, S),
                 (K, V, 8, P + 2, 4, N, S)):
        assert f(ref, *args, None) == abi.KIVI_EINVAL, args


def test_workspace_bytes(kivi_lib):
    from kivi_bit_kv_gb300 import abi
    cache = type("c", (), {"desc": _desc()})()
    assert abi.kivi_attend_workspace_bytes(cache, 4) > 0
    assert abi.kivi_attend_workspace_bytes(cache, 4, 256) >= abi.kivi_attend_workspace_bytes(cache, 4, 1)
    for Hq, N in ((4, 0), (4, 257), (5, 8), (4 * 17, 8), (0, 8)):
        assert abi.kivi_attend_workspace_bytes(cache, Hq, N) == 0
    assert abi.kivi_attend_workspace_bytes(type("c", (), {"desc": _desc(D=96)})(), 4, 1) == 0


class FakeCache:
    """What the wrappers read of a cache, without device memory."""

    def __init__(self):
        self.desc = _with_ptrs(_desc())
        self.B, self.H, self.D, self.G, self.Tmax = 2, 4, 128, 32, 4096
        self.device = torch.device("cuda", 0)


def test_wrappers_check_shapes_and_types(kivi_lib):
    from kivi_bit_kv_gb300 import abi
    c = FakeCache()
    q = torch.zeros(2, 4, 128, dtype=torch.float16)
    blocks, scores = torch.zeros(2, 4, 3, dtype=torch.int32), torch.zeros(2, 4, 128)
    out, ws = torch.zeros(2, 4, 128), torch.zeros(64)
    with pytest.raises(ValueError):                     # CPU tensors
        abi.kivi_block_select(c, q, blocks, scores)
    with pytest.raises(ValueError):
        abi.kivi_block_select(c, q[:1], blocks, scores)
    with pytest.raises(ValueError):
        abi.kivi_block_select(c, q, blocks[:, :2], scores)
    with pytest.raises(ValueError):
        abi.kivi_block_select(c, q, blocks, scores[..., :5])
    with pytest.raises(TypeError):
        abi.kivi_block_select(c, q.float(), blocks, scores)
    with pytest.raises(ValueError):
        abi.kivi_sparse_attention(c, q, blocks, out[:, :3], ws)
    tq, kv = torch.zeros(2, 4, 5, 128, dtype=torch.float16), torch.zeros(2, 4, 5, 128, dtype=torch.float16)
    mask, to = torch.zeros(2, 5, 1, dtype=torch.int64), torch.zeros(2, 4, 5, 128)
    for bad in (dict(mask=mask[:, :4]), dict(k=kv[:, :2]), dict(out=to[:, :, :3]), dict(q=tq[:, :, 0]),
                dict(n_draft=torch.zeros(3, dtype=torch.int32))):
        a = dict(q=tq, k=kv, v=kv, mask=mask, out=to, n_draft=None) | bad
        with pytest.raises(ValueError):
            abi.kivi_tree_attention(c, a["q"], a["k"], a["v"], a["mask"], a["out"], ws, n_draft=a["n_draft"])
    path, cnt, st = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        abi.kivi_append_path(c, kv, kv, path[:1], cnt, st)
    with pytest.raises(ValueError):
        abi.kivi_append_path(c, kv, kv, path, cnt[:1], st)
    with pytest.raises(ValueError):
        abi.kivi_append_path(c, kv, kv, path, cnt, st[:0])
