"""Host-side checks of the entry points around a speculative step that need no
GPU: argument errors, the binding's layout of its arguments, and the plain form
of the verification against a distribution.  No call here reaches a launch."""
import ctypes as C
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import _step
from conftest import ROOT
from test_abi import _desc, _with_ptrs
from test_attend_host import FakeCache

Q, K, V, OQ, OK, OV, F = (0x20000 + 0x10000 * i for i in range(7))


def heads(**kw):
    """Packed kivi_heads of 5 fp16 tokens a sequence of a fused projection."""
    from kivi_bit_kv_gb300 import abi
    row = (4 + 8) * 128
    a = dict(Hq=4, N=5, dtype=abi.KIVI_F16, rot=128, interleaved=0, n_axes=1, eps=1e-6, reserved=0, q_in=Q, k_in=K,
             v_in=V, qs=(5 * row, row, 128), ks=(5 * row, row, 128), vs=(5 * row, row, 128), q_weight=0, k_weight=0,
             inv_freq=F, axis=0, pos=0, base=0, n_tok=0, q=OQ, k=OK, v=OV)
    a.update(kw)
    flat = []
    for x in a.values():
        flat += x if isinstance(x, tuple) else (x,)
    return abi._HEADS.pack(*flat)


@pytest.mark.parametrize("change,needle", [
    (dict(Hq=6), "multiple of H"), (dict(N=0), "N=0"), (dict(N=1 << 27), "2^27"), (dict(dtype=3), "dtype=3"),
    (dict(dtype=-1), "dtype=-1"), (dict(rot=8), "rot=8"), (dict(rot=144), "rot=144"), (dict(rot=-16), "rot=-16"),
    (dict(n_axes=0), "n_axes=0"), (dict(n_axes=9), "n_axes=9"), (dict(eps=-1e-6), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(eps=float("inf")), "eps"), (dict(q_in=0), "q: an input"), (dict(k=0), "k: an input"),
    (dict(reserved=1), "reserved=1"), (dict(q_in=0, k_in=0, v_in=0, q=0, k=0, v=0), "all NULL"), (dict(q_in=Q + 8), "q: the input"),
    (dict(v=OV + 2), "v: the input"), (dict(qs=(5 * 1536, 1535, 128)), "dimension 1"),
    (dict(ks=(5 * 1536 + 4, 1536, 128)), "dimension 0"), (dict(vs=(5 * 1536, 1536, 132)), "dimension 2"),
    (dict(q=Q), "q overlaps input q_in"), (dict(k=Q + 1024), "k overlaps"), (dict(v=Q + 28672 - 16), "v overlaps"),
    (dict(q_weight=0x90004), "q_weight"), (dict(inv_freq=0), "inv_freq is NULL"), (dict(inv_freq=F + 2), "inv_freq is not"),
    (dict(axis=0x90002), "axis"), (dict(pos=0x90001), "pos"), (dict(base=0x90002), "base"), (dict(n_tok=0x90003), "n_tok"),
])
def test_norm_rope_refusals(kivi_lib, change, needle):
    from kivi_bit_kv_gb300 import abi
    d = _with_ptrs(_desc())
    assert kivi_lib.kivi_norm_rope(C.byref(d), heads(**change), None) == abi.KIVI_EINVAL
    assert needle in abi.kivi_last_error(), abi.kivi_last_error()


def test_norm_rope_refuses_a_bad_descriptor(kivi_lib):
    from kivi_bit_kv_gb300 import abi
    assert kivi_lib.kivi_norm_rope(None, heads(), None) == abi.KIVI_EINVAL
    d = _with_ptrs(_desc(D=96))
    assert kivi_lib.kivi_norm_rope(C.byref(d), heads(), None) == abi.KIVI_EINVAL
    d = _with_ptrs(_desc())
    assert kivi_lib.kivi_norm_rope(C.byref(d), None, None) == abi.KIVI_EINVAL
    assert "NULL" in abi.kivi_last_error()


def test_packed_arguments_match_the_header(tmp_path):
    """The binding's packed kivi_heads has the C struct's offsets."""
    from kivi_bit_kv_gb300 import abi
    if shutil.which("gcc") is None:
        pytest.skip("gcc not found")
    names = "Hq N dtype rot interleaved n_axes eps reserved q_in k_in v_in q_strides k_strides v_strides q_weight k_weight inv_freq axis pos base n_tok q k v".split()
    src = tmp_path / "o.c"
    src.write_text('#include <stdio.h>\n#include "kivi.h"\nint main(void) {\n' +
                   "".join(f'printf("%zu ", offsetof(kivi_heads, {n}));\n' for n in names) +
                   'printf("%zu\\n", sizeof(kivi_heads)); return 0; }\n')
    exe = tmp_path / "o"
    subprocess.run(["gcc", "-std=c99", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    want = [4 * i for i in range(8)] + [32, 40, 48, 56, 80, 104] + [128 + 8 * i for i in range(10)]
    assert got == want + [abi._HEADS.size]


def test_token_probs_refusals(kivi_lib):
    from kivi_bit_kv_gb300 import abi
    f = kivi_lib.kivi_token_probs
    good = dict(l=Q, dtype=abi.KIVI_F16, B=2, N=3, V=1000, sb=3000, sn=1000, t=K, n=V, p=OQ)
    for change, needle in ((dict(l=None), "logits is NULL"), (dict(l=Q + 1), "logits is not"),
                           (dict(l=Q + 2, dtype=abi.KIVI_F32), "logits is not"), (dict(dtype=3), "dtype=3"),
                           (dict(B=0), "B=0"), (dict(N=0), "N=0"), (dict(N=1 << 26), "2^27"), (dict(V=0), "V=0"),
                           (dict(V=abi.KIVI_MAX_VOCAB + 1), "vocabulary"), (dict(t=K + 2), "temperature"),
                           (dict(p=Q), "probs overlaps"), (dict(p=Q + 11984), "probs overlaps"), (dict(p=Q - 23984), "probs overlaps"),
                           (dict(n=V + 1), "n_rows"), (dict(p=None), "probs is NULL"), (dict(p=OQ + 8), "probs is not")):
        assert f(*(good | change).values(), None) == abi.KIVI_EINVAL, change
        assert needle in abi.kivi_last_error(), abi.kivi_last_error()


def test_verify_tree_refusals(kivi_lib):
    from kivi_bit_kv_gb300 import abi
    f = kivi_lib.kivi_verify_tree
    good = dict(B=2, N=8, V=1000, tokens=Q, parent=K, n=V, u=OQ, target=OK, draft=OV, path=F, counts=F + 64, next=F + 128)
    for change, needle in ((dict(B=0), "B=0"), (dict(N=0), "N=0"), (dict(N=257), "N=257"), (dict(V=0), "V=0"),
                           (dict(V=abi.KIVI_MAX_VOCAB + 1), "vocabulary"), (dict(tokens=None), "tokens is NULL"),
                           (dict(parent=K + 2), "parent is not"), (dict(n=V + 2), "n_draft"), (dict(u=None), "u is NULL"),
                           (dict(target=None), "target is NULL"), (dict(target=OK + 4), "target is not"),
                           (dict(draft=OV + 8), "draft is not"), (dict(path=None), "path is NULL"),
                           (dict(counts=F + 1), "counts is not"), (dict(next=None), "next is NULL")):
        assert f(*(good | change).values(), None) == abi.KIVI_EINVAL, change
        assert needle in abi.kivi_last_error(), abi.kivi_last_error()


def test_wrappers_check_shapes_and_types(kivi_lib):
    """On CPU tensors: each wrong shape and type is named before the device is,
    and the right ones are refused for their device."""
    from kivi_bit_kv_gb300 import abi
    c = FakeCache()
    x = torch.zeros(2, 5, 4, 128, dtype=torch.float16)
    y = torch.zeros(2, 4, 5, 128, dtype=torch.float16)
    f = torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):
        abi.kivi_norm_rope(c, x, x, x, y, y, y, f)
    for kw in (dict(q=y[:, :, :4]), dict(q=None), dict(v_in=x[:1]), dict(k_in=x[:, :4]), dict(inv_freq=f.view(1, 64)),
               dict(pos=torch.zeros(2, 4, dtype=torch.int32)), dict(axis=torch.zeros(63, dtype=torch.int32)),
               dict(base=torch.zeros(3, dtype=torch.int32)), dict(n_tok=torch.zeros(1, dtype=torch.int32)),
               dict(q_weight=torch.zeros(64)), dict(q_in=None, k_in=None, v_in=None, q=None, k=None, v=None),
               dict(q_in=x.transpose(2, 3))):
        a = dict(q_in=x, k_in=x, v_in=x, q=y, k=y, v=y, inv_freq=f) | kw
        with pytest.raises(ValueError):
            abi.kivi_norm_rope(c, **a)
    with pytest.raises(TypeError):
        abi.kivi_norm_rope(c, x.double(), None, None, y, None, None, f)
    l, p = torch.zeros(2, 3, 10), torch.zeros(2, 3, 10)
    for args in ((l[0], p), (l, p[:1]), (l[..., ::2], p[..., :5].contiguous()), (l, p)):
        with pytest.raises(ValueError):
            abi.kivi_token_probs(*args)
    for kw in (dict(temperature=torch.zeros(3)), dict(n_rows=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            abi.kivi_token_probs(l, p, **kw)
    with pytest.raises(TypeError):
        abi.kivi_token_probs(l.double(), p)
    i2, i1 = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    good = dict(tokens=i2, parent=i2, u=torch.zeros(2, 3), target=p, draft=p, path=i2, counts=i1, next=i1, n_draft=i1)
    for kw in (dict(tokens=i2[:, :2]), dict(u=torch.zeros(2, 4)), dict(draft=p[:, :2]), dict(path=i2[:1]),
               dict(counts=i1[:1]), dict(n_draft=i1[:1]), dict(target=p[0]), {}):
        with pytest.raises(ValueError):
            abi.kivi_verify_tree(**(good | kw))


@pytest.mark.parametrize("kind", ["sampled", "best"])
def test_plain_verification_follows_the_target(kind):
    """The first new token's distribution is the target's at node 0, whatever the
    draft.  4000 draws: a frequency is off by more than 5 standard deviations
    with a chance below 10^-6 a cell."""
    rng = np.random.default_rng(7)
    V, n = 6, 4000
    target = rng.dirichlet(np.ones(V), size=3).astype(np.float32)
    draft = rng.dirichlet(np.ones(V), size=3).astype(np.float32)
    seen = np.zeros(V)
    for _ in range(n):
        if kind == "sampled":
            tokens = np.array([0, *rng.choice(V, 2, p=draft[0].astype(np.float64) / draft[0].astype(np.float64).sum())])
        else:
            tokens = np.array([0, 4, 1])
        path, nxt = _step.verify(tokens, np.array([-1, 0, 0]), rng.random(3).astype(np.float32), target,
                                 draft if kind == "sampled" else None)
        seen[tokens[path[1]] if len(path) > 1 else nxt] += 1
    p = target[0].astype(np.float64)
    assert (np.abs(seen - n * p) <= 5 * np.sqrt(n * p * (1 - p)) + 1).all(), (seen / n, p)
