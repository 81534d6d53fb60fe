"""Head norms and token probabilities of inputs with negative strides (sequences,
tokens, heads or rows from the last to the first) through the C interface, in the
default and in the bounds-checked build: the results of a contiguous copy, and
no check fails."""
import ctypes as C
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def run_cases():
    sys.path[:0] = [ROOT, HERE]
    import torch
    from kivi_bit_kv_gb300 import KiviCache, abi
    dev, lib = torch.device("cuda", 0), abi.load()
    g = torch.Generator(device=dev).manual_seed(81)
    stream = C.c_void_p(torch.cuda.current_stream().cuda_stream)

    def start(t, flip):
        """Address of the element that comes first, and strides with signs."""
        at, st = t.data_ptr(), list(t.stride())
        for d in flip:
            at += (t.shape[d] - 1) * st[d] * t.element_size()
            st[d] = -st[d]
        return at, st

    for dtype, code in ((torch.float16, abi.KIVI_F16), (torch.float32, abi.KIVI_F32)):
        for V, pad in ((1000, 0), (4099, 2)):
            for flip in ((0,), (1,), (0, 1)):
                x = torch.randn((3, 4, V + pad), generator=g, device=dev).to(dtype)[..., :V]
                out, want = (torch.zeros((3, 4, V), device=dev) for _ in range(2))
                at, st = start(x, flip)
                assert lib.kivi_token_probs(at, code, 3, 4, V, st[0], st[1], None, None, out.data_ptr(), stream) == 0
                abi.kivi_token_probs(x.flip(flip).contiguous(), want)
                assert abi.kivi_check_status() == 0 and torch.equal(out, want)
        B, N, H, D = 2, 5, 3, 64
        cache = KiviCache(B, H, D, 2, 2, 32, 32, 32, device=dev)
        f = (10000.0 ** (-torch.arange(0, D, 2, device=dev) / D)).float()
        for flip in ((0,), (1,), (2,), (0, 1, 2)):
            xs = [torch.randn((B, N, H, D), generator=g, device=dev).to(dtype) for _ in range(3)]
            outs = [torch.zeros((B, H, N, D), dtype=torch.float16, device=dev) for _ in range(3)]
            want = [torch.zeros_like(o) for o in outs]
            at, st = zip(*(start(x, flip) for x in xs))
            args = abi._HEADS.pack(H, N, code, D, 0, 1, 1e-6, 0, *at, *(s for row in st for s in row[:3]), 0, 0, f.data_ptr(),
                                   0, 0, 0, 0, *(o.data_ptr() for o in outs))
            assert lib.kivi_norm_rope(C.byref(cache.desc), args, stream) == 0
            abi.kivi_norm_rope(cache, *(x.flip(flip).contiguous() for x in xs), *want, f)
            assert abi.kivi_check_status() == 0
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
    print("same")


@pytest.mark.gpu
@pytest.mark.parametrize("variant", ["", "checked"])
def test_from_the_last_to_the_first(variant):
    sys.path.insert(0, ROOT)
    from kivi_bit_kv_gb300 import build
    env = dict(os.environ)
    if variant:
        env["KIVI_LIB"] = build.build(variant=variant)
    out = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, capture_output=True, text=True, timeout=900)
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr[-2000:]


if __name__ == "__main__":
    run_cases()
