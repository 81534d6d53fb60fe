"""Head norms with rotary positions, token probabilities and verification in the
bounds-checked build of the library (KIVI_CHECKS defined): no check fails, and all
results agree with the default build's bit for bit."""
import os
import subprocess
import sys

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def run_cases(path):
    sys.path.insert(0, ROOT)
    sys.path.insert(0, HERE)
    import torch
    import test_gpu_norm_rope as rope
    import test_gpu_verify_tree as ver
    from kivi_bit_kv_gb300 import abi
    dev = torch.device("cuda", 0)
    res, words = {}, []
    for name, (B, N, H, gq, D, dtype, rot, inter, axes, norm, base, ragged) in rope.CASES.items():
        for fused in (True, False):
            xs, w, f, pos, axis, b, n = rope.inputs(dev, name, 5, fused)
            outs = [torch.zeros((B, h, N, D), dtype=torch.float16, device=dev) for h in (H * gq, H, H)]
            abi.kivi_norm_rope(rope.small_cache(dev, B, H, D), *xs, *outs, f, pos=pos, base=b, axis=axis, interleaved=inter,
                               q_weight=w[0], k_weight=w[1], n_tok=n)
            for k, o in zip("qkv", outs):
                res[f"rope_{name}_{int(fused)}_{k}"] = o.view(torch.int16).cpu().numpy()
    words.append(abi.kivi_check_status())
    g = torch.Generator().manual_seed(40)
    for dtype in (torch.float16, torch.bfloat16, torch.float32):
        for V, pad, skip in ((1, 0, 0), (33, 0, 0), (1000, 24, 0), (50001, 3, 1), (131072, 0, 0), (131071, 1, 1), (600001, 0, 0)):
            buf = torch.randn((3, 2, V + pad + skip), generator=g).to(dtype).to(dev)
            x = buf[..., skip:skip + V]
            out = torch.zeros((3, 2, V), device=dev)
            n = torch.tensor([2, 1, 2], dtype=torch.int32, device=dev)
            abi.kivi_token_probs(x, out, temperature=torch.tensor([1.0, 0.5, 0.0], device=dev), n_rows=n)
            res[f"probs_{V}_{str(dtype)[6:]}"] = out.view(torch.int32).cpu().numpy()
    words.append(abi.kivi_check_status())
    for i, (B, N, V, shape) in enumerate(((3, 5, 1000, "tree"), (2, 9, 50001, "star"), (4, 3, 131072, "chain"), (40, 20, 77, "tree"))):
        for kind in ("sampled", "best"):
            p = ver.problem(50 + i, B, N, V, shape, kind)
            for k, o in zip(("path", "counts", "next"), ver.run(dev, *p, n=[N - b % 3 for b in range(B)])):
                res[f"verify_{i}_{kind}_{k}"] = o
    words.append(abi.kivi_check_status())
    np.savez(path, words=np.array(words), **res)


@pytest.mark.gpu
def test_checked_build_agrees_bit_for_bit(tmp_path):
    sys.path.insert(0, ROOT)
    from kivi_bit_kv_gb300 import build
    checked = build.build(variant="checked")
    paths = {}
    for name, lib in (("checked", checked), ("default", None)):
        env = dict(os.environ)
        env.pop("KIVI_LIB", None)
        if lib:
            env["KIVI_LIB"] = lib
        paths[name] = str(tmp_path / f"{name}.npz")
        subprocess.run([sys.executable, os.path.abspath(__file__), paths[name]], env=env, check=True, timeout=900)
    a, b = np.load(paths["checked"]), np.load(paths["default"])
    assert not a["words"].any() and not b["words"].any()
    assert sorted(a.files) == sorted(b.files)
    for key in a.files:
        assert np.array_equal(a[key], b[key]), key


if __name__ == "__main__":
    run_cases(sys.argv[1])
