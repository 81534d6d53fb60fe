"""Block selection, sparse and tree attention and path appends in the
bounds-checked build of the library (KIVI_CHECKS defined), where every global
access and copy is checked against the cache's arrays and the call's buffers.

Each case runs through both builds, each in a process of its own: no check
fails, and all results agree bit for bit (the operators' order of sums depends
on sizes only)."""
import os
import subprocess
import sys

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

# (B, H, gq, D, bits_k, bits_v, G, R, lengths, N, n_keep)
CASES = [
    (3, 2, 4, 128, 2, 2, 32, 128, [700, 1, 4000], 4, 9),        # 16 rows
    (2, 2, 4, 128, 2, 2, 32, 128, [700, 2100], 5, 200),         # 20 rows, every group listed
    (1, 1, 1, 128, 2, 2, 32, 128, [60000], 7, 1500),            # one row in many pieces
    (1, 1, 1, 128, 4, 2, 64, 128, [30000], 40, 300),            # the same, 64-row tiles
    (4, 4, 2, 64, 4, 4, 32, 32, [513, 2048, 0, 95], 3, 3),      # an empty sequence
    (2, 2, 8, 64, 2, 8, 32, 32, [513, 300], 33, 5),             # two row tiles of 128
    (2, 2, 1, 256, 8, 8, 64, 64, [3000, 1500], 6, 11),          # D = 256, int8
    (2, 1, 4, 256, 2, 4, 128, 128, [3000, 1500], 11, 8),        # D = 256, 44 rows
    (90, 8, 1, 64, 2, 2, 32, 32, [40 + 9 * i for i in range(90)], 2, 4),  # a warp a row chooses
]


def run_cases(path):
    sys.path.insert(0, ROOT)
    sys.path.insert(0, HERE)
    import torch
    from _attend import f16, make_cache, mask_words, random_tree
    from kivi_bit_kv_gb300 import abi
    dev = torch.device("cuda", 0)
    res = {}
    for i, (B, H, gq, D, bk, bv, G, R, lens, N, keep) in enumerate(CASES):
        g = torch.Generator().manual_seed(200 + i)
        cache = make_cache(dev, B, H, D, bk, bv, G, R, lens, seed=300 + i, room=3 * N)
        Hq = H * gq
        q1, q = f16(g, B, Hq, D).to(dev), f16(g, B, Hq, N, D).to(dev)
        k, v = f16(g, B, H, N, D).to(dev), f16(g, B, H, N, D).to(dev)
        rng = np.random.default_rng(400 + i)
        mask = torch.stack([mask_words(random_tree(rng, N), N) for _ in range(B)]).to(dev)
        blocks = torch.full((B, H, keep), -1, dtype=torch.int32, device=dev)
        scores = torch.zeros((B, H, cache.Tmax // G), device=dev)
        abi.kivi_block_select(cache, q1, blocks, scores)
        ws = cache.attend_workspace(Hq, N)
        out1 = torch.zeros((B, Hq, D), device=dev)
        ws1 = cache.attend_workspace(Hq)
        abi.kivi_sparse_attention(cache, q1, blocks, out1, ws1)
        out = torch.zeros((B, Hq, N, D), device=dev)
        nd = torch.tensor([max(N - b % 3, 0) for b in range(B)], dtype=torch.int32, device=dev)
        abi.kivi_tree_attention(cache, q, k, v, mask, out, ws, n_draft=nd)
        P = min(N, 4)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        pth = torch.arange(P, dtype=torch.int32, device=dev).expand(B, P).contiguous()
        counts = torch.tensor([b % (P + 1) for b in range(B)], dtype=torch.int32, device=dev)
        for _ in range(3):
            abi.kivi_append_path(cache, k, v, pth, counts, status)
        torch.cuda.synchronize(dev)
        for name, t in (("blocks", blocks), ("scores", scores.view(torch.int32)), ("sparse", out1.view(torch.int32)),
                        ("tree", out.view(torch.int32)), ("kq", cache.kq), ("vq", cache.vq),
                        ("kres", cache.kres.view(torch.int16)), ("vres", cache.vres.view(torch.int16)),
                        ("lens", cache.lens)):
            res[f"{name}{i}"] = t.cpu().numpy()
        assert torch.isfinite(out).all() and torch.isfinite(out1).all()
        res[f"words{i}"] = np.array([int(status.item()), int(ws[:1].view(torch.int32).item()),
                                     int(ws1[:1].view(torch.int32).item()), abi.kivi_check_status()])
    np.savez(path, **res)


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
    for i in range(len(CASES)):
        assert not a[f"words{i}"].any(), f"case {i}: status words {a[f'words{i}']} in the checked build"
        assert not b[f"words{i}"].any(), f"case {i}: status words {b[f'words{i}']}"
    assert sorted(a.files) == sorted(b.files)
    for key in a.files:
        assert np.array_equal(a[key], b[key]), key


if __name__ == "__main__":
    run_cases(sys.argv[1])
