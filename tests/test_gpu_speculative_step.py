"""Whole speculative steps of a one-layer model over the quantized cache:

    projections -> kivi_norm_rope -> kivi_tree_attention -> logits ->
    kivi_token_probs -> kivi_verify_tree -> kivi_append_path

each call on what the call before it left on the device, several steps in a
row, eagerly and as one captured graph."""
import numpy as np
import pytest
import torch

import _step
from _attend import attend_ref, make_cache, mask_words, materialized, check_rows
from test_gpu_append_path import BUFS, clone_row
from test_gpu_norm_rope import check as check_heads, freqs, magnitudes
from test_gpu_token_probs import check as check_probs
from kivi_bit_kv_gb300 import abi

pytestmark = pytest.mark.gpu


class Model:
    """Random weights, a draft tree of N nodes per sequence and the step's buffers."""

    def __init__(self, dev, B, H, gq, D, N, V, bits, G, R, lens, drawn, seed):
        g = torch.Generator().manual_seed(seed)
        self.dims, self.dev, self.rng = (B, H, gq, D, N, V), dev, np.random.default_rng(seed)
        Hq, E = H * gq, 64
        self.cache = make_cache(dev, B, H, D, bits, bits, G, R, lens, seed=seed, room=8 * N)

        def w(*shape):
            return (torch.randn(shape, generator=g) / shape[0] ** 0.5).half().to(dev)

        self.emb, self.proj, self.head = w(V, E) * V ** 0.5, w(E, (Hq + 2 * H) * D), w(Hq * D, V) * 3
        self.q_weight, self.k_weight = ((1 + 0.2 * torch.randn(D, generator=g)).to(dev) for _ in range(2))
        self.inv_freq = freqs(D).to(dev)
        self.drawn = drawn
        z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device=dev)  # noqa: E731
        f16, f32 = torch.float16, torch.float32
        self.tokens, self.parent, self.depth, self.u = z(B, N), z(B, N), z(B, N), z(B, N, dtype=f32)
        self.mask = z(B, N, (N + 63) // 64, dtype=torch.int64)
        self.n = torch.tensor([max(1, N - 2 * b) for b in range(B)], dtype=torch.int32, device=dev)
        self.q, self.k, self.v = z(B, Hq, N, D, dtype=f16), z(B, H, N, D, dtype=f16), z(B, H, N, D, dtype=f16)
        self.out, self.ws = z(B, Hq, N, D, dtype=f32), self.cache.attend_workspace(Hq, N)
        self.draft_logits, self.draft = z(B, N, V, dtype=f16), z(B, N, V, dtype=f32)
        self.logits, self.target = z(B, N, V, dtype=f32), z(B, N, V, dtype=f32)
        self.temperature = torch.tensor([(0.8, 0.0, 1.3)[b % 3] for b in range(B)], device=dev)
        self.path, self.counts, self.next, self.status = z(B, N), z(B), z(B), z(1)
        self.next.random_(0, V, generator=torch.Generator(device=dev).manual_seed(seed))

    def new_tree(self):
        """Random drafted tokens below the pending one."""
        B, H, gq, D, N, V = self.dims
        r = self.rng
        parent, depth = np.full((B, N), -1, np.int32), np.zeros((B, N), np.int32)
        for i in range(1, N):
            parent[:, i] = r.integers(max(0, i - 3), i, size=B)
            depth[:, i] = depth[np.arange(B), parent[:, i]] + 1
        masks = []
        for b in range(B):
            rows = [1]
            for i in range(1, N):
                rows.append(rows[parent[b, i]] | 1 << i)
            masks.append(mask_words(rows, N))
        self.parent.copy_(torch.from_numpy(parent))
        self.depth.copy_(torch.from_numpy(depth))
        self.mask.copy_(torch.stack(masks))
        self.u.copy_(torch.from_numpy(r.random((B, N)).astype(np.float32)))
        self.draft_logits.copy_(torch.from_numpy(r.normal(size=(B, N, V)).astype(np.float32)))
        self.tokens.copy_(torch.from_numpy(r.integers(0, V, size=(B, N)).astype(np.int32)))

    def step(self):
        B, H, gq, D, N, V = self.dims
        Hq = H * gq
        abi.kivi_token_probs(self.draft_logits, self.draft, n_rows=self.n)
        self.tokens[:, 0].copy_(self.next)
        x = self.emb[self.tokens.long()]
        qkv = (x @ self.proj).view(B, N, Hq + 2 * H, D)
        self.qkv = qkv
        abi.kivi_norm_rope(self.cache, qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:], self.q, self.k, self.v,
                           self.inv_freq, pos=self.depth, base=self.cache.lens, q_weight=self.q_weight,
                           k_weight=self.k_weight, n_tok=self.n)
        abi.kivi_tree_attention(self.cache, self.q, self.k, self.v, self.mask, self.out, self.ws, n_draft=self.n)
        self.logits.copy_(self.out.permute(0, 2, 1, 3).reshape(B, N, Hq * D).half() @ self.head)
        abi.kivi_token_probs(self.logits, self.target, temperature=self.temperature, n_rows=self.n)
        abi.kivi_verify_tree(self.tokens, self.parent, self.u, self.target, self.draft if self.drawn else None, self.path,
                             self.counts, self.next, n_draft=self.n)
        abi.kivi_append_path(self.cache, self.k, self.v, self.path, self.counts, self.status)


CASES = {
    "tree_int4": (3, 2, 2, 64, 6, 211, 4, 32, 32, [40, 0, 333], True),
    "tree_int2": (4, 1, 4, 128, 9, 1000, 2, 32, 32, [95, 63, 700, 1], False),
    "rows_of_many_heads": (2, 2, 8, 128, 5, 97, 8, 64, 64, [130, 300], True),
}


@pytest.mark.parametrize("name", CASES)
def test_steps_in_a_row(cuda, name):
    m = Model(cuda, *CASES[name], seed=31)
    B, H, gq, D, N, V = m.dims
    sm = D ** -0.5
    kept = 0
    for _ in range(5):
        m.new_tree()
        lens = m.cache.lens.tolist()
        before = [clone_row(m.cache, b) for b in range(B)]
        K, Vc = materialized(m.cache, 0), materialized(m.cache, 1)
        m.step()
        torch.cuda.synchronize()
        n = m.n.tolist()
        # queries, keys and values
        pos = (m.depth.cpu().long() + torch.tensor(lens).view(B, 1)).view(1, B, N)
        Hq = H * gq
        for x, y, w, turned in ((m.qkv[:, :, :Hq], m.q, m.q_weight, True), (m.qkv[:, :, Hq:Hq + H], m.k, m.k_weight, True),
                                (m.qkv[:, :, Hq + H:], m.v, None, False)):
            want = _step.norm_rope64(x, w, 1e-6, m.inv_freq.cpu(), pos, None, False, turned)
            h = magnitudes(x, w, 1e-6, D // 2 if turned else 0, False)
            for b in range(B):
                check_heads(y[b, :, :n[b]], want[b, :, :n[b]], h[b, :, :n[b]], 2.0 ** -18 if turned else 0.0)
        # attention, probabilities, path
        path, counts, nxt = m.path.cpu().numpy(), m.counts.tolist(), m.next.tolist()
        tokens = m.tokens.cpu().numpy()
        for b in range(B):
            for i in range(n[b]):
                sees = [j for j in range(n[b]) if int(m.mask[b, i, 0]) >> j & 1]
                for hq in range(Hq):
                    k = torch.cat([K[b, hq // gq, :lens[b]], m.k[b, hq // gq, sees].cpu().double()])
                    v = torch.cat([Vc[b, hq // gq, :lens[b]], m.v[b, hq // gq, sees].cpu().double()])
                    want, bound = attend_ref(m.q[b, hq, i].cpu().double(), k, v, sm)
                    check_rows(m.out[b, hq, i].cpu(), want, bound, f"sequence {b} node {i} head {hq}")
                check_probs(m.target[b, i], m.logits[b, i], float(m.temperature[b]))
            want, last = _step.verify(tokens[b], m.parent[b].cpu().numpy(), m.u[b].cpu().numpy(), m.target[b].cpu().numpy(),
                                      m.draft[b].cpu().numpy() if m.drawn else None, n[b])
            assert path[b, :counts[b]].tolist() == want and nxt[b] == last and (path[b, counts[b]:] == -1).all()
            kept += counts[b] - 1
        # the cache holds the path as single appends would have put it there
        assert int(m.status.item()) == 0 and m.cache.lens.tolist() == [a + c for a, c in zip(lens, counts)]
        st = torch.zeros(1, dtype=torch.int32, device=cuda)
        for b, one in enumerate(before):
            for i in path[b, :counts[b]].tolist():
                abi.kivi_append_token(one, m.k[b:b + 1, :, i].contiguous(), m.v[b:b + 1, :, i].contiguous(), st)
            for buf in BUFS:
                got, ref = getattr(m.cache, buf)[b:b + 1], getattr(one, buf)
                assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8)), f"{buf} of sequence {b}"


def test_a_captured_step_equals_the_eager_one(cuda):
    eager, graphed = (Model(cuda, *CASES["tree_int4"], seed=32) for _ in range(2))
    for m in (eager, graphed):                                  # the libraries' first calls
        m.new_tree()
        m.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for _ in range(6):
        eager.new_tree()
        graphed.new_tree()
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("q", "k", "v", "out", "target", "path", "counts", "next"):
            assert torch.equal(getattr(eager, name), getattr(graphed, name)), name
        for buf in BUFS:
            assert torch.equal(getattr(eager.cache, buf), getattr(graphed.cache, buf)), buf


FIRST = """
import sys
sys.path[:0] = [{root!r}, {here!r}]
import torch
from kivi_bit_kv_gb300 import KiviCache, abi
dev = torch.device("cuda", 0)
B, N, H, D, V = 3, 4, 2, 128, 40001
cache = KiviCache(B, H, D, 2, 2, 32, 32, 64, device=dev)
g = torch.Generator(device=dev).manual_seed(1)
x = torch.randn((B, N, H, D), generator=g, device=dev).bfloat16()
f = (10000.0 ** (-torch.arange(0, D, 2, device=dev) / D)).float()
logits = torch.randn((B, N, V), generator=g, device=dev)
parent = (torch.arange(N, device=dev, dtype=torch.int32) - 1).expand(B, N).contiguous()
tokens = torch.randint(0, V, (B, N), generator=g, device=dev, dtype=torch.int32)
u = torch.rand((B, N), generator=g, device=dev)
def buffers():
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    return torch.zeros((B, H, N, D), dtype=torch.float16, device=dev), torch.zeros((B, N, V), device=dev), i(B, N), i(B), i(B)
def step(q, probs, path, counts, nxt):
    abi.kivi_norm_rope(cache, x, None, None, q, None, None, f)
    abi.kivi_token_probs(logits, probs)
    abi.kivi_verify_tree(tokens, parent, u, probs, None, path, counts, nxt)
held, eager = buffers(), buffers()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step(*held)
graph.replay()
step(*eager)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(held, eager))
assert int(held[3].min()) >= 1
print("same")
"""


def test_the_first_call_of_a_process_may_be_captured(cuda):
    """What a launcher sets up on its first call does not disturb a capture."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(root=os.path.dirname(here), here=here)
    out = subprocess.run([sys.executable, "-c", code], check=True, capture_output=True, text=True, timeout=300)
    assert out.stdout.strip() == "same"


def test_two_host_threads_on_streams_of_their_own(cuda):
    """Calls at once from two threads, each with its own inputs, give what they
    give one after the other."""
    import threading
    models = [Model(cuda, *CASES["tree_int4"], seed=33 + i) for i in range(2)]
    want = []
    for m in models:
        m.new_tree()
        first, cached = m.next.clone(), [getattr(m.cache, b).clone() for b in BUFS]
        m.step()
        torch.cuda.synchronize()
        want.append([getattr(m, n).clone() for n in ("q", "k", "v", "out", "target", "path", "counts", "next")])
        m.next.copy_(first)
        for b, t in zip(BUFS, cached):
            getattr(m.cache, b).copy_(t)
    torch.cuda.synchronize()

    def work(m):
        with torch.cuda.stream(torch.cuda.Stream()):
            for i in range(20):
                abi.kivi_token_probs(m.draft_logits, m.draft, n_rows=m.n)
            m.step()

    threads = [threading.Thread(target=work, args=(m,)) for m in models]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for m, w in zip(models, want):
        for name, t in zip(("q", "k", "v", "out", "target", "path", "counts", "next"), w):
            assert torch.equal(getattr(m, name), t), name


def test_a_captured_fork_and_join(cuda):
    """Calls on two branches of a graph, joined before a third, between kernels of
    other libraries: every call waits for all that it reads."""
    B, N, V = 4, 5, 40000
    g = torch.Generator(device=cuda).manual_seed(35)
    logits, draft_logits = (torch.randn((B, N, V), generator=g, device=cuda) for _ in range(2))
    tokens = torch.randint(0, V, (B, N), generator=g, device=cuda, dtype=torch.int32)
    parent = torch.tensor([-1, 0, 0, 1, 2], dtype=torch.int32, device=cuda).expand(B, N).contiguous()
    u = torch.rand((B, N), generator=g, device=cuda)

    def buffers():
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device=cuda)  # noqa: E731
        return [torch.zeros((B, N, V), device=cuda) for _ in range(4)] + [z(B, N), z(B), z(B)]

    def run(b, fork):
        x, y, p, q, path, counts, nxt = b
        side, main = torch.cuda.Stream(), torch.cuda.current_stream()
        if fork:
            side.wait_stream(main)
        with torch.cuda.stream(side if fork else main):
            torch.mul(draft_logits, 3.0, out=y)
            abi.kivi_token_probs(y, q)
        torch.mul(logits, 3.0, out=x)
        abi.kivi_token_probs(x, p)
        if fork:
            main.wait_stream(side)
        abi.kivi_verify_tree(tokens, parent, u, p, q, path, counts, nxt)
        counts.add_(100)
        p.zero_()
        q.zero_()

    eager, held = buffers(), buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(held, True)
    for _ in range(20):
        u.uniform_()
        logits.normal_()
        run(eager, False)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager[4:], held[4:]):
            assert torch.equal(a, b)
        assert int(held[5].min()) >= 101
