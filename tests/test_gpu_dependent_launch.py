"""Head norms, token probabilities and verification directly behind calls whose kernels
let the next one start early: every result is that of the same call on a copy made
after all work has ended.  The attentions' outputs stand in for logits,
projections and probabilities."""
import pytest
import torch

from _attend import f16, make_cache
from test_gpu_norm_rope import freqs
from kivi_bit_kv_gb300 import abi

pytestmark = pytest.mark.gpu


class Chain:
    """An attention of N tokens a sequence (0: decode attention), and the three
    calls on its output; then an append, and positions from the new lengths."""

    def __init__(self, dev, B, H, gq, D, N, lens):
        self.dims, self.N = (B, H, H * gq, D), N
        n, Hq = max(N, 1), H * gq
        self.cache = make_cache(dev, B, H, D, 4, 4, 32, 32, lens, seed=7, room=32 + 40 * n)
        z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device=dev)  # noqa: E731
        i32, f16_ = torch.int32, torch.float16
        self.q, self.k, self.v = z(B, Hq, n, D, dtype=f16_), z(B, H, n, D, dtype=f16_), z(B, H, n, D, dtype=f16_)
        self.mask = torch.full((B, n, (n + 63) // 64), -1, dtype=torch.int64, device=dev)
        self.out = z(B, Hq, n, D)
        self.ws = self.cache.attend_workspace(Hq, n) if N else self.cache.workspace(Hq)
        self.f = freqs(D).to(dev)
        self.tokens = torch.randint(0, D, (B, Hq * n), device=dev, dtype=i32)
        self.parent = (torch.arange(Hq * n, device=dev, dtype=i32) // 2).expand(B, Hq * n).contiguous()
        self.u = torch.rand((B, Hq * n), device=dev)
        self.path, self.counts, self.status = z(B, n, dtype=i32), z(B, dtype=i32), z(1, dtype=i32)
        self.got, self.want = self.buffers(z), self.buffers(z)

    def buffers(self, z):
        (B, H, Hq, D), n = self.dims, max(self.N, 1)
        i32 = torch.int32
        return dict(rows=z(B, Hq * n, D), long=z(B, Hq, n * D), heads=z(B, Hq, n, D, dtype=torch.float16),
                    path=z(B, Hq * n, dtype=i32), counts=z(B, dtype=i32), next=z(B, dtype=i32),
                    after=z(B, H, n, D, dtype=torch.float16))

    def attend(self):
        if self.N:
            abi.kivi_tree_attention(self.cache, self.q, self.k, self.v, self.mask, self.out, self.ws)
        else:
            abi.kivi_decode_attention(self.cache, self.q, self.out.view(*self.dims[:1], self.dims[2], self.dims[3]), self.ws)

    def use(self, which, x, o):
        (B, H, Hq, D), n = self.dims, max(self.N, 1)
        if which == "rows":
            abi.kivi_token_probs(x.view(B, Hq * n, D), o["rows"])
        elif which == "long":
            abi.kivi_token_probs(x.view(B, Hq, n * D), o["long"])
        elif which == "heads":
            abi.kivi_norm_rope(self.cache, x.transpose(1, 2), None, None, o["heads"], None, None, self.f)
        elif which == "path":
            abi.kivi_verify_tree(self.tokens, self.parent, self.u, x.view(B, Hq * n, D), None, o["path"], o["counts"], o["next"])

    def append(self):
        abi.kivi_append_path(self.cache, self.k, self.v, self.path, self.counts, self.status)

    def after(self, base, o):
        abi.kivi_norm_rope(self.cache, None, self.k.transpose(1, 2), None, None, o["after"], None, self.f, base=base)

    def step(self):
        for which in ("rows", "long", "heads", "path"):
            self.attend()
            self.use(which, self.out, self.got)
        if self.N:
            self.append()
            self.after(self.cache.lens, self.got)

    def fill(self, g):
        (B, H, Hq, D), n = self.dims, max(self.N, 1)
        self.q.copy_(3 * f16(g, B, Hq, n, D))
        self.k.copy_(f16(g, B, H, n, D))
        self.v.copy_(2 * f16(g, B, H, n, D))
        self.path.copy_(torch.arange(n).expand(B, n))
        self.counts.copy_(torch.randint(0, min(n, 3) + 1, (B,), generator=g))
        self.out.fill_(float("nan"))

    def check(self):
        torch.cuda.synchronize()
        x = self.out.clone()
        torch.cuda.synchronize()
        assert bool(x.isfinite().all()) and int(self.status.item()) == 0
        for which in ("rows", "long", "heads", "path"):
            self.use(which, x, self.want)
            torch.cuda.synchronize()
        if self.N:
            self.after(self.cache.lens.clone(), self.want)
        torch.cuda.synchronize()
        for name in self.want:
            assert torch.equal(self.got[name], self.want[name]), name


# (B, H, gq, D, N, lens): decode; few rows by warps, in one range and cut; many rows on
# the tensor cores, in one range and cut
CASES = {
    "decode": (3, 2, 4, 128, 0, [70, 3, 2000]),
    "warp": (6, 2, 2, 64, 4, [40, 0, 333, 95, 700, 1]),
    "warp_cut": (1, 2, 4, 128, 2, [9000]),
    "tree": (4, 2, 4, 128, 12, [300, 31, 0, 129]),
    "tree_cut": (1, 1, 8, 64, 24, [12000]),
}


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_directly_behind_a_kernel_that_lets_the_next_start(cuda, name, captured):
    g = torch.Generator().manual_seed(71)
    c = Chain(cuda, *CASES[name])
    c.fill(g)
    c.counts.zero_()
    c.step()                                                     # the libraries' first calls
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.step()
    for _ in range(25):
        c.fill(g)
        torch.cuda.synchronize()
        graph.replay() if captured else c.step()
        c.check()


def test_decode_behind_the_call_that_writes_its_queries(cuda):
    """Fused decode, itself a dependent of the call before it, on queries that
    kivi_norm_rope has just written, over and over."""
    B, H, gq, D = 4, 2, 4, 128
    g = torch.Generator(device=cuda).manual_seed(72)
    cache = make_cache(cuda, B, H, D, 2, 2, 32, 32, [500, 33, 0, 1200], seed=8)
    q = torch.zeros((B, H * gq, 1, D), dtype=torch.float16, device=cuda)
    out, want = (torch.zeros((B, H * gq, D), device=cuda) for _ in range(2))
    ws, f = cache.workspace(H * gq), freqs(D).to(cuda)
    xs = [torch.randn((B, 1, H * gq, D), generator=g, device=cuda).bfloat16() for _ in range(50)]
    for x in xs:
        torch.cuda.synchronize()
        for y in (xs[0], x):
            abi.kivi_norm_rope(cache, y, None, None, q, None, None, f, base=cache.lens)
            abi.kivi_decode_attention(cache, q, out, ws)
        torch.cuda.synchronize()
        abi.kivi_decode_attention(cache, q.clone(), want, ws)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
