"""The two ends of a speculative decoding step around the quantized cache, as
measurable cases.

    rope    projections to the queries, keys and values of the cache's entry
            points: head norms, rotary positions of one or several axes and the
            head-major layout in one pass (kivi_norm_rope)
    probs   logits to probabilities, one temperature per sequence
            (kivi_token_probs)
    verify  drafted tokens against the target's probabilities from given random
            numbers: the accepted path and the next token (kivi_verify_tree)

With ``own`` false every operator runs in its plain form (elementary torch
operations); with ``own`` true the library's entry points run on the same
tensors.
"""
import math
from types import SimpleNamespace

import numpy as np
import torch

own = False

ONE = 1 << 42            # the weight of probability 1 in a sum of weights
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one new token of one short sequence, where only latency counts
        dict(name="rope_tiny", op="rope", B=1, N=1, H=4, Hq=4, D=64, dtype="fp16", rot=64, axes=1, pairs="half",
             norm=True, place="next", ragged=False, layout="fused"),
        # 32 drafts after each of four long grouped-query contexts, at the depths of a tree
        dict(name="rope_tree_gqa", op="rope", B=4, N=32, H=8, Hq=32, D=128, dtype="bf16", rot=128, axes=1, pairs="half",
             norm=True, place="tree", ragged=True, layout="fused"),
        # the prompts of a layer: eight of 4096 tokens, 32 heads
        dict(name="rope_layer", op="rope", B=8, N=4096, H=32, Hq=32, D=128, dtype="fp16", rot=128, axes=1, pairs="half",
             norm=True, place="prompt", ragged=False, layout="fused"),
        # prompts with images or video: three axes, neighbouring channels paired, half of them rotated
        dict(name="rope_video", op="rope", B=3, N=2065, H=8, Hq=32, D=256, dtype="fp32", rot=128, axes=3, pairs="next",
             norm=True, place="axes", ragged=True, layout="split"),
        # one row of one sequence
        dict(name="probs_tiny", op="probs", B=1, N=1, V=32000, dtype="fp16", temp="one", ragged=False, pad=0),
        # 32 drafts of four sequences, each with its temperature, one of them 0
        dict(name="probs_tree", op="probs", B=4, N=32, V=32000, dtype="fp32", temp="mixed", ragged=True, pad=0),
        # an odd vocabulary, rows that start at any element
        dict(name="probs_odd", op="probs", B=16, N=5, V=100003, dtype="bf16", temp="mixed", ragged=True, pad=2),
        # a serving batch of 64 sequences with eight rows each over a large vocabulary
        dict(name="probs_batch", op="probs", B=64, N=8, V=131072, dtype="bf16", temp="mixed", ragged=False, pad=0),
        # a chain of five drafts of one sequence
        dict(name="verify_tiny", op="verify", B=1, N=6, V=32000, shape="chain", draft="sampled", ragged=False),
        # trees of 16 sampled nodes: rejected siblings change the distribution that the next is tested against
        dict(name="verify_tree", op="verify", B=16, N=16, V=131072, shape="tree", draft="sampled", ragged=True),
        # trees of the draft's best tokens, odd vocabulary
        dict(name="verify_best", op="verify", B=32, N=24, V=50001, shape="tree", draft="best", ragged=True),
        # a serving batch: chains of seven drafts
        dict(name="verify_batch", op="verify", B=64, N=8, V=131072, shape="chain", draft="sampled", ragged=False),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    op = rng.choice(["rope", "probs", "verify"])
    if op == "rope":
        D = rng.choice([64, 128, 128, 256])
        H, gq = log_int(1, 32), rng.choice([1, 1, 2, 4, 7, 8])
        dtype = rng.choice(["fp16", "bf16", "bf16", "fp32"])
        most = (1 << 28) // ((gq + 2) * H * D)               # tokens
        if dtype == "fp32":
            most //= 2
        place = rng.choice(["next", "tree", "prompt", "axes"])
        N = log_int(1, {"next": 1, "tree": 256, "prompt": 8192, "axes": 8192}[place])
        N = max(1, min(N, most))
        B = log_int(1, max(1, min(64, most // N)))
        rot = rng.choice([D, D, D // 2, D // 4, 16])
        return dict(op=op, B=B, N=N, H=H, Hq=H * gq, D=D, dtype=dtype, rot=rot, axes=3 if place == "axes" else 1,
                    pairs=rng.choice(["half", "half", "next"]), norm=rng.random() < 0.7, place=place,
                    ragged=rng.random() < 0.5, layout=rng.choice(["fused", "split"]))
    V = log_int(1000, 262144)
    N = log_int(1, 64)
    B = log_int(1, max(1, min(64, (1 << 26) // (N * V))))
    if op == "probs":
        return dict(op=op, B=B, N=N, V=V, dtype=rng.choice(["fp16", "bf16", "fp32"]), temp=rng.choice(["one", "mixed"]),
                    ragged=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 3]))
    return dict(op=op, B=B, N=N, V=V, shape=rng.choice(["chain", "tree"]), draft=rng.choice(["sampled", "best"]),
                ragged=rng.random() < 0.5)


def _rows(case):
    """Tokens (drafts, rows) of each sequence: N, or fewer for some."""
    N = case["N"]
    return [N - (5 * i * N // 16) % N if case["ragged"] else N for i in range(case["B"])]


# ----------------------------------------------------------------- inputs ---

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    st = SimpleNamespace(case=case)
    st.n = torch.tensor(_rows(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
    {"rope": _prepare_rope, "probs": _prepare_probs, "verify": _prepare_verify}[case["op"]](st, gen, int(seed))
    return st


def _prepare_rope(st, gen, seed):
    c, dev = st.case, "cuda"
    B, N, H, Hq, D, rot = (c[k] for k in ("B", "N", "H", "Hq", "D", "rot"))
    dtype = TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def projection(heads):
        out = torch.empty((B, N, heads, D), dtype=dtype, device=dev)
        for b in range(B):
            out[b] = normal(N, heads, D)
        return out

    if c["layout"] == "fused":      # one projection's output: queries, keys and values of a token side by side
        st.qkv = projection(Hq + 2 * H)
        st.q_in, st.k_in, st.v_in = st.qkv[:, :, :Hq], st.qkv[:, :, Hq:Hq + H], st.qkv[:, :, Hq + H:]
    else:
        st.q_in, st.k_in, st.v_in = projection(Hq), projection(H), projection(H)
    hot = 1 + 4 * torch.rand(D, generator=gen, device=dev)
    st.q_weight, st.k_weight = (1 + 0.2 * normal(D), hot) if c["norm"] else (None, None)
    st.eps = 1e-6
    st.inv_freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(dev)
    st.base = st.pos = st.axis = None
    if c["place"] in ("next", "tree"):   # after the cached tokens of each sequence
        st.base = torch.randint(0, 32768, (B,), generator=gen, device=dev, dtype=torch.int32)
    if c["place"] == "tree":             # each node one deeper than a parent of lower index
        g = np.random.default_rng(seed)
        depth = np.zeros((B, N), dtype=np.int32)
        for i in range(1, N):
            parent = g.integers(max(0, i - 6), i, size=B)
            depth[:, i] = depth[np.arange(B), parent] + 1
        st.pos = torch.from_numpy(depth).to(dev)
    if c["place"] == "axes":             # frames of 16 rows and columns: time, height, width
        i = torch.arange(N, device=dev, dtype=torch.int32)
        st.pos = torch.stack([i // 256, i // 16 % 16, i % 16]).view(3, 1, N).expand(3, B, N).contiguous()
        st.base = torch.randint(0, 4096, (B,), generator=gen, device=dev, dtype=torch.int32)
        st.axis = (torch.arange(rot // 2, device=dev) * 3 // max(1, rot // 2)).int()

    def out(heads):
        return torch.zeros((B, heads, N, D), dtype=torch.float16, device=dev)

    st.q, st.k, st.v = out(Hq), out(H), out(H)
    if own:
        from kivi_bit_kv_gb300 import KiviCache
        # the layer's cache; its codec and capacity play no part here
        st.cache = KiviCache(B, H, D, 2, 2, 32, 32, 32, device=dev)


def _prepare_probs(st, gen, seed):
    c, dev = st.case, "cuda"
    B, N, V = c["B"], c["N"], c["V"]
    ld = V + c["pad"]
    rows = torch.empty((B, N, ld), dtype=TYPES[c["dtype"]], device=dev)
    for b in range(B):
        rows[b] = 2.5 * torch.randn((N, ld), generator=gen, device=dev)
    st.logits = rows[..., :V]
    # a row whose grammar allows a few tokens only, now and then
    few = torch.rand((B, N, 1), generator=gen, device=dev) < 0.1
    for b in range(B):
        st.logits[b].masked_fill_(few[b] & (torch.rand((1, V), generator=gen, device=dev) < 0.99), -math.inf)
    st.temperature = None
    if c["temp"] == "mixed":
        t = 0.3 + 1.2 * torch.rand((B,), generator=gen, device=dev)
        st.temperature = torch.where(torch.arange(B, device=dev) % 4 == 3, 0.0, t)
    st.probs = torch.zeros((B, N, V), device=dev)


def _prepare_verify(st, gen, seed):
    c, dev = st.case, "cuda"
    B, N, V = c["B"], c["N"], c["V"]
    g = np.random.default_rng(seed)
    parent = np.zeros((B, N), dtype=np.int32)
    for i in range(1, N):
        parent[:, i] = i - 1 if c["shape"] == "chain" else g.integers(max(0, i - 4), i, size=B)
    parent[:, 0] = -1
    st.parent = torch.from_numpy(parent).to(dev)
    up = st.parent.long().clamp(min=0)
    st.u = torch.rand((B, N), generator=gen, device=dev)
    st.target = torch.empty((B, N, V), device=dev)
    st.draft = torch.empty((B, N, V), device=dev) if c["draft"] == "sampled" else None
    st.tokens = torch.zeros((B, N), dtype=torch.int32, device=dev)
    # the how-manieth child of its parent a node is
    rank = torch.from_numpy(np.array([[sum(parent[b, :i] == parent[b, i]) for i in range(N)] for b in range(B)])).to(dev)
    for b in range(B):
        z = 2.5 * torch.randn((N, V), generator=gen, device=dev)
        st.target[b] = torch.softmax(z, -1)
        near = torch.softmax(z + 0.5 * torch.randn((N, V), generator=gen, device=dev), -1)
        if b % 4 == 3:              # a sequence that decodes greedily
            st.target[b] = torch.nn.functional.one_hot(z.argmax(-1), V).float()
        if c["draft"] == "sampled":
            st.draft[b] = near
            race = torch.empty((N, V), device=dev).exponential_(generator=gen)
            st.tokens[b] = (near[up[b]] / race).argmax(-1).int()
        else:
            best = near[up[b]].topk(min(V, N), -1).indices
            st.tokens[b] = best.gather(1, rank[b].clamp(max=min(V, N) - 1).view(N, 1)).view(N).int()
    st.path = torch.zeros((B, N), dtype=torch.int32, device=dev)
    st.counts = torch.zeros((B,), dtype=torch.int32, device=dev)
    st.next = torch.zeros((B,), dtype=torch.int32, device=dev)


# ------------------------------------------------------------ plain forms ---

def _rope(st):
    c = st.case
    B, N, D, rot = (c[k] for k in ("B", "N", "D", "rot"))
    dev = st.q.device
    i = torch.arange(N, device=dev)
    # positions [axes, B, N], angles [B, N, rot/2] in 64 bits: a far position's lose too much in 32
    pos = i.view(1, 1, N).expand(1, B, N) if st.pos is None else st.pos.view(-1, B, N)
    if st.base is not None:
        pos = pos + st.base.view(1, B, 1)
    axis = torch.zeros(rot // 2, dtype=torch.long, device=dev) if st.axis is None else st.axis.long()
    angle = pos[axis].permute(1, 2, 0).double() * st.inv_freq.double()
    cos, sin = angle.cos().float().unsqueeze(2), angle.sin().float().unsqueeze(2)     # [B, N, 1, rot/2]
    here = None if st.n is None else (i < st.n.view(B, 1)).view(B, 1, N, 1)

    def heads(x, weight, turn):
        y = x.float()
        if weight is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + st.eps) * weight
        if turn and rot:
            if c["pairs"] == "half":
                a, b = y[..., :rot // 2], y[..., rot // 2:rot]
                y = torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], -1)
            else:
                a, b = y[..., 0:rot:2], y[..., 1:rot:2]
                y = torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), y[..., rot:]], -1)
        y = y.to(torch.float16).transpose(1, 2)
        return y.contiguous() if here is None else torch.where(here, y, 0.0)

    return {"q": heads(st.q_in, st.q_weight, True), "k": heads(st.k_in, st.k_weight, True),
            "v": heads(st.v_in, None, False)}


def _probs(st):
    B, N, V = st.logits.shape
    x = st.logits.float()
    m = x.amax(-1, keepdim=True)
    if st.temperature is None:
        e = torch.exp(x - m)
    else:
        t = st.temperature.view(B, 1, 1)
        e = torch.exp((x - m) / torch.where(t > 0, t, 1.0))
    p = e / e.sum(-1, keepdim=True)
    if st.temperature is not None:       # temperature 0: all on the first of the largest
        j = torch.arange(V, device=x.device)
        first = torch.where(x == m, j, V).amin(-1, keepdim=True)
        p = torch.where(t > 0, p, (j == first).float())
    if st.n is not None:
        p = torch.where((torch.arange(N, device=x.device) < st.n.view(B, 1)).unsqueeze(-1), p, 0.0)
    return p


def _weights(r):
    """Probabilities as multiples of 2^-42, so that their sums are exact in any order."""
    return torch.round(r.double() * ONE).long()


def _inverse(z):
    """2^42 / z in fp32 (0 for 0)."""
    return torch.where(z > 0, ONE / torch.where(z > 0, z, 1).double(), 0.0).float()


def _verify(st):
    """All sequences side by side.  A node has a higher index than its parent
    and its elder siblings, so one walk over the nodes is the walk down the
    tree: a node is tested if its parent is the last accepted one."""
    B, N, V = st.target.shape
    dev, rows = st.u.device, torch.arange(B, device=st.u.device)
    n = torch.full((B,), N, device=dev) if st.n is None else st.n.clamp(0, N)
    tok, par = st.tokens.long(), st.parent.long()
    cur = torch.zeros(B, dtype=torch.long, device=dev)
    rho = st.target[:, 0].clamp(0, 1)                # residual before its scale inv
    inv = torch.ones(B, device=dev)
    z = _weights(rho).sum(-1)
    count = (n > 0).int()
    path = torch.full((B, N), -1, dtype=torch.int32, device=dev)
    path[:, 0] = torch.where(n > 0, 0, -1)
    for i in range(1, N):
        x = tok[:, i]
        fits = (par[:, i] == cur) & (x >= 0) & (x < V) & (i < n)
        x = x.clamp(0, V - 1)
        there = rho[rows, x] * inv
        if st.draft is None:
            ok = fits & (st.u[:, i] < there)
            w = torch.where(fits & ~ok, _weights(rho[rows, x]), 0)
            z = z - w
            rho[rows, x] = torch.where(fits & ~ok, 0.0, rho[rows, x])
            inv = torch.where(fits & ~ok, _inverse(z), inv)
        else:
            q = st.draft[rows, cur].clamp(0, 1)
            ok = fits & (st.u[:, i] * q[rows, x] < there)
            no = fits & ~ok
            rho = torch.where(no.view(B, 1), (rho * inv.view(B, 1) - q).clamp(min=0), rho)
            z = torch.where(no, _weights(rho).sum(-1), z)
            inv = torch.where(no, _inverse(z), inv)
        cur = torch.where(ok, i, cur)
        rho = torch.where(ok.view(B, 1), st.target[:, i].clamp(0, 1), rho)
        z = torch.where(ok, _weights(rho).sum(-1), z)
        inv = torch.where(ok, 1.0, inv)
        path.scatter_(1, torch.where(ok, count, 0).long().view(B, 1), torch.where(ok, i, path[:, 0]).int().view(B, 1))
        count = count + ok.int()
    # nothing left of the residual: the node's own distribution
    rho = torch.where((z > 0).view(B, 1), rho, st.target[rows, cur].clamp(0, 1))
    cum = _weights(rho).cumsum(-1)
    total = cum[:, -1]
    draw_ = (st.u[:, 0].double() * 2.0 ** 32).floor().clamp(0, 2.0 ** 32 - 1).long()
    hi, lo = total >> 31, total & (2 ** 31 - 1)
    t = (hi * draw_ + ((lo * draw_) >> 31)) >> 1     # floor(total draw_ / 2^32)
    nxt = (cum <= t.view(B, 1)).sum(-1)
    nxt = torch.where((total > 0) & (n > 0), nxt, -1).int()
    return {"path": path, "counts": count, "next": nxt}


# -------------------------------------------------------------------- run ---

def run(st):
    op = st.case["op"]
    if not own:
        return {"rope": _rope, "probs": _probs, "verify": _verify}[op](st)
    from kivi_bit_kv_gb300 import abi
    if op == "rope":
        abi.kivi_norm_rope(st.cache, st.q_in, st.k_in, st.v_in, st.q, st.k, st.v, st.inv_freq, pos=st.pos, base=st.base,
                           axis=st.axis, interleaved=st.case["pairs"] == "next", q_weight=st.q_weight,
                           k_weight=st.k_weight, eps=st.eps, n_tok=st.n)
        return {"q": st.q, "k": st.k, "v": st.v}
    if op == "probs":
        abi.kivi_token_probs(st.logits, st.probs, temperature=st.temperature, n_rows=st.n)
        return st.probs
    abi.kivi_verify_tree(st.tokens, st.parent, st.u, st.target, st.draft, st.path, st.counts, st.next, n_draft=st.n)
    return {"path": st.path, "counts": st.counts, "next": st.next}


# ------------------------------------------------------------------- work ---

def work(case):
    rows = sum(_rows(case))
    if case["op"] == "rope":
        heads, D = case["Hq"] + 2 * case["H"], case["D"]
        size = 4 if case["dtype"] == "fp32" else 2
        turned = (case["Hq"] + case["H"]) * D
        # each value once in and once out; a square, two products and a pair's four for a rotated one
        return {"bytes": rows * (heads * D * (size + 2) + 4 * case["axes"]),
                "flops": rows * turned * (3 + (4 if case["norm"] else 0))}
    V = case["V"]
    if case["op"] == "probs":
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": rows * V * (size + 4), "flops": 5 * rows * V}
    # one row of the target's probabilities, and of the draft's where they matter, for each sequence; the rest of the
    # rows is read at single values only
    B = case["B"]
    kinds = 2 if case["draft"] == "sampled" else 1
    return {"bytes": kinds * 4 * B * V + rows * (16 + 4 * kinds), "flops": (kinds + 1) * B * V}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "probs": _exact_probs, "verify": _exact_verify}[case["op"]](st)


def _exact_rope(st):
    c = st.case
    B, N, H, Hq, D, rot = (c[k] for k in ("B", "N", "H", "Hq", "D", "rot"))
    dev = st.q.device
    out = {k: torch.zeros((B, h, N, D), dtype=torch.float64, device=dev) for k, h in (("q", Hq), ("k", H), ("v", H))}
    first = torch.arange(rot // 2, device=dev) * (2 if c["pairs"] == "next" else 1)
    second = first + (1 if c["pairs"] == "next" else rot // 2)
    for b, n in enumerate(_rows(c)):
        at = torch.zeros((N, rot // 2), dtype=torch.float64, device=dev)
        for j in range(rot // 2):
            a = 0 if st.axis is None else int(st.axis[j])
            p = torch.arange(N, device=dev) if st.pos is None else st.pos.reshape(-1, B, N)[a, b]
            at[:, j] = p.double() + (0 if st.base is None else int(st.base[b]))
        turn = torch.polar(torch.ones_like(at), at * st.inv_freq.double())       # e^(i angle)
        for name, src, w in (("q", st.q_in, st.q_weight), ("k", st.k_in, st.k_weight), ("v", st.v_in, None)):
            x = src[b].double()
            if w is not None:
                x = x / ((x ** 2).sum(-1, keepdim=True) / D + st.eps).sqrt() * w.double()
            if name != "v" and rot:
                zz = torch.complex(x[..., first], x[..., second]) * turn.unsqueeze(1)
                x = x.index_copy(-1, first, zz.real).index_copy(-1, second, zz.imag)
            out[name][b, :, :n] = x.permute(1, 0, 2)[:, :n]
    return out


def _exact_probs(st):
    B, N, V = st.logits.shape
    out = torch.zeros((B, N, V), dtype=torch.float64, device=st.probs.device)
    for b, n in enumerate(_rows(st.case)):
        t = 1.0 if st.temperature is None else float(st.temperature[b])
        for i in range(n):
            x = st.logits[b, i].double()
            if t > 0:
                out[b, i] = torch.softmax(x / t, 0)
            else:
                out[b, i, int((x == x.max()).nonzero()[0])] = 1.0
    return out


def _exact_verify(st):
    """Sequence by sequence down the tree, with whole numbers for the sums."""
    c = st.case
    B, N, V = c["B"], c["N"], c["V"]
    tok, par, u = st.tokens.cpu().numpy(), st.parent.cpu().numpy(), st.u.cpu().numpy()
    path, counts, nxt = np.full((B, N), -1, np.int32), np.zeros(B, np.int32), np.full(B, -1, np.int32)
    f = np.float32

    def row(t, b, i):
        return np.clip(t[b, i].cpu().numpy(), f(0), f(1))

    def whole(r):
        return np.rint(r.astype(np.float64) * ONE).astype(np.int64)

    for b, n in enumerate(_rows(c)):
        node, path[b, 0], counts[b] = 0, 0, 1
        while True:
            left, scale = row(st.target, b, node), f(1)
            q = None if st.draft is None else row(st.draft, b, node)
            taken = None
            for i in range(node + 1, n):
                if par[b, i] != node or not 0 <= tok[b, i] < V:
                    continue
                x = tok[b, i]
                if u[b, i] * (f(1) if q is None else q[x]) < left[x] * scale:
                    taken = i
                    break
                if q is None:
                    left[x] = 0
                else:
                    left = np.maximum(left * scale - q, f(0))
                z = int(whole(left).sum())
                scale = f(ONE / float(z)) if z else f(0)
            if taken is None:
                break
            node = taken
            path[b, counts[b]] = node
            counts[b] += 1
        w = whole(left)
        if not w.any():
            w = whole(row(st.target, b, node))
        total = int(w.sum())
        if total:
            t = total * min(int(float(u[b, 0]) * 2.0 ** 32), 2 ** 32 - 1) >> 32
            nxt[b] = int(np.searchsorted(np.cumsum(w), t, side="right"))
    return {"path": path, "counts": counts, "next": nxt}
