"""The operators that read and extend a quantized cache during speculative and
sparse decoding, as measurable cases.

    select   the cached groups a query may attend, chosen by an upper bound of
             their logits (kivi_block_select)
    sparse   decode attention over the chosen groups and the fp16 residual
             (kivi_sparse_attention)
    tree     attention of a tree of drafted tokens over the cache
             (kivi_tree_attention)
    append   the accepted path of a tree appended to the cache, with group
             flushes (kivi_append_path)

With ``own`` false every operator runs in its plain form (elementary torch
operations on the cache's tensors); with ``own`` true the library's entry
points run on the same tensors.
"""
import math
from types import SimpleNamespace

import torch

own = False

WORD = 64  # draft tokens per word of a tree mask


# ------------------------------------------------------------------ cases ---

def listed():
    tiny = dict(B=1, H=4, Hq=4, D=64, bits_k=4, bits_v=4, G=32, R=32, T=256, lo=256)
    gqa = dict(B=4, H=8, Hq=32, D=128, bits_k=2, bits_v=2, G=32, R=128, T=32768, lo=32768)
    ragged = dict(B=64, H=32, Hq=32, D=128, bits_k=2, bits_v=2, G=32, R=128, T=8192, lo=1024)
    layer = dict(B=8, H=32, Hq=32, D=128, bits_k=2, bits_v=2, G=32, R=128, T=4096, lo=4096)
    store = dict(B=32, H=32, Hq=32, D=128, bits_k=4, bits_v=4, G=32, R=0, T=2065, lo=2065)
    return [
        # one short sequence, where only latency counts
        dict(name="select_tiny", op="select", keep=4, N=1, P=1, **tiny),
        # four long grouped-query contexts: 1/16 of each is kept
        dict(name="select_gqa", op="select", keep=64, N=1, P=1, **gqa),
        # a full serving batch of ragged sequences
        dict(name="select_ragged", op="select", keep=32, N=1, P=1, **ragged),
        dict(name="sparse_tiny", op="sparse", keep=4, N=1, P=1, **tiny),
        # 2048 of 32768 tokens and the residual, four query heads a KV head
        dict(name="sparse_gqa", op="sparse", keep=64, N=1, P=1, **gqa),
        # 1024 tokens of every sequence of the batch and its residual
        dict(name="sparse_ragged", op="sparse", keep=32, N=1, P=1, **ragged),
        dict(name="tree_tiny", op="tree", keep=1, N=6, P=1, **tiny),
        # a 16-token draft tree verified over a layer of eight sequences
        dict(name="tree_layer", op="tree", keep=1, N=16, P=1, **layer),
        # 32 drafts x 4 heads: 128 query rows share each KV head's cache
        dict(name="tree_gqa", op="tree", keep=1, N=32, P=1, **gqa),
        # eight drafts after a stored int4 prefix, all layers of one model
        dict(name="tree_store", op="tree", keep=1, N=8, P=1, **store),
        dict(name="append_tiny", op="append", keep=1, N=6, P=4, **tiny),
        # the serving batch after a verification: 0 to 8 tokens accepted each
        dict(name="append_ragged", op="append", keep=1, N=16, P=8, **dict(ragged, T=2048)),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["select", "sparse", "tree", "append"])
    D = rng.choice([64, 128, 128, 256])
    G = rng.choice([g for g in (32, 32, 64, 128) if D % g == 0])
    R = G * rng.choice([0, 1, 2, 4])
    gq = rng.choice([1, 1, 2, 4, 7, 8])
    H = log_int(1, 32)
    T = log_int(1, 32768 if op != "append" else 2048)
    if op == "select":
        T = max(T, R + G)                      # at least one quantized group to choose from
    N = log_int(1, 64)
    most = (1 << 27) // (H * T * D)            # tokens x channels of the cache
    if op == "tree":
        most = min(most, (60 * 10 ** 9) // (4 * H * gq * N * T * D))
    B = log_int(1, max(1, min(48, most)))
    lo = T if rng.random() < 0.4 else rng.randint(0, T)
    P = rng.randint(1, min(N, 16))
    keep = log_int(1, max(1, T // G))
    return dict(op=op, B=B, H=H, Hq=H * gq, D=D, bits_k=rng.choice([2, 2, 4, 8]),
                bits_v=rng.choice([2, 2, 4, 8]), G=G, R=R, T=T, lo=lo, N=N, P=P, keep=keep)


def _lens(case):
    """Tokens of each sequence, spread over [lo, T] (T for a single one)."""
    B, lo, T = case["B"], case["lo"], case["T"]
    return [T if B == 1 else lo + (T - lo) * i // (B - 1) for i in range(B)]


def _drafts(case):
    """Drafted tokens of each sequence: every one drafts N, but each fourth fewer."""
    N = case["N"]
    return [N if i % 4 != 3 else max(1, N - 1 - i % N) for i in range(case["B"])]


def _accepted(case):
    """Tokens each sequence accepts, 0 .. P."""
    return [(3 * i + case["P"]) % (case["P"] + 1) for i in range(case["B"])]


def _quantized(n, G, R):
    return max(0, (n - R) // G * G)


def _tmax(case):
    """Capacity: the tokens, one path and room for the groups it flushes."""
    return (case["T"] + case["P"] + case["R"] + 2 * case["G"] + case["G"] - 1) // case["G"] * case["G"]


# ----------------------------------------------------------------- inputs ---

def _pack(codes, bits, dim):
    """int codes packed little-endian along dim into int32 words."""
    P = 32 // bits
    shape = list(codes.shape)
    shape[dim:dim + 1] = [shape[dim] // P, P]
    sh = [1] * len(shape)
    sh[dim + 1] = P
    shifts = (torch.arange(P, device=codes.device) * bits).view(sh)
    return (codes.long().view(shape) << shifts).sum(dim + 1).to(torch.int32)


def _quantize(x, bits, dim):
    """(codes, scale, zero) of fp32 x with statistics over dim (kept)."""
    M = (1 << bits) - 1
    mn, mx = x.amin(dim, keepdim=True) + 0.0, x.amax(dim, keepdim=True) + 0.0
    scale = (mx - mn) / torch.full_like(mx, M)          # a quotient: a Python divisor would become a product
    code = torch.round((x - mn) / torch.where(scale == 0, 1.0, scale)).clamp(0, M)
    return torch.where(scale == 0, 0.0, code).int(), scale, mn


def prepare(case, seed):
    B, H, Hq, D, G, R = (case[k] for k in ("B", "H", "Hq", "D", "G", "R"))
    bk, bv, N, P, keep = (case[k] for k in ("bits_k", "bits_v", "N", "P", "keep"))
    Tm, RG, dev = _tmax(case), R + G, "cuda"
    lens = _lens(case)
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    st = SimpleNamespace(case=case, sm=D ** -0.5)
    if own:
        from kivi_bit_kv_gb300 import KiviCache
        cache = KiviCache(B, H, D, bk, bv, G, R, Tm, device=dev)
    else:
        def zeros(*shape, dtype):
            return torch.zeros(shape, dtype=dtype, device=dev)
        cache = SimpleNamespace(
            kq=zeros(B, H, Tm * bk // 32, D, dtype=torch.int32),
            kscale=zeros(B, H, Tm // G, D, dtype=torch.float32),
            kzero=zeros(B, H, Tm // G, D, dtype=torch.float32),
            vq=zeros(B, H, Tm, D * bv // 32, dtype=torch.int32),
            vscale=zeros(B, H, Tm, D // G, dtype=torch.float32),
            vzero=zeros(B, H, Tm, D // G, dtype=torch.float32),
            kres=zeros(B, H, RG, D, dtype=torch.float16),
            vres=zeros(B, H, RG, D, dtype=torch.float16),
            lens=zeros(B, dtype=torch.int32))
    st.cache = cache
    # keys: N(0, 1) with a few outlier channels per head, the reason keys are
    # quantized per channel; values N(0, 1)
    amp = torch.ones(H, 1, D, device=dev)
    hot = max(1, round(0.04 * D))
    pick = torch.rand(H, 1, D, generator=gen, device=dev).topk(hot, -1).indices
    amp.scatter_(2, pick, 5 + 15 * torch.rand(H, 1, hot, generator=gen, device=dev))
    for b, n in enumerate(lens):
        Tq = _quantized(n, G, R)
        K, V = (normal(H, n, D) * amp).half(), normal(H, n, D).half()
        if Tq:
            code, sc, ze = _quantize(K[:, :Tq].float().view(H, Tq // G, G, D), bk, 2)
            cache.kq[b, :, :Tq * bk // 32] = _pack(code.view(H, Tq, D), bk, 1)
            cache.kscale[b, :, :Tq // G], cache.kzero[b, :, :Tq // G] = sc[:, :, 0], ze[:, :, 0]
            code, sc, ze = _quantize(V[:, :Tq].float().view(H, Tq, D // G, G), bv, 3)
            cache.vq[b, :, :Tq] = _pack(code.view(H, Tq, D), bv, 2)
            cache.vscale[b, :, :Tq], cache.vzero[b, :, :Tq] = sc[..., 0], ze[..., 0]
        slots = torch.arange(Tq, n, device=dev) % RG
        cache.kres[b, :, slots], cache.vres[b, :, slots] = K[:, Tq:], V[:, Tq:]
    st.lens0 = torch.tensor(lens, dtype=torch.int32, device=dev)
    cache.lens.copy_(st.lens0)

    if case["op"] in ("select", "sparse"):
        st.q = normal(B, Hq, D).half()
        st.blocks = torch.zeros(B, H, keep, dtype=torch.int32, device=dev)
        st.scores = torch.zeros(B, H, Tm // G, device=dev)
        if case["op"] == "sparse":
            st.blocks.copy_(_select(st)["blocks"])
            st.out = torch.zeros(B, Hq, D, device=dev)
    else:
        st.k, st.v = (normal(B, H, N, D) * amp).half(), normal(B, H, N, D).half()
    if case["op"] == "tree":
        st.q = normal(B, Hq, N, D).half()
        st.n_draft = torch.tensor(_drafts(case), dtype=torch.int32, device=dev)
        st.mask = _tree_mask(B, N, seed).to(dev)
        st.out = torch.zeros(B, Hq, N, D, device=dev)
    if case["op"] == "append":
        # the accepted path: P increasing nodes of the tree
        order = torch.rand(B, N, generator=gen, device=dev).topk(P, -1).indices
        st.path = order.sort(-1).values.int()
        st.counts = torch.tensor(_accepted(case), dtype=torch.int32, device=dev)
        st.status = torch.zeros(1, dtype=torch.int32, device=dev)
    if own and case["op"] in ("sparse", "tree"):
        st.ws = cache.attend_workspace(Hq, N if case["op"] == "tree" else 1)
    return st


def _tree_mask(B, N, seed):
    """int64 [B, N, ceil(N/64)]: bit j % 64 of word j / 64 of row i is set
    where token i attends token j -- itself and its ancestors in a random tree."""
    import random
    r = random.Random(int(seed) * 31 + N)
    W = (N + WORD - 1) // WORD
    rows = []
    for _ in range(B):
        bits = []
        for i in range(N):
            parent = r.randint(max(-1, i - 6), i - 1)
            bits.append((1 << i) | (bits[parent] if parent >= 0 else 0))
        rows.append([[((m >> (64 * w)) & (2 ** 64 - 1)) - (2 ** 64 if (m >> (64 * w + 63)) & 1 else 0)
                      for w in range(W)] for m in bits])
    return torch.tensor(rows, dtype=torch.int64)


# ------------------------------------------------------------ plain forms ---

def _unpack(words, bits, dim):
    P = 32 // bits
    sh = [1] * (words.dim() + 1)
    sh[dim + 1] = P
    shifts = (torch.arange(P, device=words.device, dtype=torch.int32) * bits).view(sh)
    shape = list(words.shape)
    shape[dim] *= P
    return ((words.unsqueeze(dim + 1) >> shifts) & ((1 << bits) - 1)).reshape(shape)


def _hat(code, scale, zero):
    """fp16 code * scale + zero; the product and sum in 64 bits, because the
    value is next to a rounding border of fp16 wherever fp32 would round twice."""
    return (code * scale.double() + zero.double()).float().half()


def _dense(st, which):
    """fp32 [B, H, Tmax, D] keys or values as kivi_dequant defines them
    (residual tokens from the ring; anything past a sequence's end is masked
    by the caller)."""
    c, x = st.case, st.cache
    B, H, D, G, R = (c[k] for k in ("B", "H", "D", "G", "R"))
    Tm = x.vq.shape[2]
    if which == 0:
        code = _unpack(x.kq, c["bits_k"], 2).view(B, H, Tm // G, G, D)
        hat = _hat(code, x.kscale.unsqueeze(3), x.kzero.unsqueeze(3))
    else:
        code = _unpack(x.vq, c["bits_v"], 3).view(B, H, Tm, D // G, G)
        hat = _hat(code, x.vscale.unsqueeze(4), x.vzero.unsqueeze(4))
    t = torch.arange(Tm, device=hat.device)
    res = (x.kres if which == 0 else x.vres)[:, :, t % (R + G)]
    Tq = ((x.lens.long() - R).clamp(min=0) // G * G).view(B, 1, 1, 1)
    return torch.where(t.view(1, 1, Tm, 1) < Tq, hat.view(B, H, Tm, D), res).float()


def _attend(q, K, V, seen, sm):
    """softmax over the seen tokens (0 where none is) times V; q [B, H, M, D],
    K, V [B, H, T, D], seen broadcastable to [B, H, M, T]."""
    s = (q @ K.transpose(-1, -2) * sm).masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    return torch.where(l > 0, (p @ V) / torch.where(l > 0, l, 1.0), 0.0)


def _select(st):
    """Scores and kept groups.  A group's score is the largest, over the query
    heads of its KV head, of sum_d max(q_d lo_d, q_d hi_d) -- an upper bound of
    q . k for every key of the group, lo = zero and hi = zero + M scale being
    its smallest and largest key.  The bound is fp32 with its sum taken
    pairwise over neighbouring channels, so that the kept groups are the same
    bit for bit wherever it is computed."""
    c, x = st.case, st.cache
    B, H, D, G, R, keep = (c[k] for k in ("B", "H", "D", "G", "R", "keep"))
    lo = x.kzero.unsqueeze(2)
    hi = x.kscale.unsqueeze(2) * float((1 << c["bits_k"]) - 1)
    hi = lo + hi
    q = st.q.float().view(B, H, -1, 1, D)
    v = torch.maximum(q * lo, q * hi)
    while v.shape[-1] > 1:
        v = v[..., 0::2] + v[..., 1::2]
    nb = ((x.lens.long() - R).clamp(min=0) // G).view(B, 1, 1)
    g = torch.arange(lo.shape[3], device=lo.device).view(1, 1, -1)
    score = v[..., 0].amax(2)
    ranked = torch.sort(score.masked_fill(g >= nb, -math.inf), dim=-1, descending=True, stable=True).indices
    first = ranked[..., :keep]
    none = torch.iinfo(torch.int32).max
    first = torch.where(torch.arange(first.shape[-1], device=g.device) < nb, first, none).sort(-1).values
    blocks = torch.full((B, H, keep), -1, dtype=torch.int32, device=g.device)
    blocks[..., :first.shape[-1]] = torch.where(first == none, -1, first).int()
    return {"blocks": blocks, "scores": score.masked_fill(g >= nb, 0.0)}


def _sparse(st):
    c, x = st.case, st.cache
    B, H, Hq, D, G, R, keep = (c[k] for k in ("B", "H", "Hq", "D", "G", "R", "keep"))
    Tm, RG, gq = x.vq.shape[2], R + G, Hq // H
    nb = ((x.lens.long() - R).clamp(min=0) // G).view(B, 1, 1)
    blk = st.blocks.long()
    listed_ = (torch.arange(keep, device=blk.device) < nb) & (blk >= 0) & (blk < nb)
    blk = torch.where(listed_, blk, 0)

    def groups(t, per):  # the listed groups of a buffer with `per` rows a group
        t = t.view(B, H, Tm // G, per, t.shape[-1])
        return t.gather(2, blk.view(B, H, keep, 1, 1).expand(-1, -1, -1, per, t.shape[-1]))

    K = _hat(_unpack(groups(x.kq, G * c["bits_k"] // 32), c["bits_k"], 3),
             groups(x.kscale, 1), groups(x.kzero, 1)).view(B, H, keep * G, D)
    V = _hat(_unpack(groups(x.vq, G), c["bits_v"], 4).view(B, H, keep, G, D // G, G),
             groups(x.vscale, G).unsqueeze(-1), groups(x.vzero, G).unsqueeze(-1)).view(B, H, keep * G, D)
    tok = nb * G + torch.arange(RG, device=blk.device)             # residual tokens [B, 1, RG]
    slot = (tok % RG).view(B, 1, RG, 1).expand(-1, H, -1, D)
    K = torch.cat([K, x.kres.gather(2, slot)], 2).float()
    V = torch.cat([V, x.vres.gather(2, slot)], 2).float()
    seen = torch.cat([listed_.repeat_interleave(G, -1),
                      (tok < x.lens.view(B, 1, 1)).expand(-1, H, -1)], -1).unsqueeze(2)
    return _attend(st.q.float().view(B, H, gq, D), K, V, seen, st.sm).view(B, Hq, D)


def _tree(st):
    c, x = st.case, st.cache
    B, H, Hq, D, N = (c[k] for k in ("B", "H", "Hq", "D", "N"))
    gq, Tm = Hq // H, x.vq.shape[2]
    K = torch.cat([_dense(st, 0), st.k.float()], 2)
    V = torch.cat([_dense(st, 1), st.v.float()], 2)
    past = (torch.arange(Tm, device=K.device) < x.lens.view(B, 1, 1)).expand(-1, N, -1)
    j = torch.arange(N, device=K.device)
    drafts = ((st.mask[:, :, j // 64] >> (j % 64)) & 1).bool() & (j < st.n_draft.view(B, 1, 1))
    seen = torch.cat([past, drafts], -1).repeat(1, gq, 1).unsqueeze(1)   # [B, 1, gq N, Tm + N]
    V = V.masked_fill(~seen.any(2).unsqueeze(-1), 0.0)
    o = _attend(st.q.float().view(B, H, gq * N, D), K, V, seen, st.sm).view(B, Hq, N, D)
    return torch.where(j.view(1, 1, N, 1) < st.n_draft.view(B, 1, 1, 1), o, 0.0)


def _append(st):
    """The first counts[b] nodes of path[b] become tokens len .. of sequence b:
    into the ring, and each time the residual reaches R + G its oldest G tokens
    into the packed cache.  Returns the cache's updated buffers."""
    c, x = st.case, st.cache
    B, H, D, G, R, P = (c[k] for k in ("B", "H", "D", "G", "R", "P"))
    RG, Tm, dev = R + G, x.vq.shape[2], x.kq.device
    L = x.lens.long()
    n = torch.where(L + st.counts <= Tm, st.counts, 0).long()
    L2 = L + n
    Tq, Tq2 = (L - R).clamp(min=0) // G * G, (L2 - R).clamp(min=0) // G * G
    # tokens Tq .. of each sequence in order: the ring's, then the path's
    Lx = (RG + P + G - 1) // G * G
    t = Tq.view(B, 1) + torch.arange(Lx, device=dev)
    node = st.path.long().gather(1, (t - L.view(B, 1)).clamp(0, P - 1))
    # the newest token of every ring slot
    s = torch.arange(RG, device=dev)
    last = L2.view(B, 1) - 1 - (L2.view(B, 1) - 1 - s) % RG
    newest = st.path.long().gather(1, (last - L.view(B, 1)).clamp(0, P - 1))

    def take(src, idx):
        return src.gather(2, idx.view(B, 1, -1, 1).expand(-1, H, -1, D))

    flushed = torch.arange(Lx // G, device=dev) < ((Tq2 - Tq) // G).view(B, 1)   # [B, groups]

    def put(buf, new, per):  # new [B, H, groups, per, .] into the flushed groups of buf
        old = buf.view(B, H, Tm // G, per, buf.shape[-1])
        at = ((Tq // G).view(B, 1) + torch.arange(Lx // G, device=dev)).view(B, 1, -1, 1, 1).expand(new.shape)
        ok = flushed.view(B, 1, -1, 1, 1)
        at = at.clamp(max=Tm // G - 1)
        old.scatter_(2, at, torch.where(ok, new.view(at.shape), old.gather(2, at)))

    for which, (src, ring) in enumerate(((st.k, x.kres), (st.v, x.vres))):
        tok = torch.where((t < L.view(B, 1)).view(B, 1, -1, 1), take(ring, t % RG), take(src, node))
        tok = tok.float().view(B, H, Lx // G, G, D)
        if which == 0:
            code, sc, ze = _quantize(tok, c["bits_k"], 3)
            put(x.kq, _pack(code, c["bits_k"], 3), G * c["bits_k"] // 32)
            put(x.kscale, sc, 1)
            put(x.kzero, ze, 1)
        else:
            code, sc, ze = _quantize(tok.view(B, H, Lx // G, G, D // G, G), c["bits_v"], 5)
            put(x.vq, _pack(code.view(B, H, Lx // G, G, D), c["bits_v"], 4), G)
            put(x.vscale, sc.squeeze(-1), G)
            put(x.vzero, ze.squeeze(-1), G)
        ring.copy_(torch.where((last >= L.view(B, 1)).view(B, 1, RG, 1), take(src, newest), ring))
    x.lens.copy_(L2)


def _state(x):
    return {k: getattr(x, k) for k in ("kq", "kscale", "kzero", "vq", "vscale", "vzero", "kres", "vres", "lens")}


# -------------------------------------------------------------------- run ---

def run(st):
    op = st.case["op"]
    if op == "append":
        # the same step each time: the lengths go back to those before it
        st.cache.lens.copy_(st.lens0)
    if not own:
        if op == "append":
            _append(st)
            return _state(st.cache)
        return {"select": _select, "sparse": _sparse, "tree": _tree}[op](st)
    from kivi_bit_kv_gb300 import abi
    x = st.cache
    if op == "select":
        abi.kivi_block_select(x, st.q, st.blocks, st.scores)
        return {"blocks": st.blocks, "scores": st.scores}
    if op == "sparse":
        abi.kivi_sparse_attention(x, st.q, st.blocks, st.out, st.ws)
        return st.out
    if op == "tree":
        abi.kivi_tree_attention(x, st.q, st.k, st.v, st.mask, st.out, st.ws, n_draft=st.n_draft)
        return st.out
    abi.kivi_append_path(x, st.k, st.v, st.path, st.counts, st.status)
    return _state(x)


# ------------------------------------------------------------------- work ---

def work(case):
    B, H, Hq, D, G, R, N = (case[k] for k in ("B", "H", "Hq", "D", "G", "R", "N"))
    bk, bv, keep = case["bits_k"], case["bits_v"], case["keep"]
    group_k = G * D * bk // 8 + 8 * D                   # bytes of a group of G tokens: codes, statistics
    group_v = G * (D * bv // 8 + 8 * (D // G))
    nbytes = flops = 0
    for n, nd, acc in zip(_lens(case), _drafts(case), _accepted(case)):
        nb = _quantized(n, G, R) // G
        res = n - nb * G
        if case["op"] == "select":      # every group's statistics once; a product and a sum per channel
            nbytes += H * nb * (8 * D + 4) + H * keep * 4 + Hq * D * 2
            flops += 2 * Hq * nb * D
        elif case["op"] == "sparse":
            m = min(keep, nb)
            nbytes += H * (m * (group_k + group_v + 4) + res * D * 4) + Hq * D * 6
            flops += 4 * Hq * D * (m * G + res)
        elif case["op"] == "tree":
            nbytes += H * (nb * (group_k + group_v) + (res + nd) * D * 4) + Hq * nd * D * 6 + 8 * nd
            flops += 4 * Hq * nd * D * (n + 1)
        else:                           # the tokens once in and once out; flushed groups read and packed
            flushed = _quantized(n + acc, G, R) // G - nb
            nbytes += H * (acc * D * 8 + flushed * (G * D * 4 + group_k + group_v)) + 8
            flops += 8 * H * flushed * G * D
    return {"bytes": nbytes + 4 * B, "flops": flops}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    if case["B"] * case["H"] > 4096:
        return None
    st = prepare(case, seed)
    return {"select": _exact_select, "sparse": _exact_sparse, "tree": _exact_tree, "append": _exact_append}[case["op"]](st)


def _codes64(words, bits):
    """Codes of int32 words as float64, the word axis last and expanded."""
    w = words.long() & 0xFFFFFFFF
    return torch.stack([(w >> (bits * i)) % (1 << bits) for i in range(32 // bits)], -1).flatten(-2).double()


def _rows64(st, b, h, g=None):
    """The keys and values of one sequence and head in 64 bits: quantized
    groups g (all of them for None), then the residual."""
    c, x = st.case, st.cache
    G, R, D = c["G"], c["R"], c["D"]
    n = int(st.lens0[b])
    nb = _quantized(n, G, R) // G
    g = torch.arange(nb, device=x.kq.device) if g is None else g
    kw = x.kq[b, h].view(-1, G * c["bits_k"] // 32, D)[g]                     # [g, words, D]
    kc = _codes64(kw.transpose(1, 2), c["bits_k"]).transpose(1, 2)             # [g, G, D]
    K = kc * x.kscale[b, h, g].double().unsqueeze(1) + x.kzero[b, h, g].double().unsqueeze(1)
    vw = x.vq[b, h].view(-1, G, D * c["bits_v"] // 32)[g]
    vc = _codes64(vw, c["bits_v"]).view(len(g), G, D // G, G)
    vs = x.vscale[b, h].view(-1, G, D // G)[g].double().unsqueeze(3)
    vz = x.vzero[b, h].view(-1, G, D // G)[g].double().unsqueeze(3)
    V = vc * vs + vz
    slots = torch.arange(nb * G, n, device=K.device) % (R + G)
    K = torch.cat([K.reshape(-1, D).float().half(), x.kres[b, h, slots]])
    V = torch.cat([V.reshape(-1, D).float().half(), x.vres[b, h, slots]])
    return K.double(), V.double()


def _soft64(s, V):
    return torch.softmax(s, -1) @ V if s.shape[-1] else torch.zeros(s.shape[0], V.shape[1], dtype=torch.float64, device=V.device)


def _exact_select(st):
    c, x = st.case, st.cache
    q = st.q.double().view(c["B"], c["H"], -1, c["D"])
    out = torch.zeros(st.scores.shape, dtype=torch.float64, device=q.device)
    for b, n in enumerate(_lens(c)):
        nb = _quantized(n, c["G"], c["R"]) // c["G"]
        lo = x.kzero[b, :, :nb].double()
        hi = lo + x.kscale[b, :, :nb].double() * ((1 << c["bits_k"]) - 1)
        up = q[b].clamp(min=0) @ hi.transpose(1, 2) + q[b].clamp(max=0) @ lo.transpose(1, 2)
        out[b, :, :nb] = up.amax(1)
    return {"blocks": None, "scores": out}


def _exact_sparse(st):
    c = st.case
    gq = c["Hq"] // c["H"]
    out = torch.zeros(st.out.shape, dtype=torch.float64, device=st.q.device)
    for b in range(c["B"]):
        nb = _quantized(_lens(c)[b], c["G"], c["R"]) // c["G"]
        for h in range(c["H"]):
            g = st.blocks[b, h, :min(nb, c["keep"])].long()
            K, V = _rows64(st, b, h, g)
            q = st.q[b, h * gq:(h + 1) * gq].double()
            out[b, h * gq:(h + 1) * gq] = _soft64(q @ K.T * st.sm, V)
    return out


def _exact_tree(st):
    c = st.case
    gq, N = c["Hq"] // c["H"], c["N"]
    out = torch.zeros(st.out.shape, dtype=torch.float64, device=st.q.device)
    words = st.mask.cpu().tolist()
    for b in range(c["B"]):
        nd = _drafts(c)[b]
        see = torch.tensor([[(words[b][i][j // 64] >> (j % 64)) & 1 for j in range(nd)] for i in range(nd)],
                           dtype=torch.bool, device=out.device)
        for h in range(c["H"]):
            K, V = _rows64(st, b, h)
            K = torch.cat([K, st.k[b, h, :nd].double()])
            V = torch.cat([V, st.v[b, h, :nd].double()])
            s = st.q[b, h * gq:(h + 1) * gq, :nd].double() @ K.T * st.sm
            s[..., K.shape[0] - nd:].masked_fill_(~see, -math.inf)
            out[b, h * gq:(h + 1) * gq, :nd] = torch.softmax(s, -1) @ V
    return out


def _exact_append(st):
    c, x = st.case, st.cache
    G, R, D = c["G"], c["R"], c["D"]
    RG = R + G
    out = {k: getattr(x, k).double() for k in ("kscale", "kzero", "vscale", "vzero", "kres", "vres")}
    for b, (n, acc) in enumerate(zip(_lens(c), _accepted(c))):
        a, z = _quantized(n, G, R), _quantized(n + acc, G, R)
        nodes = st.path[b, :acc].long()
        slots = torch.arange(a, n, device=nodes.device) % RG
        K = torch.cat([x.kres[b][:, slots], st.k[b][:, nodes]], 1).double()
        V = torch.cat([x.vres[b][:, slots], st.v[b][:, nodes]], 1).double()
        for g in range(a // G, z // G):
            kk, vv = (y[:, (g * G - a):(g * G - a) + G] for y in (K, V))
            vv = vv.view(-1, G, D // G, G)
            out["kzero"][b, :, g], out["vzero"][b, :, g * G:g * G + G] = kk.amin(1), vv.amin(-1)
            out["kscale"][b, :, g] = (kk.amax(1) - kk.amin(1)) / ((1 << c["bits_k"]) - 1)
            out["vscale"][b, :, g * G:g * G + G] = (vv.amax(-1) - vv.amin(-1)) / ((1 << c["bits_v"]) - 1)
        for i in range(acc):
            out["kres"][b, :, (n + i) % RG] = st.k[b][:, nodes[i]].double()
            out["vres"][b, :, (n + i) % RG] = st.v[b][:, nodes[i]].double()
    return {k: out.get(k) for k in ("kq", "kscale", "kzero", "vq", "vscale", "vzero", "kres", "vres", "lens")}
