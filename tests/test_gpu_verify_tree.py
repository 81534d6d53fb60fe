"""kivi_verify_tree against its definition, value for value: paths, counts and
next tokens are whole numbers, the same on any implementation."""
import numpy as np
import pytest
import torch

import _step
from kivi_bit_kv_gb300 import abi

pytestmark = pytest.mark.gpu


def trees(rng, B, N, shape):
    parent = np.full((B, N), -1, np.int32)
    for i in range(1, N):
        parent[:, i] = {"chain": i - 1, "star": 0, "tree": rng.integers(max(0, i - 4), i, size=B)}[shape]
    return parent


def problem(seed, B, N, V, shape, kind, spread=2.0, near=0.5):
    """Rows of the target, drafts near it, and drafted tokens."""
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(B, N, V)) * spread
    target = np.exp(z - z.max(-1, keepdims=True))
    target = (target / target.sum(-1, keepdims=True)).astype(np.float32)
    z = z + rng.normal(size=(B, N, V)) * near
    draft = np.exp(z - z.max(-1, keepdims=True))
    draft = (draft / draft.sum(-1, keepdims=True)).astype(np.float32)
    parent = trees(rng, B, N, shape)
    tokens = np.zeros((B, N), np.int32)
    for b in range(B):
        rank = {}
        for i in range(1, N):
            row = draft[b, parent[b, i]].astype(np.float64)
            if kind == "sampled":
                tokens[b, i] = rng.choice(V, p=row / row.sum())
            else:
                r = rank[parent[b, i]] = rank.get(parent[b, i], -1) + 1
                tokens[b, i] = np.argsort(-row, kind="stable")[min(r, V - 1)]
    u = rng.random((B, N)).astype(np.float32)
    return tokens, parent, u, target, draft if kind == "sampled" else None


def run(dev, tokens, parent, u, target, draft, n=None, stream=None):
    B, N, V = target.shape
    t = [torch.from_numpy(np.ascontiguousarray(x)).to(dev) for x in (tokens, parent, u, target)]
    d = None if draft is None else torch.from_numpy(draft).to(dev)
    path = torch.full((B, N), 55, dtype=torch.int32, device=dev)
    counts, nxt = (torch.full((B,), 55, dtype=torch.int32, device=dev) for _ in range(2))
    nd = None if n is None else torch.tensor(n, dtype=torch.int32, device=dev)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    abi.kivi_verify_tree(*t, d, path, counts, nxt, n_draft=nd, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    return path.cpu().numpy(), counts.cpu().numpy(), nxt.cpu().numpy()


def compare(dev, tokens, parent, u, target, draft, n=None):
    path, counts, nxt = run(dev, tokens, parent, u, target, draft, n)
    B, N, V = target.shape
    for b in range(B):
        want, last = _step.verify(tokens[b], parent[b], u[b], target[b], None if draft is None else draft[b],
                                  None if n is None else n[b])
        assert counts[b] == len(want) and path[b].tolist() == want + [-1] * (N - len(want)), (b, path[b], want)
        assert nxt[b] == last, (b, nxt[b], last)
    return counts


@pytest.mark.parametrize("kind", ["sampled", "best"])
@pytest.mark.parametrize("shape", ["chain", "tree", "star"])
@pytest.mark.parametrize("B,N,V", [(1, 1, 1000), (7, 6, 33), (5, 12, 1000), (3, 9, 32000), (2, 5, 50001), (2, 40, 4099),
                                   (300, 3, 64), (1, 256, 2048), (2, 3, 262207)])
def test_against_the_definition(cuda, B, N, V, shape, kind):
    compare(cuda, *problem(B * 1000 + N, B, N, V, shape, kind, spread=2.0 if V < 5000 else 3.0))


def test_largest_vocabulary(cuda):
    compare(cuda, *problem(3, 1, 2, 1 << 20, "chain", "sampled", spread=1.0))


@pytest.mark.parametrize("V", [1, 2, 3, 5, 127, 129, 1023, 1025, 8191])
@pytest.mark.parametrize("kind", ["sampled", "best"])
def test_small_and_odd_vocabularies(cuda, V, kind):
    compare(cuda, *problem(40 + V, 9, 5, V, "tree", kind))


def test_offsets_past_32_bits(cuda):
    """Rows that begin past 2^31 elements, 2^33 bytes: 2.7e9 probabilities, of which
    the last sequence's are looked at."""
    B, N, V = 64, 41, 1 << 20
    tokens, parent, u, target, _ = problem(29, 1, N, 4099, "tree", "best")
    rows = torch.zeros((B, N, V), device=cuda)
    rows[B - 1, :, V - 4099:] = torch.from_numpy(target[0]).to(cuda)
    full = np.zeros((N, V), np.float32)
    full[:, V - 4099:] = target[0]
    ids = [torch.from_numpy(np.ascontiguousarray(np.broadcast_to(x, (B, N)))).to(cuda)
           for x in (tokens[0] + V - 4099, parent[0], u[0])]
    path = torch.zeros((B, N), dtype=torch.int32, device=cuda)
    counts, nxt = (torch.zeros(B, dtype=torch.int32, device=cuda) for _ in range(2))
    abi.kivi_verify_tree(*ids, rows, None, path, counts, nxt)
    want, last = _step.verify(tokens[0] + V - 4099, parent[0], u[0], full, None)
    assert path[B - 1].tolist() == want + [-1] * (N - len(want)) and int(nxt[B - 1]) == last
    assert int(counts[B - 1]) == len(want)
    assert counts[:B - 1].eq(1).all() and nxt[:B - 1].eq(-1).all()        # empty rows


@pytest.mark.parametrize("kind", ["sampled", "best"])
def test_ragged_trees(cuda, kind):
    p = problem(21, 8, 10, 777, "tree", kind)
    counts = compare(cuda, *p, n=[10, 0, 1, -5, 99, 4, 2, 7])
    assert counts[1] == counts[3] == 0 and counts[2] == 1


def test_all_accepted_and_none(cuda):
    tokens, parent, u, target, draft = problem(22, 6, 9, 500, "chain", "sampled")
    u[:3] = 0.0                                                  # 0 < p: every node is kept, the first token drawn last
    u[3:, 1:] = 1.0                                              # kept only where the target's is larger
    counts = compare(cuda, tokens, parent, u, target, draft)
    assert (counts[:3] == 9).all()
    same = target.copy()                                         # draft and target equal: all kept for u < 1
    u[:, 1:] = np.float32(1 - 2.0 ** -24)
    counts = compare(cuda, tokens, parent, u, target, same)


def test_residual_of_nothing(cuda):
    """A rejection where the draft is nowhere below the target leaves nothing: the
    next token comes from the target's row; an empty row gives -1."""
    V = 300
    target = np.zeros((4, 3, V), np.float32)
    target[0, 0, 7] = 0.25
    target[1, 0, [5, 250]] = 0.5
    draft = np.ones((4, 3, V), np.float32)
    target[2, 0, 3] = 1.0                                         # accepted, then an empty row
    tokens = np.array([[0, 7, 7], [0, 5, 250], [0, 3, 0], [0, 1, 2]], np.int32)
    parent = np.tile(np.array([-1, 0, 0], np.int32), (4, 1))
    parent[2] = [-1, 0, 1]
    for u0 in (0.0, 0.49999, 0.5, 0.999999):
        u = np.full((4, 3), 0.75, np.float32)
        u[:, 0] = u0
        for d in (draft, None):
            compare(cuda, tokens, parent, u, target, d)


@pytest.mark.parametrize("kind", ["sampled", "best"])
def test_bad_nodes_change_nothing(cuda, kind):
    """Parents of higher index, of none, tokens outside the vocabulary."""
    tokens, parent, u, target, draft = problem(23, 4, 8, 100, "tree", kind)
    parent[0, 2], parent[0, 3], parent[1, 1], parent[1, 5] = 2, 7, -1, -2 ** 31
    parent[3, 4] = 2 ** 31 - 1
    tokens[2, 1:4] = [-1, 100, 2 ** 31 - 1]
    tokens[3, 2] = -2 ** 31
    tokens[:, 0] = -9                                            # not read
    parent[:, 0] = 3
    compare(cuda, tokens, parent, u, target, draft)


def test_values_outside_zero_to_one(cuda):
    """NaN and negative probabilities count as 0, those above 1 as 1."""
    for kind in ("sampled", "best"):
        tokens, parent, u, target, draft = problem(24, 5, 7, 200, "tree", kind)
        for x in (target, draft):
            if x is not None:
                x[0, :, ::3], x[1, :, 1::3], x[2, :, 5], x[3, :, 9] = np.nan, -0.5, np.inf, -np.inf
                x[4] = np.nan
        u[0, 0], u[1, 0], u[2, 0], u[3, 0] = np.nan, 1.0, -1.0, 7.0
        compare(cuda, tokens, parent, u, target, draft)


def test_same_token_twice_among_siblings(cuda):
    for kind in ("sampled", "best"):
        tokens, parent, u, target, draft = problem(25, 64, 6, 12, "star", kind)
        tokens[:, 3], tokens[:, 5] = tokens[:, 2], tokens[:, 1]
        u[:, 1:] = np.maximum(u[:, 1:], np.float32(0.6))
        compare(cuda, tokens, parent, u, target, draft)


def test_tiny_probabilities(cuda):
    """Rows that sum to far less than 1 down to single multiples of 2^-42."""
    rng = np.random.default_rng(26)
    tokens, parent, u, target, draft = problem(26, 12, 6, 900, "star", "sampled")
    for b in range(12):
        target[b] *= np.float32(2.0 ** -(3 * b))
        draft[b] *= np.float32(2.0 ** -(3 * b + b % 3))
    compare(cuda, tokens, parent, u, target, draft)
    compare(cuda, tokens, parent, u, target, None)


def test_every_token_can_be_drawn(cuda):
    """u_0 at each border between two tokens' shares of a flat row, and just below."""
    V = 97
    target = np.full((1, 1, V), 1 / 128, np.float32)
    u = np.repeat(np.arange(V, dtype=np.float64) / V, 2)
    u[1::2] = np.nextafter(u[1::2].astype(np.float32), np.float32(-1))
    B = len(u)
    compare(cuda, np.zeros((B, 1), np.int32), np.zeros((B, 1), np.int32), u.astype(np.float32).reshape(B, 1),
            np.repeat(target, B, 0), None)


@pytest.mark.parametrize("kind", ["sampled", "best"])
def test_tokens_follow_the_target(cuda, kind):
    """40000 sequences of one small problem: the first new token has the target's
    distribution.  A cell is off by over 6 standard deviations with a chance below
    2e-9."""
    rng = np.random.default_rng(27)
    V, B, N = 8, 40000, 3
    row, near = rng.dirichlet(np.ones(V), size=2).astype(np.float32)
    target = np.tile(row, (B, N, 1))
    draft = np.tile(near, (B, N, 1)) if kind == "sampled" else None
    tokens = np.zeros((B, N), np.int32)
    p64 = near.astype(np.float64) / near.astype(np.float64).sum()
    tokens[:, 1:] = rng.choice(V, size=(B, 2), p=p64) if kind == "sampled" else [6, 2]
    parent = np.tile(np.array([-1, 0, 0], np.int32), (B, 1))
    path, counts, nxt = run(cuda, tokens, parent, rng.random((B, N)).astype(np.float32), target, draft)
    first = np.where(counts > 1, tokens[np.arange(B), np.maximum(path[:, 1], 0)], nxt)
    p = row.astype(np.float64) / row.astype(np.float64).sum()
    seen = np.bincount(first, minlength=V)
    assert (np.abs(seen - B * p) <= 6 * np.sqrt(B * p * (1 - p)) + 1).all(), (seen / B, p)


def test_other_stream_and_graph(cuda):
    p = problem(28, 6, 8, 5001, "tree", "sampled")
    tokens, parent, u, target, draft = (torch.from_numpy(x).to(cuda) for x in p)
    path = torch.zeros((6, 8), dtype=torch.int32, device=cuda)
    counts, nxt = (torch.zeros(6, dtype=torch.int32, device=cuda) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.kivi_verify_tree(tokens, parent, u, target, draft, path, counts, nxt)
    side = torch.cuda.Stream()
    for seed in (1, 2):
        fresh = np.random.default_rng(seed).random((6, 8)).astype(np.float32)
        u.copy_(torch.from_numpy(fresh))
        graph.replay()
        want = run(cuda, p[0], p[1], fresh, p[3], p[4])
        other = run(cuda, p[0], p[1], fresh, p[3], p[4], stream=side)
        for a, b, c in zip((path, counts, nxt), want, other):
            assert np.array_equal(a.cpu().numpy(), b) and np.array_equal(b, c)
