"""kivi_verify_tree with random numbers outside [0, 1): the acceptance test is the
plain comparison of its definition, for repeated siblings too."""
import numpy as np
import pytest

import _step
from test_gpu_verify_tree import problem, run

pytestmark = pytest.mark.gpu


def compare(dev, tokens, parent, u, target, draft):
    """As in test_gpu_verify_tree.py, whose plain form takes no infinite u_0: it gets the
    1 that stands for all larger ones (u_0 is clamped)."""
    path, counts, nxt = run(dev, tokens, parent, u, target, draft)
    B, N, V = target.shape
    plain = u.copy()
    plain[:, 0] = np.where(u[:, 0] > 1, np.float32(1), u[:, 0])
    for b in range(B):
        want, last = _step.verify(tokens[b], parent[b], plain[b], target[b], None if draft is None else draft[b])
        assert counts[b] == len(want) and path[b].tolist() == want + [-1] * (N - len(want)), (b, path[b], want)
        assert nxt[b] == last, (b, nxt[b], last)
    return counts


@pytest.mark.parametrize("kind", ["sampled", "best"])
@pytest.mark.parametrize("shape", ["star", "tree"])
def test_any_numbers(cuda, shape, kind):
    tokens, parent, u, target, draft = problem(61, 48, 7, 40, shape, kind)
    rng = np.random.default_rng(62)
    odd = np.array([-1.0, -0.0, -1e-30, 1.0, 2.0, np.inf, -np.inf, np.nan], np.float32)
    swap = rng.random(u.shape) < 0.5
    u[swap] = odd[rng.integers(0, len(odd), size=u.shape)][swap]
    compare(cuda, tokens, parent, u, target, draft)


@pytest.mark.parametrize("kind", ["sampled", "best"])
def test_a_rejected_token_again_with_a_negative_number(cuda, kind):
    """Nothing is left of a token that was rejected, and a number below 0 accepts it
    all the same: among the first 32 nodes and beyond, directly after and later."""
    B, N, V = 6, 70, 50
    tokens, parent, u, target, draft = problem(63, B, N, V, "star", kind)
    u[:, 1:] = np.float32(2.0)                                    # rejected
    for b, at in enumerate((2, 3, 31, 32, 45, 69)):
        tokens[b, at] = tokens[b, 1]
        u[b, at] = -0.5
    counts = compare(cuda, tokens, parent, u, target, draft)
    if kind == "best":
        assert (counts == 2).all()
