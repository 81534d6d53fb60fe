"""kivi_verify_tree where the definition alone says how many nodes are kept."""
import numpy as np
import pytest

from test_gpu_verify_tree import problem, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [500, 32000])
def test_a_draft_equal_to_the_target_is_kept(cuda, V):
    """u p < p for every u below 1 whose product is rounded below p: all of a chain."""
    tokens, parent, u, target, _ = problem(71, 4, 9, V, "chain", "sampled")
    rows, up = np.arange(4)[:, None], np.maximum(parent, 0)
    p = target[rows, up, tokens]
    u[:] = 1 - 2.0 ** -22
    assert bool((u * p < p).all())
    path, counts, _ = run(cuda, tokens, parent, u, target, target.copy())
    assert (counts == 9).all() and (path == np.arange(9)).all()


def test_nothing_is_kept_with_the_largest_numbers_and_a_far_draft(cuda):
    """The target gives the drafted tokens nothing."""
    tokens, parent, u, target, draft = problem(72, 5, 6, 300, "star", "sampled")
    for b in range(5):
        target[b, 0, tokens[b, 1:]] = 0
    path, counts, nxt = run(cuda, tokens, parent, u, target, draft)
    assert (counts == 1).all() and not any(nxt[b] in tokens[b, 1:] for b in range(5))
