"""The reference of the tree attention against sequential decode (no GPU): a token's result is that of
decode steps along its own path."""
import numpy as np
import pytest

from oracle import kvcache as ref


@pytest.mark.parametrize("W,S", [(1, 0), (3, 0), (3, 2), (5, 9), (100, 0)])
def test_tree_is_decode_along_the_path(W, S):
    rng = np.random.default_rng(W + S)
    base, n, Hq, Hkv, d = 6, 9, 4, 2, 8
    parents = [-1, 0, 1, -1, 3, 1, 5, 6, 7]
    gates = rng.integers(0, 2, n)
    q = rng.standard_normal((n, Hq, d))
    k, v = rng.standard_normal((2, 1, base + n, Hkv, d))
    o, lse, *_ = ref.decode_tree(q, k, v, [base + n], [0, n], parents, gates, W, S, 0.4)
    for t in range(n):
        path = ref.tree_path(parents, t)
        along = np.concatenate([np.arange(base), base + np.array(path)])
        exps = np.full((1, len(along), Hkv), 127)
        want, want_lse, *_ = ref.decode(q[None, t], k[:, along], v[:, along], exps, [len(along)], [gates[t]], W, S, 0.4)
        np.testing.assert_allclose(o[t], want[0], atol=1e-12)
        np.testing.assert_allclose(lse[t], want_lse[0], atol=1e-12)


def test_tree_visible_by_hand():
    seen = ref.tree_visible([-1, 0, 0, -1], [0, 1, 0, 0], 3, 2, 1)
    assert seen.astype(int).tolist() == [
        [1, 0, 1, 1, 0, 0, 0],    # position 3: window {2, 3}, anchor 0
        [1, 1, 1, 1, 1, 0, 0],    # routed
        [1, 0, 0, 1, 0, 1, 0],    # position 4: window {3, 4}
        [1, 0, 1, 0, 0, 0, 1]]


def test_tree_path_ends_at_a_bad_parent():
    assert ref.tree_path([5, 0, 2, 1], 3) == [0, 1, 3]
    assert ref.tree_path([5, 0, 2, 1], 2) == [2]
