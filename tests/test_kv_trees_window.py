"""kv_trees with a window: the bits of the ancestors that lie within it (no GPU)."""
import random

import pytest

import nvfp4_block_scaled_amd as nv


def ancestors(sequence, d, window):
    found = []
    while d >= 0 and (not window or len(found) < window):
        found.append(d)
        d = sequence[d]
    return set(found)


@pytest.mark.parametrize("window", [0, 1, 2, 5, 64, 200])
def test_ancestors_within_the_window(window):
    rng = random.Random(window)
    parents = [list(range(-1, 129)), [], [-1], [rng.randint(max(-1, d - 3), d - 1) for d in range(90)],
               [rng.randint(-1, d - 1) for d in range(40)]]
    tree, depths = nv.kv_trees(parents, window)
    plain, same = nv.kv_trees(parents)
    assert depths.tolist() == same.tolist() and tree.shape == plain.shape
    assert window or tree.equal(plain)
    at = 0
    for sequence in parents:
        for d in range(len(sequence)):
            row = [int(w) for w in tree[at]]
            assert {i for i in range(64 * len(row)) if row[i // 64] >> i % 64 & 1} == ancestors(sequence, d, window), (window, d)
            at += 1


def test_refusals():
    with pytest.raises(ValueError, match="window"):
        nv.kv_trees([[-1]], window=-1)
