"""Masks of drafted trees under a window: what tree_masks leaves visible, by the rule of vh_tree_attn in include/vh.h, is what
a windowed model sees when it takes each branch one token after the other."""
import random

import pytest

import paged_len_decode_gb300 as v


def seen_by_the_call(masks, n, base, window, sinks):
    """Slots that token i of one row sees, by the header's rule."""
    rows = []
    for i in range(n):
        bits = sum((w & (1 << 64) - 1) << 64 * k for k, w in enumerate(masks[i].tolist())) & (1 << i) - 1
        at = base + bits.bit_count()
        rows.append([j for j in range(base) if not window or at - j < window or j < sinks] +
                    [base + k for k in range(i) if bits >> k & 1] + [base + i])
    return rows


def seen_by_a_branch(parents, base, window, sinks):
    """The same of a model that decodes the context and then each token's branch: positions are places in that sequence."""
    rows = []
    for i in range(len(parents)):
        branch, up = [], i
        while up >= 0:
            branch.append(base + up)
            up = parents[up]
        slots = list(range(base)) + branch[::-1]
        last = len(slots) - 1
        rows.append([s for pos, s in enumerate(slots) if not window or last - pos < window or pos < sinks])
    return rows


@pytest.mark.parametrize("window", [0, 1, 2, 3, 8, 16, 64, 65, 200])
@pytest.mark.parametrize("sinks", [0, 1, 4, 20, 100])
def test_masks_hide_what_a_window_hides(window, sinks):
    rng = random.Random(window * 101 + sinks)
    for base in (0, 1, 3, 15, 40):
        for n, kind in ((1, "chain"), (70, "chain"), (130, "chain"), (40, "deep"), (90, "random")):
            parents = [i - 1 if kind == "chain" else rng.randint(max(-1, i - 3) if kind == "deep" else -1, i - 1) for i in range(n)]
            masks = v.tree_masks([[-1], parents], device="cpu", window=window, sinks=sinks, contexts=[7, base])[1:]
            assert seen_by_the_call(masks, n, base, window, sinks) == seen_by_a_branch(parents, base, window, sinks)


def test_a_window_wider_than_the_tree_changes_nothing():
    parents = [list(range(-1, 15)), [-1, 0, 0, 1]]
    assert (v.tree_masks(parents, device="cpu", window=16) == v.tree_masks(parents, device="cpu")).all()
    assert (v.tree_masks(parents, device="cpu", window=15) != v.tree_masks(parents, device="cpu")).sum() == 1


def test_refusals():
    for bad in (dict(window=-1), dict(window=4, sinks=-1), dict(window=4, sinks=2), dict(window=4, sinks=2, contexts=[1])):
        with pytest.raises(ValueError):
            v.tree_masks([[-1, 0], [-1]], device="cpu", **bad)
