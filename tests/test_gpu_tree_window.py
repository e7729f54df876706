"""Drafted trees as deep as the window, with masks that the window cuts, against float64 and against the calls that take
the same tokens one after the other."""
import pytest
import torch

import quant_ref as Q
import window_ref as R
from test_gpu_tree import BF, FP, fill_drafts, i32, run, vh

pytestmark = pytest.mark.gpu


def masks(r, parents):
    return vh().tree_masks(parents, device="cpu", window=r.window, sinks=r.sinks, contexts=[n - m for n, m in zip(r.lens, r.news)])


@pytest.mark.parametrize("window", [1, 16, 64, 65, 100])
@pytest.mark.parametrize("sinks", [0, 4])
def test_a_chain_under_a_window_is_the_prompt_attention(window, sinks):
    """Chains shorter, as long as and longer than the window."""
    for dtype, heads in ((BF, (8, 2)), (FP, (32, 4))):
        r = R.make([300, 64, 90, 70], [64, 64, 15, 70], *heads, window=window, sinks=sinks, dtype=dtype, seed=window + sinks)
        q = R.queries(r, dtype)
        parents = [Q.parents(n, r.extra["gen"], "chain") for n in r.news]
        ref = R.attention(r, q)
        # (the tree's lists of keys go back from its root's place: what only they reach is filled with numbers)
        fill_drafts(r)
        ours, err = run(r, q, masks(r, parents))
        theirs, _ = run(r, q, None)
        assert err == 0
        for out in (ours, theirs):
            bad = R.close(out, ref, dtype, r.D, False)
            assert bad is None, bad


@pytest.mark.parametrize("depth", [7, 15, 16, 40])
def test_a_chain_under_a_window_is_its_decode_steps(depth):
    """Less deep than the window of 16, and deeper."""
    v = vh()
    r = R.make([120], [depth], Hq=8, Hkv=2, window=16, sinks=3, seed=depth)
    fill_drafts(r)
    q = R.queries(r, BF)
    tree, err = run(r, q, masks(r, [list(range(-1, depth - 1))]))
    assert err == 0
    pool, ws = r.pool.cuda(), v.alloc_workspace(1, 8, 2, r.D, r.P)
    for i in range(depth):
        one = R.Ragged(**{**r.__dict__, "lens": [120 - depth + i + 1], "news": [1]})
        out = torch.empty(1, 8, r.D, dtype=BF, device="cuda")
        v.vh_window_decode_attn(q[i:i + 1].float().cuda(), r.view(pool, 0), r.view(pool, 1), r.table.cuda(), i32(one.lens), i32([1]),
                                out, ws, window=16, sinks=3)
        ref = R.attention(one, q[i:i + 1])
        for got, split in ((out.cpu(), True), (tree[i:i + 1], False)):
            bad = R.close(got, ref, BF, r.D, split)
            assert bad is None, bad


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (5, 0), (5, 40), (9, 4)])
def test_branches_under_a_window(window, sinks):
    """Every token of a tree against its own branch as a sequence; contexts shorter than the sinks, and none."""
    r = R.make([120, 40, 70, 33], [60, 40, 50, 1], Hq=8, Hkv=2, P=8, window=window, sinks=sinks, seed=window)
    fill_drafts(r)
    q = R.queries(r, BF)
    g = r.extra["gen"]
    parents = [[int(torch.randint(max(-1, i - 3), i, (1,), generator=g)) if i else -1 for i in range(n)] for n in r.news]
    out, err = run(r, q, masks(r, parents))
    assert err == 0
    k, val = r.view(r.pool, 0), r.view(r.pool, 1)
    for b in range(r.B):
        base = r.lens[b] - r.news[b]
        slots = [(int(r.table[b, j // r.P]), j % r.P) for j in range(r.lens[b])]
        for i in range(r.news[b]):
            branch, up = [], i
            while up >= 0:
                branch.append(base + up)
                up = parents[b][up]
            seq = list(range(base)) + branch[::-1]
            # the branch as a row of its own, in one page a token
            s = R.Ragged(r.Hq, r.Hkv, r.D, 1, torch.stack([torch.stack([x[slots[j]] for x in (k, val)]).unsqueeze(1) for j in seq]),
                         "NHD", torch.arange(len(seq), dtype=torch.int32).view(1, -1), [len(seq)], [1], [1], window, sinks)
            t = r.starts[b] + i
            bad = R.close(out[t:t + 1], R.attention(s, q[t:t + 1]), BF, r.D, False)
            assert bad is None, (b, i, bad)
