"""Attention of drafted trees on a GB300 against the float64 definition (tests/quant_ref.py's tree, tolerances of
tests/window_ref.py)."""
import pytest
import torch

import quant_ref as Q
import window_ref as R

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def vh():
    import paged_len_decode_gb300 as v
    return v


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(r, q, mask, splits=0, extra=0, scale=0.0, call=None):
    v = vh()
    pool = r.pool.cuda()
    T = r.starts[-1] + extra
    qq = torch.cat([q, torch.full((extra, r.Hq, r.D), float("nan"), dtype=q.dtype)]).cuda()
    out = torch.full((T, r.Hq, r.D), 7.0, dtype=r.pool.dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = v.alloc_prompt_workspace(T, r.B, r.Hq, r.Hkv, r.D)
    if mask is not None:
        mask = torch.cat([mask, torch.full((extra, mask.shape[1]), -1, dtype=torch.int64)]).cuda()
    args = (qq, r.view(pool, 0), r.view(pool, 1), r.table.cuda(), i32(r.starts), i32(r.lens), i32(r.active))
    more = dict(window=r.window, sinks=r.sinks, sm_scale=scale, num_splits=splits, err_flag=err)
    if mask is None:
        v.vh_window_prompt_attn(*args, out, ws, **more)
    else:
        v.vh_tree_attn(*args, mask, out, ws, **more)
    torch.cuda.synchronize()
    assert not ws[:256].any(), "the workspace is left zero for the next call"
    out = out.cpu()
    assert (out[r.starts[-1]:] == 7.0).all(), "tokens behind the last row were written"
    return out[:r.starts[-1]], int(err)


def trees(r, kind="random"):
    parents = [Q.parents(n, r.extra["gen"], kind) for n in r.news]
    return parents, vh().tree_masks(parents, device="cpu")


def check(r, kind="random", noise=True, **kw):
    parents, mask = trees(r, kind)
    q = R.queries(r, r.pool.dtype)
    if noise:
        # bits from a token's own number on do not count
        g = r.extra["gen"]
        for b in range(r.B):
            for i in range(r.news[b]):
                t = r.starts[b] + i
                for w in range(mask.shape[1]):
                    above = max(0, min(64, i - 64 * w))
                    junk = int(torch.randint(0, 1 << 62, (1,), generator=g)) * 3 & (1 << 64) - 1 & ~((1 << above) - 1)
                    x = (int(mask[t, w]) & (1 << 64) - 1) | junk
                    mask[t, w] = x - (1 << 64) if x >> 63 else x
    out, err = run(r, q, mask, **kw)
    assert err == 0
    bad = R.close(out, Q.tree(parents, r, q, kw.get("scale", 0.0)), r.pool.dtype, r.D, False)
    assert bad is None, bad


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 4), (33, 40), (100, 5), (1000, 4)])
@pytest.mark.parametrize("P", [8, 16, 48, 256])
def test_tree_windows(window, sinks, P):
    lens, news = [300, 5, 1, 140, 64, 200], [30, 5, 1, 20, 0, 62]
    # (every drafted slot is seen, by itself at least; windows hide no drafted token)
    r = R.make(lens, news, Hq=8, Hkv=2, P=P, window=window, sinks=sinks, seed=window + sinks + P)
    fill_drafts(r)
    check(r, extra=3)


def fill_drafts(r):
    """Drafted slots that a window of tests/window_ref.py would hide hold numbers too, and their pages are there; and so
    are the context's slots from the root's window on."""
    g = r.extra["gen"]
    for b in range(r.B):
        base = r.lens[b] - r.news[b]
        low = max(0, base - r.window + 1) if r.window else 0
        for j in range(low, r.lens[b]):
            if r.active[b] and int(r.table[b, j // r.P]) < 0:
                pool = torch.cat([r.pool, torch.full_like(r.pool[:1], float("nan"))])
                r.table[b, j // r.P] = pool.shape[0] - 1
                r.pool = pool
            if not r.active[b]:
                continue
            for i in (0, 1):
                at = r.view(r.pool, i)[int(r.table[b, j // r.P]), j % r.P]
                if torch.isnan(at).any():
                    at.copy_(torch.randn(r.Hkv, r.D, generator=g).to(at.dtype))


@pytest.mark.parametrize("heads", [(1, 1), (8, 1), (6, 3), (5, 5), (32, 4)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_tree_heads(heads, D, dtype):
    check(R.make([150, 77, 290], [16, 3, 40], *heads, D=D, dtype=dtype, layout="HND", seed=D + heads[0]))


@pytest.mark.parametrize("splits", [1, 2, 4, 8, 16])
def test_tree_splits(splits):
    check(R.make([1500, 700, 90], [9, 64, 1], Hq=8, Hkv=2, seed=splits), splits=splits)
    check(R.make([333, 40], [1, 40], Hq=8, Hkv=1, D=64, dtype=FP, active=[1, 0], seed=splits), splits=splits, extra=2)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 700, 1024])
@pytest.mark.parametrize("context", [0, 1, 100, 127, 128])
def test_tree_sizes(n, context):
    # several blocks of queries, words at the masks' borders, trees that cross key tiles, no context at all
    check(R.make([n + context, 7], [n, 7], Hq=8, Hkv=4, D=64, seed=n + context))


@pytest.mark.parametrize("kind", ["chain", "flat", "random"])
def test_tree_shapes(kind):
    check(R.make([260, 90], [90, 66], Hq=4, Hkv=2, seed=3), kind)
    r = R.make([260, 90], [90, 66], Hq=4, Hkv=2, window=20, sinks=2, seed=4)
    fill_drafts(r)
    check(r, kind)


def test_tree_of_one_chain_is_causal_attention():
    """The same bits as the prompt attention where both calls take blocks of the same size (the second batch) and share no
    keys; the same numbers in any case."""
    for heads, news, same in (((8, 2), [40, 64, 1], False), ((32, 4), [300, 64, 500], True)):
        r = R.make([900, 64, 700], news, *heads, seed=6)
        q = R.queries(r, BF)
        parents, mask = trees(r, "chain")
        ours, err = run(r, q, mask, splits=1)
        theirs, _ = run(r, q, None, splits=1)
        assert err == 0 and (torch.equal(ours, theirs) or not same)
        ref = R.attention(r, q)
        for out in (ours, theirs):
            bad = R.close(out, ref, BF, 128, False)
            assert bad is None, bad


def test_tree_large_blocks_and_many_rows():
    lens = [1 + (37 * b) % 150 for b in range(70)]
    news = [min(n, (13 * b) % 40) for b, n in enumerate(lens)]
    check(R.make(lens, news, Hq=4, Hkv=2, active=[int(b % 7 != 2) for b in range(70)], seed=9), extra=4)
    # more blocks than SMs
    check(R.make([400] * 24, [64] * 24, Hq=32, Hkv=8, D=64, dtype=FP, seed=10))


def test_tree_inactive_and_bad_rows():
    v = vh()
    r = R.make([40, 9, 70], [40, 9, 8], active=[1, 0, 1], seed=5)
    q = R.queries(r, BF)
    parents, mask = trees(r)
    out, err = run(r, q, mask)
    assert err == 0 and (out[40:49] == 0).all()
    assert R.close(out, Q.tree(parents, r, q), BF, 128, False) is None
    for bad in (7, -1, 10 ** 6):  # fewer tokens than the row brings, or more than its pages
        r2 = R.Ragged(**{**r.__dict__, "lens": [40, 9, bad]})
        out2, err = run(r2, q, mask)
        assert err == v.VH_ERR_SEQLEN and (out2[49:] == 0).all() and torch.equal(out2[:49], out[:49])
    # more drafted tokens than the masks have bits: zeros and a flag, the others as they are
    for B in (2, 40):
        r = R.make([100, 90] + [3] * (B - 2), [65, 64] + [1] * (B - 2), Hq=4, Hkv=2, seed=B)
        q = R.queries(r, BF)
        parents, mask = trees(r)
        full, err = run(r, q, mask)
        assert err == 0
        cut, err = run(r, q, mask[:, :1].contiguous())
        assert err == v.VH_ERR_SEQLEN and (cut[:65] == 0).all() and torch.equal(cut[65:], full[65:])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_tree_unseen_keys_and_values_never_count(value):
    """What a drafted token holds reaches its descendants only."""
    for news, heads in ((70, (4, 2)), (100, (8, 1))):
        r = R.make([260], [news], *heads, seed=31)
        q = R.queries(r, BF)
        parents, mask = trees(r)
        base, odd = 260 - news, 3
        for i in (0, 1):
            r.view(r.pool, i)[int(r.table[0, (base + odd) // 16]), (base + odd) % 16] = value
        out, err = run(r, q, mask)
        assert err == 0
        ref = Q.tree(parents, r, q)
        reached = torch.isnan(ref[0]).any(-1).any(-1)
        assert reached[odd] and not reached.all()
        assert torch.isnan(out[reached].float()).any(-1).any(-1).all()
        bad = R.close(out[~reached], tuple(x[~reached] for x in ref), BF, 128, False)
        assert bad is None, bad


def test_tree_bad_page_ids_are_flagged_and_read_as_zeros():
    r = R.make([40, 60], [1, 6], seed=12)
    q = R.queries(r, BF)
    parents, mask = trees(r)
    bad = R.Ragged(**{**r.__dict__, "table": r.table.clone()})
    page = int(bad.table[1, 2])
    bad.table[1, 2] = 1 << 28
    out, err = run(bad, q, mask)
    assert err == vh().VH_ERR_PAGE
    r.pool[page] = 0
    assert R.close(out, Q.tree(parents, r, q), BF, 128, False) is None
