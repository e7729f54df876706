"""Infinities and NaN in the cache under the windowed decode and the prompt
attention, against float64: they have to reach the outputs whose queries see
them, as they would in float64, and no others; and a call must stay about as fast."""
import math
import os
import random
import statistics

import pytest
import torch

import test_gpu_window as W
import test_gpu_window_fuzz as F
import window_batch as X
import window_ref as R

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
INF, NAN = math.inf, math.nan
KINDS = {"inf": [INF], "minus": [-INF], "nan": [NAN], "both": [INF, -INF], "all": [INF, -INF, NAN]}


def plant(r, which, values, count, seed, heads=None):
    """`count` elements of K (0) or V (1), at slots that some query sees."""
    rng = random.Random(seed)
    x = r.view(r.pool, which)
    rows = [b for b in range(r.B) if r.active[b] and r.news[b]]
    for c in range(count):
        b = rng.choice(rows)
        j = rng.choice(r.seen(b))
        x[int(r.table[b, j // r.P]), j % r.P, rng.randrange(r.Hkv), rng.randrange(r.D)] = values[c % len(values)]


def column(r, b, j, head, value, dims=slice(None), which=1):
    r.view(r.pool, which)[int(r.table[b, j // r.P]), j % r.P, head, dims] = value


def check(r, decode, scale=0.0, **kw):
    q = R.queries(r, torch.float32 if decode else r.pool.dtype)
    out, err = (W.decode if decode else W.prompt)(r, q, scale=scale, **kw)
    assert err == 0
    ref = X.attention(r, q, scale)
    bad = X.differs(out, ref, R.tolerance(ref, r.pool.dtype, r.D, decode, 8.0))
    assert bad is None, bad
    return out, ref


# small blocks (128 rows), shares of the keys, and blocks of 256 rows (more than 152 of the small ones)
PROMPTS = {
    "causal": (dict(lens=[260, 31], news=[260, 31], Hq=4, Hkv=2), {}),
    "window": (dict(lens=[300, 90], news=[200, 90], Hq=8, Hkv=2, window=40, sinks=5, P=48), {}),
    "shared": (dict(lens=[1500, 700], news=[20, 3], Hq=8, Hkv=2, window=1100, sinks=10, P=8), dict(splits=4)),
    "shared_all": (dict(lens=[900], news=[30], Hq=8, Hkv=1), dict(splits=2)),
    "large": (dict(lens=[900, 800], news=[900, 740], Hq=16, Hkv=8, window=300, sinks=7), {}),
    "large_all": (dict(lens=[700, 600, 300], news=[700, 600, 300], Hq=8, Hkv=8, P=64), {}),
    "large_shared": (dict(lens=[900, 900], news=[800, 700], Hq=16, Hkv=8, window=500, sinks=130), dict(splits=2)),
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (64, FP), (128, FP)])
@pytest.mark.parametrize("shape", PROMPTS)
def test_prompt_values(shape, D, dtype, kind):
    make, call = PROMPTS[shape]
    for seed, count in ((1, 1), (2, 7)):
        r = R.make(**make, D=D, dtype=dtype, layout="HND" if seed == 2 else "NHD", seed=seed)
        plant(r, 1, KINDS[kind], count, seed)
        check(r, False, **call)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape", PROMPTS)
def test_prompt_values_seen_by_all_some_and_none(shape, dtype):
    """The first slot (all, or a sink, or nobody), the last (one query), and whole tokens of NaN."""
    make, call = PROMPTS[shape]
    for j in (0, -1, -17):
        r = R.make(**make, dtype=dtype, seed=5)
        seen = r.seen(0)
        column(r, 0, seen[j], 0, INF, 3)
        column(r, 0, seen[j], 1 % r.Hkv, NAN)
        check(r, False, **call)


@pytest.mark.parametrize("shape", PROMPTS)
def test_prompt_keys_and_values(shape):
    """One infinite element of a key: scores of +inf (NaN rows) and -inf (no weight), the latter also with an
    infinite value; and weights far below the largest."""
    make, call = PROMPTS[shape]
    r = R.make(**make, seed=6)
    plant(r, 0, [INF, -INF], 2, 6)
    check(r, False, **call)
    r = R.make(**make, seed=7)
    j = r.seen(0)[len(r.seen(0)) // 2]
    column(r, 0, j, 0, -INF, 5, which=0)
    column(r, 0, j, 0, INF, 9)
    plant(r, 1, [NAN, INF], 2, 7)
    check(r, False, **call)
    for dtype in (BF, FP):
        r = R.make(**make, dtype=dtype, seed=8)
        plant(r, 1, [INF, -INF, INF], 9, 8)
        check(r, False, scale=0.7, **call)


def test_prompt_bad_page_beside_an_infinity():
    v = W.vh()
    r = R.make([200, 40], [200, 40], Hq=4, Hkv=2, window=100, sinks=2, seed=12)
    q = R.queries(r, BF)
    plant(r, 1, [INF, NAN], 4, 3)
    bad = R.Ragged(**{**r.__dict__, "table": r.table.clone()})
    page = int(bad.table[0, 5])
    bad.table[0, 5] = 1 << 28
    out, err = W.prompt(bad, q)
    assert err == v.VH_ERR_PAGE
    r.pool[page] = 0
    ref = X.attention(r, q)
    assert X.differs(out, ref, R.tolerance(ref, BF, 128, False, 8.0)) is None


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("splits", [1, 2])
def test_rows_whose_scores_are_all_minus_infinity(splits, large):
    """NaN, whichever way the keys are shared, in the prompt as in the decode."""
    lens = [700, 900] if large else [90]
    r = R.make(lens, lens, Hq=16 if large else 4, Hkv=8 if large else 2, window=1, seed=3)
    q = R.queries(r, BF)
    q[..., 5] = 1.0
    for j in (7, 80):
        column(r, 0, j, 1, -INF, 5, which=0)
    ref = X.attention(r, q)
    assert torch.isnan(ref[0]).any() and not torch.isnan(ref[0]).all()
    out, err = W.prompt(r, q, splits=splits)
    assert err == 0 and X.differs(out, ref, R.tolerance(ref, BF, 128, False, 8.0)) is None
    if not large:
        d = R.make([90, 8], [1, 1], Hq=4, Hkv=2, window=1, seed=4)
        qd = R.queries(d, torch.float32)
        qd[..., 5] = 1.0
        column(d, 1, 7, 0, -INF, 5, which=0)
        ref = X.attention(d, qd)
        out, err = W.decode(d, qd)
        assert err == 0 and X.differs(out, ref, R.tolerance(ref, BF, 128, True, 8.0)) is None


DECODES = {
    "rows": (dict(lens=[1, 2, 15, 16, 17, 333, 90], Hq=16, Hkv=8, window=64, sinks=5, P=8), {}),
    "whole": (dict(lens=[333, 90, 12], Hq=8, Hkv=2, P=48), dict(num_ctas=1)),
    "split": (dict(lens=[900, 3, 411], Hq=8, Hkv=4, window=700, sinks=20), dict(num_ctas=40)),
    "one_head": (dict(lens=[3000, 17], Hq=8, Hkv=1, window=2500, sinks=40), {}),
    "three": (dict(lens=[700, 60], Hq=3, Hkv=3, P=64), dict(num_ctas=7)),
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (64, FP), (128, FP)])
@pytest.mark.parametrize("shape", DECODES)
def test_decode_values(shape, D, dtype, kind):
    make, call = DECODES[shape]
    for seed, count in ((1, 1), (2, 7)):
        r = R.make(**make, news=[1] * len(make["lens"]), D=D, dtype=dtype, layout="HND" if seed == 2 else "NHD", seed=seed)
        plant(r, 1, KINDS[kind], count, seed)
        check(r, True, **call)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape", DECODES)
def test_decode_keys_and_values(shape, dtype):
    make, call = DECODES[shape]
    make = dict(make, news=[1] * len(make["lens"]), dtype=dtype)
    r = R.make(**make, seed=6)
    plant(r, 0, [INF, -INF], 2, 6)
    check(r, True, **call)
    r = R.make(**make, seed=7)
    j = r.seen(0)[len(r.seen(0)) // 2] if len(r.seen(0)) > 1 else 0
    column(r, 0, j, 0, -INF, 5, which=0)
    column(r, 0, j, 0, INF, 9)
    plant(r, 1, [NAN, INF], 2, 7)
    check(r, True, **call)
    r = R.make(**make, seed=8)
    plant(r, 1, [INF, -INF, INF], 9, 8)
    check(r, True, scale=0.7, **call)
    r = R.make(**make, seed=9)          # a whole token
    column(r, 0, r.seen(0)[0], 0, NAN)
    column(r, 1, r.seen(1)[-1], r.Hkv - 1, INF)
    check(r, True, **call)


def test_small_fp16_weights_count():
    """One key far above the others, each of which has 2^-27 of its weight: 4000 of them count together.  fp16
    weights are at least 2^7 at a row's maximum, so one loses at most 2^-25 2^-7 = 2^-32 of it.  (One CTA a block:
    a share of the keys without the first would have a maximum of its own.)"""
    lens, D = [4000], 64
    r = R.make(lens, [70], Hq=2, Hkv=1, D=D, dtype=FP, seed=2)
    k, v = r.view(r.pool, 0), r.view(r.pool, 1)
    k.zero_()
    v.fill_(1.0)
    column(r, 0, 0, 0, 18.75, 0, which=0)
    column(r, 0, 0, 0, 0.0)
    q = torch.zeros(70, 2, D, dtype=FP)
    q[..., 0] = 1.0
    out, err = W.prompt(r, q, scale=1.0, splits=1)
    ref = X.attention(r, q, 1.0)
    o, A, a, n = ref
    half = 2.0 ** -11
    tol = half * o.abs() + A * (2 * (a * (D + 4) * 2.0 ** -23 + 2.0 ** -20) + half + n * 2.0 ** -23) * (1 + half) + 2.0 ** -25 + n * 2.0 ** -32
    assert (ref[0] > 20 * tol).all()      # weights lost would show
    assert err == 0 and X.differs(out, ref, tol) is None


@pytest.mark.parametrize("shape", PROMPTS)
def test_values_near_the_end_of_bf16(shape):
    """Finite outputs although sums of unnormalised products would overflow fp32."""
    make, call = PROMPTS[shape]
    for big in (2.0 ** 121, 2.0 ** 124):    # (a merge of up to 8 pieces stays finite)
        r = R.make(**make, D=64, seed=11)
        v = r.view(r.pool, 1)
        v.copy_(torch.where(torch.isfinite(v.float()), v.float().sign() * big, v.float()).to(BF))
        out, ref = check(r, False, **call)
        assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("shape", DECODES)
def test_decode_values_near_the_end_of_bf16(shape):
    make, call = DECODES[shape]
    r = R.make(**make, news=[1] * len(make["lens"]), seed=11)
    v = r.view(r.pool, 1)
    v.copy_(torch.where(torch.isfinite(v.float()), v.float().sign() * 2.0 ** 120, v.float()).to(BF))
    out, ref = check(r, True, **call)
    assert torch.isfinite(out.float()).all()


CASES = int(os.environ.get("VH_NONFINITE_CASES", "24"))


def planted(rng, r):
    for which, count in ((1, rng.choice([0, 1, 3, 20])), (0, rng.choice([0, 0, 1, 2]))):
        values = KINDS[rng.choice(list(KINDS))] if which else [INF, -INF, NAN][:rng.choice([2, 2, 3])]
        plant(r, which, values, count, rng.randrange(1 << 20))
    if rng.random() < 0.3:
        b = rng.choice([b for b in range(r.B) if r.active[b] and r.news[b]])
        column(r, b, rng.choice(r.seen(b)), rng.randrange(r.Hkv), rng.choice([INF, -INF, NAN]))
    return r


def alive(make):
    if not any(a and n for a, n in zip(make["active"], make["news"])):
        make["active"], make["news"] = [1] * len(make["active"]), [max(1, n) for n in make["news"]]
    return make


@pytest.mark.parametrize("case", range(CASES))
def test_random_decode_cases(case):
    rng = random.Random(31000 + case)
    r = planted(rng, R.make(**alive(F.pick(rng, True))))
    check(r, True, scale=rng.choice([0.0, 0.05, 0.5]), num_ctas=rng.choice([0, 0, 1, 2, 5, 33]), pdl=rng.random() < 0.5)


@pytest.mark.parametrize("case", range(CASES))
def test_random_prompt_cases(case):
    rng = random.Random(32000 + case)
    r = planted(rng, R.make(**alive(F.pick(rng, False))))
    check(r, False, scale=rng.choice([0.0, 0.05, 0.5]), splits=rng.choice([0, 0, 0, 1, 2, 4, 8]), extra=rng.choice([0, 3]))


@pytest.mark.parametrize("D", [64, 128])
def test_more_than_32_requests(D):
    lens = [1 + (37 * b) % 250 for b in range(70)]
    news = [min(n, (13 * b) % 90) for b, n in enumerate(lens)]
    r = R.make(lens, news, Hq=16, Hkv=8, D=D, window=100, sinks=3, active=[int(b % 7 != 2) for b in range(70)], seed=D)
    plant(r, 1, [INF, NAN, -INF], 40, 5)
    check(r, False, extra=2)


def test_replayed_graph_with_values_that_come_and_go():
    """A captured prompt and decode call, replayed with finite values, bad ones and finite ones again."""
    v = W.vh()
    r = R.make([700, 500], [700, 450], Hq=16, Hkv=8, window=300, sinks=4, seed=3)
    d = R.make([700, 500], [1, 1], Hq=16, Hkv=8, window=300, sinks=4, seed=4)
    gp, gd = W.on_gpu(r), W.on_gpu(d)
    q, qd = R.queries(r, BF).cuda(), R.queries(d, torch.float32).cuda()
    out, outd = torch.zeros_like(q), torch.zeros(2, 16, 128, dtype=BF, device="cuda")
    ws, wd = v.alloc_prompt_workspace(1150, 2, 16, 8, 128), v.alloc_workspace(2, 16, 8, 128, 16)

    def call():
        v.vh_window_prompt_attn(q, gp["k"], gp["v"], gp["table"], gp["starts"], gp["lens"], gp["active"], out, ws, window=300,
                                sinks=4, err_flag=gp["err"])
        v.vh_window_decode_attn(qd, gd["k"], gd["v"], gd["table"], gd["lens"], gd["active"], outd, wd, window=300, sinks=4,
                                err_flag=gd["err"])

    call()
    torch.cuda.synchronize()
    first = out.clone(), outd.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    places = [(gp, r, 0, 1, 3), (gp, r, 1, 60, 90), (gp, r, 0, 650, 100), (gd, d, 0, 2, 5), (gd, d, 1, 499, 7)]
    for _ in range(3):
        kept = []
        for (t, x, b, j, e), value in zip(places, (NAN, INF, -INF, INF, NAN)):
            at = t["v"][int(x.table[b, j // 16]), j % 16, :, e]
            kept.append((at, at.clone()))
            at.fill_(value)
            x.view(x.pool, 1)[int(x.table[b, j // 16]), j % 16, :, e] = value
        g.replay()
        torch.cuda.synchronize()
        for o, x, y, split in ((out, r, q, False), (outd, d, qd, True)):
            ref = X.attention(x, y.cpu())
            bad = X.differs(o, ref, R.tolerance(ref, BF, 128, split, 8.0))
            assert bad is None, bad
        for (at, was), (t, x, b, j, e) in zip(kept, places):
            at.copy_(was)
            x.view(x.pool, 1)[int(x.table[b, j // 16]), j % 16, :, e] = was.cpu()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(outd, first[1])
        assert not ws.any() and int(gp["err"]) == 0 and int(gd["err"]) == 0


def timed(call):
    for _ in range(3):
        call()
    ms = []
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        ms.append(a.elapsed_time(b))
    return statistics.median(ms)


@pytest.mark.parametrize("where", ["all", "some", "none"])
@pytest.mark.parametrize("value", [INF, NAN])
def test_time_with_a_bad_value(where, value):
    """A value that is no number costs a block a second run and one for each kind of value, not a
    run of its own for each query: the second filters V at up to four times the time of the first,
    the others take the key tiles that hold such a value, so six times the time of finite values (and
    50 us of start)."""
    v = W.vh()
    r = R.make([4160], [4096], Hq=16, Hkv=8, window=1024 if where == "none" else 0, seed=2)
    g = W.on_gpu(r)
    q = R.queries(r, BF).cuda()
    out = torch.zeros_like(q)
    ws = v.alloc_prompt_workspace(4096, 1, 16, 8, 128)
    call = lambda: v.vh_window_prompt_attn(q, g["k"], g["v"], g["table"], g["starts"], g["lens"], g["active"], out, ws,  # noqa: E731
                                           window=r.window, err_flag=g["err"])
    plain = timed(call)
    j = {"all": 3, "some": 2000, "none": 3000}[where]
    g["v"][int(r.table[0, j // 16]), j % 16, :, 7] = value
    bad = timed(call)
    assert int(g["err"]) == 0 and not ws.any()
    assert bad < 6 * plain + 0.05, f"{bad * 1e3:.0f} us against {plain * 1e3:.0f} us"


@pytest.mark.parametrize("value", [INF, NAN])
def test_long_context_with_a_bad_value(value):
    """No wait runs out over a context of 120,000 tokens, and a request beside it is served."""
    lens, news = [120000, 500], [512, 300]
    r = R.make(lens, news, Hq=8, Hkv=1, D=64, P=64, seed=4)
    column(r, 0, 3, 0, value, 7)
    column(r, 0, 119900, 0, value, 9)
    check(r, False)
    d = R.make([120000, 500], [1, 1], Hq=8, Hkv=1, D=64, P=64, seed=5)
    column(d, 0, 3, 0, value, 7)
    check(d, True)
    check(d, True, num_ctas=1)
