"""Decode over the 8-bit cache where early keys with large value scales lose their weight to later ones, against float64
(tests/quant_ref.py).

What a weight p_j vs_j loses beside its rounding: the kernel multiplies the weights by a power of two c that puts the
largest one so far at 2^13 at least (and the sum's later rescaling keeps it there), and rounds the product to fp16, whose
last half step is 2^-25.  So a weight loses at most 2^-38 of the largest one, and a value is at most 448:
448 n 2^-38 max_j w_j beside the tolerance of quant_ref.attention, which has 2^-40 in that term.  Every rise of the
maximum multiplies what is there by one more 2^x, off by 2^-22 and, for the difference of two scores of up to 2^8, 2^-17
times log 2: below 2^-17 together, for sums and outputs alike.
The kernel's fp32 arithmetic has no numbers below 2^-126.  With p relative to the running maximum a p_j vs_j below that may
count as zero, and so may an output: with values of at most 448 and a sum of weights of at least 1, that is
(448 n + 1) 2^-126 at most.  (The last of the falling values with rise 30.5 lie there: their scale is the least one, 2^-126,
and their outputs are about 2^-139.)
"""
import math
import random

import pytest
import torch

import quant_ref as Q
import window_ref as R
from test_gpu_quant import BF, FP, decode

pytestmark = pytest.mark.gpu

def batch(lens, groups, seed=0, heads=(8, 2), D=128, **kw):
    """A batch whose keys have the scores and value scales of `groups`: (slots, lowest and highest score in base 2, log2 of
    the values' size); the last group goes on to the row's end.  Queries are 4 everywhere, so a key of the constant x
    has the score 4 D x / sqrt(D) log2(e)."""
    HQ, HKV = heads
    r = Q.make(lens, [1] * len(lens), Hq=HQ, Hkv=HKV, D=D, seed=seed, **kw)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(r.pool.shape, generator=g)
    k, v = r.view(x, 0), r.view(x, 1)
    for b, L in enumerate(lens):
        ends = torch.tensor([n for n, *_ in groups]).cumsum(0)
        for j in range(L):
            i = min(int((ends <= j).sum()), len(groups) - 1)
            _, lo, hi, size = groups[i]
            at = int(r.table[b, j // r.P]), j % r.P
            if at[0] < 0:  # behind the window
                continue
            score = lo + (hi - lo) * torch.rand(HKV, 1, generator=g)
            k[at] = score * math.sqrt(D) / (4 * D * math.log2(math.e))
            v[at] *= 2.0 ** size
    Q.set_pool(r, *Q.quantised(x))
    return r, torch.full((len(lens), HQ, D), 4.0)


def check(r, q, dtype, num_ctas, raises=1):
    HQ, HKV, D = r.Hq, r.Hkv, r.D
    out, err = decode(r, q, dtype, num_ctas=num_ctas)
    assert err == 0
    ref, tol = Q.attention(r, q, dtype=dtype)
    k, v = r.view(r.pool, 0), r.view(r.pool, 1)
    vs = r.extra["scale"][:, 1].double()
    for b in range(r.B):
        at = torch.tensor(r.seen(b))
        pages = r.table[b].long()[at // r.P]
        qq = q[b].double().view(HKV, HQ // HKV, D)
        p = torch.softmax(torch.einsum("hgd,nhd->hgn", qq, k[pages, at % r.P]) / math.sqrt(D), -1)
        top = (p * vs[pages, :, at % r.P].t()[:, None]).amax(-1).reshape(HQ, 1)
        A = torch.einsum("hgn,nhd->hgd", p, v[pages, at % r.P].abs()).reshape(HQ, D)
        tol[b] += 448 * len(at) * 2.0 ** -38 * top + 2 * raises * 2.0 ** -17 * A + (448 * len(at) + 1) * 2.0 ** -126
    bad = Q.differs(out, (ref, tol), dtype)
    assert bad is None, bad


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("num_ctas", [1, 2, 3, 7])
@pytest.mark.parametrize("drop", [16, 22, 26, 30, 38, 44, 60])
def test_large_scales_lose_their_weight_to_later_small_ones(dtype, num_ctas, drop):
    """The first pair of tiles holds the large values under low scores; from the third on, keys whose scores are 60 above
    have all the weight."""
    high = 0 if dtype == BF else min(drop, 12)   # (fp16 holds outputs down to 2^-24)
    r, q = batch([96, 130, 420], [(32, 0, 1, high), (32, 0, 7.9, high), (1, 60, 64, high - drop)], seed=drop)
    if dtype == FP and high - drop < -20:
        r.extra["scale"][:, 1] *= 2.0 ** (drop - 20)  # outputs where fp16 is normal, the early values up to 2^40 beside them
        sc = r.extra["scale"] if r.layout == "HND" else r.extra["scale"].transpose(2, 3)
        Q.set_pool(r, r.extra["q8"], sc.contiguous())
    check(r, q, dtype, num_ctas, 2)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("num_ctas", [1, 4])
@pytest.mark.parametrize("rise", [7.0, 8.5, 9.0, 30.5])
def test_the_maximum_rises_in_steps_while_scales_fall(dtype, num_ctas, rise):
    """Every two tiles the scores are higher by `rise`, and the values smaller by half or all of what that brings."""
    for share in (0.5, 1.0):
        fall = round(rise * share)
        groups = [(32, i * rise, i * rise + 0.5, 12 - i * fall if dtype == BF else 10 - i * min(fall, 4)) for i in range(6)]
        r, q = batch([192, 175, 33, 600], groups, seed=int(rise * 4))
        check(r, q, dtype, num_ctas, 6)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_scales_rise_again_after_the_maximum(dtype):
    """The factor that rose with the maximum is lowered for the next large values."""
    groups = [(32, 0, 1, 8), (32, 40, 41, -8), (32, 41, 44, 10), (32, 70, 71, -12), (1, 71, 72, 9)]
    r, q = batch([96, 128, 161, 400], groups, seed=5, window=390, sinks=4)
    for num_ctas in (1, 5):
        check(r, q, dtype, num_ctas, 4)


def test_a_window_hides_the_large_values_and_sinks_keep_them():
    for sinks in (0, 8):
        r, q = batch([300, 96], [(32, 0, 1, 20), (32, 0, 7, 0), (1, 50, 55, -12)], seed=sinks, window=200, sinks=sinks)
        check(r, q, BF, 1, 2)


@pytest.mark.parametrize("seed", range(24))
def test_random_runs_of_scores_and_scales(seed):
    rng = random.Random(seed)
    dtype = rng.choice([BF, FP])
    groups, most = [], 40 if dtype == BF else 10
    for _ in range(rng.randint(2, 8)):
        low = rng.choice([0, rng.uniform(-60, 60)])
        groups.append((rng.choice([1, 5, 16, 32, 33, 70]), low, low + rng.choice([0.0, 1.0, 9.0]), rng.randint(-most, most)))
    hkv = rng.choice([1, 2, 3, 8])
    heads = (hkv * rng.choice([1, 2, 4, 8]), hkv)
    lens = [rng.randint(1, 500) for _ in range(rng.randint(1, 6))]
    r, q = batch(lens, groups, seed, heads, rng.choice([64, 128]), P=rng.choice([8, 16, 48]), layout=rng.choice(["NHD", "HND"]),
                 window=rng.choice([0, 0, 100, 300]), sinks=rng.choice([0, 4, 20]))
    for num_ctas in (0, 1, rng.randint(2, 20)):
        check(r, q, dtype, num_ctas, len(groups))
