"""The prompt attention's blocks of 256 (token, head) rows, which long and many
prompts take (more than 152 blocks of 128 rows), against float64: both head
dimensions and types, windows of many key tiles and none, page sizes, more than
32 requests, shares of the keys; and seeded random cases above that border."""
import random

import pytest
import torch

import test_gpu_window as W
import window_batch as X
import window_ref as R

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
TYPES = [(64, BF), (64, FP), (128, BF), (128, FP)]


def blocks_of_128(r):
    """(token, head) blocks of 128 rows that the call's T and B make likely, over all kv heads."""
    per = 128 // (r.Hq // r.Hkv)
    return (-(-r.starts[-1] // per) + (r.B - 1) // 2) * r.Hkv


def check(r, scale=0.0, **kw):
    assert blocks_of_128(r) > 152
    q = R.queries(r, r.pool.dtype)
    out, err = W.prompt(r, q, scale=scale, **kw)
    assert err == 0
    ref = X.attention(r, q, scale)
    bad = R.close(out, ref, r.pool.dtype, r.D, False)
    assert bad is None, bad


@pytest.mark.parametrize("D,dtype", TYPES)
@pytest.mark.parametrize("heads,window,sinks", [((8, 8), 0, 0), ((16, 8), 900, 4), ((32, 4), 0, 0), ((8, 1), 2500, 200)])
def test_many_key_tiles(heads, window, sinks, D, dtype):
    T = 160 * 128 * heads[1] // heads[0] // heads[1] + 37
    T = max(T, 152 * 128 // heads[0] + 200)
    check(R.make([T + 1300, 900], [T, 5], *heads, D=D, dtype=dtype, window=window, sinks=sinks, layout="HND", seed=D + window), extra=2)


@pytest.mark.parametrize("P", [8, 48, 64, 1024])
@pytest.mark.parametrize("D,dtype", TYPES)
def test_page_sizes(P, D, dtype):
    lens, news = [1111, 700, 1, 130], [1000, 333, 1, 2]
    check(R.make(lens, news, 16, 8, D=D, dtype=dtype, P=P, window=400, sinks=33, seed=P + D), extra=1)
    check(R.make(lens, news, 16, 8, D=D, dtype=dtype, P=P, seed=P + D + 1))


@pytest.mark.parametrize("D,dtype", TYPES)
def test_more_than_32_requests(D, dtype):
    lens = [1 + (37 * b) % 250 for b in range(70)]
    news = [min(n, (13 * b) % 90) for b, n in enumerate(lens)]
    check(R.make(lens, news, 16, 8, D=D, dtype=dtype, window=100, sinks=3, active=[int(b % 7 != 2) for b in range(70)], seed=D), extra=4)


@pytest.mark.parametrize("splits", [2, 4, 8])
@pytest.mark.parametrize("D,dtype", TYPES)
def test_shares_of_the_keys(D, dtype, splits):
    check(R.make([1500, 600], [900, 600], 16, 8, D=D, dtype=dtype, window=700, sinks=20, seed=splits), splits=splits)


@pytest.mark.parametrize("case", range(12))
def test_random_cases(case):
    rng = random.Random(9000 + case)
    hkv = rng.choice([1, 2, 3, 5, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    need = 160 * 128 // hq
    B = rng.choice([1, 2, 5, 12, 40])
    cuts = sorted(rng.randrange(need + 1) for _ in range(B - 1))
    news = [b - a for a, b in zip([0, *cuts], [*cuts, need])]
    lens = [max(1, n + rng.choice([0, 0, 1, 77, 500])) for n in news]
    active = [int(rng.random() > 0.1) for _ in range(B)]
    check(R.make(lens, news, hq, hkv, D=rng.choice([64, 128]), P=rng.choice([8, 16, 48, 64, 256]), dtype=rng.choice([BF, FP]),
                 window=rng.choice([0, 1, 17, 200, 1000]), sinks=rng.choice([0, 0, 4, 100, 1000]), layout=rng.choice(["NHD", "HND"]),
                 active=active, seed=case), scale=rng.choice([0.0, 0.05]), splits=rng.choice([0, 0, 1, 2]), extra=rng.choice([0, 3]))
