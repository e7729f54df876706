"""Seeded random cases of the windowed decode and the prompt attention against
float64: shapes, pages, windows, sinks, ragged rows, idle rows, key shares.
VH_WINDOW_FUZZ_CASES sets how many (24 by default)."""
import os
import random

import pytest
import torch

import test_gpu_window as W
import window_ref as R

pytestmark = pytest.mark.gpu
CASES = int(os.environ.get("VH_WINDOW_FUZZ_CASES", "24"))


def pick(rng, decode):
    hkv = rng.choice([1, 1, 2, 3, 4, 8])
    heads = (hkv * rng.choice([1, 2, 4, 8]), hkv)
    B = rng.choice([1, 1, 2, 3, 5, 9, 40 if heads[0] <= 8 else 6])
    most = rng.choice([3, 17, 64, 130, 300, 900]) if B <= 5 else rng.choice([3, 40, 130])
    news = [1 if decode else rng.choice([0, 1, 2, rng.randint(1, most)]) for _ in range(B)]
    if not decode:   # (the reference takes token by token)
        while sum(news) > 500:
            news[news.index(max(news))] //= 2
        if sum(news) == 0:
            news[0] = 1
    lens = [max(n, rng.randint(1, most), 1) for n in news]
    return dict(lens=lens, news=news, Hq=heads[0], Hkv=heads[1], D=rng.choice([64, 128]), P=rng.choice([8, 16, 32, 48, 64, 128, 1024]),
                window=rng.choice([0, 0, 1, 2, 15, 16, 17, 64, 100, 500]), sinks=rng.choice([0, 0, 1, 4, 16, 33, 100, 1000]),
                dtype=rng.choice([torch.bfloat16, torch.float16]), layout=rng.choice(["NHD", "HND"]), seed=rng.randrange(1 << 30),
                active=[int(rng.random() > 0.1) for _ in range(B)], dead=rng.choice([-1, 1 << 30]))


@pytest.mark.parametrize("case", range(CASES))
def test_decode_cases(case):
    rng = random.Random(1000 + case)
    r = R.make(**pick(rng, True))
    W.check_decode(r, num_ctas=rng.choice([0, 0, 1, 2, 5, 33]), scale=rng.choice([0.0, 0.05]), pdl=rng.random() < 0.5)


@pytest.mark.parametrize("case", range(CASES))
def test_prompt_cases(case):
    rng = random.Random(5000 + case)
    r = R.make(**pick(rng, False))
    W.check_prompt(r, splits=rng.choice([0, 0, 0, 1, 2, 4, 8]), scale=rng.choice([0.0, 0.05]), extra=rng.choice([0, 0, 3]))
