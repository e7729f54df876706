"""Windowed decode and prompt attention on a GB300 against the float64
reference (tests/window_ref.py, which derives the tolerance)."""
import pytest
import torch

import window_ref as R

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def vh():
    import paged_len_decode_gb300 as v
    return v


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def on_gpu(r):
    pool = r.pool.cuda()
    return dict(k=r.view(pool, 0), v=r.view(pool, 1), table=r.table.cuda(), starts=i32(r.starts), lens=i32(r.lens),
                active=i32(r.active), err=torch.zeros(1, dtype=torch.int32, device="cuda"))


def decode(r, q, num_ctas=0, scale=0.0, pdl=False, table=True, ws=None, repeat=1):
    v, g = vh(), on_gpu(r)
    out = torch.full((r.B, r.Hq, r.D), float("nan"), dtype=r.pool.dtype, device="cuda")
    if ws is None:
        ws = v.alloc_workspace(r.B, r.Hq, r.Hkv, r.D, r.P, num_ctas)
    for _ in range(repeat):
        v.vh_window_decode_attn(q.cuda().float().contiguous(), g["k"], g["v"], g["table"] if table else None, g["lens"],
                                g["active"], out, ws, window=r.window, sinks=r.sinks, sm_scale=scale,
                                num_ctas=num_ctas, err_flag=g["err"], pdl=pdl)
    torch.cuda.synchronize()
    return out.cpu(), int(g["err"])


def prompt(r, q, scale=0.0, splits=0, table=True, extra=0):
    """extra: tokens behind the last row's, which must stay as they are."""
    v, g = vh(), on_gpu(r)
    T = r.starts[-1] + extra
    qq = torch.cat([q, torch.full((extra, r.Hq, r.D), float("nan"), dtype=q.dtype)]).cuda()
    out = torch.full((T, r.Hq, r.D), 7.0, dtype=r.pool.dtype, device="cuda")
    ws = v.alloc_prompt_workspace(T, r.B, r.Hq, r.Hkv, r.D)
    v.vh_window_prompt_attn(qq, g["k"], g["v"], g["table"] if table else None, g["starts"], g["lens"], g["active"], out,
                            ws, window=r.window, sinks=r.sinks, sm_scale=scale, num_splits=splits, err_flag=g["err"])
    torch.cuda.synchronize()
    assert not ws.any(), "the workspace is left zero for the next call"
    out = out.cpu()
    assert (out[r.starts[-1]:] == 7.0).all(), "tokens behind the last row were written"
    return out[:r.starts[-1]], int(g["err"])


def check_decode(r, **kw):
    q = R.queries(r, torch.float32)
    out, err = decode(r, q, **kw)
    assert err == 0
    bad = R.close(out, R.attention(r, q, kw.get("scale", 0.0), contiguous=not kw.get("table", True)), r.pool.dtype, r.D, True)
    assert bad is None, bad


def check_prompt(r, **kw):
    q = R.queries(r, r.pool.dtype)
    out, err = prompt(r, q, **kw)
    assert err == 0
    bad = R.close(out, R.attention(r, q, kw.get("scale", 0.0), contiguous=not kw.get("table", True)), r.pool.dtype, r.D, False)
    assert bad is None, bad


LENS = [1, 2, 15, 16, 17, 31, 33, 64, 100, 129, 200, 333]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 4), (17, 16), (64, 5), (100, 33), (1000, 4), (50, 1000)])
@pytest.mark.parametrize("P", [8, 16, 48])
def test_decode_windows(window, sinks, P):
    check_decode(R.make(LENS, [1] * len(LENS), P=P, window=window, sinks=sinks, seed=window * 7 + sinks + P))


@pytest.mark.parametrize("heads", [(1, 1), (8, 1), (6, 3), (20, 5), (8, 8), (32, 4), (64, 8)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_decode_heads(heads, D, dtype):
    check_decode(R.make([5, 77, 190], [1] * 3, *heads, D=D, window=60, sinks=3, dtype=dtype, layout="HND", seed=D + heads[0]))


@pytest.mark.parametrize("num_ctas", [1, 2, 3, 7, 40, 1000])
def test_decode_split_rows(num_ctas):
    check_decode(R.make([900, 3, 411, 1], [1] * 4, window=700, sinks=20, seed=num_ctas), num_ctas=num_ctas)


@pytest.mark.parametrize("B", [128, 129, 700])
def test_decode_many_rows(B):
    # more rows than the producer warp sums up alone, and more than CTAs
    lens = [1 + (29 * b) % 75 for b in range(B)]
    lens[B // 2] = 1500
    check_decode(R.make(lens, [1] * B, Hq=2, Hkv=1, D=64, window=40, sinks=3, active=[int(b % 9 != 4) for b in range(B)], seed=B))
    check_decode(R.make(lens, [1] * B, Hq=2, Hkv=1, D=64, seed=B))


def test_offsets_beyond_32_bits():
    """Pages whose elements lie more than 2^32 into the pool: the same bits as in a small pool."""
    v = vh()
    P, HKV, D, lens = 16, 8, 128, [70, 33]
    far = (1 << 32) // (2 * P * HKV * D) + 3
    small = R.make(lens, [1, 1], P=P, seed=4)
    big = torch.empty(far + small.pool.shape[0], 2, P, HKV, D, dtype=BF, device="cuda")
    big[far:] = small.pool.cuda()
    table = torch.where(small.table > 0, small.table + far, small.table).cuda()
    x = torch.randn(2, 32, D).to(BF).cuda()
    cs = v.vh_rope_table(torch.empty(128, D, device="cuda"))
    got = []
    for pool, t in ((small.pool.cuda(), small.table.cuda()), (big, table)):
        k, val = pool[:, 0], pool[:, 1]
        q32 = torch.empty(2, 16, D, device="cuda")
        q16 = torch.empty(2, 16, D, dtype=BF, device="cuda")
        rows = (t, i32(lens), i32([1, 1]))
        o1, o2 = torch.zeros(2, 16, D, dtype=BF, device="cuda"), torch.zeros(2, 16, D, dtype=BF, device="cuda")
        for q in (q32, q16):
            v.vh_mrope_kv_append(x[:, :16], x[:, 16:24], x[:, 24:], cs, k, val, *rows, q)
        v.vh_window_decode_attn(q32, k, val, *rows, o1, v.alloc_workspace(2, 16, HKV, D, P))
        v.vh_window_prompt_attn(q16, k, val, t, i32([0, 1, 2]), *rows[1:], o2, v.alloc_prompt_workspace(2, 2, 16, HKV, D))
        torch.cuda.synchronize()
        n = small.pool.shape[0]
        got.append((o1, o2, pool[-n:].clone().view(torch.int16)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.isfinite(got[0][0].float()).all() and torch.isfinite(got[0][1].float()).all()


def test_decode_many_pieces_and_repeated_calls():
    r = R.make([6000, 17], [1, 1], Hq=8, Hkv=1, window=5500, sinks=40, seed=3)
    check_decode(r)
    q = R.queries(r, torch.float32)
    v = vh()
    ws = v.alloc_workspace(2, 8, 1, 128, 16)
    a, _ = decode(r, q, ws=ws)
    b, _ = decode(r, q, ws=ws, repeat=3, pdl=True)
    assert torch.equal(a, b), "the same call gives other bits"


def test_decode_padding_rows_and_bad_rows():
    r = R.make([40, 9, 70], [1] * 3, window=32, sinks=2, active=[1, 0, 1], seed=5)
    q = R.queries(r, torch.float32)
    out, err = decode(r, q)
    assert err == 0 and (out[1] == 0).all()
    assert R.close(out, R.attention(r, q), BF, 128, True) is None
    v = vh()
    for bad in (0, -4, 10 ** 6):  # a length out of range: zeros and a flag, the others as before
        r2 = R.Ragged(**{**r.__dict__, "lens": [40, 9, bad], "active": [1, 0, 1]})
        out2, err = decode(r2, q)
        assert err == v.VH_ERR_SEQLEN and (out2[2] == 0).all() and torch.equal(out2[0], out[0])


def test_decode_contiguous_cache():
    lens = [11, 3, 7]
    r = R.make(lens, [1] * 3, D=64, P=11, window=6, sinks=1, table_extra=0, seed=8)
    pool = torch.randn(3, 2, 11, 8, 64).to(BF)
    r.pool, r.table = pool, torch.arange(3, dtype=torch.int32).view(3, 1)
    check_decode(r, table=False)
    check_prompt(R.Ragged(**{**r.__dict__, "news": [5, 3, 1]}), table=False)


def test_bad_page_ids_are_flagged_and_read_as_zeros():
    v = vh()
    for fn, news, dt, split in ((decode, [1, 1], torch.float32, True), (prompt, [1, 6], BF, False)):
        r = R.make([40, 60], news, window=40, sinks=0, seed=12)
        q = R.queries(r, dt)
        bad = R.Ragged(**{**r.__dict__, "table": r.table.clone()})
        page = int(bad.table[1, 2])
        bad.table[1, 2] = 1 << 28
        out, err = fn(bad, q)
        assert err == v.VH_ERR_PAGE
        zero = R.Ragged(**{**r.__dict__, "pool": r.pool.clone()})
        zero.pool[page] = 0
        assert R.close(out, R.attention(zero, q), BF, 128, split) is None


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 4), (33, 40), (100, 5), (1000, 4)])
@pytest.mark.parametrize("P", [8, 16, 48, 256])
def test_prompt_windows(window, sinks, P):
    lens = [300, 5, 1, 140, 64, 200]
    news = [300, 5, 1, 20, 0, 130]
    check_prompt(R.make(lens, news, Hq=8, Hkv=2, P=P, window=window, sinks=sinks, seed=window + sinks + P), extra=3)


@pytest.mark.parametrize("heads", [(1, 1), (8, 1), (6, 3), (5, 5), (32, 4)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_prompt_heads(heads, D, dtype):
    check_prompt(R.make([150, 77, 290], [150, 3, 140], *heads, D=D, window=90, sinks=3, dtype=dtype, layout="HND", seed=D + heads[0]))


@pytest.mark.parametrize("splits", [1, 2, 4, 8, 16])
def test_prompt_splits(splits):
    check_prompt(R.make([1500, 700, 90], [9, 150, 1], Hq=8, Hkv=2, window=1100, sinks=10, seed=splits), splits=splits)
    check_prompt(R.make([333, 40], [1, 40], Hq=8, Hkv=1, D=64, dtype=FP, sinks=0, active=[1, 0], seed=splits), splits=splits, extra=2)


@pytest.mark.parametrize("heads", [(8, 1), (2, 2), (8, 8)])
def test_prompt_large_blocks(heads):
    # more blocks than SMs: blocks of 256 (token, head) rows, drawn one after the other
    T = 152 * 128 // heads[0] + 700
    r = R.make([T // 2 + 3, T // 2, 5], [T // 2 + 3, T // 2 - 9, 5], *heads, D=64, window=70, sinks=3, dtype=FP, seed=heads[0])
    check_prompt(r, extra=1)


def test_prompt_many_rows():
    # more requests than one a lane of the drawing warp
    lens = [1 + (37 * b) % 150 for b in range(70)]
    news = [min(n, (13 * b) % 40) for b, n in enumerate(lens)]
    check_prompt(R.make(lens, news, Hq=4, Hkv=2, window=50, sinks=3, active=[int(b % 7 != 2) for b in range(70)], seed=9), extra=4)


def test_prompt_large_scores_and_scale():
    for dt in (BF, FP):
        r = R.make([400], [200], Hq=4, Hkv=2, dtype=dt, window=150, sinks=4, seed=21)
        check_prompt(r, scale=0.7)
        check_decode(R.make([400, 21], [1, 1], Hq=4, Hkv=2, dtype=dt, window=150, sinks=4, seed=22), scale=0.7)


def test_prompt_inactive_and_bad_rows():
    v = vh()
    r = R.make([40, 9, 70], [40, 9, 8], window=32, sinks=2, active=[1, 0, 1], seed=5)
    q = R.queries(r, BF)
    out, err = prompt(r, q)
    assert err == 0 and (out[40:49] == 0).all()
    assert R.close(out, R.attention(r, q), BF, 128, False) is None
    for bad in (7, -1, 10 ** 6):  # fewer tokens than the row brings, or more than its pages
        r2 = R.Ragged(**{**r.__dict__, "lens": [40, 9, bad]})
        out2, err = prompt(r2, q)
        assert err == v.VH_ERR_SEQLEN and (out2[49:] == 0).all() and torch.equal(out2[:49], out[:49])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("window", [0, 20])
def test_unseen_keys_and_values_never_count(value, window):
    """A key and a value that later queries see, and earlier ones do not."""
    r = R.make([260], [260], Hq=4, Hkv=2, window=window, sinks=0, seed=31)
    q = R.queries(r, BF)
    at = 150
    k, v = r.view(r.pool, 0), r.view(r.pool, 1)
    k[int(r.table[0, at // 16]), at % 16] = value
    v[int(r.table[0, at // 16]), at % 16] = value
    out, err = prompt(r, q)
    ref = R.attention(r, q)
    blind = torch.ones(260, dtype=torch.bool)
    blind[at:at + window if window else 260] = False
    assert err == 0
    assert torch.isnan(out[~blind].float()).all() == torch.isnan(ref[0][~blind]).all()
    part = tuple(x[blind] for x in ref)
    bad = R.close(out[blind], part, BF, 128, False)
    assert bad is None, bad
