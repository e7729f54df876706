"""The 8-bit cache on a GB300: append, attention and read-back against the float64 definitions (tests/quant_ref.py)."""
import math

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


# ---- append ------------------------------------------------------------------------------------------------------------

def append_case(lens, news, Hq=8, Hkv=2, D=128, P=16, dtype=BF, q16=False, norm=False, interleaved=False, layout="NHD", packed=False,
                active=None, one_each=False, axes=None, seed=0, extra=0, change=None):
    """Runs an append; checks q_rot, bytes and scales; returns what the cache holds."""
    v, g = vh(), torch.Generator().manual_seed(seed)
    r = Q.make(lens, news, Hq=Hq, Hkv=Hkv, D=D, P=P, layout=layout, seed=seed, active=active)
    c = Q.on_gpu(r, pad=1)
    T, most, half = r.starts[-1], 300, D // 2
    x = torch.randn(T + extra, Hq + 2 * Hkv, D, generator=g).to(dtype)
    if change:
        change(x)
    pos = torch.randint(0, most, ((len(set(axes)) if axes else 1), T + extra), generator=g, dtype=torch.int32)
    wq, wk = ((1 + 0.1 * torch.randn(D, generator=g), 1 + 0.1 * torch.randn(D, generator=g)) if norm else (None, None))
    cs = v.vh_rope_table(torch.empty(most, D, device="cuda"))
    xg = x.cuda()
    q, kn, vn = xg[:, :Hq], xg[:, Hq:Hq + Hkv], xg[:, Hq + Hkv:]
    if not packed:
        q, kn, vn = q.contiguous(), kn.contiguous(), vn.contiguous()
    q_rot = torch.full((T + extra, Hq, D), 7.0, dtype=dtype if q16 else torch.float32, device="cuda")
    before = c["pool"].view(torch.uint8).cpu().clone(), c["ks"].cpu().clone(), c["vs"].cpu().clone()
    v.vh_quant_kv_append(q, kn, vn, cs, c["k"], c["v"], c["ks"], c["vs"], c["table"], c["lens"], c["active"], q_rot,
                         token_start=None if one_each else c["starts"], positions=pos.cuda(), pair_axis=axes, err_flag=c["err"],
                         q_norm_w=None if wq is None else wq.cuda(), k_norm_w=None if wk is None else wk.cuda(),
                         interleaved=interleaved)
    torch.cuda.synchronize()
    err = int(c["err"])
    at = pos.long()[torch.tensor(axes if axes else [0] * half)].t()
    csc = cs.cpu()
    cos, sin = csc[at, torch.arange(half)], csc[at, half + torch.arange(half)]
    qr, qe = R.rope(x[:, :Hq], cos, sin, wq, 1e-6, interleaved)
    kr, ke = R.rope(x[:, Hq:Hq + Hkv], cos, sin, wk, 1e-6, interleaved)
    got_q, pool = q_rot.cpu().double(), c["pool"].cpu()
    ks, vs = c["ks"].cpu(), c["vs"].cpu()
    written = torch.zeros(pool.shape[0], P, dtype=torch.bool)
    for b in range(r.B):
        for i in range(r.news[b]):
            t, j = r.starts[b] + i, r.lens[b] - r.news[b] + i
            page, off = int(r.table[b, j // P]), j % P
            if not r.active[b]:
                assert (got_q[t] == 7.0).all()
                continue
            written[page, off] = True
            step = torch.finfo(dtype).eps / 2 if q16 else 2.0 ** -24
            fine = torch.isfinite(qr[t])
            assert ((got_q[t] - qr[t]).abs() <= qe[t] + step * (qr[t].abs() + qe[t]) + (2.0 ** -25 if q16 else 0))[fine].all()
            # values: bits of the rule, which has no other rounding
            want, sc = Q.quantised(x[t, Hq + Hkv:].float())
            have = r.view(pool, 1)[page, off]
            assert torch.equal(torch.nan_to_num(vs[page, :, off], -1), torch.nan_to_num(sc, -1)), (vs[page, :, off], sc)
            ok = torch.isfinite(sc)
            assert torch.equal(have.view(torch.uint8)[ok], want.view(torch.uint8)[ok])
            # keys: the scale to fp32's error of the rotation, the value to half a step of e4m3 and that
            top = kr[t].abs().amax(-1)
            s = ks[page, :, off].double()
            ok = torch.isfinite(kr[t]).all(-1)
            assert torch.equal(torch.isnan(s), ~ok)
            exact = (top / 448).clamp(min=2.0 ** -126)
            assert ((s - exact).abs() <= ke[t].amax(-1) / 448 + 2.0 ** -23 * exact)[ok].all()
            y = r.view(pool, 0)[page, off].double() * s[:, None]
            tol = 2.0 ** -4 * (kr[t].abs() + ke[t]) * (1 + 2.0 ** -20) + ke[t] + (exact * 2.0 ** -10 * (1 + 2.0 ** -20))[:, None]
            assert ((y - kr[t]).abs() <= tol)[ok].all()
    assert (got_q[T:] == 7.0).all()
    # nothing else was written
    old, now = before[0], pool.view(torch.uint8)
    for i in (0, 1):
        same = (r.view(old, i) == r.view(now, i)).all(-1).all(-1) | written
        assert same.all()
        a, b = (before[1], ks) if i == 0 else (before[2], vs)
        assert ((torch.nan_to_num(a, -1) == torch.nan_to_num(b, -1)).all(1) | written).all()
    return r, c, err


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_append_forms(D, dtype, interleaved, norm):
    assert append_case([40, 3, 17], [40, 3, 5], D=D, dtype=dtype, interleaved=interleaved, norm=norm, q16=norm, seed=D, packed=norm)[2] == 0


@pytest.mark.parametrize("heads", [(1, 1), (8, 1), (6, 3), (20, 5), (16, 8), (64, 8)])
@pytest.mark.parametrize("P,layout", [(8, "NHD"), (16, "HND"), (48, "NHD")])
def test_append_heads_and_pages(heads, P, layout):
    assert append_case([33, 1, 9, 100], [20, 1, 9, 2], *heads, P=P, layout=layout, active=[1, 1, 0, 1], extra=2, seed=P + heads[0])[2] == 0


def test_append_one_token_a_row_and_many_rows():
    append_case([5, 16, 17, 1], [1] * 4, one_each=True, active=[1, 1, 0, 1])
    lens = [1 + (7 * b) % 40 for b in range(140)]
    append_case(lens, [1] * 140, Hq=2, Hkv=1, D=64, one_each=True)
    append_case(lens, [min(n, b % 4) for b, n in enumerate(lens)], Hq=4, Hkv=2, D=64, dtype=FP)
    append_case([700, 800], [700, 700], Hq=4, Hkv=2, D=64)   # (a warp a token)


def test_append_axes():
    append_case([50], [50], axes=[0] * 16 + [1] * 24 + [2] * 24, seed=2)
    append_case([50], [50], D=64, axes=[i % 3 for i in range(32)], seed=3, interleaved=True)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_append_zero_small_large_and_nonfinite_heads(dtype):
    def change(x):
        x[0] = 0
        x[1] *= 1e-4
        x[2] *= 1000 if dtype == FP else 1e30
        x[3, :, 5] = math.inf
        x[4, :, 64] = math.nan
        x[5, :, :] = 0
        x[5, :, 9] = -2.0
        x[6] = x[6] * (2.0 ** -20 if dtype == FP else 1e-30)
    r, c, err = append_case([20], [20], dtype=dtype, change=change, seed=7)
    assert err == 0
    page = int(r.table[0, 0])
    assert (c["vs"][page, :, 0] == 2.0 ** -126).all() and not r.view(c["pool"].cpu(), 1)[page, 0].float().any()
    assert torch.isnan(c["vs"][page, :, 3:5]).all() and torch.isnan(c["ks"][page, :, 3:5]).all()


def test_append_bad_pages_positions_and_lengths():
    v = vh()
    r = Q.make([20, 20], [3, 3], Hq=4, Hkv=2, D=64, seed=1)
    c = Q.on_gpu(r)
    x = torch.randn(6, 8, 64).to(BF).cuda()
    cs = v.vh_rope_table(torch.empty(64, 64, device="cuda"))
    old = c["pool"].view(torch.uint8).clone(), torch.nan_to_num(c["ks"], -1), torch.nan_to_num(c["vs"], -1)

    def call(table, lens, pos):
        out = torch.full((6, 4, 64), 7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        v.vh_quant_kv_append(x[:, :4], x[:, 4:6], x[:, 6:], cs, c["k"], c["v"], c["ks"], c["vs"], table, i32(lens), c["active"], out,
                             token_start=c["starts"], positions=i32(pos), err_flag=err)
        torch.cuda.synchronize()
        return out, int(err)

    bad = c["table"].clone()
    bad[:, 1] = torch.tensor([-1, 1 << 30], dtype=torch.int32)
    out, err = call(bad, [20, 20], [0] * 6)
    assert err == v.VH_ERR_PAGE and (out != 7.0).any(-1).all()
    out, err = call(c["table"], [2, 10 ** 6], [0] * 6)
    assert err == v.VH_ERR_SEQLEN and (out == 7.0).all()
    out, err = call(c["table"], [20, 20], [-1, 64, 1 << 30] * 2)
    assert err == v.VH_ERR_POS and (out == 7.0).all()
    assert torch.equal(old[0], c["pool"].view(torch.uint8)) and torch.equal(old[1], torch.nan_to_num(c["ks"], -1))
    assert torch.equal(old[2], torch.nan_to_num(c["vs"], -1))


# ---- attention -----------------------------------------------------------------------------------------------------------

def decode(r, q, dtype=BF, num_ctas=0, scale=0.0, table=True, pad=0, ws=None, repeat=1, pdl=False):
    v, c = vh(), Q.on_gpu(r, pad)
    out = torch.full((r.B, r.Hq, r.D), math.nan, dtype=dtype, device="cuda")
    if ws is None:
        ws = v.alloc_workspace(r.B, r.Hq, r.Hkv, r.D, r.P, num_ctas)
    for _ in range(repeat):
        v.vh_quant_decode_attn(q.cuda(), c["k"], c["v"], c["ks"], c["vs"], c["table"] if table else None, c["lens"], c["active"], out,
                               ws, window=r.window, sinks=r.sinks, sm_scale=scale, num_ctas=num_ctas, err_flag=c["err"], pdl=pdl)
    torch.cuda.synchronize()
    return out.cpu(), int(c["err"])


def check_decode(r, dtype=BF, q=None, **kw):
    q = R.queries(r, torch.float32) if q is None else q
    out, err = decode(r, q, dtype, **kw)
    assert err == 0
    bad = Q.differs(out, Q.attention(r, q, kw.get("scale", 0.0), not kw.get("table", True), dtype), dtype)
    assert bad is None, bad


LENS = [1, 2, 15, 16, 17, 31, 33, 64, 100, 129, 200, 333]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 4), (17, 16), (64, 5), (100, 33), (1000, 4), (50, 1000)])
@pytest.mark.parametrize("P", [8, 16, 48])
def test_decode_windows(window, sinks, P):
    check_decode(Q.make(LENS, [1] * len(LENS), P=P, window=window, sinks=sinks, seed=window * 7 + sinks + P))


@pytest.mark.parametrize("heads", [(1, 1), (8, 1), (6, 3), (20, 5), (8, 8), (32, 4), (64, 8), (44, 11)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_decode_heads(heads, D, dtype):
    check_decode(Q.make([5, 77, 190], [1] * 3, Hq=heads[0], Hkv=heads[1], D=D, window=60, sinks=3, layout="HND", seed=D + heads[0]), dtype,
                 pad=1)


def test_one_head_or_page_with_any_stride():
    """torch gives dimensions of one element strides of its own: they are not looked at."""
    v = vh()
    for lens, P in (([40, 9], 16), ([7], 8)):
        r = Q.make(lens, [1] * len(lens), Hq=4, Hkv=1, P=P, seed=P, spare=0 if len(lens) > 1 else -1, table_extra=0)
        if len(lens) == 1:
            r.table.zero_()
            Q.set_pool(r, *Q.quantised(torch.randn(r.pool.shape)))
        c, q = Q.on_gpu(r), R.queries(r, torch.float32).cuda()
        NP = c["k"].shape[0]
        scale = [s.squeeze(1).contiguous().as_strided((NP, 1, P), (P if NP > 1 else 1, 1, 1)) for s in (c["ks"], c["vs"])]
        cache = [x.squeeze(2).contiguous().as_strided((NP, P, 1, 128), (P * 128 if NP > 1 else 3, 128, 1, 1)) for x in (c["k"], c["v"])]
        out = torch.zeros(len(lens), 4, 128, dtype=BF, device="cuda")
        v.vh_quant_decode_attn(q, *cache, *scale, c["table"], c["lens"], c["active"], out, v.alloc_workspace(len(lens), 4, 1, 128, P))
        bad = Q.differs(out, Q.attention(r, q.cpu()), BF)
        assert bad is None, bad


@pytest.mark.parametrize("num_ctas", [1, 2, 3, 7, 40, 1000])
def test_decode_split_rows(num_ctas):
    check_decode(Q.make([900, 3, 411, 1], [1] * 4, window=700, sinks=20, seed=num_ctas), num_ctas=num_ctas)


@pytest.mark.parametrize("B", [128, 129, 700])
def test_decode_many_rows(B):
    lens = [1 + (29 * b) % 75 for b in range(B)]
    lens[B // 2] = 1500
    check_decode(Q.make(lens, [1] * B, Hq=2, Hkv=1, D=64, window=40, sinks=3, active=[int(b % 9 != 4) for b in range(B)], seed=B))
    check_decode(Q.make(lens, [1] * B, Hq=2, Hkv=1, D=64, seed=B))


def test_decode_long_row_and_repeated_calls():
    r = Q.make([6000, 17], [1, 1], Hq=8, Hkv=1, window=5500, sinks=40, seed=3)
    check_decode(r)
    q = R.queries(r, torch.float32)
    ws = vh().alloc_workspace(2, 8, 1, 128, 16)
    a, _ = decode(r, q, ws=ws)
    b, _ = decode(r, q, ws=ws, repeat=3, pdl=True)
    assert torch.equal(a, b), "the same call gives other bits"


def test_decode_padding_rows_and_bad_rows():
    v = vh()
    r = Q.make([40, 9, 70], [1] * 3, window=32, sinks=2, active=[1, 0, 1], seed=5)
    q = R.queries(r, torch.float32)
    out, err = decode(r, q)
    assert err == 0 and (out[1] == 0).all()
    assert Q.differs(out, Q.attention(r, q), BF) is None
    for bad in (0, -4, 10 ** 6):  # a length out of range: zeros and a flag, the others as before
        r2 = R.Ragged(**{**r.__dict__, "lens": [40, 9, bad], "active": [1, 0, 1]})
        out2, err = decode(r2, q)
        assert err == v.VH_ERR_SEQLEN and (out2[2] == 0).all() and torch.equal(out2[0], out[0])


def test_decode_contiguous_cache():
    r = Q.make([11, 3, 7], [1] * 3, D=64, P=11, window=6, sinks=1, table_extra=0, seed=8, spare=-1)
    x = torch.randn(3, 2, 11, 8, 64)
    r.table = torch.arange(3, dtype=torch.int32).view(3, 1)
    Q.set_pool(r, *Q.quantised(x))
    check_decode(r, table=False)


def test_decode_bad_page_ids_are_flagged_and_read_as_zeros():
    for P in (16, 8):
        r = Q.make([40, 60], [1, 1], P=P, window=40, sinks=0, seed=12)
        q = R.queries(r, torch.float32)
        bad = R.Ragged(**{**r.__dict__, "table": r.table.clone()})
        page = int(bad.table[1, 32 // P])
        bad.table[1, 32 // P] = 1 << 28
        out, err = decode(bad, q)
        assert err == vh().VH_ERR_PAGE
        r.pool[page] = 0
        r.extra["scale"][page] = 0
        bad = Q.differs(out, Q.attention(r, q), BF)
        assert bad is None, bad


@pytest.mark.parametrize("dtype", [BF, FP])
def test_decode_scales_far_apart(dtype):
    """Keys, values and queries of very different sizes."""
    r = Q.make([300, 90], [1, 1], Hq=8, Hkv=2, seed=17)
    g = torch.Generator().manual_seed(1)
    sc = r.extra["scale"]
    by = torch.randint(-40, 41, sc[:, 1].shape, generator=g).double()
    sc[:, 1] *= (2.0 ** (by if dtype == BF else by / 8)).float()
    sc[:, 0] *= (2.0 ** torch.randint(-30, 3, sc[:, 0].shape, generator=g).double()).float()
    order = sc if r.layout == "HND" else sc.transpose(2, 3)
    Q.set_pool(r, r.extra["q8"], order.contiguous())
    q = R.queries(r, torch.float32)
    q *= (2.0 ** torch.randint(-20, 2, (2, 8, 1), generator=g).double()).float()
    q[0, 3, :100] *= 1e-6
    check_decode(r, dtype, q=q)


def test_decode_sharp_softmax_and_scale():
    check_decode(Q.make([400, 33], [1, 1], Hq=4, Hkv=2, window=150, sinks=4, seed=21, sigma=3.0), scale=0.7)
    r = Q.make([400, 33], [1, 1], Hq=4, Hkv=2, seed=22)
    check_decode(r, q=R.queries(r, torch.float32) * 40)


def test_decode_all_zero_heads():
    r = Q.make([50, 17], [1, 1], Hq=4, Hkv=2, seed=23)
    Q.set_pool(r, *Q.quantised(torch.zeros(r.pool.shape)))
    check_decode(r)
    check_decode(r, q=torch.zeros(2, 4, 128))


def test_decode_large_value_without_weight_among_tiny_ones():
    """Values near the least scale, and a huge one under a score that leaves it no weight."""
    r = Q.make([40], [1], Hq=4, Hkv=2, seed=24)
    x = torch.randn(r.pool.shape, generator=torch.Generator().manual_seed(2))
    x[:, 1] *= 2.0 ** -112
    page = int(r.table[0, 0])
    q = torch.full((1, 4, 128), 4.0)
    x[page, 0, 3], x[page, 1, 3] = -64.0, 2.0 ** 60   # (its score: 128 * 4 * -64 / sqrt(128) = -2896)
    x[:, 0][x[:, 0].abs() < 64] = 0.0
    Q.set_pool(r, *Q.quantised(x))
    check_decode(r, q=q)


def test_decode_nonfinite_scales_and_queries():
    """A key whose scale is NaN makes its rows NaN, a value its outputs, a query its head; others stay."""
    base = Q.make([300, 90, 40], [1, 1, 1], Hq=8, Hkv=2, window=200, sinks=4, seed=25)
    q = R.queries(base, torch.float32)
    order = lambda: (base.extra["scale"] if base.layout == "HND" else base.extra["scale"].transpose(2, 3)).clone()  # noqa: E731
    sc = order()
    page = int(base.table[0, 250 // 16])
    sc[page, 0, 250 % 16, 1] = math.nan       # row 0, kv head 1: its keys
    sc[int(base.table[1, 1]), 1, 3, 0] = math.nan   # row 1, kv head 0: its values
    Q.set_pool(base, base.extra["q8"], sc)
    q[2, 5, 17] = math.inf
    q[2, 2, 17] = math.nan
    out, err = decode(base, q)
    assert err == 0
    nan = torch.zeros(3, 8, dtype=torch.bool)
    nan[0, 4:] = nan[1, :4] = nan[2, 5] = nan[2, 2] = True
    assert torch.equal(torch.isnan(out).all(-1), nan) and torch.equal(torch.isnan(out).any(-1), nan)
    q[2, 5, 17] = q[2, 2, 17] = 0
    ref = Q.attention(base, q)
    for b in range(3):
        keep = ~nan[b]
        bad = Q.differs(out[b][keep], (ref[0][b][keep], ref[1][b][keep]), BF)
        assert bad is None, bad


def test_offsets_beyond_32_bits():
    """Pages whose bytes lie more than 2^32 into the pool: the same bits as in a small pool, in every call."""
    v = vh()
    P, HKV, D, lens = 16, 8, 128, [70, 33]
    far = (1 << 32) // (2 * P * HKV * D) + 3
    small = Q.make(lens, [1, 1], P=P, seed=4)
    n = small.pool.shape[0]
    by, sc = small.extra["q8"].view(torch.uint8).cuda(), small.extra["scale"].cuda()
    big = torch.zeros(far + n, 2, P, HKV, D, dtype=torch.uint8, device="cuda")
    big[far:] = by
    big_sc = torch.zeros(far + n, 2, HKV, P, device="cuda")
    big_sc[far:] = sc
    table = torch.where(small.table > 0, small.table + far, small.table).cuda()
    x = torch.randn(2, 32, D).to(BF).cuda()
    cs = v.vh_rope_table(torch.empty(128, D, device="cuda"))
    got = []
    for pool, scale, t in ((by.clone(), sc.clone(), small.table.cuda()), (big, big_sc, table)):
        k, val = (pool.view(Q.E4M3)[:, i] for i in (0, 1))
        cache = (k, val, scale[:, 0], scale[:, 1])
        q32 = torch.empty(2, 16, D, device="cuda")
        rows = (t, i32(lens), i32([1, 1]))
        out = torch.zeros(2, 16, D, dtype=BF, device="cuda")
        v.vh_quant_kv_append(x[:, :16], x[:, 16:24], x[:, 24:], cs, *cache, *rows, q32)
        v.vh_quant_decode_attn(q32, *cache, *rows, out, v.alloc_workspace(2, 16, HKV, D, P))
        back = torch.zeros(2, 2, 80, HKV, D, dtype=BF, device="cuda")
        v.vh_quant_kv_read(*cache, *rows, back[:, 0], back[:, 1], None)
        torch.cuda.synchronize()
        got.append((out, back, pool[-n:].clone(), scale[-n:].nan_to_num(-1)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.isfinite(got[0][0].float()).all()


# ---- read-back -------------------------------------------------------------------------------------------------------------

def check_read(r, dtype=BF, P2=16, sinks=0, first=None, contiguous=False, layout2="NHD", bad=None):
    """bad: (row, page number) of 16-bit pages without a place."""
    v, c = vh(), Q.on_gpu(r)
    per_row = max(1, -(-max(r.lens) // P2)) if not contiguous else 1
    if contiguous:
        P2 = max(r.lens)
        table, NP = None, r.B
    else:
        NP = r.B * per_row + 1
        table = (1 + torch.randperm(NP - 1, generator=r.extra["gen"])).view(r.B, per_row).to(torch.int32)
        if bad:
            table[bad] = NP
    shape = (NP, 2, P2, r.Hkv, r.D) if layout2 == "NHD" else (NP, 2, r.Hkv, P2, r.D)
    out = torch.full(shape, 7.0, dtype=dtype, device="cuda")
    view = lambda x, i: x[:, i] if layout2 == "NHD" else x[:, i].transpose(1, 2)  # noqa: E731
    v.vh_quant_kv_read(c["k"], c["v"], c["ks"], c["vs"], c["table"], c["lens"], c["active"], view(out, 0), view(out, 1),
                       None if table is None else table.cuda(), first_slot=None if first is None else i32(first), sinks=sinks,
                       err_flag=c["err"])
    torch.cuda.synchronize()
    want = torch.full(shape, 7.0, dtype=dtype)
    for b in range(r.B):
        if not r.active[b]:
            continue
        for j in range(r.lens[b]):
            if first is not None and j < first[b] and j >= sinks:
                continue
            page, off = int(r.table[b, j // r.P]), j % r.P
            to, to_off = (b, j) if contiguous else (int(table[b, j // P2]), j % P2)
            if not 0 <= to < NP:
                continue
            for i in (0, 1):
                # e4m3 times the scale, one rounding to fp32 and one to 16 bits
                y = r.view(r.extra["q8"], i)[page, off].float() * r.extra["scale"][page, i, :, off][:, None]
                view(want, i)[to, to_off] = y.to(dtype)
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))
    return int(c["err"])


@pytest.mark.parametrize("P", [8, 16, 48])
@pytest.mark.parametrize("P2,contiguous", [(16, False), (8, False), (64, False), (0, True)])
def test_read_pages(P, P2, contiguous):
    assert check_read(Q.make([1, 16, 40, 200, 129], [1] * 5, P=P, seed=P, active=[1, 1, 0, 1, 1]), P2=P2, contiguous=contiguous) == 0


@pytest.mark.parametrize("heads", [1, 3, 5, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_read_heads(heads, D, dtype):
    check_read(Q.make([70, 33], [1, 1], Hq=heads, Hkv=heads, D=D, layout="HND", seed=D + heads), dtype, layout2="HND" if heads == 5 else "NHD")


@pytest.mark.parametrize("sinks", [0, 1, 4, 40])
def test_read_windows(sinks):
    r = Q.make([100, 300, 5, 64], [1] * 4, window=30, sinks=sinks, seed=sinks)
    first = [max(0, n - 30) for n in r.lens]
    assert check_read(r, first=first, sinks=sinks) == 0


def test_read_many_rows_and_bad_ones():
    lens = [1 + (11 * b) % 90 for b in range(300)]
    assert check_read(Q.make(lens, [1] * 300, Hq=1, Hkv=1, D=64, seed=1, active=[int(b % 7 != 3) for b in range(300)])) == 0
    v = vh()
    r = Q.make([40, 60], [1, 1], seed=2)
    assert check_read(r, bad=(1, 2)) == v.VH_ERR_PAGE
    c = Q.on_gpu(r)
    out = torch.full((10, 2, 16, 8, 128), 7.0, dtype=BF, device="cuda")
    table = torch.arange(1, 9, dtype=torch.int32, device="cuda").view(2, 4)
    for lens, first in (([0, -1], None), ([65, 10 ** 6], None), ([40, 60], [-1, -5]), ([40, 60], [40, 100])):
        c["err"].zero_()
        v.vh_quant_kv_read(c["k"], c["v"], c["ks"], c["vs"], c["table"], i32(lens), c["active"], out[:, 0], out[:, 1], table,
                           first_slot=None if first is None else i32(first), err_flag=c["err"])
        torch.cuda.synchronize()
        assert int(c["err"]) == (0 if first == [40, 100] else v.VH_ERR_SEQLEN) and (out == 7.0).all()
    bad = c["table"].clone()
    bad[0, 1] = -3
    v.vh_quant_kv_read(c["k"], c["v"], c["ks"], c["vs"], bad, c["lens"], c["active"], out[:, 0], out[:, 1], table, err_flag=c["err"])
    torch.cuda.synchronize()
    assert int(c["err"]) == v.VH_ERR_PAGE and not out[2].any() and (out[1] != 7.0).any()
