"""RoPE with several axes and the ragged append on a GB300, against float64."""
import pytest
import torch

import window_ref as R

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def vh():
    import paged_len_decode_gb300 as v
    return v


def run(lens, news, heads=(16, 8), D=128, P=16, dtype=BF, layout="NHD", axes=None, axis_count=3, q16=False, norm=False,
        interleaved=False, packed=False, one_each=False, active=None, positions=True, seed=0, extra=0, max_pos=4096):
    """Run the append and check every output; returns the error bits."""
    v = vh()
    Hq, Hkv = heads
    r = R.make(lens, news, Hq, Hkv, D=D, P=P, dtype=dtype, layout=layout, active=active, seed=seed)
    g = r.extra["gen"]
    T = r.starts[-1] + extra
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dtype)
    pos = torch.randint(0, max_pos, (axis_count, T), generator=g, dtype=torch.int32) if positions else None
    w = [1 + 0.2 * torch.randn(D, generator=g) for _ in range(2)] if norm else [None, None]
    before = r.pool.clone()
    pool, xc = r.pool.cuda(), x.cuda()
    q, k, val = xc[:, :Hq], xc[:, Hq:Hq + Hkv], xc[:, Hq + Hkv:]
    if not packed:
        q, k, val = q.contiguous(), k.contiguous(), val.contiguous()
    cs = v.vh_rope_table(torch.empty(max_pos, D, device="cuda"))
    q_rot = torch.full((T, Hq, D), 7.0, dtype=dtype if q16 else torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    v.vh_mrope_kv_append(q, k, val, cs, r.view(pool, 0), r.view(pool, 1), r.table.cuda(), i32(r.lens), i32(r.active), q_rot,
                         token_start=None if one_each else i32(r.starts), positions=None if pos is None else pos.cuda(),
                         pair_axis=axes, err_flag=err, q_norm_w=None if w[0] is None else w[0].cuda(),
                         k_norm_w=None if w[1] is None else w[1].cuda(), interleaved=interleaved)
    torch.cuda.synchronize()
    q_rot, pool, cs = q_rot.cpu(), pool.cpu(), cs.cpu()
    # the reference
    ax = torch.tensor(axes if axes is not None else [0] * (D // 2))
    slot = torch.zeros(T, dtype=torch.long)
    row = torch.zeros(T, dtype=torch.long)
    live = torch.zeros(T, dtype=torch.bool)
    for b in range(r.B):
        a, e = r.starts[b], r.starts[b + 1]
        slot[a:e] = torch.arange(lens[b] - news[b], lens[b])
        row[a:e] = b
        live[a:e] = bool(r.active[b])
    p = (pos.long()[ax] if pos is not None else slot.expand(D // 2, T)).t()  # [T, D/2]
    p = torch.where(live[:, None], p, torch.zeros_like(p))
    i = torch.arange(D // 2)
    cos, sin = cs[p, i], cs[p, D // 2 + i]
    half = torch.finfo(dtype).eps / 2
    yq, eq = R.rope(x[:, :Hq], cos, sin, w[0], 1e-6, interleaved)
    yk, ek = R.rope(x[:, Hq:Hq + Hkv], cos, sin, w[1], 1e-6, interleaved)
    tiny = 2.0 ** -25  # half of the least fp16
    tq = eq + (half * (yq.abs() + eq) + tiny if q16 else 0)
    assert ((q_rot[live].double() - yq[live]).abs() <= tq[live]).all()
    assert (q_rot[~live] == 7.0).all()
    want = before.clone()
    kw, vw = r.view(want, 0), r.view(want, 1)
    kg = r.view(pool, 0)
    pages = r.table[row, slot // P].long()
    got_k = kg[pages[live], slot[live] % P]
    assert ((got_k.double() - yk[live]).abs() <= (ek + half * (yk.abs() + ek) + tiny)[live]).all()
    kw[pages[live], slot[live] % P] = got_k
    vw[pages[live], slot[live] % P] = x[live][:, Hq + Hkv:]
    assert torch.equal(want.view(torch.int16), pool.view(torch.int16)), "values differ, or another slot was written"
    return int(err)


SECTIONS = [0] * 16 + [1] * 24 + [2] * 24


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("q16", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_prompt_tokens(dtype, q16, interleaved, norm):
    assert run([37, 1, 200, 16], [37, 1, 9, 0], dtype=dtype, q16=q16, interleaved=interleaved, norm=norm, axes=SECTIONS, extra=5) == 0


@pytest.mark.parametrize("heads,D", [((1, 1), 64), ((8, 1), 128), ((6, 3), 64), ((40, 5), 128), ((64, 8), 64)])
@pytest.mark.parametrize("P,layout", [(8, "NHD"), (16, "HND"), (48, "NHD"), (1024, "HND")])
def test_heads_pages_packed(heads, D, P, layout):
    v = vh()
    axes = v.mrope_pair_axis([D // 2 - 20, 10, 10], D, cyclic=True)
    assert run([70, 3], [64, 2], heads=heads, D=D, P=P, layout=layout, axes=axes, packed=True, q16=True) == 0


@pytest.mark.parametrize("B", [1, 5, 33, 64])
def test_one_token_a_row(B):
    lens = [1 + (37 * b) % 90 for b in range(B)]
    assert run(lens, [1] * B, one_each=True, axes=SECTIONS, active=[int(b % 5 != 3) for b in range(B)], packed=True) == 0


def test_many_rows_and_many_tokens():
    # more rows than one round of the row search probes, and more tokens than one a CTA
    news = [(b * 7) % 4 for b in range(1300)]
    assert run([n + 3 for n in news], news, heads=(2, 1), D=64, P=8, axes=None, axis_count=1) == 0
    news = [700, 1, 0, 1999]
    assert run(news, news, heads=(4, 2), axes=SECTIONS, q16=True) == 0


def test_positions_from_slots_and_four_axes():
    assert run([90, 17], [60, 17], positions=False) == 0
    assert run([90, 17], [60, 17], axes=[i % 4 for i in range(64)], axis_count=4) == 0


def test_same_bits_as_the_single_axis_append():
    """One token a row, one axis: what vh_rope_kv_append gives."""
    v = vh()
    r = R.make([5, 40, 17], [1] * 3, seed=4)
    g = r.extra["gen"]
    q, k, val = (torch.randn(3, h, 128, generator=g).to(BF).cuda() for h in (16, 8, 8))
    cs = v.vh_rope_table(torch.empty(64, 128, device="cuda"))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    got = []
    for f in (v.vh_rope_kv_append, v.vh_mrope_kv_append):
        pool, out = r.pool.cuda(), torch.zeros(3, 16, 128, device="cuda")
        f(q, k, val, cs, r.view(pool, 0), r.view(pool, 1), r.table.cuda(), i32(r.lens), i32(r.active), out)
        got.append((pool.cpu().view(torch.int16), out.cpu()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_bad_positions_pages_and_rows_are_flagged():
    v = vh()
    r = R.make([20, 20, 20], [2, 2, 2], Hq=2, Hkv=1, D=64, seed=6)
    x = torch.randn(6, 4, 64).to(BF).cuda()
    cs = v.vh_rope_table(torch.empty(64, 64, device="cuda"))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731

    def call(pos=None, table=None, lens=None, starts=None):
        pool, out = r.pool.cuda(), torch.full((6, 2, 64), 7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        v.vh_mrope_kv_append(x[:, :2], x[:, 2:3], x[:, 3:], cs, r.view(pool, 0), r.view(pool, 1),
                             i32(table if table is not None else r.table.tolist()), i32(lens or r.lens), i32([1] * 3), out,
                             token_start=i32(starts or r.starts), positions=i32(pos or [[1] * 6] * 2),
                             pair_axis=[0] * 32, err_flag=err)
        torch.cuda.synchronize()
        wrote = (out != 7.0).flatten(1).any(1).tolist()
        slots = (pool.cpu().view(torch.int16) != r.pool.view(torch.int16)).flatten(2).any(2)[:, 0].sum().item()
        return int(err), wrote, slots

    yes = [True] * 6
    assert call()[:2] == (0, yes)
    for axis in (0, 1):  # the second axis is checked although no pair takes it
        for bad in (-1, 64):
            pos = [[1] * 6, [1] * 6]
            pos[axis][3] = bad
            assert call(pos=pos)[:2] == (v.VH_ERR_POS, [True, True, True, False, True, True])
    t = r.table.clone()
    t[2, 1] = 10 ** 8
    assert call(table=t.tolist())[:2] == (v.VH_ERR_PAGE, yes)
    for lens in ([20, 1, 20], [20, 10 ** 7, 20], [20, -3, 20]):
        assert call(lens=lens)[:2] == (v.VH_ERR_SEQLEN, [True, True, False, False, True, True])
    err, wrote, _ = call(starts=[0, 2, 4, 9])  # tokens past the arrays
    assert err == v.VH_ERR_SEQLEN and wrote == [True, True, True, True, False, False]


def test_no_tokens():
    """An empty batch of tokens is accepted by the append and the prompt attention, and writes nothing."""
    v = vh()
    r = R.make([5, 7], [0, 0], Hq=4, Hkv=2, D=64, seed=2)
    pool = r.pool.cuda()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.zeros(0, 8, 64, dtype=BF, device="cuda")
    q_rot = torch.zeros(0, 4, 64, dtype=BF, device="cuda")
    k, val = r.view(pool, 0), r.view(pool, 1)
    rows = (r.table.cuda(), i32(r.lens), i32(r.active))
    v.vh_mrope_kv_append(x[:, :4], x[:, 4:6], x[:, 6:], v.vh_rope_table(torch.empty(8, 64, device="cuda")), k, val, *rows, q_rot,
                         token_start=i32(r.starts))
    ws = v.alloc_prompt_workspace(0, 2, 4, 2, 64)
    v.vh_window_prompt_attn(q_rot, k, val, rows[0], i32(r.starts), *rows[1:], torch.zeros_like(q_rot), ws)
    torch.cuda.synchronize()
    assert torch.equal(pool.cpu().view(torch.int16), r.pool.view(torch.int16))


def test_offsets_out_of_order_write_no_foreign_slots():
    """With more than 32 rows a token's row is searched; offsets out of order (not allowed, but data) may lead the
    search to a row that starts behind the token.  Nothing may be written then but slots of the rows' own new tokens."""
    v = vh()
    B, T, P, Hq, Hkv, D = 40, 200, 16, 4, 2, 64
    g = torch.Generator().manual_seed(9)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(BF).cuda()
    cs = v.vh_rope_table(torch.empty(256, D, device="cuda"))
    per = 16  # pages a row: up to 256 tokens
    table = torch.arange(B * per, dtype=torch.int32).view(B, per).cuda()
    for _ in range(8):
        starts = torch.randint(0, T + 1, (B + 1,), generator=g).tolist()
        lens = [max(0, e - a) for a, e in zip(starts, starts[1:])]
        pool = torch.full((B * per + 2, 2, P, Hkv, D), 5.0, dtype=BF, device="cuda")
        inner = pool[1:-1]  # a page on either side that no table entry names
        q_rot = torch.full((T, Hq, D), 7.0, device="cuda")
        v.vh_mrope_kv_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cs, inner[:, 0], inner[:, 1], table, i32(lens),
                             i32([1] * B), q_rot, token_start=i32(starts))
        torch.cuda.synchronize()
        wrote = (pool != 5.0).flatten(3).any(3)[:, 0].cpu()
        assert not wrote[0].any() and not wrote[-1].any()
        by_row = wrote[1:-1].reshape(B, per * P)
        for b in range(B):
            assert not by_row[b, lens[b]:].any()
