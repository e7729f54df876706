"""The 8-bit cache and drafted trees together, as a model's layer calls them: prompts in chunks whose context is read
back into 16-bit pages, single tokens over the 8-bit cache, drafted tokens as a tree over what is read back; eager on a side
stream, captured in CUDA graphs and replayed with other lengths, and two at once.  Every attention is compared with float64
over what the cache holds at that moment (what the appends write has tests of its own)."""
import math
import os
import random
import re

import pytest
import torch

import quant_ref as Q
import test_gpu_quant as TQ
import test_gpu_tree as TT
import window_ref as R

pytestmark = pytest.mark.gpu
HQ, HKV, D, P, W, S = 8, 2, 128, 16, 40, 3
CASES = int(os.environ.get("VH_QUANT_FUZZ_CASES", "24"))


def vh():
    import paged_len_decode_gb300 as v
    return v


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Layer:
    """One layer's two caches, with page tables of their own, and B requests."""

    def __init__(self, B, most, dtype, seed, head_major=False):
        v, g = vh(), torch.Generator().manual_seed(seed)
        self.B, self.dtype, self.g = B, dtype, g
        per_row = -(-most // P)
        tables = [(1 + torch.randperm(B * per_row, generator=g)).view(B, per_row).to(torch.int32) for _ in range(2)]
        self.table, self.table16 = (t.cuda() for t in tables)
        NP = B * per_row + 1
        self.k, self.v, self.ks, self.vs = v.alloc_quant_cache(NP, P, HKV, D, head_major)
        for t in (self.k, self.v):
            t.view(torch.uint8).fill_(Q.NAN_BYTE)
        self.ks.fill_(math.nan)
        self.vs.fill_(math.nan)
        self.pool16 = torch.full((NP, 2, P, HKV, D), math.nan, dtype=dtype, device="cuda")
        self.k16, self.v16 = self.pool16[:, 0], self.pool16[:, 1]
        self.cos_sin = v.vh_rope_table(torch.empty(500, D, device="cuda"))
        self.active = i32([1] * B)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    @property
    def cache(self):
        return self.k, self.v, self.ks, self.vs

    def tokens(self, T):
        return torch.randn(T, HQ + 2 * HKV, D, generator=self.g).to(self.dtype).cuda()

    def held8(self, lens, news, window, sinks):
        """tests/quant_ref.py's batch of the 8-bit cache as it is now (its pool in the layout [NP, 2, P, Hkv, D])."""
        torch.cuda.synchronize()
        r = R.Ragged(HQ, HKV, D, P, None, "NHD", self.table.cpu(), lens, news, [1] * self.B, window, sinks)
        q8 = torch.stack([self.k.view(torch.uint8).cpu(), self.v.view(torch.uint8).cpu()], 1)
        scale = torch.stack([self.ks.cpu(), self.vs.cpu()], 1)
        Q.set_pool(r, q8.view(Q.E4M3), scale.transpose(2, 3).contiguous())
        return r

    def held16(self, lens, news, window, sinks):
        torch.cuda.synchronize()
        return R.Ragged(HQ, HKV, D, P, self.pool16.cpu(), "NHD", self.table16.cpu(), lens, news, [1] * self.B, window, sinks)

    def check8(self, q_rot, out, lens, window=0, sinks=0):
        r = self.held8(lens, [1] * self.B, window, sinks)
        bad = Q.differs(out, Q.attention(r, q_rot.cpu(), dtype=self.dtype), self.dtype)
        assert bad is None, bad


def starts_of(news):
    s = [0]
    for n in news:
        s.append(s[-1] + n)
    return s


def append8(m, x, lens, q_rot, starts=None, positions=None):
    vh().vh_quant_kv_append(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], m.cos_sin, *m.cache, m.table, lens, m.active, q_rot,
                            token_start=starts, positions=positions, err_flag=m.err)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("head_major", [False, True])
def test_prompts_single_tokens_and_drafts_on_a_side_stream(dtype, head_major):
    v = vh()
    m = Layer(3, 300, dtype, 3, head_major)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lens = [0, 0, 0]
        for news in ([100, 3, 64], [1, 61, 0], [33, 8, 90]):   # chunks of prompts under a window
            lens = [a + b for a, b in zip(lens, news)]
            T, start = sum(news), i32(starts_of(news))
            x, q = m.tokens(T), torch.empty(T, HQ, D, dtype=dtype, device="cuda")
            out, ws = torch.zeros_like(q), v.alloc_prompt_workspace(T, 3, HQ, HKV, D)
            append8(m, x, i32(lens), q, start)
            first = [max(0, n - k - W + 1) for n, k in zip(lens, news)]
            v.vh_quant_kv_read(*m.cache, m.table, i32(lens), m.active, m.k16, m.v16, m.table16, first_slot=i32(first), sinks=S,
                               err_flag=m.err)
            v.vh_window_prompt_attn(q, m.k16, m.v16, m.table16, start, i32(lens), m.active, out, ws, window=W, sinks=S, err_flag=m.err)
            bad = R.close(out, R.attention(m.held16(lens, news, W, S), q.cpu()), dtype, D, False)
            assert bad is None, bad
        ws = v.alloc_workspace(3, HQ, HKV, D, P)
        for window, sinks in ((W, S), (0, 0), (W, S)):
            lens = [n + 1 for n in lens]
            q, out = torch.empty(3, HQ, D, device="cuda"), torch.zeros(3, HQ, D, dtype=dtype, device="cuda")
            append8(m, m.tokens(3), i32(lens), q)
            v.vh_quant_decode_attn(q, *m.cache, m.table, i32(lens), m.active, out, ws, window=window, sinks=sinks, err_flag=m.err, pdl=True)
            m.check8(q, out, lens, window, sinks)
        # drafted tokens, positions by their depth, over the context read back
        v.vh_quant_kv_read(*m.cache, m.table, i32(lens), m.active, m.k16, m.v16, m.table16, err_flag=m.err)
        parents = [Q.parents(n, m.g) for n in (17, 1, 40)]
        news = [len(p) for p in parents]
        T, start, drafted = sum(news), i32(starts_of(news)), [a + b for a, b in zip(lens, news)]
        mask = v.tree_masks(parents)
        depth = torch.tensor([bin(int(x) & (1 << 64) - 1).count("1") for x in mask.cpu()[:, 0]], dtype=torch.int32)
        pos = (torch.tensor([n for n, k in zip(lens, news) for _ in range(k)], dtype=torch.int32) + depth).cuda()
        x, q = m.tokens(T), torch.empty(T, HQ, D, dtype=dtype, device="cuda")
        out = torch.zeros_like(q)
        v.vh_mrope_kv_append(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], m.cos_sin, m.k16, m.v16, m.table16, i32(drafted), m.active, q,
                             token_start=start, positions=pos, err_flag=m.err)
        for window, sinks in ((0, 0), (W, S)):
            v.vh_tree_attn(q, m.k16, m.v16, m.table16, start, i32(drafted), m.active, mask, out, v.alloc_prompt_workspace(T, 3, HQ, HKV, D),
                           window=window, sinks=sinks, err_flag=m.err)
            bad = R.close(out, Q.tree(parents, m.held16(drafted, news, window, sinks), q.cpu()), dtype, D, False)
            assert bad is None, bad
    assert int(m.err) == 0


def test_captured_steps_with_other_lengths():
    """One graph of append and attention, one of read-back and tree attention, with static shapes; two of the first on one
    workspace, one after the other."""
    v = vh()
    m = Layer(4, 200, torch.bfloat16, 9)
    B, T = 4, 64
    lens, drafted, starts = i32([1] * B), i32([1] * B), i32([0] * (B + 1))
    x, xt = m.tokens(B), m.tokens(T)
    q, qt = torch.empty(B, HQ, D, device="cuda"), torch.empty(T, HQ, D, dtype=m.dtype, device="cuda")
    out, out2, ot = (torch.zeros(n, HQ, D, dtype=m.dtype, device="cuda") for n in (B, B, T))
    mask, ws, wt = torch.zeros(T, 1, dtype=torch.int64, device="cuda"), v.alloc_workspace(B, HQ, HKV, D, P), v.alloc_prompt_workspace(T, B, HQ, HKV, D)

    def step(o):
        append8(m, x, lens, q)
        v.vh_quant_decode_attn(q, *m.cache, m.table, lens, m.active, o, ws, err_flag=m.err)

    def draft():
        v.vh_quant_kv_read(*m.cache, m.table, lens, m.active, m.k16, m.v16, m.table16, err_flag=m.err)
        v.vh_mrope_kv_append(xt[:, :HQ], xt[:, HQ:HQ + HKV], xt[:, HQ + HKV:], m.cos_sin, m.k16, m.v16, m.table16, drafted, m.active, qt,
                             token_start=starts, err_flag=m.err)
        v.vh_tree_attn(qt, m.k16, m.v16, m.table16, starts, drafted, m.active, mask, ot, wt, err_flag=m.err)

    step(out)   # first calls, outside any capture
    draft()
    torch.cuda.synchronize()
    s, graphs = torch.cuda.Stream(), []
    for f in (lambda: step(out), lambda: step(out2), draft):
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            f()
        graphs.append(g)
    torch.cuda.current_stream().wait_stream(s)
    for held in range(2, 120):
        lens.copy_(i32([held, max(1, held // 2), 1 + held % 17, held]))
        x.copy_(m.tokens(B))
        graphs[held % 2].replay()
        if held in (2, 15, 16, 17, 60, 119):
            m.check8(q, (out, out2)[held % 2], lens.tolist())
    at = lens.tolist()
    # the rows' slots that no step wrote hold NaN: they are written first
    for n in range(1, max(at) + 1):
        lens.copy_(i32([min(n, k) for k in at]))
        x.copy_(m.tokens(B))
        graphs[0].replay()
    lens.copy_(i32(at))
    m.check8(q, out, at)
    for news in ([1, 1, 1, 1], [20, 0, 3, 41], [64, 0, 0, 0]):
        parents = [Q.parents(n, m.g) for n in news]
        mine = v.tree_masks(parents)
        mask[:mine.shape[0]] = mine
        starts.copy_(i32(starts_of(news)))
        drafted.copy_(i32([a + b for a, b in zip(at, news)]))
        xt.copy_(m.tokens(T))
        ot.fill_(9.0)
        graphs[2].replay()
        t = sum(news)
        bad = R.close(ot[:t], Q.tree(parents, m.held16(drafted.tolist(), news, 0, 0), qt[:t].cpu()), m.dtype, D, False)
        assert bad is None, bad
        assert (ot[t:] == 9.0).all()
    assert int(m.err) == 0


def test_two_calls_at_once_with_workspaces_of_their_own():
    v = vh()
    cases = []
    for seed, heads in ((1, (16, 8)), (2, (8, 1))):
        r = Q.make([900, 77, 1500], [1] * 3, Hq=heads[0], Hkv=heads[1], seed=seed)
        q = R.queries(r, torch.float32)
        cases.append((r, q, Q.on_gpu(r), q.cuda(), torch.zeros(3, heads[0], 128, dtype=torch.bfloat16, device="cuda"),
                      v.alloc_workspace(3, *heads, 128, 16), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for r, q, c, qg, out, ws, s in cases:
            with torch.cuda.stream(s):
                v.vh_quant_decode_attn(qg, c["k"], c["v"], c["ks"], c["vs"], c["table"], c["lens"], c["active"], out, ws, err_flag=c["err"])
    torch.cuda.synchronize()
    for r, q, c, qg, out, ws, s in cases:
        assert int(c["err"]) == 0
        bad = Q.differs(out, Q.attention(r, q), torch.bfloat16)
        assert bad is None, bad


def test_small_workspaces_are_refused():
    v = vh()
    r = Q.make([40, 9], [1, 1], seed=1)
    c, q = Q.on_gpu(r), R.queries(r, torch.float32).cuda()
    out = torch.full((2, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = v.alloc_workspace(2, 16, 8, 128, 16)
    need = v.vh_decode_workspace_bytes(2, 16, 8, 128, 16, 5)
    args = (q, c["k"], c["v"], c["ks"], c["vs"], c["table"], c["lens"], c["active"], out)
    with pytest.raises(v.VHError):
        v.vh_quant_decode_attn(*args, ws[:need - 1].contiguous(), num_ctas=5)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
    v.vh_quant_decode_attn(*args, ws[:need].contiguous(), num_ctas=5)
    assert Q.differs(out, Q.attention(r, q.cpu()), torch.bfloat16) is None
    with pytest.raises(ValueError):
        v.vh_quant_decode_attn(q, c["k"], c["v"], c["ks"].cpu(), c["vs"].cpu(), *args[5:], ws)


@pytest.mark.parametrize("P", [1, 3, 15, 100])
def test_caches_of_one_small_page_a_row(P):
    """Contiguous caches whose page, and so their tiles' boxes, are of any size."""
    v = vh()
    B, D_ = 3, 64
    cache = v.alloc_quant_cache(B, P, 2, D_)
    g = torch.Generator().manual_seed(P)
    lens = [P, max(1, P // 2), 1]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lens), 8, D_, generator=g).to(torch.bfloat16).cuda()
    cs = v.vh_rope_table(torch.empty(128, D_, device="cuda"))
    q16 = torch.empty(sum(lens), 4, D_, dtype=torch.bfloat16, device="cuda")
    starts, act = i32(starts_of(lens)), i32([1] * B)
    v.vh_quant_kv_append(x[:, :4], x[:, 4:6], x[:, 6:], cs, *cache, None, i32(lens), act, q16, token_start=starts, err_flag=err)
    q, out = torch.randn(B, 4, D_, generator=g), torch.zeros(B, 4, D_, dtype=torch.bfloat16, device="cuda")
    v.vh_quant_decode_attn(q.cuda(), *cache, None, i32(lens), act, out, v.alloc_workspace(B, 4, 2, D_, P), err_flag=err)
    back = torch.zeros(B, 2, P, 2, D_, dtype=torch.bfloat16, device="cuda")
    v.vh_quant_kv_read(*cache, None, i32(lens), act, back[:, 0], back[:, 1], None, err_flag=err)
    mask = v.tree_masks([list(range(-1, n - 1)) for n in lens])
    tree_out = torch.zeros_like(q16)
    v.vh_tree_attn(q16, back[:, 0], back[:, 1], None, starts, i32(lens), act, mask, tree_out,
                   v.alloc_prompt_workspace(sum(lens), B, 4, 2, D_), err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    r = R.Ragged(4, 2, D_, P, None, "NHD", torch.arange(B, dtype=torch.int32).view(B, 1), lens, [1] * B, [1] * B, 0, 0)
    q8 = torch.stack([c.view(torch.uint8).cpu() for c in cache[:2]], 1)
    Q.set_pool(r, q8.view(Q.E4M3), torch.stack([c.cpu() for c in cache[2:]], 1).transpose(2, 3).contiguous())
    bad = Q.differs(out, Q.attention(r, q, contiguous=True), torch.bfloat16)
    assert bad is None, bad
    assert torch.equal(back.cpu().double()[0], r.pool[0].float().to(torch.bfloat16).double())
    r16 = R.Ragged(4, 2, D_, P, back.cpu(), "NHD", r.table, lens, lens, [1] * B, 0, 0)
    bad = R.close(tree_out, R.attention(r16, q16.cpu()), torch.bfloat16, D_, False)
    assert bad is None, bad


def test_thousands_of_rows():
    lens = [1 + b % 3 for b in range(9000)]
    lens[4321] = 700
    r = Q.make(lens, [1] * 9000, Hq=1, Hkv=1, D=64, seed=1, table_extra=0, active=[int(b % 11 != 5) for b in range(9000)])
    TQ.check_decode(r)
    assert TQ.check_read(r, contiguous=False, P2=16) == 0


def test_empty_calls():
    v = vh()
    cache, dev = v.alloc_quant_cache(4, 16, 2, 64), dict(device="cuda")
    table, rows, act = i32([[1, 2]]), i32([0]), i32([0])
    none = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, **dev)  # noqa: E731
    cs = v.vh_rope_table(torch.empty(8, 64, **dev))
    v.vh_quant_kv_append(none(0, 4, 64), none(0, 2, 64), none(0, 2, 64), cs, *cache, table, rows, act, none(0, 4, 64, dt=torch.float32),
                         token_start=i32([0, 0]))
    out = torch.full((1, 4, 64), 7.0, dtype=torch.bfloat16, **dev)
    v.vh_quant_decode_attn(none(1, 4, 64, dt=torch.float32), *cache, table, rows, act, out, v.alloc_workspace(1, 4, 2, 64, 16))
    pool = torch.full((4, 2, 16, 2, 64), 7.0, dtype=torch.bfloat16, **dev)
    v.vh_quant_kv_read(*cache, table, rows, act, pool[:, 0], pool[:, 1], table)
    v.vh_tree_attn(none(0, 4, 64), pool[:, 0], pool[:, 1], table, i32([0, 0]), rows, act, none(0, 1, dt=torch.int64), none(0, 4, 64),
                   v.alloc_prompt_workspace(0, 1, 4, 2, 64))
    torch.cuda.synchronize()
    assert (out == 0).all() and (pool == 7.0).all() and not cache[0].float().any()


# ---- seeded random cases ---------------------------------------------------------------------------------------------

def pick(rng, one_each):
    hkv = rng.choice([1, 1, 2, 3, 4, 8])
    heads = (hkv * rng.choice([1, 2, 4, 8]), hkv)
    B = rng.choice([1, 1, 2, 3, 5, 9, 40 if heads[0] <= 8 else 6])
    most = rng.choice([3, 17, 64, 130, 300, 900]) if B <= 5 else rng.choice([3, 40, 130])
    news = [1 if one_each else rng.choice([0, 1, 2, rng.randint(1, min(most, 150))]) for _ in range(B)]
    if sum(news) == 0:
        news[0] = 1
    lens = [max(n, rng.randint(1, most), 1) for n in news]
    return dict(lens=lens, news=news, Hq=heads[0], Hkv=heads[1], D=rng.choice([64, 128]), P=rng.choice([8, 16, 32, 48, 64, 128, 1024]),
                window=rng.choice([0, 0, 1, 2, 15, 16, 17, 64, 100, 500]), sinks=rng.choice([0, 0, 1, 4, 16, 33, 100, 1000]),
                layout=rng.choice(["NHD", "HND"]), seed=rng.randrange(1 << 30), active=[int(rng.random() > 0.1) for _ in range(B)],
                dead=rng.choice([-1, 1 << 30]))


DTYPES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("case", range(CASES))
def test_decode_cases(case):
    rng = random.Random(2000 + case)
    r = Q.make(**pick(rng, True), spread=rng.choice([0.0, 0.5, 2.0]), sigma=rng.choice([0.3, 1.0, 2.0]))
    TQ.check_decode(r, rng.choice(DTYPES), num_ctas=rng.choice([0, 0, 1, 2, 5, 33]), scale=rng.choice([0.0, 0.05]), pdl=rng.random() < 0.5,
                    pad=rng.choice([0, 1, 3]))


@pytest.mark.parametrize("case", range(CASES))
def test_tree_cases(case):
    rng = random.Random(3000 + case)
    r = R.make(**pick(rng, False), dtype=rng.choice(DTYPES))
    TT.fill_drafts(r)
    TT.check(r, rng.choice(["random", "random", "chain", "flat"]), splits=rng.choice([0, 0, 0, 1, 2, 4, 8]), scale=rng.choice([0.0, 0.05]),
             extra=rng.choice([0, 0, 3]))


@pytest.mark.parametrize("case", range(CASES))
def test_append_cases(case):
    rng = random.Random(4000 + case)
    k = pick(rng, rng.random() < 0.3)
    one = all(n == 1 for n in k["news"])
    err = TQ.append_case(k["lens"], k["news"], k["Hq"], k["Hkv"], k["D"], k["P"], rng.choice(DTYPES), q16=rng.random() < 0.5,
                         norm=rng.random() < 0.5, interleaved=rng.random() < 0.3, layout=k["layout"], packed=rng.random() < 0.5,
                         active=k["active"], one_each=one and rng.random() < 0.7, seed=k["seed"], extra=0 if one else rng.choice([0, 3]))[2]
    assert err == 0


@pytest.mark.parametrize("case", range(CASES))
def test_read_cases(case):
    rng = random.Random(6000 + case)
    k = pick(rng, True)
    r = Q.make(**k)
    first = [max(0, n - k["window"]) if k["window"] else 0 for n in k["lens"]]
    err = TQ.check_read(r, rng.choice(DTYPES), P2=rng.choice([8, 16, 48, 128]), sinks=k["sinks"], first=first,
                        contiguous=rng.random() < 0.2, layout2=rng.choice(["NHD", "HND"]))
    assert err == 0


def test_readme_example_runs_as_written():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    first, _, code = re.findall(r"```python\n(.*?)```", text, re.S)[:3]
    torch.manual_seed(8)
    e = {}
    exec(first, e)
    exec(code, e)
    torch.cuda.synchronize()
    held = e["held"].tolist()
    r = R.Ragged(e["Hq"], e["Hkv"], e["D"], e["P"], None, "NHD", e["page_table"].cpu(), held, [1] * 8, [1] * 8, 0, 0)
    q8 = torch.stack([e["k8"].view(torch.uint8).cpu(), e["v8"].view(torch.uint8).cpu()], 1)
    Q.set_pool(r, q8.view(Q.E4M3), torch.stack([e["ks"].cpu(), e["vs"].cpu()], 1).transpose(2, 3).contiguous())
    bad = Q.differs(e["out"], Q.attention(r, e["q8_rot"].cpu()), torch.bfloat16)
    assert bad is None, bad
    news = [len(p) for p in e["parents"]]
    r = R.Ragged(e["Hq"], e["Hkv"], e["D"], e["P"], e["pool"].cpu(), "NHD", e["page_table"].cpu(), e["drafted"].tolist(), news, [1] * 8, 0, 0)
    bad = R.close(e["tree_out"], Q.tree(e["parents"], r, e["q_tree"].cpu()), torch.bfloat16, e["D"], False)
    assert bad is None, bad
