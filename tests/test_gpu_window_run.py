"""The ragged append, the prompt attention and the windowed decode together, as
a model's layer calls them: a prompt in chunks, then single tokens, pages given
back behind the window; eager on a side stream, and captured in CUDA graphs."""
import pytest
import torch

import window_ref as R

pytestmark = pytest.mark.gpu
HQ, HKV, D, P, W, S = 8, 2, 128, 16, 40, 3
PAIRS = [0] * 16 + [1] * 24 + [2] * 24


def vh():
    import paged_len_decode_gb300 as v
    return v


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """One layer over a paged cache: its raw tokens, and what float64 makes of them."""

    def __init__(self, chunks, dtype, seed, layout="NHD"):
        v = vh()
        g = torch.Generator().manual_seed(seed)
        self.chunks = chunks                    # per call: new tokens of every row
        B = len(chunks[0])
        self.B, self.dtype = B, dtype
        total = [sum(c[b] for c in chunks) for b in range(B)]
        per_row = max(-(-t // P) for t in total)
        self.raw = [torch.randn(t, HQ + 2 * HKV, D, generator=g).to(dtype) for t in total]
        self.pos = [torch.randint(0, 500, (3, t), generator=g, dtype=torch.int32) for t in total]
        self.table = (1 + torch.randperm(B * per_row, generator=g)).view(B, per_row).to(torch.int32)
        NP = B * per_row + 1
        shape = (NP, 2, P, HKV, D) if layout == "NHD" else (NP, 2, HKV, P, D)
        pool = torch.empty(shape, dtype=dtype)
        pool.view(torch.int16).fill_(R.NAN_BITS)
        self.pool = pool.cuda()
        self.k, self.v = (self.pool[:, i] if layout == "NHD" else self.pool[:, i].transpose(1, 2) for i in (0, 1))
        self.cos_sin = v.vh_rope_table(torch.empty(500, D, device="cuda"))
        torch.cuda.synchronize()
        cs, half, ax = self.cos_sin.cpu(), D // 2, torch.tensor(PAIRS)
        self.q, self.keys, self.vals = [], [], []
        for b in range(B):
            at = self.pos[b].long()[ax].t()
            i = torch.arange(half)
            cos, sin = cs[at, i], cs[at, half + i]
            self.q.append(R.rope(self.raw[b][:, :HQ], cos, sin, None, 0, False)[0])
            self.keys.append(R.rope(self.raw[b][:, HQ:HQ + HKV], cos, sin, None, 0, False)[0].to(dtype))
            self.vals.append(self.raw[b][:, HQ + HKV:])

    def lens(self, c):
        return [sum(x[b] for x in self.chunks[:c + 1]) for b in range(self.B)]

    def call_inputs(self, c):
        """Tensors of call c: packed projection, positions, lengths, token starts."""
        n, lens = self.chunks[c], self.lens(c)
        x = torch.cat([self.raw[b][lens[b] - n[b]:lens[b]] for b in range(self.B)])
        pos = torch.cat([self.pos[b][:, lens[b] - n[b]:lens[b]] for b in range(self.B)], 1).contiguous()
        starts = [0]
        for k in n:
            starts.append(starts[-1] + k)
        return dict(x=x.cuda(), pos=pos.cuda(), lens=i32(lens), starts=i32(starts))

    def give_back(self, table, lens, n):
        """Pages that no query of the next call sees hold garbage ids and NaN."""
        table = table.clone()
        for b in range(self.B):
            low = max(0, lens[b] - n[b] + 1 - W)
            for j in range(-(-S // P), low // P):
                page = int(self.table[b, j])
                table[b, j] = -7 if j % 2 else 1 << 30
                self.pool[page].view(torch.int16).fill_(R.NAN_BITS)
        return table.cuda()

    def reference(self, c, q_dtype):
        """Float64 attention of call c's tokens and its bounds, per token in order."""
        outs = []
        for b in range(self.B):
            n, L = self.chunks[c][b], self.lens(c)[b]
            r = R.Ragged(HQ, HKV, D, max(1, L), torch.stack([self.keys[b][:L], self.vals[b][:L]])[None], "NHD",
                         torch.zeros(1, 1, dtype=torch.int32), [L], [n], [1], W, S)
            q = self.q[b][L - n:L]
            outs.append(R.attention(r, q.to(q_dtype) if q_dtype is not None else q.float()))
        return tuple(torch.cat([o[i] for o in outs]) for i in range(4))


def slack(ref, model):
    """The cache's keys (and a rounded q) may sit one step beside the reference's: a
    rotation that ends within fp32's error of a rounding boundary.  One step of one
    factor moves a score by at most eps |q| |k|, hence a weight by 2 eps a relatively."""
    eps = torch.finfo(model.dtype).eps
    return ref[1] * 4 * eps * ref[2]


def step(model, inp, table, out, q_rot, ws, one_each, err):
    v = vh()
    x = inp["x"]
    v.vh_mrope_kv_append(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], model.cos_sin, model.k, model.v, table, inp["lens"],
                         inp["active"], q_rot, token_start=None if one_each else inp["starts"], positions=inp["pos"],
                         pair_axis=PAIRS, err_flag=err)
    if one_each:
        v.vh_window_decode_attn(q_rot, model.k, model.v, table, inp["lens"], inp["active"], out, ws, window=W, sinks=S,
                                err_flag=err, pdl=True)
    else:
        v.vh_window_prompt_attn(q_rot, model.k, model.v, table, inp["starts"], inp["lens"], inp["active"], out, ws,
                                window=W, sinks=S, err_flag=err)


def buffers(model, T, one_each):
    v = vh()
    q_rot = torch.empty(T, HQ, D, dtype=torch.float32 if one_each else model.dtype, device="cuda")
    out = torch.zeros(T, HQ, D, dtype=model.dtype, device="cuda")
    ws = (v.alloc_workspace(model.B, HQ, HKV, D, P) if one_each else v.alloc_prompt_workspace(T, model.B, HQ, HKV, D))
    return q_rot, out, ws


def check(model, c, out, one_each):
    ref = model.reference(c, None if one_each else model.dtype)
    d = (out.double().cpu() - ref[0]).abs()
    tol = R.tolerance(ref, model.dtype, D, one_each, 8.0) + slack(ref, model)
    assert (d <= tol).all(), f"call {c}: {d.max().item()}"


CHUNKS = [[100, 3, 64], [1, 61, 0], [33, 8, 90], [1, 1, 1], [1, 1, 1], [1, 1, 1]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
def test_prompt_chunks_then_single_tokens_on_a_side_stream(dtype, layout):
    m = Model(CHUNKS, dtype, 5, layout)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c, n in enumerate(CHUNKS):
            one_each = all(k == 1 for k in n)
            inp = m.call_inputs(c)
            inp["active"] = torch.ones(m.B, dtype=torch.int32, device="cuda")
            table = m.give_back(m.table, m.lens(c), n)
            q_rot, out, ws = buffers(m, sum(n), one_each)
            step(m, inp, table, out, q_rot, ws, one_each, err)
            side.synchronize()
            check(m, c, out, one_each)
    assert int(err) == 0


def test_captured_steps_with_other_lengths_and_a_shared_workspace():
    """A prompt graph and a decode graph, captured once with static shapes, replayed
    with other tokens, lengths and row borders; two decode graphs on one workspace."""
    m = Model(CHUNKS, torch.bfloat16, 8)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    T = 190                                                  # room for every prompt call
    big = dict(x=torch.zeros(T, HQ + 2 * HKV, D, dtype=m.dtype, device="cuda"), pos=torch.zeros(3, T, dtype=torch.int32, device="cuda"),
               lens=i32([0] * 3), starts=i32([0] * 4), active=i32([1] * 3))
    one = dict(x=torch.zeros(3, HQ + 2 * HKV, D, dtype=m.dtype, device="cuda"), pos=torch.zeros(3, 3, dtype=torch.int32, device="cuda"),
               lens=i32([1] * 3), starts=None, active=i32([0] * 3))
    table = m.table.cuda()
    qb, ob, wb = buffers(m, T, False)
    qo, oo, wo = buffers(m, 3, True)
    o2 = torch.zeros_like(oo)
    step(m, big, table, ob, qb, wb, False, err)              # first calls, outside any capture
    step(m, one, table, oo, qo, wo, True, err)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graphs = []
    for inp, o, q, w, each in ((big, ob, qb, wb, False), (one, oo, qo, wo, True), (one, o2, qo, wo, True)):
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            step(m, inp, table, o, q, w, each, err)
        graphs.append(g)
    torch.cuda.current_stream().wait_stream(s)
    one["active"].fill_(1)
    for c, n in enumerate(CHUNKS):
        inp, t = m.call_inputs(c), sum(n)
        dst = one if all(k == 1 for k in n) else big
        dst["x"][:t] = inp["x"]
        dst["pos"][:, :t] = inp["pos"]
        dst["lens"].copy_(inp["lens"])
        if dst is big:
            dst["starts"].copy_(inp["starts"])
            ob.fill_(9.0)
            graphs[0].replay()
            torch.cuda.synchronize()
            assert (ob[t:] == 9.0).all()
            check(m, c, ob[:t], False)
        else:
            for g, o in ((graphs[1], oo), (graphs[2], o2), (graphs[1], oo)):   # (the append writes the same again)
                g.replay()
                torch.cuda.synchronize()
                check(m, c, o, True)
    assert int(err) == 0


def test_readme_example_runs_as_written():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    first, second = re.findall(r"```python\n(.*?)```", text, re.S)[:2]
    torch.manual_seed(6)
    e = {}
    exec(first, e)
    prompt, single = second.split("seq_lens += 1", 1)
    exec(prompt, e)
    torch.cuda.synchronize()
    starts = e["token_start"].tolist()
    news = [b - a for a, b in zip(starts, starts[1:])]

    def reference(q, lens, n):
        r = R.Ragged(e["Hq"], e["Hkv"], e["D"], e["P"], e["pool"].cpu(), "NHD", e["page_table"].cpu(), lens, n, [1] * len(lens),
                     e["window"], e["sinks"])
        return R.attention(r, q.cpu())

    assert R.close(e["prompt_out"], reference(e["q_rot"], news, news), torch.bfloat16, e["D"], False) is None
    exec("seq_lens += 1" + single, e)
    torch.cuda.synchronize()
    assert R.close(e["out"], reference(e["q_rot32"], [n + 1 for n in news], [1] * 8), torch.bfloat16, e["D"], True) is None
