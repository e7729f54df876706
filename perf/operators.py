"""The prompt and sliding-window operators of the paged cache, as they are measured.

Three operators that a decode or prompt step of a language model calls one after the other on a paged KV cache:

  append   rotary positions with several axes (time, height, width) on the new queries and keys of a ragged batch, the
           rotated keys and the values written into the cache's pages
  decode   attention of one new token a row over the last `window` cached tokens and the first `sinks` ones
  prompt   the same attention for many new tokens a row (a prompt, or a chunk of one)

`run` computes each in plain torch operations, or, where `own` is true, through paged_len_decode_gb300.
"""
import math
import random

import torch

own = False

# A full model's table of angles: theta 10000, one row a position, cos in the first half and sin in the second.
THETA = 10000.0


# ---- cases ---------------------------------------------------------------------------------------------------------

def _case(op, name, rows, heads, dim, page, lens, new, window=0, sinks=0, idle=0, fp16=False, layout="NHD", norm=False,
          packed=False, cyclic=False, interleaved=False, q16=False, lens_seed=1):
    """lens: least and most tokens a row holds, the new ones among them; new: least and most new tokens a row (0, 0: one
    each, a decode step); window 0: every earlier token is seen; idle: rows that hold no request."""
    c = dict(op=op, rows=rows, hq=heads[0], hkv=heads[1], dim=dim, page=page, len_lo=lens[0], len_hi=lens[1],
             new_lo=new[0], new_hi=new[1], window=window, sinks=sinks, idle=idle, fp16=fp16, layout=layout, norm=norm,
             packed=packed, cyclic=cyclic, interleaved=interleaved, q16=q16, lens_seed=lens_seed)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # a decode step's new tokens of 64 requests, one each: the smallest call, where latency counts
        _case("append", "append_step", 64, (16, 8), 128, 16, (200, 1200), (0, 0)),
        # four prompts of a few hundred tokens each (text and an image's rows and columns), heads normalised first
        _case("append", "append_prompts", 4, (16, 8), 128, 16, (300, 900), (300, 900), norm=True, q16=True),
        # one long prompt out of a packed projection, axes that take the frequencies in turn
        _case("append", "append_long", 1, (32, 8), 128, 64, (16384, 16384), (16384, 16384), packed=True, cyclic=True, q16=True),
        # a handful of short requests of a small model
        _case("decode", "decode_tiny", 4, (8, 2), 64, 16, (17, 200), (0, 0), window=64, sinks=4, fp16=True),
        # 64 requests of a speech model, some of the batch idle
        _case("decode", "decode_step", 64, (16, 8), 128, 16, (200, 1200), (0, 0), window=512, sinks=4, idle=9),
        # few requests of long context: the window is what is read
        _case("decode", "decode_long", 16, (32, 8), 128, 16, (2048, 8192), (0, 0), window=4096, sinks=16, layout="HND"),
        # a full batch of long contexts in large pages
        _case("decode", "decode_full", 256, (32, 8), 128, 64, (1024, 32768), (0, 0), window=2048, sinks=64),
        # a handful of tokens checked at once against a cached context: few rows, the cache's length is the work
        _case("prompt", "prompt_verify", 1, (16, 8), 128, 16, (5000, 5000), (16, 16), window=4096, sinks=4),
        # ragged short prompts of a small model
        _case("prompt", "prompt_ragged", 24, (16, 8), 64, 16, (3, 800), (3, 800), window=256, sinks=4, fp16=True),
        # one prompt of ordinary length
        _case("prompt", "prompt_one", 1, (16, 8), 128, 16, (4096, 4096), (4096, 4096), window=1024, sinks=4),
        # chunks of 512 tokens of 16 requests, no window: every earlier token is seen
        _case("prompt", "prompt_chunks", 16, (32, 8), 128, 64, (600, 8192), (512, 512)),
        # one long prompt under a wide window
        _case("prompt", "prompt_long", 1, (32, 8), 128, 64, (16384, 16384), (16384, 16384), window=4096, sinks=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prompt"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    heads = (hkv * rng.choice([g for g in (1, 2, 4, 8) if g * hkv <= 40]), hkv)
    dim = rng.choice([64, 128, 128])
    page = rng.choice([8, 16, 16, 32, 48, 64, 128, 256])
    more = dict(fp16=rng.random() < 0.4, layout=rng.choice(["NHD", "HND"]), lens_seed=rng.randrange(1 << 20),
                interleaved=rng.random() < 0.3)
    if op == "append":
        if rng.random() < 0.4:
            rows = _log(rng, 1, 512)
            return _case(op, None, rows, heads, dim, page, (1, _log(rng, 2, 4000)), (0, 0), norm=rng.random() < 0.5,
                         packed=rng.random() < 0.5, cyclic=rng.random() < 0.5, idle=rng.randrange(0, rows // 3 + 1), **more)
        rows = _log(rng, 1, 24)
        most = _log(rng, 2, 16384 // rows)
        return _case(op, None, rows, heads, dim, page, (1, most), (1, most), norm=rng.random() < 0.5, q16=True,
                     packed=rng.random() < 0.5, cyclic=rng.random() < 0.5, **more)
    window = 0 if rng.random() < 0.25 else _log(rng, 1, 4096)
    sinks = rng.choice([0, 0, 1, 4, 5, 16, 64, 100])
    if op == "decode":
        rows = _log(rng, 1, 128)
        most = _log(rng, 20, 8000 if window == 0 and rows > 32 else 30000)
        return _case(op, None, rows, heads, dim, page, (1, most), (0, 0), window=window, sinks=sinks,
                     idle=rng.randrange(0, rows // 3 + 1), **more)
    rows = _log(rng, 1, 16)
    new = _log(rng, 2, 6000 // rows)
    most = max(new, _log(rng, 20, 8192))
    return _case(op, None, rows, heads, dim, page, (min(most, new), most), (1, new), window=window, sinks=sinks, **more)


# ---- what a case's rows hold: from the case alone, so that a pass's work is known --------------------------------------

def _rows(case):
    """(tokens held, new tokens) of every row; an idle row holds and brings none."""
    rng = random.Random(case["lens_seed"])
    held, new = [], []
    for b in range(case["rows"]):
        n = 1 if case["new_hi"] == 0 else rng.randint(case["new_lo"], case["new_hi"])
        held.append(max(n, rng.randint(case["len_lo"], case["len_hi"])))
        new.append(n)
    if case["op"] == "append" and case["new_hi"]:
        held = list(new)  # whole prompts
    for b in rng.sample(range(case["rows"]), case["idle"]):
        held[b] = 0
    return held, new


def _seen(case, held, new):
    """(pairs of query and key, keys read) of one row's attention."""
    if not held:
        return 0, 0
    w = case["window"] or held
    first = held - new
    pairs = 0
    for i in (range(first, held) if w < held else ()):
        lo = max(0, i - w + 1)
        pairs += i + 1 - lo + min(case["sinks"], lo)
    if w >= held:
        pairs = (first + 1 + held) * new // 2
    lo = max(0, first - w + 1)
    return pairs, held - lo + min(case["sinks"], lo)


def work(case):
    held, new = _rows(case)
    size, dim, hq, hkv = 2, case["dim"], case["hq"], case["hkv"]
    live = sum(n for h, n in zip(held, new) if h)
    if case["op"] == "append":
        # q, k and v in; q (16 or 32 bits), k and v out; the angles' rows of three axes are few distinct ones
        out = size if case["q16"] else 4
        return {"bytes": live * dim * (hq * (size + out) + 4 * hkv * size), "flops": live * dim * (hq + hkv) * (7 if case["norm"] else 3)}
    pairs = keys = 0
    for h, n in zip(held, new):
        p, k = _seen(case, h, n)
        pairs, keys = pairs + p, keys + k
    q = 4 if case["op"] == "decode" else size
    return {"bytes": keys * hkv * dim * 2 * size + sum(new) * hq * dim * (q + size), "flops": 4 * pairs * hq * dim}


# ---- inputs --------------------------------------------------------------------------------------------------------

def _axes(case):
    """The axis of every rotated pair: time, height and width, in sections or in turn."""
    half = case["dim"] // 2
    h = w = 3 * half // 8
    t = half - h - w
    if case["cyclic"]:
        return [1 if i % 3 == 1 and i < 3 * h else 2 if i % 3 == 2 and i < 3 * w else 0 for i in range(half)]
    return [0] * t + [1] * h + [2] * w


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    et = torch.float16 if case["fp16"] else torch.bfloat16
    rows, hq, hkv, dim, page = case["rows"], case["hq"], case["hkv"], case["dim"], case["page"]
    held, new = _rows(case)
    one_each = case["new_hi"] == 0
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    tokens = starts[-1]

    # pages: a random order, page 0 belongs to nobody; pages that no query sees any more have been given back (-1)
    per_row = max(1, max(-(-h // page) for h in held))
    wanted, dead = [], []
    for b, (h, n) in enumerate(zip(held, new)):
        lo = max(0, h - n + 1 - case["window"]) if case["window"] and case["op"] != "append" else 0
        for j in range(-(-h // page)):
            (dead if j * page >= case["sinks"] and (j + 1) * page <= lo else wanted).append(b * per_row + j)
    order = torch.randperm(len(wanted), generator=gen, device=dev).to(torch.int32) + 1
    table = torch.zeros(rows * per_row, dtype=torch.int32, device=dev)
    table[torch.tensor(wanted, dtype=torch.int64, device=dev)] = order
    if dead:
        table[torch.tensor(dead, dtype=torch.int64, device=dev)] = -1
    shape = (len(wanted) + 1, 2, page, hkv, dim) if case["layout"] == "NHD" else (len(wanted) + 1, 2, hkv, page, dim)
    pool = torch.empty(shape, dtype=et, device=dev).normal_(generator=gen)
    k, v = (pool[:, i] if case["layout"] == "NHD" else pool[:, i].transpose(1, 2) for i in (0, 1))
    s = dict(case=case, table=table.view(rows, per_row), pool=pool, k=k, v=v,
             held=torch.tensor(held, dtype=torch.int32, device=dev),
             active=torch.tensor([int(h > 0) for h in held], dtype=torch.int32, device=dev),
             starts=torch.tensor(starts, dtype=torch.int32, device=dev), tokens=tokens)
    randn = lambda *d: torch.randn(*d, generator=gen, device=dev)  # noqa: E731
    if case["op"] == "append":
        # positions: text runs, then an image's grid, whose time stands still while its rows and columns advance
        most = max(1, max(held))
        at = torch.arange(tokens, device=dev) - s["starts"][:-1].long().repeat_interleave(torch.tensor(new, device=dev))
        base = torch.randint(0, most + 1, (rows,), generator=gen, device=dev).repeat_interleave(torch.tensor(new, device=dev))
        side = 24
        grid = (at // 97) % 2 == 1
        pos = torch.stack([base + torch.where(grid, at // 97 * 97, at), base + torch.where(grid, at % 97 // side, at),
                           base + torch.where(grid, at % side, at)])
        s["positions"] = pos.to(torch.int32)
        half = torch.arange(dim // 2, dtype=torch.float64, device=dev)
        angle = torch.arange(2 * most + 128, dtype=torch.float64, device=dev)[:, None] * THETA ** (-2 * half / dim)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["axes"] = _axes(case)
        s["axes_dev"] = torch.tensor(s["axes"], device=dev)
        if case["packed"]:
            qkv = randn(tokens, hq + 2 * hkv, dim).to(et)  # one projection's output: q, k and v side by side
            s["q"], s["k_new"], s["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k_new"], s["v_new"] = randn(tokens, hq, dim).to(et), randn(tokens, hkv, dim).to(et), randn(tokens, hkv, dim).to(et)
        s["wq"], s["wk"] = (1 + 0.1 * randn(dim), 1 + 0.1 * randn(dim)) if case["norm"] else (None, None)
        s["out"] = torch.zeros(tokens, hq, dim, dtype=et if case["q16"] else torch.float32, device=dev)
    else:
        s["q"] = randn(tokens, hq, dim) if one_each else randn(tokens, hq, dim).to(et)
        s["out"] = torch.zeros(tokens, hq, dim, dtype=et, device=dev)
        if own:
            import paged_len_decode_gb300 as vh

            if one_each:
                s["ws"] = vh.alloc_workspace(rows, hq, hkv, dim, page)
            else:
                s["ws"] = vh.alloc_prompt_workspace(tokens, rows, hq, hkv, dim)
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return _plain_append(s) if s["case"]["op"] == "append" else _plain_attention(s)


def _own(s):
    import paged_len_decode_gb300 as vh

    c = s["case"]
    ragged = None if c["new_hi"] == 0 else s["starts"]
    if c["op"] == "append":
        vh.vh_mrope_kv_append(s["q"], s["k_new"], s["v_new"], s["cos_sin"], s["k"], s["v"], s["table"], s["held"], s["active"],
                              s["out"], token_start=ragged, positions=s["positions"], pair_axis=s["axes"], q_norm_w=s["wq"],
                              k_norm_w=s["wk"], interleaved=c["interleaved"])
        return s["out"], s["pool"]
    if c["op"] == "decode":
        return vh.vh_window_decode_attn(s["q"], s["k"], s["v"], s["table"], s["held"], s["active"], s["out"], s["ws"],
                                        window=c["window"], sinks=c["sinks"])
    return vh.vh_window_prompt_attn(s["q"], s["k"], s["v"], s["table"], s["starts"], s["held"], s["active"], s["out"], s["ws"],
                                    window=c["window"], sinks=c["sinks"])


def _plain_append(s):
    c = s["case"]
    half, dev = c["dim"] // 2, s["q"].device
    t = torch.arange(s["tokens"], device=dev)
    row = torch.searchsorted(s["starts"][1:].long(), t, right=True)
    live = s["active"][row] != 0
    slot = s["held"].long()[row] - s["starts"].long()[row + 1] + t
    # cos and sin of every pair, each from its axis's position
    pos = s["positions"].long()[s["axes_dev"]].t()
    pair = torch.arange(half, device=dev)
    cos, sin = s["cos_sin"][pos, pair].unsqueeze(1), s["cos_sin"][pos, half + pair].unsqueeze(1)

    def rotated(x, w):
        x = x.float()
        if w is not None:
            x = w * (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6))
        if c["interleaved"]:
            a, b = x[..., 0::2], x[..., 1::2]
            return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    s["out"][live] = rotated(s["q"], s["wq"]).to(s["out"].dtype)[live]
    page, off = s["table"][row, (slot // c["page"]).clamp(min=0)].long()[live], (slot % c["page"])[live]
    s["k"][page, off] = rotated(s["k_new"], s["wk"]).to(s["k"].dtype)[live]
    s["v"][page, off] = s["v_new"][live]
    return s["out"], s["pool"]


def _plain_attention(s):
    """Queries in blocks of one row each; a block's keys are the sinks and the span from its first query's window to its last
    query, gathered through the page table."""
    c = s["case"]
    dev, hkv, dim, page = s["q"].device, c["hkv"], c["dim"], c["page"]
    group = c["hq"] // hkv
    size = 1 if c["new_hi"] == 0 else 128
    rows, most = s["table"].shape[0], s["table"].shape[1] * page
    starts, held = s["starts"].long(), s["held"].long()
    window, sinks = min(c["window"] or most, most), min(c["sinks"], most)
    # block i belongs to the last row b with starts[b] // size + b <= i
    blocks = torch.arange(s["tokens"] // size + rows if size > 1 else rows, device=dev)
    row = torch.searchsorted(starts[:-1] // size + torch.arange(rows, device=dev), blocks, right=True) - 1 if size > 1 else blocks
    first = starts[row] + (blocks - starts[row] // size - row if size > 1 else 0) * size
    tok = first[:, None] + torch.arange(size, device=dev)
    real = (tok < starts[row + 1, None]) & (s["active"][row, None] != 0)
    at = held[row, None] - starts[row + 1, None] + tok  # the queries' places in their rows
    low = (at[:, :1] - window + 1).clamp(min=sinks)
    n = min(window + size - 1, most)
    j = torch.cat([torch.arange(sinks, device=dev).expand(len(blocks), sinks), low + torch.arange(n, device=dev)], 1)
    inside = j.clamp(max=most - 1)
    pg, off = s["table"][row[:, None], inside // page].long().clamp(min=0), inside % page
    k, v = s["k"][pg, off].float().transpose(1, 2), s["v"][pg, off].float().transpose(1, 2)  # [block, kv head, key, dim]
    q = s["q"].float()[tok.clamp(max=s["tokens"] - 1)].view(len(blocks), size, hkv, group, dim)
    q = q.permute(0, 2, 3, 1, 4).reshape(len(blocks), hkv, group * size, dim)
    j = j[:, None, :]
    seen = (j <= at[:, :, None]) & ((j < sinks) | (j > at[:, :, None] - window)) & real[:, :, None]
    score = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(dim)).view(len(blocks), hkv, group, size, -1)
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(len(blocks), hkv, group * size, -1) @ v).view(len(blocks), hkv, group, size, dim)
    o = (o / torch.where(total == 0, 1, total)).permute(0, 3, 1, 2, 4).reshape(len(blocks), size, c["hq"], dim)
    mine = tok < starts[row + 1, None]  # an idle row's output is zero
    s["out"][tok[mine]] = o[mine].to(s["out"].dtype)
    return s["out"]


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    held, new = _rows(case)
    if case["op"] == "append":
        return _exact_append(s, held, new)
    dim, page, hkv = case["dim"], case["page"], case["hkv"]
    out = torch.zeros(s["tokens"], case["hq"], dim, dtype=torch.float64, device=s["q"].device)
    t0 = 0
    for b, (h, n) in enumerate(zip(held, new)):
        for a in range(0, n if h else 0, 512):
            m = min(512, n - a)
            at = torch.arange(h - n + a, h - n + a + m, device=out.device)
            lo = max(0, h - n + a + 1 - case["window"]) if case["window"] else 0
            j = torch.cat([torch.arange(0, min(case["sinks"], lo), device=out.device), torch.arange(lo, h - n + a + m, device=out.device)])
            pages = s["table"][b].long()[j // page]
            keys, vals = s["k"][pages, j % page].double(), s["v"][pages, j % page].double()
            see = j[None] <= at[:, None]
            if case["window"]:
                see &= (at[:, None] - j[None] < case["window"]) | (j[None] < case["sinks"])
            for g in range(hkv):
                each = case["hq"] // hkv
                q = s["q"][t0 + a:t0 + a + m, g * each:(g + 1) * each].double()
                sc = torch.einsum("mgd,jd->gmj", q, keys[:, g]) / dim ** 0.5
                sc = torch.softmax(sc.masked_fill(~see, -math.inf), -1)
                out[t0 + a:t0 + a + m, g * each:(g + 1) * each] = torch.einsum("gmj,jd->mgd", sc, vals[:, g])
        t0 += n
    return out


def _exact_append(s, held, new):
    c = s["case"]
    half, page = c["dim"] // 2, c["page"]
    first = torch.arange(half, device=s["q"].device) * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else half)
    out, pool = s["out"].double(), s["pool"].double()
    k, v = (pool[:, i] if c["layout"] == "NHD" else pool[:, i].transpose(1, 2) for i in (0, 1))
    t0 = 0
    for b, (h, n) in enumerate(zip(held, new)):
        if h:
            t = torch.arange(t0, t0 + n, device=out.device)
            j = t - t0 + h - n
            pages = s["table"][b].long()[j // page]
            pos = s["positions"].long()[:, t][s["axes_dev"]].t()
            cos = torch.gather(s["cos_sin"][:, :half].double(), 0, pos)[:, None]
            sin = torch.gather(s["cos_sin"][:, half:].double(), 0, pos)[:, None]
            for src, w, to in ((s["q"], s["wq"], "q"), (s["k_new"], s["wk"], "k")):
                x = src[t].double()
                if w is not None:
                    x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
                y = torch.empty_like(x)
                y[..., first] = x[..., first] * cos - x[..., second] * sin
                y[..., second] = x[..., second] * cos + x[..., first] * sin
                if to == "q":
                    out[t] = y
                else:
                    k[pages, j % page] = y
            v[pages, j % page] = s["v_new"][t].double()
        t0 += n
    return out, pool
