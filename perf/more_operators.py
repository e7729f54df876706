"""The operators of an 8-bit cache and of drafted trees, as they are measured.

Four operators of a serving loop over a paged KV cache:

  append   rotary positions on the new queries and keys of a ragged batch, the rotated keys and the values written into the
           cache in 8 bits (e4m3), with a scale for every slot and kv head
  decode   attention of one new token a row over that cache, or over its last `window` tokens and the first `sinks` ones
  read     slots of that cache back into a cache of 16 bits
  tree     attention of drafted tokens that form a tree over a cache of 16 bits: a token sees the context, and of the
           drafted ones its ancestors and itself

`run` computes each in plain torch operations, or, where `own` is true, through paged_len_decode_gb300.
"""
import math
import random

import torch

own = False

THETA = 10000.0  # of a full model's table of angles: one row a position, cos in the first half and sin in the second
E4M3 = torch.float8_e4m3fn
MOST = 448.0     # the largest e4m3 value


# ---- cases ---------------------------------------------------------------------------------------------------------

def _case(op, name, rows, heads, dim, page, lens, new=(0, 0), window=0, sinks=0, idle=0, fp16=False, layout="NHD",
          norm=False, packed=False, interleaved=False, q16=False, branch=3, lens_seed=1):
    """lens: least and most tokens a row holds, the new ones among them; new: least and most new tokens a row (0, 0: one
    each, a decode step); window 0: every earlier token is seen; idle: rows that hold no request; branch: children that a
    drafted token has at most."""
    c = dict(op=op, rows=rows, hq=heads[0], hkv=heads[1], dim=dim, page=page, len_lo=lens[0], len_hi=lens[1],
             new_lo=new[0], new_hi=new[1], window=window, sinks=sinks, idle=idle, fp16=fp16, layout=layout, norm=norm,
             packed=packed, interleaved=interleaved, q16=q16, branch=branch, lens_seed=lens_seed)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # a decode step's new tokens of 64 requests, one each: the smallest call, where latency counts
        _case("append", "quant_append_step", 64, (16, 8), 128, 16, (200, 1200)),
        # four prompts of a few hundred tokens each, heads normalised first
        _case("append", "quant_append_prompts", 4, (16, 8), 128, 16, (300, 900), (300, 900), norm=True, q16=True),
        # one long prompt out of a packed projection
        _case("append", "quant_append_long", 1, (32, 8), 128, 64, (16384, 16384), (16384, 16384), packed=True, q16=True),
        # a handful of short requests of a small model
        _case("decode", "quant_decode_tiny", 4, (8, 2), 64, 16, (17, 200), window=64, sinks=4, fp16=True),
        # 64 requests of a speech model, some of the batch idle
        _case("decode", "quant_decode_step", 64, (16, 8), 128, 16, (200, 1200), idle=9),
        # few requests of long context, all of it seen
        _case("decode", "quant_decode_long", 16, (32, 8), 128, 16, (4096, 32768), layout="HND"),
        # a full batch of long contexts in large pages under a window
        _case("decode", "quant_decode_full", 256, (32, 8), 128, 64, (1024, 32768), window=2048, sinks=64),
        # what a small model's window leaves of eight requests, for their next chunks of a prompt
        _case("read", "quant_read_window", 8, (16, 8), 64, 16, (300, 4000), window=512, sinks=4, fp16=True),
        # whole contexts of sixteen requests
        _case("read", "quant_read_long", 16, (32, 8), 128, 64, (2048, 16384)),
        # one request's drafted tokens against a cached context: few rows, the cache's length is the work
        _case("tree", "tree_one", 1, (16, 8), 128, 16, (5000, 5000), (16, 16)),
        # ragged trees of a small model's batch, a window over the context
        _case("tree", "tree_batch", 32, (16, 8), 64, 16, (200, 4000), (5, 64), window=1024, sinks=4, fp16=True, branch=4),
        # large trees over long contexts
        _case("tree", "tree_long", 8, (32, 8), 128, 64, (8192, 32768), (64, 64)),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "read", "tree"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    heads = (hkv * rng.choice([g for g in (1, 2, 4, 8) if g * hkv <= 40]), hkv)
    dim = rng.choice([64, 128, 128])
    page = rng.choice([8, 16, 16, 32, 48, 64, 128, 256])
    more = dict(fp16=rng.random() < 0.4, layout=rng.choice(["NHD", "HND"]), lens_seed=rng.randrange(1 << 20))
    if op == "append":
        more.update(norm=rng.random() < 0.5, packed=rng.random() < 0.5, interleaved=rng.random() < 0.3)
        if rng.random() < 0.4:
            rows = _log(rng, 1, 512)
            return _case(op, None, rows, heads, dim, page, (1, _log(rng, 2, 4000)), idle=rng.randrange(0, rows // 3 + 1), **more)
        rows = _log(rng, 1, 24)
        most = _log(rng, 2, 16384 // rows)
        return _case(op, None, rows, heads, dim, page, (1, most), (1, most), q16=True, **more)
    window = 0 if rng.random() < 0.4 else _log(rng, 1, 4096)
    sinks = rng.choice([0, 0, 1, 4, 5, 16, 64, 100])
    if op == "decode":
        rows = _log(rng, 1, 128)
        most = _log(rng, 20, 8000 if window == 0 and rows > 32 else 30000)
        return _case(op, None, rows, heads, dim, page, (1, most), window=window, sinks=sinks,
                     idle=rng.randrange(0, rows // 3 + 1), **more)
    if op == "read":
        rows = _log(rng, 1, 64)
        most = _log(rng, 20, 250000 // rows)
        return _case(op, None, rows, heads, dim, page, (1, most), window=window, sinks=sinks,
                     idle=rng.randrange(0, rows // 3 + 1), **more)
    rows = _log(rng, 1, 32)
    new = _log(rng, 1, 128 if rows <= 8 else 48)
    most = max(new, _log(rng, 20, 100000 // rows if rows > 4 else 24000))
    return _case(op, None, rows, heads, dim, page, (min(most, new), most), (1, new), window=window, sinks=sinks,
                 branch=rng.randint(1, 6), idle=rng.randrange(0, rows // 3 + 1), **more)


# ---- what a case's rows hold: from the case alone, so that a pass's work is known --------------------------------------

def _rows(case):
    """(tokens held, new tokens) of every row; an idle row holds none."""
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


def _trees(case):
    """The ancestors of every drafted token of every row, as bits over the row's drafted tokens (itself left out)."""
    rng = random.Random(case["lens_seed"] + 1)
    rows = []
    for n in _rows(case)[1]:
        above, children, opened = [], [], 0
        for i in range(n):
            # breadth first, mostly: below one of the oldest tokens that may have another child
            while opened < i and children[opened] >= case["branch"]:
                opened += 1
            parent = -1 if i == 0 else min(i - 1, opened + rng.choice([0, 0, 1, 2, 3]))
            if i and parent >= 0:
                children[parent] += 1
            above.append(0 if parent < 0 else above[parent] | 1 << parent)
            children.append(0)
        rows.append(above)
    return rows


def _first(case, held):
    """The first slot behind the sinks that a row's next token, or the first of its drafted ones, sees."""
    return [max(0, h - case["window"]) if case["window"] else 0 for h in held]


def work(case):
    held, new = _rows(case)
    dim, hq, hkv = case["dim"], case["hq"], case["hkv"]
    live = sum(n for h, n in zip(held, new) if h)
    if case["op"] == "append":
        # q, k and v in; q (16 or 32 bits), k and v (8 bits and scales) out
        out = 2 if case["q16"] else 4
        return {"bytes": live * (hq * dim * (2 + out) + hkv * (dim * (4 + 2) + 8)),
                "flops": live * dim * (hq * (7 if case["norm"] else 3) + hkv * ((7 if case["norm"] else 3) + 4))}
    if case["op"] in ("decode", "read"):
        slots = sum(h - f + min(case["sinks"], f) for h, f in zip(held, _first(case, held)))
        if case["op"] == "read":
            return {"bytes": slots * hkv * (dim * 2 * (1 + 2) + 8), "flops": slots * hkv * dim * 2}
        return {"bytes": slots * hkv * (dim * 2 + 8) + case["rows"] * hq * dim * (4 + 2), "flops": 4 * slots * hq * dim}
    pairs = slots = 0
    for h, n, above in zip(held, new, _trees(case)):
        if not h:
            continue
        base, w = h - n, case["window"] or h + 1
        low = max(0, base - w + 1)
        slots += h - low + min(case["sinks"], low)
        for a in above:
            low = max(0, base + a.bit_count() - w + 1)
            pairs += max(0, base - low) + min(case["sinks"], low, base) + a.bit_count() + 1
    return {"bytes": slots * hkv * dim * 4 + sum(new) * hq * dim * 4, "flops": 4 * pairs * hq * dim}


# ---- inputs --------------------------------------------------------------------------------------------------------

def _quantised(x):
    """e4m3 values and the scale of every head of x [..., dim]."""
    scale = (x.abs().amax(-1) / MOST).clamp(min=2.0 ** -126)
    return (x * (1 / scale)[..., None]).to(E4M3), scale


def _pages(case, gen, held, keep_from, per_row):
    """A page table [rows, per_row] in a random order (page 0 belongs to nobody), and how many pages there are. Pages that
    lie behind the sinks and before slot keep_from[b] have been given back (-1)."""
    page, wanted, dead = case["page"], [], []
    for b, (h, lo) in enumerate(zip(held, keep_from)):
        for j in range(-(-h // page)):
            (dead if j * page >= case["sinks"] and (j + 1) * page <= lo else wanted).append(b * per_row + j)
    dev = torch.device("cuda")
    table = torch.zeros(case["rows"] * per_row, dtype=torch.int32, device=dev)
    order = torch.randperm(len(wanted), generator=gen, device=dev).to(torch.int32) + 1
    table[torch.tensor(wanted, dtype=torch.int64, device=dev)] = order
    if dead:
        table[torch.tensor(dead, dtype=torch.int64, device=dev)] = -1
    return table.view(case["rows"], per_row), len(wanted) + 1


def _views(case, pool):
    return (pool[:, i] if case["layout"] == "NHD" else pool[:, i].transpose(1, 2) for i in (0, 1))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    et = torch.float16 if case["fp16"] else torch.bfloat16
    rows, hq, hkv, dim, page, op = case["rows"], case["hq"], case["hkv"], case["dim"], case["page"], case["op"]
    held, new = _rows(case)
    one_each = case["new_hi"] == 0
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    tokens = starts[-1]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    randn = lambda *d: torch.randn(*d, generator=gen, device=dev)    # noqa: E731

    first = _first(case, held) if op != "append" else [0] * rows
    if op == "tree":  # the root's place is the first one behind the context
        first = [max(0, h - n - case["window"] + 1) if case["window"] else 0 for h, n in zip(held, new)]
    per_row = max(1, max(-(-h // page) for h in held))
    table, pages = _pages(case, gen, held, first, per_row)
    shape = (pages, 2, page, hkv, dim) if case["layout"] == "NHD" else (pages, 2, hkv, page, dim)
    s = dict(case=case, table=table, held=ints(held), active=ints([int(h > 0) for h in held]), starts=ints(starts),
             tokens=tokens, first=ints(first))
    if op == "tree":
        s["pool"] = torch.empty(shape, dtype=et, device=dev).normal_(generator=gen)
    else:
        # heads of different sizes: their scales differ
        x = torch.empty(shape, device=dev).normal_(generator=gen).mul_(randn(*shape[:-1], 1).mul_(0.5).exp_())
        s["pool"], scale = _quantised(x)
        del x
        # scales lie [page, k or v, head, slot], whatever the cache's layout
        s["scale"] = scale.transpose(2, 3).contiguous() if case["layout"] == "NHD" else scale
        s["k_scale"], s["v_scale"] = s["scale"][:, 0], s["scale"][:, 1]
    s["k"], s["v"] = _views(case, s["pool"])

    if op == "append":
        most = max(1, max(held))
        at = torch.arange(tokens, device=dev) - s["starts"][:-1].long().repeat_interleave(ints(new))
        s["positions"] = (torch.randint(0, most + 1, (rows,), generator=gen, device=dev).repeat_interleave(ints(new)) + at).to(torch.int32)
        half = torch.arange(dim // 2, dtype=torch.float64, device=dev)
        angle = torch.arange(2 * most + 2, dtype=torch.float64, device=dev)[:, None] * THETA ** (-2 * half / dim)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        if case["packed"]:
            qkv = randn(tokens, hq + 2 * hkv, dim).to(et)  # one projection's output: q, k and v side by side
            s["q"], s["k_new"], s["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k_new"], s["v_new"] = randn(tokens, hq, dim).to(et), randn(tokens, hkv, dim).to(et), randn(tokens, hkv, dim).to(et)
        s["wq"], s["wk"] = (1 + 0.1 * randn(dim), 1 + 0.1 * randn(dim)) if case["norm"] else (None, None)
        s["out"] = torch.zeros(tokens, hq, dim, dtype=et if case["q16"] else torch.float32, device=dev)
        return s
    if op == "read":
        # the other cache has its own pages, in its own order
        s["out_table"], n = _pages(case, gen, held, first, per_row)
        s["out_pool"] = torch.zeros((n,) + shape[1:], dtype=et, device=dev)
        s["k_out"], s["v_out"] = _views(case, s["out_pool"])
        return s
    s["q"] = randn(tokens, hq, dim) if one_each else randn(tokens, hq, dim).to(et)
    s["out"] = torch.zeros(tokens, hq, dim, dtype=et, device=dev)
    if op == "tree":
        words = -(-max(new) // 64)
        mask = [[(a >> 64 * w & (1 << 64) - 1) for w in range(words)] for row in _trees(case) for a in (x | 1 << i for i, x in enumerate(row))]
        s["mask"] = torch.tensor([[x - (1 << 64) if x >> 63 else x for x in m] for m in mask], dtype=torch.int64, device=dev)
    if own:
        import paged_len_decode_gb300 as vh

        s["ws"] = vh.alloc_workspace(rows, hq, hkv, dim, page) if op == "decode" else vh.alloc_prompt_workspace(tokens, rows, hq, hkv, dim)
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return {"append": _plain_append, "decode": _plain_decode, "read": _plain_read, "tree": _plain_tree}[s["case"]["op"]](s)


def _own(s):
    import paged_len_decode_gb300 as vh

    c = s["case"]
    if c["op"] == "append":
        vh.vh_quant_kv_append(s["q"], s["k_new"], s["v_new"], s["cos_sin"], s["k"], s["v"], s["k_scale"], s["v_scale"],
                              s["table"], s["held"], s["active"], s["out"], token_start=s["starts"] if c["new_hi"] else None,
                              positions=s["positions"], q_norm_w=s["wq"], k_norm_w=s["wk"], interleaved=c["interleaved"])
        return s["out"], s["pool"], s["scale"]
    if c["op"] == "decode":
        return vh.vh_quant_decode_attn(s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["held"], s["active"],
                                       s["out"], s["ws"], window=c["window"], sinks=c["sinks"])
    if c["op"] == "read":
        vh.vh_quant_kv_read(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["held"], s["active"], s["k_out"], s["v_out"],
                            s["out_table"], first_slot=s["first"], sinks=c["sinks"])
        return s["out_pool"]
    return vh.vh_tree_attn(s["q"], s["k"], s["v"], s["table"], s["starts"], s["held"], s["active"], s["mask"], s["out"], s["ws"],
                           window=c["window"], sinks=c["sinks"])


def _plain_append(s):
    c = s["case"]
    half, dev = c["dim"] // 2, s["q"].device
    t = torch.arange(s["tokens"], device=dev)
    row = torch.searchsorted(s["starts"][1:].long(), t, right=True)
    live = s["active"][row] != 0
    slot = s["held"].long()[row] - s["starts"].long()[row + 1] + t
    angles = s["cos_sin"][s["positions"].long()].unsqueeze(1)
    cos, sin = angles[..., :half], angles[..., half:]

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
    k, v = _views(c, s["pool"].view(torch.uint8))
    for to, scales, x in ((k, s["k_scale"], rotated(s["k_new"], s["wk"])), (v, s["v_scale"], s["v_new"].float())):
        values, scale = _quantised(x[live])
        to[page, off] = values.view(torch.uint8)
        scales[page, :, off] = scale
    return s["out"], s["pool"], s["scale"]


def _dequantised(s, page, off):
    """Keys and values [..., kv head, dim] of slot `off` of page `page`."""
    k8, v8 = (x[page, off].view(E4M3).float() for x in _views(s["case"], s["pool"].view(torch.uint8)))
    heads = torch.arange(s["case"]["hkv"], device=page.device)
    at = page[..., None], heads, off[..., None]
    return k8.mul_(s["k_scale"][at][..., None]), v8.mul_(s["v_scale"][at][..., None])


def _plain_read(s):
    c = s["case"]
    slot = torch.arange(s["table"].shape[1] * c["page"], device=s["table"].device)
    held, first = s["held"][:, None], s["first"][:, None]
    row, slot = ((s["active"][:, None] != 0) & (slot < held) & ((slot >= first) | (slot < c["sinks"]))).nonzero(as_tuple=True)
    of_row, off = slot // c["page"], slot % c["page"]
    k, v = _dequantised(s, s["table"][row, of_row].long(), off)
    page = s["out_table"][row, of_row].long()
    s["k_out"][page, off] = k.to(s["out_pool"].dtype)
    s["v_out"][page, off] = v.to(s["out_pool"].dtype)
    return s["out_pool"]


def _softmax_product(s, q, k, v, seen, live):
    """out [rows, new, q head, dim] of q [rows, new, q head, dim] over k, v [rows, keys, kv head, dim]."""
    c = s["case"]
    rows, size, hkv, dim = q.shape[0], q.shape[1], c["hkv"], c["dim"]
    group = c["hq"] // hkv
    q = q.float().view(rows, size, hkv, group, dim).permute(0, 2, 3, 1, 4).reshape(rows, hkv, group * size, dim)
    score = (q @ k.permute(0, 2, 3, 1)).mul_(1 / math.sqrt(dim)).view(rows, hkv, group, size, -1)
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(rows, hkv, group * size, -1) @ v.transpose(1, 2)).view(rows, hkv, group, size, dim)
    o = (o / torch.where(total == 0, 1, total)).permute(0, 3, 1, 2, 4).reshape(rows, size, c["hq"], dim)
    return torch.where(live[:, None, None, None], o, 0)  # an idle row's output is zero


def _plain_decode(s):
    c = s["case"]
    rows, most = s["table"].shape[0], s["table"].shape[1] * c["page"]
    dev, held, live = s["q"].device, s["held"].long()[:, None], s["active"] != 0
    window, sinks = min(c["window"] or most, most), min(c["sinks"], most)
    low = (held - window).clamp(min=sinks)
    j = torch.cat([torch.arange(sinks, device=dev).expand(rows, sinks), low + torch.arange(window, device=dev)], 1)
    inside = j.clamp(max=most - 1)
    page = s["table"].gather(1, inside // c["page"]).long().clamp(min=0)
    k, v = _dequantised(s, page, inside % c["page"])
    seen = (j < held) & ((j < sinks) | (j >= held - window)) & live[:, None]
    s["out"].copy_(_softmax_product(s, s["q"][:, None], k, v, seen[:, None], live)[:, 0])
    return s["out"]


def _plain_tree(s):
    c = s["case"]
    rows, most = s["table"].shape[0], s["table"].shape[1] * c["page"]
    dev, held, live = s["q"].device, s["held"].long()[:, None, None], s["active"] != 0
    starts = s["starts"].long()
    size = 64 * s["mask"].shape[1]
    i = torch.arange(size, device=dev)
    tok = starts[:-1, None] + i
    mine = tok < starts[1:, None]
    tok = tok.clamp(max=s["tokens"] - 1)
    n = (starts[1:] - starts[:-1])[:, None, None]
    base = held - n
    # the drafted tokens that each one sees
    bits = (s["mask"][tok][..., None] >> torch.arange(64, device=dev) & 1).view(rows, size, size) != 0
    bits &= i <= i[:, None]
    at = base + bits.sum(-1, keepdim=True) - 1  # the positions: the context and the ancestors lie before
    j = torch.arange(most, device=dev)
    draft = (j - base).clamp(0, size - 1).expand(rows, size, most)
    context = (j < base) & ((j > at - (c["window"] or most)) | (j < c["sinks"]))
    seen = (context | ((j >= base) & (j < held) & bits.gather(2, draft))) & live[:, None, None] & mine[..., None]
    page, off = s["table"].long().clamp(min=0)[:, j // c["page"]], (j % c["page"]).expand(rows, most)
    k, v = s["k"][page, off].float(), s["v"][page, off].float()
    o = _softmax_product(s, s["q"][tok], k, v, seen, live)
    s["out"][tok[mine]] = o[mine].to(s["out"].dtype)
    return s["out"]


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    held, new = _rows(case)
    if case["op"] == "append":
        return _exact_append(s, held, new)
    dim, page, hkv, dev = case["dim"], case["page"], case["hkv"], s["table"].device
    out = s["out_pool"].double() if case["op"] == "read" else torch.zeros(s["tokens"], case["hq"], dim, dtype=torch.float64, device=dev)
    t0 = 0
    for b, (h, n) in enumerate(zip(held, new)):
        if not h:
            t0 += n
            continue
        f = int(s["first"][b])
        j = torch.cat([torch.arange(0, min(case["sinks"], f), device=dev), torch.arange(f, h, device=dev)])
        pages, off = s["table"][b].long()[j // page], j % page
        keys, vals = s["k"][pages, off].double(), s["v"][pages, off].double()
        if case["op"] != "tree":
            keys, vals = keys * s["k_scale"][pages, :, off].double()[..., None], vals * s["v_scale"][pages, :, off].double()[..., None]
        if case["op"] == "read":
            k, v = _views(case, out)
            to = s["out_table"][b].long()[j // page]
            k[to, off], v[to, off] = keys, vals
            continue
        see = torch.ones(n, len(j), dtype=torch.bool, device=dev)
        if case["op"] == "tree":
            base = h - n
            for i, above in enumerate(_trees(case)[b]):
                at = base + bin(above).count("1")
                drafted = torch.tensor([base + x for x in range(n) if above >> x & 1 or x == i], device=dev)
                context = (j < base) & ((at - j < case["window"]) | (j < case["sinks"])) if case["window"] else j < base
                see[i] = context | torch.isin(j, drafted)
        each = case["hq"] // hkv
        for g in range(hkv):
            q = s["q"][t0:t0 + n, g * each:(g + 1) * each].double()
            sc = torch.einsum("mgd,jd->gmj", q, keys[:, g]) / dim ** 0.5
            sc = torch.softmax(sc.masked_fill(~see, -math.inf), -1)
            out[t0:t0 + n, g * each:(g + 1) * each] = torch.einsum("gmj,jd->mgd", sc, vals[:, g])
        t0 += n
    return out


def _exact_append(s, held, new):
    """The rotated queries, the keys and values that the 8 bits stand for, without their rounding, over their scales, and
    the scales."""
    c = s["case"]
    half, page = c["dim"] // 2, c["page"]
    first = torch.arange(half, device=s["q"].device) * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else half)
    out, pool, scale = s["out"].double(), s["pool"].double(), s["scale"].double()
    k, v = _views(c, pool)
    t0 = 0
    for b, (h, n) in enumerate(zip(held, new)):
        if h:
            t = torch.arange(t0, t0 + n, device=out.device)
            j = t - t0 + h - n
            pages, off = s["table"][b].long()[j // page], j % page
            angles = s["cos_sin"][s["positions"].long()[t]].double()[:, None]
            cos, sin = angles[..., :half], angles[..., half:]
            for src, w, to in ((s["q"], s["wq"], None), (s["k_new"], s["wk"], 0), (s["v_new"], None, 1)):
                y = src[t].double()
                if w is not None:
                    y = y / (y.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
                if to != 1:
                    x, y = y, torch.empty_like(y)
                    y[..., first] = x[..., first] * cos - x[..., second] * sin
                    y[..., second] = x[..., second] * cos + x[..., first] * sin
                if to is None:
                    out[t] = y
                    continue
                size = y.abs().amax(-1) / MOST
                (k, v)[to][pages, off] = y / size[..., None]
                scale[pages, to, :, off] = size
        t0 += n
    return out, pool, scale
