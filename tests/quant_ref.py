"""Float64 reference of the 8-bit cache and of the tree attention, on the CPU, written from the definitions in
include/vh.h, and seeded inputs for them (tests/window_ref.py's ragged batches).

Decode tolerance, elementwise.  With p the weights, w_j = p_j vs_j, A = sum_j w_j |v8_j|,
a = scale max_j ks_j sum_d |q_d| |k8_jd|, a1 the same with the head's largest |q| in the place of every |q_d|, n visible
keys and head dim D:
  * q is held to 2^-22 of the head's largest element, so a score is off by at most 2^-22 a1; its products are summed in
    fp32 and multiplied by the scales: a (D + 4) 2^-23;
  * a weight is off by that relatively, by exp2 and the maximum's subtraction (2^-20 covers both), and by its rounding
    u_p, 2^-11, or 2^-22 where the output is fp16; the sum too, hence the factor 2 on the first;
  * weights far below the largest one lose at most 2^-40 of the largest w_j each, and a value is at most 448:
    448 n 2^-40 max_j w_j;
  * n fp32 additions lose at most n 2^-23; the output is rounded once.
"""
import math

import torch

import window_ref as R

E4M3 = torch.float8_e4m3fn
NAN_BYTE = 0x7F


def quantised(x):
    """(e4m3 values, scales) of the heads x [..., D] (float32), by the header's rule; a head with a value that is no
    finite number has the scale NaN."""
    top = x.abs().amax(-1)
    scale = (top / 448).clamp(min=2.0 ** -126)
    scale = torch.where(torch.isfinite(x).all(-1), scale, math.nan)
    return (x * (1 / scale)[..., None]).to(E4M3), scale


def make(lens, news, sigma=1.0, spread=0.5, **kw):
    """A ragged batch r (tests/window_ref.py) over an 8-bit cache: r.pool holds in float64 what the cache stands for,
    r.extra["q8"] the bytes and r.extra["scale"] the scales [NP, 2, Hkv, P].  Slots that no query sees hold NaN bytes
    and NaN scales."""
    r = R.make(lens, news, dtype=torch.float32, sigma=sigma, **kw)
    x = r.pool
    x = x * (torch.randn(*x.shape[:-1], 1, generator=r.extra["gen"]) * spread).exp()
    set_pool(r, *quantised(x))
    return r


def set_pool(r, q8, scale):
    """q8 in the layout of r.pool, scale [.., slot and head in its order] without the last axis."""
    by = q8.view(torch.uint8).clone()
    by[torch.isnan(scale)[..., None].expand_as(by)] = NAN_BYTE
    q8 = by.view(E4M3)
    r.pool = q8.double() * scale.double()[..., None]
    r.extra["q8"] = q8
    r.extra["scale"] = (scale.transpose(2, 3) if r.layout == "NHD" else scale).contiguous()


def on_gpu(r, pad=0):
    """pad: floats between the pages' scales, which have to be stepped over."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = r.extra["q8"].view(torch.uint8).cuda().view(E4M3)
    sc = r.extra["scale"]
    # (slots in multiples of 4 floats: strides have to be multiples of 16 bytes)
    wide = torch.full((*sc.shape[:2], sc.shape[2] + pad, -(-sc.shape[3] // 4) * 4), math.nan)
    wide[:, :, :sc.shape[2], :sc.shape[3]] = sc
    wide = wide.cuda()[:, :, :sc.shape[2], :sc.shape[3]]
    return dict(pool=pool, k=r.view(pool, 0), v=r.view(pool, 1), ks=wide[:, 0], vs=wide[:, 1], table=r.table.cuda(),
                starts=i32(r.starts), lens=i32(r.lens), active=i32(r.active), err=torch.zeros(1, dtype=torch.int32, device="cuda"))


def attention(r, q, scale=0.0, contiguous=False, dtype=torch.bfloat16):
    """(out, tol without the output's rounding) [B, Hq, D] of one query a row, q [B, Hq, D] fp32."""
    D, G = r.D, r.Hq // r.Hkv
    f = scale if scale > 0 else 1 / math.sqrt(D)
    k, v = r.view(r.pool, 0), r.view(r.pool, 1)
    vs = r.extra["scale"][:, 1].double()
    out, tol = torch.zeros(r.B, r.Hq, D, dtype=torch.float64), torch.zeros(r.B, r.Hq, D, dtype=torch.float64)
    for b in range(r.B):
        if not r.active[b]:
            continue
        at = torch.tensor(r.seen(b))
        pages = (b * r.table.shape[1] + at // r.P) if contiguous else r.table[b].long()[at // r.P]
        kk, vv, vvs = k[pages, at % r.P], v[pages, at % r.P], vs[pages, :, at % r.P]
        qq = q[b].double().view(r.Hkv, G, D)
        p = torch.softmax(torch.einsum("hgd,nhd->hgn", qq, kk) * f, -1)
        dot = lambda x, y: torch.einsum("hgn,nhd->hgd", x, y).reshape(r.Hq, -1)  # noqa: E731
        out[b] = dot(p, vv)
        A = dot(p, vv.abs())
        a = (torch.einsum("hgd,nhd->hgn", qq.abs(), kk.abs()).amax(-1) * f).reshape(r.Hq, 1)
        a1 = (qq.abs().amax(-1)[..., None] * kk.abs().sum(-1).t()[:, None]).amax(-1).reshape(r.Hq, 1) * f
        n = len(at)
        top = (p * vvs.t()[:, None]).amax(-1).reshape(r.Hq, 1)
        delta = a * (D + 4) * 2.0 ** -23 + a1 * 2.0 ** -22 + 2.0 ** -20
        u_p = 2.0 ** -22 if dtype == torch.float16 else 2.0 ** -11
        tol[b] = A * (2 * delta + u_p + n * 2.0 ** -23) + 448 * n * 2.0 ** -40 * top
    return out, tol


def differs(got, ref, dtype):
    """None, or a sentence about the worst element; NaN where the reference has it."""
    out, tol = ref
    half = torch.finfo(dtype).eps / 2
    tol = tol * (1 + half) + half * out.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    g = got.double().cpu()
    if not torch.equal(torch.isnan(g), torch.isnan(out)):
        return f"NaN in {int(torch.isnan(g).sum())} places, expected in {int(torch.isnan(out).sum())}"
    bad = ~((g - out).abs() <= tol) & ~torch.isnan(out)
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        return f"{int(bad.sum())} of {bad.numel()} off; at {at}: {g[at].item()} against {out[at].item()}, tolerance {tol[at].item()}"
    return None


def tree(parents, r, q, scale=0.0):
    """(out, A, a, n) as tests/window_ref.py's attention, of drafted tokens whose rows have these parents."""
    T, D, G = r.starts[-1], r.D, r.Hq // r.Hkv
    scale = scale if scale > 0 else 1 / math.sqrt(D)
    k, v = r.view(r.pool, 0), r.view(r.pool, 1)
    out = torch.zeros(T, r.Hq, D, dtype=torch.float64)
    A, a, n = torch.zeros_like(out), torch.zeros(T, r.Hq, 1, dtype=torch.float64), torch.zeros(T, r.Hq, 1, dtype=torch.float64)
    for b in range(r.B):
        if not r.active[b]:
            continue
        L, m = r.lens[b], r.news[b]
        base = L - m
        at = torch.arange(L)
        pages = r.table[b].long()[at // r.P]
        for x in range(m):
            chain, up = [], parents[b][x]
            while up >= 0:
                chain.append(base + up)
                up = parents[b][up]
            pos = base + len(chain)
            vis = (at < base) & ((pos - at < r.window) | (at < r.sinks) if r.window else at < base)
            vis[chain + [base + x]] = True
            t = r.starts[b] + x
            kk, vv = k[pages[vis], at[vis] % r.P].double(), v[pages[vis], at[vis] % r.P].double()
            qq = q[t].double().view(r.Hkv, G, D)
            p = torch.softmax(torch.einsum("hgd,nhd->hgn", qq, kk) * scale, -1)
            out[t] = torch.einsum("hgn,nhd->hgd", p, vv).reshape(r.Hq, D)
            A[t] = torch.einsum("hgn,nhd->hgd", p, vv.abs()).reshape(r.Hq, D)
            a[t] = (torch.einsum("hgd,nhd->hgn", qq.abs(), kk.abs()).amax(-1) * scale).view(r.Hq, 1)
            n[t] = int(vis.sum())
    return out, A, a, n


def parents(n, gen, kind="random"):
    """Parents of n drafted tokens: a chain, all siblings, or a tree in which every token picks an earlier one."""
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "flat":
        return [-1] * n
    return [int(torch.randint(-1, i, (1,), generator=gen)) if i else -1 for i in range(n)]
