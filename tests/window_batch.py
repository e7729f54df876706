"""Float64 attention over a window and sinks for whole blocks of queries, values
that are no numbers included, and its bounds; written from the definition in
include/vh.h, apart from tests/window_ref.py.

With p the weights of the visible keys, a column of V that holds an infinity or a
NaN gives what float64 gives for sum_j p_j V_j: p_j > 0 for every score above
-inf, so +inf or -inf, NaN if both or a NaN are seen, NaN for an infinity under a
score of -inf (0 times infinity), and NaN everywhere in a row whose visible scores
hold a NaN or +inf or are all -inf.  The bounds (A, a, n of tests/window_ref.py) are
those of the finite elements.
"""
import math

import torch


def attention(r, q, scale=0.0, device="cuda", block=128):
    """(out, A, a, n) of the new tokens' queries q [T, Hq, D], on the CPU."""
    T, D, G = r.starts[-1], r.D, r.Hq // r.Hkv
    scale = scale if scale > 0 else 1 / math.sqrt(D)
    f64 = dict(dtype=torch.float64, device=device)
    out, A = torch.zeros(T, r.Hkv, G, D, **f64), torch.zeros(T, r.Hkv, G, D, **f64)
    a, n = torch.zeros(T, r.Hkv, G, 1, **f64), torch.zeros(T, r.Hkv, G, 1, **f64)
    keys, vals = r.view(r.pool, 0), r.view(r.pool, 1)
    for b in range(r.B):
        if not r.active[b] or not r.news[b]:
            continue
        L, m, first = r.lens[b], r.news[b], r.lens[b] - r.news[b]
        for x in range(0, m, block):
            c = min(block, m - x)
            i = torch.arange(first + x, first + x + c)
            low = max(0, first + x - r.window + 1) if r.window else 0
            at = torch.cat([torch.arange(0, min(r.sinks, low)), torch.arange(low, first + x + c)])
            pages = r.table[b].long()[at // r.P]
            k, v = (t[pages, at % r.P].to(**f64).transpose(0, 1) for t in (keys, vals))      # [Hkv, n, D]
            see = at[None] <= i[:, None]
            if r.window:
                see &= (i[:, None] - at[None] < r.window) | (at[None] < r.sinks)
            see = see.to(device)[None, :, None]                                              # [1, c, 1, n]
            t0 = r.starts[b] + x
            qq = q[t0:t0 + c].to(**f64).view(c, r.Hkv, G, D).permute(1, 0, 2, 3)             # [Hkv, c, G, D]
            flat = qq.reshape(r.Hkv, c * G, D)
            # (products with infinities one by one: a matrix product may order them as it likes)
            s = (flat @ torch.nan_to_num(k, 0, 0, 0).transpose(1, 2)).view(r.Hkv, c, G, -1) * scale
            odd = ~torch.isfinite(k).all(-1)
            for h, j in odd.nonzero().tolist():
                s[h, :, :, j] = (qq[h] * k[h, j]).sum(-1) * scale
            s = s.masked_fill(~see, -math.inf)
            p = torch.softmax(s, -1)
            real = torch.nan_to_num(v, 0, 0, 0)
            dot = lambda w, y: (w.reshape(r.Hkv, c * G, -1) @ y).view(r.Hkv, c, G, D)  # noqa: E731
            o = dot(torch.nan_to_num(p, 0.0), real)
            if not torch.isfinite(v).all():
                some, none = (see & (s > -math.inf)).double(), (see & (s == -math.inf)).double()
                up, down = dot(some, (v == math.inf).double()) > 0, dot(some, (v == -math.inf).double()) > 0
                bad = (dot(some + none, torch.isnan(v).double()) + dot(none, torch.isinf(v).double()) > 0) | (up & down)
                o = torch.where(up, math.inf, torch.where(down, -math.inf, o)).masked_fill(bad, math.nan)
            o = o.masked_fill(torch.isnan(p).any(-1, keepdim=True), math.nan)
            to = slice(t0, t0 + c)
            out[to] = o.permute(1, 0, 2, 3)
            A[to] = dot(torch.nan_to_num(p, 0.0), real.abs()).permute(1, 0, 2, 3)
            kk = torch.nan_to_num(k, 0, 0, 0).abs().transpose(1, 2)
            top = ((flat.abs() @ kk).view(r.Hkv, c, G, -1) * see).amax(-1, keepdim=True) * scale
            a[to] = top.permute(1, 0, 2, 3)
            n[to] = see.sum(-1, dtype=torch.float64).view(1, c, 1, 1).expand(r.Hkv, c, G, 1).permute(1, 0, 2, 3)
    return tuple(t.reshape(T, r.Hq, -1).cpu() for t in (out, A, a, n))


def differs(got, ref, tol):
    """None, or a sentence: infinities and NaN have to be where the reference has them, the rest within tol."""
    g, want = got.double().cpu(), ref[0]
    for what, x, y in (("NaN", torch.isnan(g), torch.isnan(want)), ("+inf", g == math.inf, want == math.inf),
                       ("-inf", g == -math.inf, want == -math.inf)):
        if not torch.equal(x, y):
            at = (x != y).nonzero()
            t = tuple(at[0].tolist())
            return f"{what} in {int(x.sum())} places, expected in {int(y.sum())}; {len(at)} differ, at {t}: {g[t].item()} against {want[t].item()}"
    d = (g - want).abs()
    bad = torch.isfinite(want) & ~(d <= tol)
    if bad.any():
        t = tuple(bad.nonzero()[0].tolist())
        return f"{int(bad.sum())} of {bad.numel()} off; at {t}: {g[t].item()} against {want[t].item()}, tolerance {tol[t].item()}"
    return None
