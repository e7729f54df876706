"""Float64 reference of the ragged append and the windowed attention, on the
CPU, written from the definitions in include/vh.h; and seeded inputs for them.

Attention tolerance, elementwise.  With A = sum_j p_j |v_j| (the attention of
|v|), a = scale max_j sum_d |q_d| |k_jd|, n visible keys and head dim D:
  * the score of a key is off by at most a (u_q + (D + 4) 2^-23): u_q is the
    rounding of q (2^-16 for the bf16 high part plus residual of the decode
    kernel, 2^-22 for fp16, 0 for the prompt kernel, which takes q as it is),
    the products are summed in fp32, and the scale is one more rounding;
  * a weight is off by that, relatively, by exp2 and the max's subtraction
    (2^-20 covers both), and by its rounding u_p to the element type (2^-16 and
    2^-22 for the split weights of the decode kernel; 2^-8 and 2^-11 for the
    prompt kernel); the same holds for the sum, hence the factor 2 on the first;
  * n fp32 additions lose at most n 2^-23;
  * the output is rounded once: 2^-8 |o| (bf16), 2^-11 |o| (fp16).
fp16 weights below 2^-14 lose 2^-25 absolutely (the largest weight is at least
1 before the division by the sum): n 2^-25 max|v|; subnormal outputs lose 2^-25.
"""
from __future__ import annotations

import math
from dataclasses import dataclass, field

import torch

NAN_BITS = 0x7FC0  # a quiet NaN in bf16 and in fp16


@dataclass
class Ragged:
    """A seeded ragged batch on the CPU.  pool: NHD [NP, 2, P, Hkv, D] or HND [NP, 2, Hkv, P, D]."""
    Hq: int
    Hkv: int
    D: int
    P: int
    pool: torch.Tensor
    layout: str
    table: torch.Tensor          # int32 [B, pages per row]
    lens: list
    news: list
    active: list
    window: int
    sinks: int
    extra: dict = field(default_factory=dict)

    @property
    def B(self):
        return len(self.lens)

    @property
    def starts(self):
        s = [0]
        for n in self.news:
            s.append(s[-1] + n)
        return s

    def view(self, pool, i):
        return pool[:, i] if self.layout == "NHD" else pool[:, i].transpose(1, 2)

    def seen(self, b):
        """Slots of row b that some query of the call sees."""
        L, n, W, S = self.lens[b], self.news[b], self.window, self.sinks
        lo = max(0, L - n + 1 - W) if W else 0
        return [j for j in range(L) if j >= lo or j < S]


def make(lens, news, Hq=16, Hkv=8, D=128, P=16, window=0, sinks=0, dtype=torch.bfloat16, layout="NHD", seed=0,
         active=None, sigma=1.0, table_extra=1, dead=-1, spare=3):
    """Pages in a seeded order; every slot that no query sees holds NaN, and the
    entries of pages without a seen slot hold `dead`."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    active = [1] * B if active is None else list(active)
    per_row = max(1, max(-(-L // P) for L in lens)) + table_extra
    r = Ragged(Hq, Hkv, D, P, None, layout, None, list(lens), list(news), active, window, sinks)
    want = [(b, j) for b in range(B) if active[b] for j in sorted({s // P for s in r.seen(b)})]
    NP = len(want) + 1 + spare
    ids = (1 + torch.randperm(NP - 1, generator=g))[:len(want)].tolist()
    table = torch.full((B, per_row), dead, dtype=torch.int32)
    pool = torch.empty((NP, 2, P, Hkv, D), dtype=dtype)
    pool.view(torch.int16).fill_(NAN_BITS)
    for (b, j), page in zip(want, ids):
        table[b, j] = page
    for b in range(B):
        if not active[b]:
            continue
        for s in r.seen(b):
            pool[table[b, s // P], :, s % P] = (torch.randn(2, Hkv, D, generator=g) * sigma).to(dtype)
    r.table = table
    r.pool = pool if layout == "NHD" else pool.transpose(2, 3).contiguous()
    r.extra["gen"] = g
    return r


def queries(r, dtype, sigma=1.0):
    return (torch.randn(r.starts[-1], r.Hq, r.D, generator=r.extra["gen"]) * sigma).to(dtype)


def attention(r: Ragged, q, scale=0.0, contiguous=False):
    """(out, A, a, n): float64 output [T, Hq, D], attention of |v|, score bound
    and visible keys [T, Hq, 1]; rows of inactive requests are zeros."""
    T, D, G = r.starts[-1], r.D, r.Hq // r.Hkv
    scale = scale if scale > 0 else 1 / math.sqrt(D)
    k, v = r.view(r.pool, 0), r.view(r.pool, 1)
    out = torch.zeros(T, r.Hq, D, dtype=torch.float64)
    A, a, n = torch.zeros_like(out), torch.zeros(T, r.Hq, 1, dtype=torch.float64), torch.zeros(T, r.Hq, 1, dtype=torch.float64)
    for b in range(r.B):
        if not r.active[b]:
            continue
        L, m = r.lens[b], r.news[b]
        at = torch.arange(L)
        pages = (b * r.table.shape[1] + at // r.P) if contiguous else r.table[b].long()[at // r.P]
        for x in range(m):
            i, t = L - m + x, r.starts[b] + x
            vis = (at <= i) & ((at < r.sinks) | (at > i - r.window) if r.window else at <= i)
            kk, vv = k[pages[vis], at[vis] % r.P].double(), v[pages[vis], at[vis] % r.P].double()  # [n, Hkv, D]
            qq = q[t].double().view(r.Hkv, G, D)
            s = torch.einsum("hgd,nhd->hgn", qq, kk) * scale
            p = torch.softmax(s, -1)
            out[t] = torch.einsum("hgn,nhd->hgd", p, vv).reshape(r.Hq, D)
            A[t] = torch.einsum("hgn,nhd->hgd", p, vv.abs()).reshape(r.Hq, D)
            a[t] = (torch.einsum("hgd,nhd->hgn", qq.abs(), kk.abs()).amax(-1) * scale).view(r.Hq, 1)
            n[t] = int(vis.sum())
    return out, A, a, n


def tolerance(ref, dtype, D, split: bool, vmax: float):
    """Elementwise bound (see the module's docstring); split: the decode kernel."""
    out, A, a, n = ref
    half = torch.finfo(dtype).eps / 2
    u_q = (2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -22) if split else 0.0
    u_p = (2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -22) if split else half
    delta = a * (u_q + (D + 4) * 2.0 ** -23) + 2.0 ** -20
    tol = half * out.abs() + A * (2 * delta + u_p + n * 2.0 ** -23) * (1 + half)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 * (1 + n * vmax)
    return tol


def close(got, ref, dtype, D, split, vmax=8.0):
    """None, or a sentence about the worst element."""
    d = (got.double().cpu() - ref[0]).abs()
    tol = tolerance(ref, dtype, D, split, vmax)
    bad = ~(d <= tol)
    if not bad.any():
        return None
    w = torch.where(bad, torch.nan_to_num(d / tol, nan=1e30, posinf=1e30), torch.zeros(()).double())
    i = int(w.argmax())
    at = []
    for s in reversed(d.shape):
        at.append(i % s)
        i //= s
    at = tuple(reversed(at))
    return f"{int(bad.sum())} of {d.numel()} off; at {at}: {got[at].item()} against {ref[0][at].item()}, tolerance {tol[at].item()}"


def rope(x, cos, sin, w, eps, interleaved):
    """Float64 norm and rotation of x [T, H, D], and the bound (per unit) of fp32's error.
    cos, sin [T, D/2].  fp32: the norm's mean, rsqrt and two products stay within 2^-20
    relatively (the sum of D squares D 2^-24, rsqrt and the division 2^-22), the
    rotation's two products and one sum within 3 2^-24 (|x c| + |y s|) <= 2^-22 (|x| + |y|)."""
    x = x.double()
    rel = 2.0 ** -22
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
        rel = 2.0 ** -19
    h = x.shape[-1] // 2
    i = torch.arange(h)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    c, s = cos[:, None].double(), sin[:, None].double()
    y, err = torch.empty_like(x), torch.empty_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    err[..., a] = err[..., b] = rel * (x[..., a].abs() + x[..., b].abs())
    return y, err
