"""The 8-bit projection and the 4-bit cache written out from their definitions
in 64 bits (torch on the CPU), and the bounds their GPU results are held to.

Half a step of rounding to a type t is finfo(t).eps / 2 relative to the value
(and half the smallest subnormal absolutely); U32 = 2^-24 is that of fp32."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24
LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
PAGE = 64
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ quant --

def quant_rows(x):
    """(q int8, scale float32) of rows of a bf16 or fp16 tensor."""
    x = x.cpu().double()
    top = x.abs().amax(1) if x.shape[1] else torch.zeros(x.shape[0], dtype=torch.float64)
    ok = torch.isfinite(x).all(1) & (top >= 2.0 ** -100)
    q = torch.zeros(x.shape, dtype=torch.int8)
    # numerator and quotient in 64 bits: an 18-bit by 11-bit quotient is exactly halfway or clearly off it
    q[ok] = torch.round(x[ok] * 127 / top[ok][:, None]).to(torch.int8)
    scale = (top.float() / 127).where(ok, torch.zeros(()))
    return q, scale.where(torch.isfinite(x).all(1), torch.full((), math.nan))


# -------------------------------------------------------------- projection --

def proj_quant(x, xs, w, ws, hq, hkv, D, gq, gk, eps, plain):
    """[T, N] in 64 bits."""
    y = (x.cpu().double() @ w.cpu().double().t()) * ws.cpu().double() * xs.cpu().double()[:, None]
    if not plain:
        for lo, n, g in ((0, hq, gq), (hq * D, hkv, gk)):
            if n:
                h = y[:, lo:lo + n * D].reshape(-1, n, D)
                rms = torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
                y[:, lo:lo + n * D] = (h / rms * g.cpu().double()).reshape(-1, n * D)
    return y


def proj_tolerance(y, dtype, D):
    """The output's rounding, and on the way to it: the sum's conversion, two scales,
    gamma, the norm's factor and its application (a step each), and the mean
    square (D squares and sums, halved by the root; its reciprocal root a step or two)."""
    return y.abs() * (half_step(dtype) * (1 + 2.0 ** -7) + (D / 2 + 12) * U32) + TINY[dtype]


# ------------------------------------------------------------------- cache --

def vector_codes(x):
    """(codes uint8, scales bf16) of head vectors [..., D]."""
    x = x.cpu().double()
    top = x.abs().amax(-1)
    finite = torch.isfinite(x).all(-1)
    live = finite & (top >= 2.0 ** -100)
    s = torch.where(live, top / 6, torch.ones(())).to(torch.bfloat16)
    u = torch.where(live[..., None], x, torch.zeros(())) / s.double()[..., None]
    a = u.abs().clamp(max=6.0)
    dist = (a[..., None] - LEVELS).abs()
    best = dist.amin(-1, keepdim=True)
    near = dist == best                                       # one level, or two at a halfway point
    even = torch.tensor([True, False] * 4)
    pick = torch.where((near.sum(-1, keepdim=True) > 1), near & even, near)
    code = pick.int().argmax(-1).to(torch.uint8) | ((u < 0).to(torch.uint8) << 3)
    scale = torch.where(live, s.float(), torch.zeros(())).where(finite, torch.full((), math.nan))
    return code, scale.to(torch.bfloat16)


def code_values(code):
    v = LEVELS[(code & 7).long()]
    return torch.where(code >= 8, -v, v)


def read_page(page, D):
    """(K, V) values [hkv, 64, D] in 64 bits of one page [hkv, 64*D + 256] of bytes, byte by byte
    as documented."""
    page = page.cpu()
    h = page.shape[0]
    k = torch.empty(h, PAGE, D, dtype=torch.float64)
    v = torch.empty(h, PAGE, D, dtype=torch.float64)
    for t in range(PAGE):
        kb = page[:, t * (D // 2):(t + 1) * (D // 2)]
        vb = page[:, 32 * D + t:64 * D:64]
        for out, b, at in ((k, kb, 64 * D), (v, vb, 64 * D + 128)):
            s = page[:, at + 2 * t:at + 2 * t + 2].contiguous().view(torch.bfloat16).double()
            out[:, t, 0::2] = code_values(b & 15) * s
            out[:, t, 1::2] = code_values(b >> 4) * s
    return k, v


def random_cache(pages, hkv, D, seed, vscale=1.0, stride=None):
    """A cache of random codes and scales [pages, hkv, 64*D + 256] uint8 (CPU)."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 256, (pages, hkv, 64 * D + 256), generator=g, dtype=torch.uint8)
    ks = (torch.rand(pages, hkv, PAGE, generator=g) * 0.5 + 0.2).to(torch.bfloat16)
    vs = (torch.exp2(torch.randn(pages, hkv, PAGE, generator=g) * 2) * 0.2 * vscale).to(torch.bfloat16)
    c[..., 64 * D:64 * D + 128] = ks.view(torch.uint8)
    c[..., 64 * D + 128:] = vs.view(torch.uint8)
    return c


# --------------------------------------------------------------- attention --

def attention(q, cache, table, lens, starts, hq, hkv, D, scale, window, dtype, values=None):
    """(out, lse, tolerance of out, tolerance of lse, rows that some sequence has), 64 bits.

    The tolerances, for a row that sees n tokens, from
      d    the score's error: fp32 sums of D exact products, times two factors
      2^-11  a weight's rounding to fp16, or 2^-25 below fp16's normal range (of
           weights that are at most about one times the largest V scale there)
      n    additions in fp32 of weights and of weighted values
    """
    T = q.shape[0]
    group = hq // hkv
    q = q.cpu().double()
    out = torch.zeros(T, hq, D, dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    covered = torch.zeros(T, dtype=torch.bool)
    pages = cache.shape[0]
    read = {}
    for b in range(len(lens)):
        n0, r0, r1 = lens[b], starts[b], starts[b + 1]
        covered[r0:r1] = True
        if n0 == 0 or r1 == r0:
            continue
        ks, vs, there = [], [], []
        for j in range((n0 + PAGE - 1) // PAGE):
            p = int(table[b][j])
            ok = 0 <= p < pages
            if ok and p not in read:
                read[p] = read_page(cache[p], D)
            k, v = read[p] if ok else (torch.zeros(hkv, PAGE, D, dtype=torch.float64),) * 2
            ks.append(k)
            vs.append(v)
            there += [ok] * PAGE
        k, v = torch.cat(ks, 1)[:, :n0], torch.cat(vs, 1)[:, :n0]
        there = torch.tensor(there[:n0])
        at = torch.arange(n0)
        for i in range(r1 - r0):
            pos = n0 - (r1 - r0) + i
            see = there & (at <= pos)
            if window:
                see &= at > pos - window
            n = int(see.sum())
            if n == 0:
                continue
            for h in range(hq):
                kk, vv = k[h // group][see], v[h // group][see]
                qq = q[r0 + i, h * D:(h + 1) * D]
                s = kk @ qq * scale
                l = torch.logsumexp(s, 0)
                p = torch.exp(s - l)
                o = p @ vv
                d = float(((kk.abs() @ qq.abs()) * abs(scale)).max()) * (D + 4) * U32 + 4 * U32 * float(s.abs().max() + 1)
                a = p @ vv.abs()
                out[r0 + i, h], lse[r0 + i, h] = o, l
                tol[r0 + i, h] = (a * (2.0 ** -11 + 2 * d + (2 * n + 64) * U32) + n * 2.0 ** -25 * float(vv.abs().max())
                                  + o.abs() * half_step(dtype) * (1 + 2.0 ** -7) + TINY[dtype])
                ltol[r0 + i, h] = d + (n + 16) * U32 + 4 * U32 * (abs(float(l)) + 1)
    return out, lse, tol, ltol, covered
