"""64-bit plain forms of the paged 8-bit cache's operators, on the CPU, with the error bounds
the tests hold the kernels to.

Bounds: one rounding to type t is off by at most finfo(t).eps / 2 of the value.  fp32 sums of n
terms, each rounded, are off by at most n 2^-23 of the sum of magnitudes (twice the rounding
unit, which also covers sums that the matrix instructions truncate)."""
from __future__ import annotations

import math

import torch

QMAX = {"int8": 127.0, "e4m3": 448.0}
TORCH_CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
F64 = torch.float64


def norm_rope(x, pos, inv_freq=None, interleaved=False, w=None, eps=1e-6):
    """(y, bound on |fp32 result - y| before the last rounding) of rows x [T, H, D]."""
    y = x.to(F64)
    D = y.shape[-1]
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.to(F64)
    size = y.abs()
    if inv_freq is not None:
        r = 2 * inv_freq.numel()
        th = pos.to(F64)[:, None] * inv_freq.to(F64)[None]
        co, si = torch.cos(th)[:, None], torch.sin(th)[:, None]
        ia = torch.arange(0, r, 2) if interleaved else torch.arange(r // 2)
        ib = ia + 1 if interleaved else ia + r // 2
        a, b = y[..., ia], y[..., ib]
        y, size = y.clone(), size.clone()
        y[..., ia], y[..., ib] = a * co - b * si, a * si + b * co
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    # the sum of squares (D / 2 steps count, halved by the root), rsqrt, weights, sin and cos of
    # an angle rounded to fp32 within half a turn (pi 2^-25), two products and a sum
    return y, size * (D / 8 + 16) * 2.0 ** -24


def rounded_ok(got, want, bound, dtype):
    tol = want.abs() * (torch.finfo(dtype).eps / 2) + bound * 1.01 + torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    return ((got.to(F64) - want).abs() <= tol).all().item()


def pow2_scale(amax: float, code: str) -> float:
    s = 2.0 ** -64
    while QMAX[code] * s < amax:
        s *= 2
    return s


def to_codes(x, code):
    """Codes of fp64 values (nearest, ties to even), as numbers."""
    if code == "int8":
        return x.round().clamp(-127, 127)
    return x.to(torch.float32).clamp(-448, 448).to(torch.float8_e4m3fn).to(F64)


def code_step(x, code):
    """Half the distance of neighbouring codes around x."""
    if code == "int8":
        return torch.full_like(x, 0.5)
    return torch.maximum(x.abs() * 2.0 ** -4, torch.full_like(x, 2.0 ** -10))


def attention(q, k_pool, v_pool, k_scale, v_scale, table, lens, cu, scale, window=0, page=16):
    """(out, tolerance before the last rounding) of q [T, Hq, D]; rows of no sequence are NaN.
    Pools are numbers [pages, Hkv, page, D]."""
    T, Hq, D = q.shape
    Hkv = k_pool.shape[1]
    G = Hq // Hkv
    out = torch.full((T, Hq, D), math.nan, dtype=F64)
    tol = torch.zeros((T, Hq, D), dtype=F64)
    for b in range(len(lens)):
        n, L = cu[b + 1] - cu[b], max(0, lens[b])
        if n <= 0:
            continue
        ids = [int(table[b][i]) if i < len(table[b]) else -1 for i in range((L + page - 1) // page)]
        live = torch.tensor([0 <= ids[j // page] < k_pool.shape[0] for j in range(L)], dtype=torch.bool)
        safe = torch.tensor([i if 0 <= i < k_pool.shape[0] else 0 for i in ids], dtype=torch.long)
        rows = slice(cu[b], cu[b + 1])
        at = torch.arange(L - n, L)
        j = torch.arange(L)
        see = (j[None] <= at[:, None]) & live[None]
        if window:
            see &= j[None] > at[:, None] - window
        for h in range(Hkv):
            k = (k_pool[safe, h].to(F64) * k_scale[safe, h].to(F64)[:, None, None]).reshape(-1, D)[:L]
            v = (v_pool[safe, h].to(F64) * v_scale[safe, h].to(F64)[:, None, None]).reshape(-1, D)[:L]
            for g in range(G):
                hh = h * G + g
                qq = q[rows, hh].to(F64)
                if L == 0:
                    out[rows, hh] = 0
                    continue
                some = see.any(-1, keepdim=True)
                k0 = torch.where(live[:, None], k, torch.zeros_like(k))
                v0 = torch.where(see.any(0)[:, None], v, torch.zeros_like(v))
                k0 = torch.where(see.any(0)[:, None], k0, torch.zeros_like(k0))
                qz = torch.where(some, qq, torch.zeros_like(qq))
                x = (qz @ k0.T) * scale
                x = x.masked_fill(~see, -math.inf)
                p = torch.where(some, torch.softmax(x, -1), torch.zeros_like(x)).nan_to_num(0.0)
                out[rows, hh] = p @ v0
                # logits: a sum of D terms in fp32, times scales (two more roundings) and the
                # logit's own size in exp2's argument; weights rounded to fp16 (2^-11) or better,
                # the sum of weights and the products' sum over keys (at most 2^-23 a step of
                # the running sums, of which a key takes part in few: counted as 2^-16)
                mag = ((qz.abs() @ k0.abs().T) * abs(scale)).masked_fill(~see, 0).amax(-1, keepdim=True)
                d = 2 * mag * (D + 8) * 2.0 ** -23
                vmax = v0.abs().max()
                tol[rows, hh] = (p @ v0.abs()) * (2.0 ** -11 + d + 2.0 ** -16) + L * 2.0 ** -30 * vmax
    return out, tol


def make_pool(gen, pages, hkv, page, d, code, low=-8, high=-4):
    """(codes, scales) with power-of-two scales that differ from page to page."""
    x = torch.randn((pages, hkv, page, d), generator=gen) * (60 if code == "e4m3" else 24)
    x = x.clamp(-QMAX[code], QMAX[code])
    codes = (x.round() if code == "int8" else x).to(TORCH_CODE[code])
    s = torch.exp2(torch.randint(low, high, (pages, hkv), generator=gen).float())
    return codes, s


def make_table(gen, lens, page, max_pages, extra=3):
    """(table, pages): distinct random pages for every sequence, -1 behind the last one."""
    need = [(max(0, n) + page - 1) // page for n in lens]
    perm = torch.randperm(sum(need) + extra, generator=gen).tolist()
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = perm.pop()
    return table, sum(need) + extra


def append(k, v, pools, table, lens, cu, page, code, encode):
    """Reference append.  pools: numbers (k, v) [pages, Hkv, page, D] and scales, copied.  Returns
    (values over scales unrounded, scales, bound over scales, written mask) for K and V."""
    res = []
    Hkv, D = k.shape[1], k.shape[2]
    for x, pool, scale, enc in ((k, pools[0], pools[2], encode), (v, pools[1], pools[3], None)):
        val, sc = pool.to(F64).clone(), scale.to(F64).clone()
        bound = torch.zeros_like(val)
        state = torch.zeros(val.shape[:3], dtype=torch.int8)       # 1: new token, 2: held, rescaled
        for b in range(len(lens)):
            n = cu[b + 1] - cu[b]
            if lens[b] == 0 or n == 0:
                continue
            start = lens[b] - n
            rows = x[cu[b]:cu[b + 1]].to(F64)
            err = rows.abs() * 0
            if enc is not None:
                rows, err = enc(x[cu[b]:cu[b + 1]], torch.arange(start, lens[b]))
            j = start
            while j < lens[b]:
                pg, lo = int(table[b, j // page]), j % page
                m = min(page - lo, lens[b] - j)
                for h in range(Hkv):
                    part = rows[j - start:j - start + m, h]
                    fin = part[torch.isfinite(part)].abs()
                    amax = fin.max().item() if fin.numel() else 0.0
                    new = pow2_scale(amax, code)
                    if lo:
                        old = sc[pg, h].item()
                        new = max(new, old)
                        if new != old:
                            val[pg, h, :lo] = to_codes(val[pg, h, :lo] * (old / new), code)
                            state[pg, h, :lo] = 2
                    sc[pg, h] = new
                    val[pg, h, lo:lo + m] = part / new
                    bound[pg, h, lo:lo + m] = err[j - start:j - start + m, h] / new
                    state[pg, h, lo:lo + m] = 1
                j += m
        res.append((val, sc, bound, state))
    return res
