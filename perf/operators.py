"""Cases of the paged 8-bit cache's operators and their plain forms.

norm_rope   per-head RMS norm of queries and keys and their rotation, in one pass
append      new keys (normed and rotated on the way) and values into the paged 8-bit cache, with
            the step's queries
attention   attention over that cache: single tokens, several tokens a sequence, prompt chunks

A page of the cache holds `page` tokens of every kv head as 8-bit codes [kv head][token][dim] and
one fp32 scale per (page, kv head) for the keys and one for the values."""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
SCALE_MIN_EXP = -64      # the append's smallest scale is 2^-64
EPS = 1e-6
THETA = 10000.0


def _case(name, op, **kw):
    c = dict(op=op, hkv=8, g=4, d=128, dtype="bf16", rot=128, interleaved=False, norm=True)
    c.update(kw)
    c["name"] = name
    return c


def listed():
    return [
        # one token of one sequence: the latency of a decode step's first kernel
        _case("norm_rope_step", "norm_rope", t=1, pos_max=32768),
        # a long prompt, whole heads rotated
        _case("norm_rope_prompt", "norm_rope", t=32768, pos_max=32768),
        # an odd number of tokens of a model with 64-dim heads, partly rotated in interleaved pairs, far positions
        _case("norm_rope_odd", "norm_rope", t=5003, pos_max=1 << 20, hkv=8, g=8, d=64, dtype="fp16", rot=32,
              interleaved=True),
        # one new token of each of 64 sequences, most of them inside a page that has tokens already
        _case("append_step", "append", b=64, start_min=1000, start_max=2048, new_min=1, new_max=1, page=64,
              code="e4m3"),
        # chunks of eight prompts of odd lengths, some continuing a page
        _case("append_chunks", "append", b=8, start_min=0, start_max=4000, new_min=1500, new_max=4096, page=64,
              code="e4m3"),
        # short prompts of many sequences, small pages, 64-dim heads, no norm
        _case("append_short", "append", b=96, start_min=0, start_max=40, new_min=1, new_max=200, page=16,
              code="e4m3", d=64, g=2, dtype="fp16", rot=64, interleaved=True, norm=False),
        # one short sequence: latency
        _case("attend_one", "attention", b=1, len_min=700, len_max=700, q_min=1, q_max=1, page=64, code="e4m3",
              window=0),
        # the 64 x 32k decode step
        _case("attend_b64_32k", "attention", b=64, len_min=32768, len_max=32768, q_min=1, q_max=1, page=64,
              code="e4m3", window=0),
        # one sequence of 131k tokens, 64 query heads on 8 kv heads
        _case("attend_b1_131k", "attention", b=1, len_min=131072, len_max=131072, q_min=1, q_max=1, page=128,
              code="int8", g=8, window=0),
        # a ragged batch, 64-dim heads, small pages, the last 4096 tokens of each sequence
        _case("attend_ragged_window", "attention", b=48, len_min=1, len_max=16384, q_min=1, q_max=1, page=16,
              code="int8", d=64, g=7, dtype="fp16", window=4096),
        # verification of a few drafted tokens for each sequence
        _case("attend_verify", "attention", b=16, len_min=4000, len_max=8192, q_min=3, q_max=6, page=32,
              code="e4m3", window=0),
        # prompt chunks on top of what the cache holds
        _case("attend_prompt", "attention", b=2, len_min=12000, len_max=16384, q_min=1900, q_max=2048, page=64,
              code="e4m3", window=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice([64, 128])
    c = dict(op=rng.choice(["norm_rope", "append", "attention", "attention"]), d=d, hkv=rng.choice([1, 2, 4, 8]),
             g=rng.choice([1, 2, 4, 5, 7, 8]), dtype=rng.choice(["bf16", "fp16"]), norm=rng.random() < 0.5,
             rot=8 * rng.randint(1, d // 8), interleaved=rng.random() < 0.5)
    if c["op"] == "norm_rope":
        c.update(t=_log_int(rng, 1, 16384), pos_max=rng.choice([4096, 131072, 1 << 20]))
    elif c["op"] == "append":
        b = _log_int(rng, 1, 128)
        c.update(b=b, start_min=0, start_max=_log_int(rng, 1, 4096), new_min=1,
                 new_max=_log_int(rng, 1, max(1, 16384 // b)), page=rng.choice([16, 32, 64, 128]), code="e4m3")
    else:
        b = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 32768)
        c.update(b=b, page=rng.choice([16, 32, 64, 128]), code=rng.choice(["e4m3", "int8"]), len_min=max(1, hi // 8),
                 len_max=hi, window=rng.choice([0, 0, _log_int(rng, 16, 8192)]))
        # heads x query rows x keys within the largest listed case's
        qmax = _log_int(rng, 1, max(1, min(2048, (1 << 31) // (b * hi * c["hkv"] * c["g"]))))
        c.update(q_min=max(1, qmax // 2), q_max=qmax)
    return c


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _lens(b, lo, hi, turn=0.6180339887498949):
    """b lengths in [lo, hi], spread over their logarithm in an irregular order; the first is hi. They
    are the case's own: every seed has the same shapes."""
    a, w = math.log(lo + 1), math.log(hi + 1) - math.log(lo + 1)
    return [hi] + [max(lo, min(hi, int(math.exp(a + w * (i * turn % 1.0)) - 1))) for i in range(1, b)]


def _shapes(c):
    """(tokens in the cache, new tokens or query tokens) of each sequence."""
    if c["op"] == "append":
        new = _lens(c["b"], c["new_min"], c["new_max"], 0.7548776662466927)
        return [s + n for s, n in zip(_lens(c["b"], c["start_min"], c["start_max"]), new)], new
    lens = _lens(c["b"], c["len_min"], c["len_max"])
    return lens, [min(n, q) for n, q in zip(lens, _lens(c["b"], c["q_min"], c["q_max"], 0.7548776662466927))]


def _cumulative(n):
    return torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)


def _block_table(gen, lens, page):
    """(block table [B, max pages] int32 with -1 behind a sequence's last page, pages in the pool)."""
    need = (lens + page - 1) // page
    most, total = int(need.max()), int(need.sum())
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    at = _cumulative(need).to(torch.int64)[:-1, None] + torch.arange(max(1, most), device=DEV)[None]
    live = torch.arange(max(1, most), device=DEV)[None] < need[:, None]
    return perm[at.clamp(max=total - 1)].masked_fill(~live, -1), total


def _pool(gen, pages, c):
    """Codes [pages][kv head][page][dim] and scales [pages][kv head] of values near N(0, 1) whose
    size differs from head to head and page to page."""
    shape = (pages, c["hkv"], c["page"], c["d"])
    codes = torch.empty(shape, dtype=CODES[c["code"]], device=DEV)
    unit = 64.0 if c["code"] == "e4m3" else 24.0
    step = max(1, (1 << 27) // (c["hkv"] * c["page"] * c["d"]))
    for i in range(0, pages, step):
        x = torch.randn((min(step, pages - i), *shape[1:]), generator=gen, device=DEV, dtype=torch.bfloat16) * unit
        x = x.clamp_(-QMAX[c["code"]], QMAX[c["code"]])
        codes[i:i + step] = (x.round_() if c["code"] == "int8" else x).to(codes.dtype)
    # powers of two, as the append writes them
    base = -6 if c["code"] == "e4m3" else -5
    e = torch.randint(-1, 2, shape[:2], generator=gen, device=DEV) + base
    return codes, torch.exp2(e.to(torch.float32))


def _rope_state(gen, c):
    s = {"inv_freq": None, "qw": None, "kw": None}
    dt = DTYPES[c["dtype"]]
    if c["rot"]:
        i = torch.arange(c["rot"] // 2, dtype=torch.float64)
        s["inv_freq"] = torch.pow(THETA, -2.0 * i / c["rot"]).to(torch.float32).to(DEV)
    if c["norm"]:
        s["qw"] = (1 + 0.1 * torch.randn(c["d"], generator=gen, device=DEV)).to(dt)
        s["kw"] = (1 + 0.1 * torch.randn(c["d"], generator=gen, device=DEV)).to(dt)
    return s


def _qkv(gen, t, c):
    """Queries, keys and values as views of one projection's output, as a layer has them."""
    hq, hkv, d = c["hkv"] * c["g"], c["hkv"], c["d"]
    x = torch.randn((t, hq + 2 * hkv, d), generator=gen, device=DEV, dtype=torch.float32).to(DTYPES[c["dtype"]])
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


def prepare(case, seed):
    c, gen = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "norm_rope":
        s["q"], s["k"], _ = _qkv(gen, c["t"], c)
        s["pos"] = torch.randint(0, c["pos_max"], (c["t"],), generator=gen, device=DEV, dtype=torch.int32)
        s.update(_rope_state(gen, c))
        if own:
            from reasoning_model_kv_b200 import TkvRope
            s["rope"] = TkvRope(s["inv_freq"], c["interleaved"], s["qw"], s["kw"], EPS)
        return s
    lens, new = (torch.tensor(x, device=DEV) for x in _shapes(c))
    if c["op"] == "append":
        s["cu"], s["max_new"] = _cumulative(new), c["new_max"]
        s["q"], s["k"], s["v"] = _qkv(gen, int(new.sum()), c)
        s.update(_rope_state(gen, c))
    else:
        s["max_q"] = c["q_max"]
        s["cu"] = _cumulative(new) if c["q_max"] > 1 else None
        s["q"] = _qkv(gen, int(new.sum()), c)[0].contiguous()
    s["kv_len"] = lens.to(torch.int32)
    s["block_table"], pages = _block_table(gen, lens, c["page"])
    s["k_pool"], s["k_scale"] = _pool(gen, pages, c)
    s["v_pool"], s["v_scale"] = _pool(gen, pages, c)
    if own:
        from reasoning_model_kv_b200 import TkvPagedCache, TkvRope
        s["cache"] = TkvPagedCache(c["b"], c["hkv"], c["g"], c["d"], c["page"], pages, s["block_table"].shape[1],
                                   code=c["code"], dtype=DTYPES[c["dtype"]],
                                   pools=(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"]))
        if c["op"] == "append":
            s["rope"] = TkvRope(s["inv_freq"], c["interleaved"], s["qw"], s["kw"], EPS)
    return s


# ----------------------------------------------------------------------------- plain forms
def _norm_rope(x, w, pos, inv_freq, c):
    """fp32 rows [T, H, D] of x after the norm (w not None) and the rotation."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    if inv_freq is None:
        return y
    th = pos.double()[:, None] * inv_freq.double()[None]
    cos, sin = torch.cos(th).float()[:, None], torch.sin(th).float()[:, None]
    r = c["rot"]
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if c["interleaved"] else (y[..., :r // 2], y[..., r // 2:r])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, v), -1).flatten(-2) if c["interleaved"] else torch.cat((u, v), -1)
    return torch.cat((turned, y[..., r:]), -1)


def _pow2_scale(amax, code):
    """The smallest power of two s >= 2^-64 with qmax * s >= amax."""
    m, e = torch.frexp(amax)
    qm, qe = math.frexp(QMAX[code])
    x = e - qe + (m > qm).to(e.dtype)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, x, SCALE_MIN_EXP).clamp(min=SCALE_MIN_EXP))


def _codes(x, code):
    return (x.round().clamp(-127, 127) if code == "int8" else x).to(CODES[code])


def _append_one(x, pool, scale, pages, offs, first_page, lo, code):
    """x [T, Hkv, D] fp32 into the pool's slots (pages, offs); lo [B] tokens of first_page [B], the
    first page that a sequence writes, were there before. In place."""
    amax = x.abs().amax(-1)                                                      # [T, Hkv]
    need = torch.zeros_like(scale).index_reduce_(0, pages, amax, "amax")
    need = _pow2_scale(need, code)
    old_first = scale[first_page]                                                # [B, Hkv]
    keep = torch.where((lo > 0)[:, None], old_first, torch.zeros_like(old_first))
    new = torch.maximum(need, torch.zeros_like(scale).index_copy_(0, first_page, keep))
    # the tokens that the first pages held, in the pages' new scales
    ratio = (old_first / new[first_page])[:, :, None, None]
    held = pool[first_page]
    redone = _codes(held.float() * ratio, code)
    inside = torch.arange(pool.shape[2], device=x.device)[None] < lo[:, None]
    pool[first_page] = torch.where(inside[:, None, :, None], redone.view(torch.uint8), held.view(torch.uint8)).view(pool.dtype)
    scale[pages] = new[pages]
    pool.view(torch.uint8)[pages, :, offs] = _codes(x / new[pages][..., None], code).view(torch.uint8)


def _slots(s, page):
    """Of each new token: its position, page and offset; of each sequence (all have new tokens): the
    first page written and the tokens that it held."""
    cu, lens = s["cu"].long(), s["kv_len"].long()
    start = lens - (cu[1:] - cu[:-1])
    t = torch.arange(s["k"].shape[0], device=cu.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    slot = start[b] + t - cu[b]
    rows = torch.arange(len(start), device=cu.device)
    return (slot, s["block_table"][b, slot // page].long(), slot % page,
            s["block_table"][rows, start // page].long(), start % page)


def _append(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    slot, pages, offs, first, lo = _slots(s, c["page"])
    q = _norm_rope(s["q"], s["qw"], slot, s["inv_freq"], c).to(dt)
    k = _norm_rope(s["k"], s["kw"], slot, s["inv_freq"], c)
    _append_one(k, s["k_pool"], s["k_scale"], pages, offs, first, lo, c["code"])
    _append_one(s["v"].float(), s["v_pool"], s["v_scale"], pages, offs, first, lo, c["code"])
    return q


def _seen(lens, nq, most_q, most_k, window):
    """[B, most_q, most_k]: query row i of sequence b sees key j."""
    i = torch.arange(most_q, device=lens.device)[None, :, None]
    j = torch.arange(most_k, device=lens.device)[None, None]
    at = (lens - nq)[:, None, None] + i
    ok = (j <= at) & (i < nq[:, None, None])
    return ok & (j > at - window) if window else ok


def _attention(s):
    c = s["case"]
    b, hkv, g, d, page = c["b"], c["hkv"], c["g"], c["d"], c["page"]
    lens = s["kv_len"].long()
    most_k = s["block_table"].shape[1] * page
    ids = s["block_table"].long().clamp(min=0)

    def values(pool, scale):                       # [B, Hkv, keys, D] fp32
        x = pool[ids].float() * scale[ids][..., None, None]
        return x.transpose(1, 2).reshape(b, hkv, most_k, d)

    if s["cu"] is None:
        nq, q = torch.ones_like(lens), s["q"][:, None]                            # [B, 1, Hq, D]
        rows = None
    else:
        cu = s["cu"].long()
        nq = cu[1:] - cu[:-1]
        rows = (cu[:-1, None] + torch.arange(s["max_q"], device=cu.device)[None]).clamp(max=s["q"].shape[0] - 1)
        q = s["q"][rows]
    tq = q.shape[1]
    seen = _seen(lens, nq, tq, most_k, c["window"])
    q = q.float().view(b, tq, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, tq * g, d)
    x = torch.matmul(q, values(s["k_pool"], s["k_scale"]).transpose(2, 3)).mul_(d ** -0.5).view(b, hkv, tq, g, most_k)
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hkv, tq * g, most_k), values(s["v_pool"], s["v_scale"])).view(b, hkv, tq, g, d)
    o = torch.where(z > 0, o / z, torch.zeros_like(o))
    o = o.permute(0, 2, 1, 3, 4).reshape(b, tq, hkv * g, d).to(DTYPES[c["dtype"]])
    if rows is None:
        return o[:, 0]
    live = torch.arange(tq, device=lens.device)[None] < nq[:, None]
    out = torch.zeros_like(s["q"])
    at = torch.where(live, cu[:-1, None] + torch.arange(tq, device=cu.device)[None], s["q"].shape[0])
    return torch.cat((out, out[:1])).index_copy_(0, at.flatten(), o.flatten(0, 1))[:-1]


def run(state):
    s, c = state, state["case"]
    if c["op"] == "norm_rope":
        if own:
            from reasoning_model_kv_b200 import tkv_qk_norm_rope
            return tkv_qk_norm_rope(s["q"], s["k"], s["pos"], s["rope"])
        dt = DTYPES[c["dtype"]]
        return (_norm_rope(s["q"], s["qw"], s["pos"], s["inv_freq"], c).to(dt),
                _norm_rope(s["k"], s["kw"], s["pos"], s["inv_freq"], c).to(dt))
    if c["op"] == "append":
        if own:
            q = s["cache"].append(s["k"], s["v"], s["block_table"], s["kv_len"], cu=s["cu"], max_new=s["max_new"],
                                  rope=s["rope"], q=s["q"])
        else:
            q = _append(s)
        return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"], "k_scale": s["k_scale"],
                "v_scale": s["v_scale"]}
    if own:
        return s["cache"].attention(s["q"], s["block_table"], s["kv_len"], c["d"] ** -0.5, cu=s["cu"],
                                    max_q=s["max_q"], window=c["window"])
    return _attention(s)


# ----------------------------------------------------------------------------- work and 64-bit values
def work(case):
    c = case
    hkv, hq, d = c["hkv"], c["hkv"] * c["g"], c["d"]
    if c["op"] == "norm_rope":
        t = c["t"]
        return {"bytes": t * ((hq + hkv) * d * 4 + 4), "flops": t * (hq + hkv) * d * (4 * c["norm"] + 3)}
    lens, new = _shapes(c)
    t = sum(new)
    if c["op"] == "append":
        pages = sum((n - 1) // c["page"] - (n - m) // c["page"] + 1 for n, m in zip(lens, new))
        return {"bytes": t * d * (hq * 4 + hkv * (4 + 2)) + pages * (hkv * 8 + 4),
                "flops": t * d * (hq + 2 * hkv) * (4 * c["norm"] + 6)}
    w = c["window"] or max(lens)
    keys = sum(min(n, w + m - 1) for n, m in zip(lens, new))
    # row i of m sees min(n - m + 1 + i, w) keys
    seen = sum(sum(min(n - m + 1 + i, w) for i in range(m)) for n, m in zip(lens, new))
    return {"bytes": keys * hkv * d * 2 + t * hq * d * 4 + keys // c["page"] * (hkv * 8 + 4),
            "flops": 4.0 * hq * d * seen}


def _exact_norm_rope(x, w, pos, inv_freq, c):
    y = x.to(torch.float64)
    if w is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["d"] + EPS) * w.to(torch.float64)
    if inv_freq is None:
        return y
    r, out = c["rot"], y.clone()
    for i in range(r // 2):
        th = pos.to(torch.float64) * inv_freq[i].to(torch.float64)
        co, si = th.cos()[:, None], th.sin()[:, None]
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
        out[..., a] = y[..., a] * co - y[..., b] * si
        out[..., b] = y[..., b] * co + y[..., a] * si
    return out


def _exact_append(s):
    """The pools as numbers in units of their scales: what was there, rescaled, and the new tokens
    unrounded."""
    c, page = s["case"], s["case"]["page"]
    cu, lens, table = s["cu"].tolist(), s["kv_len"].tolist(), s["block_table"].tolist()
    pos = torch.cat([torch.arange(lens[b] - (cu[b + 1] - cu[b]), lens[b]) for b in range(c["b"])]).to(DEV)
    k = _exact_norm_rope(s["k"], s["kw"], pos, s["inv_freq"], c)
    got = {"q": _exact_norm_rope(s["q"], s["qw"], pos, s["inv_freq"], c)}
    for name, x in (("k", k), ("v", s["v"].to(torch.float64))):
        pool, scale = s[name + "_pool"].float().to(torch.float64), s[name + "_scale"].to(torch.float64)
        for b in range(c["b"]):
            j = lens[b] - (cu[b + 1] - cu[b])
            while j < lens[b]:
                at, lo = table[b][j // page], j % page
                n = min(page - lo, lens[b] - j)
                rows = x[cu[b + 1] - (lens[b] - j):][:n]                              # [n, Hkv, D]
                need = torch.ceil(torch.log2(rows.abs().amax((0, 2)) / QMAX[c["code"]])).clamp(min=SCALE_MIN_EXP)
                new = torch.exp2(need)
                if lo:
                    new = torch.maximum(new, scale[at])
                    pool[at, :, :lo] *= (scale[at] / new)[:, None, None]
                pool[at, :, lo:lo + n] = rows.transpose(0, 1) / new[:, None, None]
                scale[at] = new
                j += n
        got[name + "_pool"], got[name + "_scale"] = pool, scale
    return got


def _exact_attention(s):
    c, page, d = s["case"], s["case"]["page"], s["case"]["d"]
    lens = s["kv_len"].tolist()
    cu = s["cu"].tolist() if s["cu"] is not None else list(range(c["b"] + 1))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b in range(c["b"]):
        n, n0, n1 = lens[b], cu[b], cu[b + 1]
        first = max(0, n - (n1 - n0) - c["window"] + 1) if c["window"] else 0
        p0 = first // page
        ids = s["block_table"][b, p0:(n + page - 1) // page].long()
        at = torch.arange(n - (n1 - n0), n, device=DEV)
        j = torch.arange(p0 * page, n, device=DEV)
        hide = j[None] > at[:, None]
        if c["window"]:
            hide |= j[None] <= at[:, None] - c["window"]
        for h in range(c["hkv"]):
            k, v = (((pool[ids, h].float().to(torch.float64)) * scale[ids, h].to(torch.float64)[:, None, None])
                    .reshape(-1, d)[:n - p0 * page] for pool, scale in
                    ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"])))
            heads = slice(h * c["g"], (h + 1) * c["g"])
            q = s["q"][n0:n1, heads].to(torch.float64).transpose(0, 1)                # [G, rows, D]
            x = (q @ k.T) / math.sqrt(d)
            x[:, hide] = -math.inf
            out[n0:n1, heads] = (torch.softmax(x, -1) @ v).transpose(0, 1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return (_exact_norm_rope(s["q"], s["qw"], s["pos"], s["inv_freq"], case),
                _exact_norm_rope(s["k"], s["kw"], s["pos"], s["inv_freq"], case))
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)
