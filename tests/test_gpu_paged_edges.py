"""The paged 8-bit cache's calls at the edges of what include/tkv.h allows: lengths that the block
table has no room for, windows without an end, value scales far apart, values and queries that
are not finite, other streams than the current one.  Against 64-bit forms, as in
tests/test_gpu_paged.py."""
import math
import subprocess
import sys

import pytest
import torch

import synth
from reasoning_model_kv_b200 import TkvPagedCache, TkvRope, tkv, tkv_qk_norm_rope
from tests import paged_oracle as po
from tests.conftest import ROOT, gpu_available
from tests.gpu_harness import build_pair

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA device")]

BF16, FP16, F64 = torch.bfloat16, torch.float16, torch.float64


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _cu(n):
    return [0, *torch.tensor(n).cumsum(0).tolist()]


def exact(q, pools, table, lens, nq, scale, window, page):
    """(out, bound before the last rounding) in 64 bits, from the definition: a row sees what its
    mask and the readable pages leave, nothing else touches it, whatever it is.

    Bound.  A weight p_j is rounded to fp16 as P = 2^7 p_j / (the largest so far): by 2^-11 of
    itself or, where P is below fp16's normal numbers, by half a step of 2^-24, at most P:
    min(p_j, 2^-32 of the largest).  The largest is that of the keys that a warp of the kernel for
    few rows has met, none of whose value scales is below 2^-10 of this key's (else the product is
    formed in fp32).  The kernel for many rows takes p_j times the value scale in place of p_j, of
    scales within 2^10: 2^-22 in place of 2^-32.
    A logit is a sum of D products in fp32 with two scales on it, off by (D + 8) 2^-23 of the sum of
    magnitudes (twice the rounding unit, for sums that the matrix instructions truncate) and so is
    p_j, twice: as a summand and in the sum of weights.  2^-15: a scale's logarithm beside the logit
    (up to 128, so 2^-18) and the running sums."""
    kp, vp, ks, vs = (t.cpu() for t in pools)
    T, Hq, D = q.shape
    hkv = kp.shape[1]
    g = Hq // hkv
    floor = 2.0 ** -32 if g * max(nq) <= 32 else 2.0 ** -22
    out, tol = torch.zeros((T, Hq, D), dtype=F64), torch.zeros((T, Hq, D), dtype=F64)
    cu = _cu(nq)
    for b, (n, L) in enumerate(zip(nq, lens)):
        room = min(L, table.shape[1] * page)
        ids = table[b].tolist()
        keys = [j for j in range(room) if 0 <= ids[j // page] < kp.shape[0]]
        j = torch.tensor(keys, dtype=torch.long)
        pg = torch.tensor([ids[i // page] for i in keys], dtype=torch.long)
        for i in range(n):
            at = L - n + i
            see = j <= at
            if window:
                see &= j > at - window
            if not see.any():
                continue
            js, ps = j[see], pg[see]
            for h in range(hkv):
                s = vs[ps, h].to(F64)
                k = kp[ps, h, js % page].float().to(F64) * ks[ps, h].to(F64)[:, None]
                v = vp[ps, h, js % page].float().to(F64) * s[:, None]
                qq = q[cu[b] + i, h * g:(h + 1) * g].to(F64)
                p = torch.softmax(qq @ k.T * scale, -1)
                d = 2 * (qq.abs() @ k.abs().T) * abs(scale) * (D + 8) * 2.0 ** -23
                lost = torch.zeros_like(p)
                for u in s.unique().tolist():
                    most = p[:, s >= u / 1024].amax(-1, keepdim=True)
                    lost[:, s == u] = torch.minimum(p[:, s == u], floor * most)
                o = p @ v
                out[cu[b] + i, h * g:(h + 1) * g] = o
                tol[cu[b] + i, h * g:(h + 1) * g] = ((p * (2.0 ** -11 + 2.0 ** -15 + d) + lost) @ v.abs() +
                                                     (p * d).sum(-1, keepdim=True) * o.abs())
    return out, tol


def check(got, want, tol, dtype):
    """Within the bound and the output's rounding where the formula gives a number, NaN where it
    gives NaN; infinities of the number's sign are right from the type's largest value on."""
    got = got.cpu().to(F64)
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan), (got.isnan().sum().item(), nan.sum().item())
    lim = want.abs() * (torch.finfo(dtype).eps / 2) + tol + torch.finfo(dtype).tiny
    err = (got - want).abs()
    beyond = want.abs() + tol >= torch.finfo(dtype).max * (1 + torch.finfo(dtype).eps / 4)
    err[beyond & got.isinf() & (got.sign() == want.sign())] = 0
    assert (err <= lim)[~nan].all(), ((err - lim)[~nan].max().item(), (err / want.abs())[~nan].max().item())


def _small_pools(gen, pages, hkv, page, d, code):
    kp, ks = po.make_pool(gen, pages, hkv, page, d, code)
    vp, vs = po.make_pool(gen, pages, hkv, page, d, code)
    return tuple(t.cuda() for t in (kp, vp, ks, vs))


# ------------------------------------------------------------------ lengths and windows
@pytest.mark.parametrize("length", [33, 5000, 100000, 10 ** 6, 1 << 30])
@pytest.mark.parametrize("nq", [1, 3, 45])
@pytest.mark.parametrize("window", [0, 1000])
def test_tokens_that_the_table_has_no_room_for_count_as_masked(length, nq, window):
    """A length far beyond a short table's room: the rows are written all the same, over the keys
    that the table has, and the fault is latched."""
    gen = torch.Generator().manual_seed(length + nq)
    page, hkv, g, d, mp = 16, 1, 2, 64, 2
    pools = _small_pools(gen, 5, hkv, page, d, "e4m3")
    table, lens, rows = _i32([[4, 1], [3, 0]]), [length, 30], [nq, min(nq, 30)]
    c = TkvPagedCache(2, hkv, g, d, page, 5, mp, pools=pools)
    q = torch.randn((sum(rows), hkv * g, d), generator=gen).to(BF16)
    out = torch.full_like(q, 9.0).cuda()
    for _ in range(2):
        c.attention(q.cuda(), table.cuda(), _i32(lens).cuda(), d ** -0.5, cu=_i32(_cu(rows)).cuda(), max_q=nq, window=window,
                    out=out)
        assert c.poll_error() == tkv.TKV_ERR_CAPACITY
        check(out, *exact(q, pools, table, lens, rows, d ** -0.5, window, page), BF16)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 30, 1 << 30, (1 << 30) - 1, 7])
@pytest.mark.parametrize("lens,nq", [([2, 3], [5, 1]), ([2, 0], [4, 3]), ([20, 70], [45, 60]), ([3, 200], [90, 33])])
def test_windows_without_an_end_and_rows_at_negative_positions(window, lens, nq):
    gen = torch.Generator().manual_seed(sum(lens))
    page, hkv, g, d, mp = 32, 2, 2, 128, 8
    pools = _small_pools(gen, 16, hkv, page, d, "int8")
    table = torch.randperm(16, generator=gen).to(torch.int32).view(2, mp)
    c = TkvPagedCache(2, hkv, g, d, page, 16, mp, code="int8", dtype=FP16, pools=pools)
    q = torch.randn((sum(nq), hkv * g, d), generator=gen).to(FP16)
    out = torch.full_like(q, 9.0).cuda()
    c.attention(q.cuda(), table.cuda(), _i32(lens).cuda(), d ** -0.5, cu=_i32(_cu(nq)).cuda(), max_q=max(nq), window=window,
                out=out)
    assert c.poll_error() == tkv.TKV_OK
    check(out, *exact(q, pools, table, lens, nq, d ** -0.5, window, page), FP16)


# ------------------------------------------------------------------ value scales far apart
def _scales_apart(gen, kind, r, odd, page, hkv, d, code):
    """Four pages in the sequence's order, of which page `odd` has a value scale 2^r times the
    others'.  Dim 0 of the keys pushes a token down: by 1.02 (d 128) or 1.44 log2 units a code."""
    big = 60 if code == "e4m3" else 24
    to = po.TORCH_CODE[code]
    k = (torch.randn((4, hkv, page, d), generator=gen) * 4).round()
    v = (torch.randn((4, hkv, page, d), generator=gen) * big).clamp(-po.QMAX[code], po.QMAX[code]).round()
    k[..., 0] = 0
    vs = torch.full((4, hkv), 2.0 ** -6)
    vs[odd] *= 2.0 ** r
    if kind == "far":             # nobody attends to that page
        k[odd, :, :, 0] = -96
    elif kind == "holds_all":     # all the attention is on that page
        k[:, :, :, 0] = -96
        k[odd, :, :, 0] = 0
    elif kind == "outlier":       # one token has set the page's scale, the others' values are zeros there
        v[odd] = 0
        v[odd, :, 5] = po.QMAX[code]
        k[odd, :, 5, 0] = -96
    else:                         # little weight, but values so large that they are the output
        k[odd, :, :, 0] = -40
    return k.to(to), v.to(to), torch.full((4, hkv), 2.0 ** -3), vs


@pytest.mark.parametrize("kind,r", [("far", 24), ("far", 28), ("far", 34), ("far", 60), ("far", -40), ("holds_all", -24),
                                    ("holds_all", -28), ("holds_all", -34), ("holds_all", -70), ("holds_all", 70),
                                    ("outlier", 8), ("outlier", 20), ("outlier", 34), ("outlier", 90), ("little", 70),
                                    ("little", 90)])
@pytest.mark.parametrize("odd", [0, 2])
@pytest.mark.parametrize("code,dtype,page,d", [("e4m3", BF16, 16, 128), ("int8", BF16, 64, 128), ("e4m3", BF16, 64, 64)])
@pytest.mark.parametrize("nq,g", [(1, 4), (5, 2), (12, 2), (40, 2), (150, 1)])
def test_value_scales_far_apart(kind, r, odd, code, dtype, page, d, nq, g):
    gen = torch.Generator().manual_seed(abs(r) + odd)
    hkv, L = 2, 4 * page - 3
    k, v, ks, vs = _scales_apart(gen, kind, r, odd, page, hkv, d, code)
    order = torch.tensor([2, 0, 3, 1])
    pools = tuple(torch.empty_like(t.view(torch.uint8) if t.element_size() == 1 else t) for t in (k, v, ks, vs))
    for dst, src in zip(pools, (k, v, ks, vs)):
        dst[order] = src.view(torch.uint8) if src.element_size() == 1 else src
    pools = tuple(p.view(s.dtype).cuda() for p, s in zip(pools, (k, v, ks, vs)))
    table = order.to(torch.int32)[None]
    q = torch.randn((nq, hkv * g, d), generator=gen)
    q[..., 0] = 64
    q = q.to(dtype)
    want, tol = exact(q, pools, table, [L], [nq], d ** -0.5, 0, page)
    # once, every unit of keys in another block; and many times, whole sequences in a block
    for n in (1, 300):
        c = TkvPagedCache(n, hkv, g, d, page, 4, 4, code=code, dtype=dtype, pools=pools)
        cu = torch.arange(n + 1, dtype=torch.int32) * nq
        out = c.attention(q.repeat(n, 1, 1).cuda(), table.repeat(n, 1).cuda(), _i32([L] * n).cuda(), d ** -0.5, cu=cu.cuda(),
                          max_q=nq)
        assert c.poll_error() == tkv.TKV_OK
        for i in {0, 1, n // 2, n - 1}:
            if i < n:
                check(out[i * nq:(i + 1) * nq], want, tol, dtype)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("nq,g", [(1, 4), (5, 2), (12, 2), (40, 2), (150, 1)])
def test_one_huge_value_does_not_reach_the_other_pages(code, nq, g):
    """A sequence appended with one value of 2^34 among values near one: rows of other tokens' values
    keep theirs, at decode and in chunks, over several blocks' parts."""
    gen = torch.Generator().manual_seed(3)
    page, hkv, d, L = 64, 2, 128, 3000
    k, v = (torch.randn((L, hkv, d), generator=gen).to(BF16) for _ in range(2))
    k[1234, :, 0] = -300.0
    v[1234, :, 3] = 2.0 ** 34
    c = TkvPagedCache(1, hkv, g, d, page, 48, 48, code=code)
    table = torch.randperm(48, generator=gen).to(torch.int32)[None]
    c.append(k.cuda(), v.cuda(), table.cuda(), _i32([L]).cuda(), cu=_i32([0, L]).cuda(), max_new=L)
    q = torch.randn((nq, hkv * g, d), generator=gen)
    q[..., 0] = 8.0
    q = q.to(BF16)
    out = c.attention(q.cuda(), table.cuda(), _i32([L]).cuda(), d ** -0.5, cu=_i32([0, nq]).cuda(), max_q=nq)
    pools = (c.k_pool, c.v_pool, c.k_scale, c.v_scale)
    check(out, *exact(q, pools, table, [L], [nq], d ** -0.5, 0, page), BF16)


@pytest.mark.parametrize("page,g,window,d,dtype", [(16, 3, 0, 128, BF16), (64, 4, 70, 64, FP16), (128, 1, 0, 128, FP16)])
def test_scales_apart_in_some_sequences_and_outputs_over_the_queries(page, g, window, d, dtype):
    """Many sequences, a few of which (and of their heads) have pages of far larger scales; the output
    may take the queries' place, and a replayed call gives the same bits."""
    gen = torch.Generator().manual_seed(page)
    B, hkv = 40, 2
    lens = [60 + 37 * i % 700 for i in range(B)]
    nq = [min(n, 40 + 31 * i % 90) for i, n in enumerate(lens)]
    table, pages = po.make_table(gen, lens, page, 760 // page + 1)
    pools = _small_pools(gen, pages, hkv, page, d, "int8")
    for b in range(0, B, 7):
        pools[3][int(table[b, (b // 7) % 2 * (lens[b] - 1) // page]), b % 2] *= 2.0 ** 25
    args = (table.cuda(), _i32(lens).cuda(), d ** -0.5)
    kw = dict(cu=_i32(_cu(nq)).cuda(), max_q=max(nq), window=window)
    c = TkvPagedCache(B, hkv, g, d, page, pages, table.shape[1], code="int8", dtype=dtype, pools=pools)
    q = torch.randn((sum(nq), hkv * g, d), generator=gen).to(dtype)
    out = c.attention(q.cuda(), *args, **kw)
    over, keep = q.cuda(), q.cuda()
    assert c.attention(over, *args, out=over, **kw) is over and torch.equal(over, out)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        c.attention(over, *args, out=over, **kw)
    for _ in range(2):
        over.copy_(keep)
        gr.replay()
        assert torch.equal(over, out)
    assert c.poll_error() == tkv.TKV_OK
    cu = _cu(nq)
    for b in (0, 1, 7, 21, 39):
        want, tol = exact(q[cu[b]:cu[b + 1]], pools, table[b:b + 1], lens[b:b + 1], nq[b:b + 1], d ** -0.5, window, page)
        check(out[cu[b]:cu[b + 1]], want, tol, dtype)


# ------------------------------------------------------------------ what is not finite
@pytest.mark.parametrize("nq", [1, 5, 45])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_queries_that_are_not_finite_over_pages_that_cannot_be_read(nq, page, value):
    """No key that such a row may see can be read: zeros, as for any row that sees none.  The next
    sequence, some of whose pages are missing, keeps its own values."""
    gen = torch.Generator().manual_seed(nq)
    hkv, g, d = 1, 4, 128
    pools = _small_pools(gen, 8, hkv, page, d, "e4m3")
    table = _i32([[-1, -1, -1, -1], [0, -1, 3, 7]])
    lens, rows = [4 * page - 1, 4 * page - 2], [nq, nq]
    q = torch.randn((2 * nq, hkv * g, d), generator=gen).to(BF16)
    q[:nq] = value
    c = TkvPagedCache(2, hkv, g, d, page, 8, 4, pools=pools)
    out = c.attention(q.cuda(), table.cuda(), _i32(lens).cuda(), d ** -0.5, cu=_i32(_cu(rows)).cuda(), max_q=nq)
    assert c.poll_error() == tkv.TKV_ERR_CAPACITY
    assert (out[:nq] == 0).all()
    check(out, *exact(q, pools, table, lens, rows, d ** -0.5, 0, page), BF16)


@pytest.mark.parametrize("nq", [1, 3, 12, 45, 150])
@pytest.mark.parametrize("window", [0, 20, 100])
@pytest.mark.parametrize("page,d", [(16, 128), (64, 64), (64, 128)])
def test_values_that_are_nan_reach_the_rows_that_see_them_only(nq, window, page, d):
    """NaN among the values or the keys of tokens that some rows of a call see and others do not,
    before the rows' first token and behind it, or outside a window."""
    gen = torch.Generator().manual_seed(nq + window)
    hkv, g, lens = 2, 2, [333, 200]
    mp = -(-max(lens) // page)
    pools = _small_pools(gen, 2 * mp, hkv, page, d, "e4m3")
    table = torch.randperm(2 * mp, generator=gen).to(torch.int32).view(2, mp)

    def poison(pool, b, j, h, dims):
        pool.view(torch.uint8)[int(table[b, j // page]), h, j % page, dims] = 0xff

    poison(pools[1], 0, 333 - 2, 0, slice(3, 7))
    poison(pools[1], 0, max(0, 333 - nq // 2 - window), 0, slice(d - 1, d))
    poison(pools[1], 0, 333 - nq // 3 - 20, 1, slice(0, d))
    poison(pools[0], 1, 200 - nq // 2 - 1, 0, slice(5, 6))
    poison(pools[1], 1, 200 - min(nq, 200) + nq // 3, 1, slice(8, 12))
    c = TkvPagedCache(2, hkv, g, d, page, 2 * mp, mp, pools=pools)
    q = torch.randn((2 * nq, hkv * g, d), generator=gen).to(BF16)
    out = c.attention(q.cuda(), table.cuda(), _i32(lens).cuda(), d ** -0.5, cu=_i32([0, nq, 2 * nq]).cuda(), max_q=nq,
                      window=window)
    assert c.poll_error() == tkv.TKV_OK
    check(out, *exact(q, pools, table, lens, [nq, nq], d ** -0.5, window, page), BF16)


# ------------------------------------------------------------------ streams
def _busy(n=40):
    """Some milliseconds of work on the current stream."""
    x = torch.zeros((8192, 8192), dtype=BF16, device="cuda")
    for _ in range(n):
        x = x @ x
    return x


@pytest.mark.parametrize("op", ["attention", "append", "norm_rope"])
def test_outputs_of_another_stream_are_not_the_current_streams_memory(op):
    """While the current stream still works on memory that the program has given back, a call on
    another stream makes its output: the earlier work's late writes must not end up in it."""
    gen = torch.Generator().manual_seed(1)
    c = TkvPagedCache(64, 4, 4, 128, 64, 64, 1, pools=_small_pools(gen, 64, 4, 64, 128, "e4m3"))
    q = torch.randn((64, 16, 128), generator=gen).to(BF16).cuda()
    k = torch.randn((64, 4, 128), generator=gen).to(BF16).cuda()
    table, lens, pos = torch.arange(64, dtype=torch.int32)[:, None].cuda(), _i32([40] * 64).cuda(), _i32(range(64)).cuda()
    rope = TkvRope((10000.0 ** (-torch.arange(0, 128, 2) / 128)).cuda())
    call = {"attention": lambda s: c.attention(q, table, lens, 0.1, stream=s),
            "append": lambda s: c.append(k, k, table, lens, rope=rope, q=q, stream=s),
            "norm_rope": lambda s: tkv_qk_norm_rope(q, k, pos, rope, stream=s)[0]}[op]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        keep = _busy()
        given_back = [torch.empty_like(q) for _ in range(8)]
        for t in given_back:
            t.fill_(9.0)                # runs when the products are done
        del given_back, t
        got = call(side)
        side.synchronize()
        first = got.clone()             # behind the current stream's work
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(first, want)
        del keep, got


@pytest.mark.parametrize("call", ["attention", "sparsity", "step"])
def test_decode_outputs_of_another_stream_are_not_the_current_streams_memory(call):
    """The same of the thought-adaptive cache's calls."""
    w, gpu, _, _ = build_pair("tiny_b1_ctx2k")
    state = gpu.export_state()
    k, v, cls, pos, q = (t.cuda() for t in synth.decode_inputs(w, 0))
    new = [t[:, :, 0].contiguous() for t in (k, v)] + [t[:, 0].contiguous() for t in (cls, pos)]
    run = {"attention": lambda s: [gpu.decode_attention(q, 0.1, stream=s)],
           "sparsity": lambda s: list(gpu.decode_attention_sparsity(q, 0.1, stream=s)),
           "step": lambda s: [gpu.decode_step(*new, q, 0.1, stream=s)]}[call]
    want = run(None)
    side = torch.cuda.Stream()
    for _ in range(3):
        gpu.import_state(state)
        torch.cuda.synchronize()
        keep = _busy()
        given_back = [torch.empty_like(x) for x in want for _ in range(8)]
        for t in given_back:
            t.fill_(9)
        del given_back, t
        got = run(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del keep, got


@pytest.mark.parametrize("shared", [False, True])
def test_a_new_caches_pools_are_ready_for_any_stream(shared):
    """Pools that a cache makes are zeroed when it is there, with a workspace of its own or shared:
    what another stream appends at once stays."""
    page, hkv, d = 16, 2, 64
    first = TkvPagedCache(1, hkv, 1, d, page, 512, 4)
    x = torch.ones((1, hkv, d), dtype=BF16, device="cuda")
    table, lens = _i32([[3, 2, 1, 0]]).cuda(), _i32([1]).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = _busy()
    c = TkvPagedCache(1, hkv, 1, d, page, 512, 4, share=first if shared else None)
    c.append(x, x, table, lens, stream=side)
    torch.cuda.synchronize()
    assert (c.k_pool[3, :, 0].float() * c.k_scale[3][:, None] == 1).all() and (c.v_scale[3] > 0).all()
    del keep


# ------------------------------------------------------------------ bad row offsets
@pytest.mark.parametrize("cu,good", [([0, 4, 2, 2], [0]), ([0, 4, 9, 5, 40, 40], [0, 1]), ([3, 5, -2, -2], [0]),
                                     ([0, 3, 41, 41], [0]), ([0, 0, 6, 1, 1], [1])])
def test_queries_of_usable_sequences_beside_row_offsets_that_are_not(cu, good):
    """Offsets that decrease or leave the rows behind a usable sequence: its rows are encoded and
    appended, the others' are not, and the fault is latched."""
    gen = torch.Generator().manual_seed(len(cu))
    T, B, page, hkv, g, d = 40, len(cu) - 1, 16, 1, 2, 64
    c = TkvPagedCache(B, hkv, g, d, page, 4 * B, 4)
    table = torch.arange(4 * B, dtype=torch.int32).view(B, 4)
    n = [cu[i + 1] - cu[i] if i in good else 0 for i in range(B)]
    lens = [n[i] + 7 if i in good else 50 for i in range(B)]
    k, q = torch.randn((T, hkv, d), generator=gen).to(BF16), torch.randn((T, hkv * g, d), generator=gen).to(BF16)
    out = torch.full_like(q, 9.0).cuda()
    c.append(k.cuda(), k.cuda(), table.cuda(), _i32(lens).cuda(), cu=_i32(cu).cuda(), max_new=8, q=q.cuda(), q_out=out)
    assert c.poll_error() == tkv.TKV_ERR_INVALID
    mine = torch.zeros(T, dtype=torch.bool)
    for b in good:
        mine[cu[b]:cu[b + 1]] = True
        assert (c.k_scale[4 * b] > 0).all()
    assert torch.equal(out.cpu()[mine], q[mine]) and (out.cpu()[~mine] == 9.0).all()


def test_a_cache_that_lives_until_the_interpreter_ends():
    """Its host object is freed without a word, whatever modules are gone by then."""
    code = ("from reasoning_model_kv_b200 import TkvPagedCache, paged; "
            "paged.kept = TkvPagedCache(1, 1, 1, 64, 16, 1, 1); print('made')")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "made" and "__del__" not in r.stderr, r.stderr


@pytest.mark.parametrize("nq,g", [(1, 4), (5, 2), (40, 2), (150, 1)])
@pytest.mark.parametrize("page,zeros", [(16, (32, 80)), (64, (0, 64)), (64, (128, 256))])
def test_pages_of_zero_values_beside_others(nq, g, page, zeros):
    """Values that are zeros for whole pages take the append's least scale; they count in the softmax
    and add nothing."""
    gen = torch.Generator().manual_seed(nq)
    hkv, d, L = 2, 128, 300
    k, v = (torch.randn((L, hkv, d), generator=gen).to(BF16) for _ in range(2))
    v[slice(*zeros)] = 0
    mp = -(-L // page)
    c = TkvPagedCache(1, hkv, g, d, page, mp, mp)
    table = torch.randperm(mp, generator=gen).to(torch.int32)[None]
    c.append(k.cuda(), v.cuda(), table.cuda(), _i32([L]).cuda(), cu=_i32([0, L]).cuda(), max_new=L)
    assert (c.v_scale == 2.0 ** -64).any()
    q = torch.randn((nq, hkv * g, d), generator=gen).to(BF16)
    out = c.attention(q.cuda(), table.cuda(), _i32([L]).cuda(), d ** -0.5, cu=_i32([0, nq]).cuda(), max_q=nq)
    pools = (c.k_pool, c.v_pool, c.k_scale, c.v_scale)
    check(out, *exact(q, pools, table, [L], [nq], d ** -0.5, 0, page), BF16)
