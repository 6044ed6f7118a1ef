"""The paged 8-bit cache's operators against 64-bit plain forms (tests/paged_oracle.py): norm and
rotation, append, attention, their runs together, and what they do with padding, bad pages,
streams, captured graphs and rows that belong to no sequence."""
import math

import pytest
import torch

from reasoning_model_kv_b200 import (TkvError, TkvPagedCache, TkvRope, tkv, tkv_paged_append, tkv_paged_attention,
                                     tkv_qk_norm_rope)
from tests import paged_oracle as po
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA device")]

BF16, FP16 = torch.bfloat16, torch.float16


def _gen(seed=0):
    return torch.Generator().manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _cu(n, first=0):
    c = [first]
    for x in n:
        c.append(c[-1] + x)
    return c


def _rope(gen, d, rot, dtype, norm, interleaved, eps=1e-6):
    inv = 10000.0 ** (-2.0 * torch.arange(rot // 2).double() / max(rot, 1)) if rot else None
    inv = inv.float() if rot else None
    w = [(1 + 0.2 * torch.randn(d, generator=gen)).to(dtype) for _ in range(2)] if norm else [None, None]
    dev = [None if t is None else t.cuda() for t in (inv, *w)]
    return inv, w, TkvRope(dev[0], interleaved, dev[1], dev[2], eps)


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("d,rot,norm,inter", [(128, 128, True, False), (128, 64, False, True), (128, 8, True, False),
                                              (128, 0, True, False), (64, 64, False, False), (64, 24, True, True),
                                              (64, 40, True, False), (128, 104, True, False), (64, 0, False, False)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,hq,hkv", [(1, 8, 2), (37, 5, 1), (300, 28, 4)])
def test_norm_rope(d, rot, norm, inter, dtype, T, hq, hkv):
    gen = _gen(T + d + rot)
    x = torch.randn((T, hq + 2 * hkv, d), generator=gen).to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=gen, dtype=torch.int32)
    pos[0] = 0
    inv, w, rope = _rope(gen, d, rot, dtype, norm, inter)
    xg = x.cuda()
    q, k = tkv_qk_norm_rope(xg[:, :hq], xg[:, hq:hq + hkv], pos.cuda(), rope)     # views of one projection
    for got, rows, ww in ((q, x[:, :hq], w[0]), (k, x[:, hq:hq + hkv], w[1])):
        want, bound = po.norm_rope(rows, pos, inv, inter, ww)
        assert got.is_contiguous() and po.rounded_ok(got.cpu(), want, bound, dtype)


def test_norm_rope_in_place_layouts_and_empty():
    gen = _gen(3)
    inv, w, rope = _rope(gen, 128, 96, BF16, True, False)
    x = torch.randn((6, 19, 128), generator=gen).to(BF16)       # [heads][tokens][D], seen as [tokens][heads][D]
    pos = torch.arange(19, dtype=torch.int32) * 1000 - 9000     # negative positions turn the other way
    xg = x.cuda()
    q, k = xg[:4].transpose(0, 1), xg[4:].transpose(0, 1)
    q2, k2 = tkv_qk_norm_rope(q, k, pos.cuda(), rope, q_out=q, k_out=k)
    assert q2 is q and k2 is k
    for sl, ww in ((slice(0, 4), w[0]), (slice(4, 6), w[1])):
        want, bound = po.norm_rope(x[sl].transpose(0, 1), pos, inv, False, ww)
        assert po.rounded_ok(xg[sl].transpose(0, 1).cpu(), want, bound, BF16)
    e = tkv_qk_norm_rope(xg[:0, :4], xg[:0, 4:8], _i32([]).cuda(), rope)
    assert e[0].shape == (0, 4, 128)
    # no keys
    q3, k3 = tkv_qk_norm_rope(x.cuda()[:, :5], x.cuda()[:, :0], _i32(range(6)).cuda(), rope)
    want, bound = po.norm_rope(x[:, :5], torch.arange(6), inv, False, w[0])
    assert k3.shape == (6, 0, 128) and po.rounded_ok(q3.cpu(), want, bound, BF16)
    # a zero row stays finite, an infinity stays in its own row
    z = torch.zeros((2, 3, 128), dtype=BF16)
    z[1, 1, 5] = math.inf
    q4, _ = tkv_qk_norm_rope(z.cuda(), z.cuda(), _i32([4, 5]).cuda(), rope)
    assert (q4[0] == 0).all() and (q4[1, 0] == 0).all() and (q4[1, 2] == 0).all()


# ------------------------------------------------------------------ append
def _check_append(code, page, lens, new, d=128, hkv=2, g=2, dtype=BF16, rot=64, norm=True, inter=False, seed=0,
                  with_q=True, first=0, behind=0, mul=1.0):
    gen = _gen(seed)
    B = len(lens)
    max_pages = max(1, max((n + page - 1) // page for n in lens)) + 1
    table, pages = po.make_table(gen, lens, page, max_pages)
    kp, ks = po.make_pool(gen, pages, hkv, page, d, code, -14, -4)
    vp, vs = po.make_pool(gen, pages, hkv, page, d, code, -14, -4)
    cu = _cu(new, first)
    T = cu[-1] + behind
    inv, w, rope = _rope(gen, d, rot, dtype, norm, inter)
    x = (torch.randn((T, hkv * (g + 2), d), generator=gen) * mul).to(dtype)
    q, k, v = x[:, :hkv * g], x[:, hkv * g:hkv * (g + 1)], x[:, hkv * (g + 1):]
    dev = [t.cuda() for t in (kp, vp, ks, vs)]
    c = TkvPagedCache(B, hkv, g, d, page, pages, max_pages, code=code, dtype=dtype, pools=tuple(dev))
    xg = x.cuda()
    one = new == [1] * B and first == 0 and behind == 0
    q_out = torch.full((T, hkv * g, d), 7.0, dtype=dtype, device="cuda") if with_q else None
    got_q = c.append(xg[:, hkv * g:hkv * (g + 1)], xg[:, hkv * (g + 1):], table.cuda(), _i32(lens).cuda(),
                     cu=None if one else _i32(cu).cuda(), max_new=max(1, max(new)), rope=rope,
                     q=xg[:, :hkv * g] if with_q else None, q_out=q_out)
    assert c.poll_error() == tkv.TKV_OK
    enc = lambda r, pos: po.norm_rope(r, pos, inv, inter, w[1])
    ref = po.append(k, v, (kp.to(po.F64), vp.to(po.F64), ks, vs), table, lens, cu, page, code, enc)
    for pool, scale, (val, sc, bound, state), before in zip(dev[:2], dev[2:], ref, (kp, vp)):
        assert torch.equal(scale.cpu().to(po.F64), sc)
        p = pool.cpu()
        new_t, held = state == 1, state == 2
        num = p.to(po.F64)
        err = (num - val).abs()
        tol = po.code_step(val, code) * (1 + 2.0 ** -6) + bound
        assert (err[new_t] <= tol[new_t]).all()
        assert torch.equal(num[held], val[held])
        rest = state == 0
        assert torch.equal(p.view(torch.uint8)[rest], before.view(torch.uint8)[rest])
    if with_q:
        want_pos = torch.zeros(T, dtype=torch.long)
        mine = torch.zeros(T, dtype=torch.bool)
        for b in range(B):
            if lens[b]:
                want_pos[cu[b]:cu[b + 1]] = torch.arange(lens[b] - new[b], lens[b])
                mine[cu[b]:cu[b + 1]] = True
        want, bound = po.norm_rope(q, want_pos, inv, inter, w[0])
        gq = got_q.cpu()
        assert po.rounded_ok(gq[mine], want[mine], bound[mine], dtype)
        assert (gq[~mine] == 7.0).all()
    else:
        assert got_q is None


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("page,d", [(16, 64), (16, 128), (32, 64), (32, 128), (64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens,new", [([1, 17, 64, 200], [1, 1, 1, 1]), ([5, 130, 0, 300, 64], [5, 67, 0, 300, 33]),
                                      ([129, 16], [129, 1])])
def test_append(code, page, d, lens, new):
    _check_append(code, page, lens, new, d=d, seed=page + d)


@pytest.mark.parametrize("kw", [
    dict(dtype=FP16, norm=False, rot=0), dict(dtype=FP16, inter=True, rot=24, hkv=1, g=7), dict(hkv=8, g=1, norm=False),
    dict(hkv=3, g=5), dict(with_q=False), dict(first=3, behind=4), dict(mul=1e-4, norm=False), dict(mul=300.0, norm=False)])
@pytest.mark.parametrize("page", [16, 64])
def test_append_variants(kw, page):
    _check_append("e4m3", page, [70, 3, 100, 0], [20, 3, 41, 0], **kw)


def test_append_padding_and_refused_sequences():
    """kv_len 0 is padding; too few tokens, too many new ones, missing and bad pages skip what
    they touch and are latched, and the other sequences are appended."""
    gen = _gen(9)
    page, hkv, g, d, B, mp = 16, 2, 2, 128, 6, 3
    kp, ks = po.make_pool(gen, 12, hkv, page, d, "e4m3")
    lens = [0, 1, 5, 20, 18, 60]
    new = [1, 2, 1, 4, 3, 1]           # padding; shorter than its rows; fine; too many; bad page; table too short
    table = _i32([[0, -1, -1], [1, -1, -1], [2, -1, -1], [3, 4, -1], [5, 12, -1], [6, 7, 8]])
    cu = _cu(new)
    x = torch.randn((cu[-1], hkv, d), generator=gen).to(BF16).cuda()
    for only, status in (([0, 2], tkv.TKV_OK), ([1], tkv.TKV_ERR_INVALID), ([3], tkv.TKV_ERR_INVALID),
                         ([4], tkv.TKV_ERR_INVALID), ([5], tkv.TKV_ERR_CAPACITY), (range(6), None)):
        dev = [t.cuda() for t in (kp, kp, ks, ks)]
        c = TkvPagedCache(B, hkv, g, d, page, 12, mp, pools=tuple(dev))
        use = [lens[b] if b in only else 0 for b in range(B)]
        qo = torch.full((cu[-1], hkv * g, d), 3.0, dtype=BF16, device="cuda")
        c.append(x, x, table.cuda(), _i32(use).cuda(), cu=_i32(cu).cuda(), max_new=3, q=x.repeat(1, g, 1), q_out=qo)
        st = c.poll_error()
        assert st == status if status is not None else st in (tkv.TKV_ERR_INVALID, tkv.TKV_ERR_CAPACITY)
        assert c.poll_error() == tkv.TKV_OK
        changed = (dev[0].view(torch.uint8).cpu() != kp.view(torch.uint8)).flatten(1).any(1).nonzero().flatten().tolist()
        # of the bad page's sequence, tokens 15, 16 and 17 are new: the first is in page 5
        assert set(changed) == {b for b, i in ((2, 2), (5, 4)) if i in only}
        assert (qo[:1] == 3.0).all() and (qo[1:3] == 3.0).all()
        if 2 in only:
            assert torch.equal(qo[3], x.repeat(1, g, 1)[3])


def test_append_values_that_are_not_finite():
    page, d = 16, 64
    for code in ("e4m3", "int8"):
        c = TkvPagedCache(1, 1, 1, d, page, 1, 1, code=code)
        x = torch.full((3, 1, d), 0.5, dtype=BF16)
        x[0, 0, 0], x[1, 0, 1], x[2, 0, 2] = math.inf, -math.inf, math.nan
        v = torch.full((3, 1, d), math.nan, dtype=BF16)
        c.append(x.cuda(), v.cuda(), _i32([[0]]).cuda(), _i32([3]).cuda(), cu=_i32([0, 3]).cuda(), max_new=3)
        s = c.k_scale.item()
        assert s == po.pow2_scale(0.5, code) and c.v_scale.item() == 2.0 ** -64
        p = c.k_pool.float().cpu()[0, 0]
        assert p[0, 0] == po.QMAX[code] and p[1, 1] == -po.QMAX[code]
        assert (p[2, 2] == 0 if code == "int8" else math.isnan(p[2, 2])) and p[0, 5] == 0.5 / s
        z = c.v_pool.float().cpu()[0, 0, :3]
        assert (z == 0).all() if code == "int8" else z.isnan().all()


# ------------------------------------------------------------------ attention
def _attend(lens, nq, page=16, d=128, hkv=2, g=4, code="e4m3", dtype=BF16, window=0, seed=0, first=0, behind=0,
            break_table=None, q_mul=1.0, scales=(-8, -4), poison=True, max_q=None, calls=1, status=tkv.TKV_OK):
    gen = _gen(seed)
    B = len(lens)
    max_pages = max(1, max((max(0, n) + page - 1) // page for n in lens)) + 1
    table, pages = po.make_table(gen, lens, page, max_pages)
    if break_table:
        for (b, i), to in break_table.items():
            table[b, i] = to
    kp, ks = po.make_pool(gen, pages, hkv, page, d, code, *scales)
    vp, vs = po.make_pool(gen, pages, hkv, page, d, code, *scales)
    if poison:         # what is behind a sequence's last token is never used: NaN codes (int8: large ones)
        for b, n in enumerate(lens):
            if n > 0 and n % page and 0 <= int(table[b, n // page]) < pages:
                for p in (kp, vp):
                    p.view(torch.uint8)[int(table[b, n // page]), :, n % page:] = 0x7f
    cu = _cu(nq, first)
    T = cu[-1] + behind
    q = (torch.randn((T, hkv * g, d), generator=gen) * q_mul).to(dtype)
    want, tol = po.attention(q, kp.to(torch.float32).to(po.F64), vp.to(torch.float32).to(po.F64), ks, vs, table, lens, cu,
                             d ** -0.5, window, page)
    c = TkvPagedCache(B, hkv, g, d, page, pages, max_pages, code=code, dtype=dtype,
                      pools=tuple(t.cuda() for t in (kp, vp, ks, vs)))
    one = nq == [1] * B and first == 0 and behind == 0
    out = torch.full((T, hkv * g, d), 9.0, dtype=dtype, device="cuda")
    for _ in range(calls):
        got = c.attention(q.cuda(), table.cuda(), _i32(lens).cuda(), d ** -0.5, cu=None if one else _i32(cu).cuda(),
                          max_q=max_q or max(1, max(nq)), window=window, out=out)
    assert got is out and c.poll_error() == status
    got = got.cpu()
    mine = ~want.isnan().any(-1)
    assert (got[~mine] == 9.0).all()
    err = (got[mine].to(po.F64) - want[mine]).abs()
    lim = want[mine].abs() * (torch.finfo(dtype).eps / 2) + tol[mine] + torch.finfo(dtype).tiny
    assert (err <= lim).all(), (err - lim).max().item()
    return got


@pytest.mark.parametrize("code,dtype", [("e4m3", BF16), ("int8", FP16)])
@pytest.mark.parametrize("page,d", [(16, 64), (16, 128), (32, 128), (64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("g", [1, 4, 7])
def test_attention_single_tokens(code, dtype, page, d, g):
    _attend([1, 2, 15, 16, 17, 63, 64, 65, 333, 0], [1] * 10, page=page, d=d, g=g, code=code, dtype=dtype)


@pytest.mark.parametrize("code,dtype", [("e4m3", FP16), ("int8", BF16)])
@pytest.mark.parametrize("g", [2, 5, 8, 16])
@pytest.mark.parametrize("window", [0, 1, 50, 1000])
def test_attention_long_single_tokens(code, dtype, g, window):
    _attend([1500, 2049, 7], [1, 1, 1], page=64, g=g, code=code, dtype=dtype, window=window)


@pytest.mark.parametrize("code,dtype,d", [("e4m3", BF16, 128), ("int8", FP16, 64), ("e4m3", FP16, 64), ("int8", BF16, 128)])
@pytest.mark.parametrize("nq", [[2, 1, 3], [5, 6, 0], [9, 17, 4], [33, 40, 7], [150, 64, 1]])
@pytest.mark.parametrize("g,window", [(1, 0), (4, 0), (5, 33), (8, 200), (16, 0)])
def test_attention_several_tokens(code, dtype, d, nq, g, window):
    _attend([200, 300, 97], nq, page=32, d=d, hkv=1, g=g, code=code, dtype=dtype, window=window, seed=g)


@pytest.mark.parametrize("page", [16, 128])
def test_attention_whole_prompts(page):
    _attend([257, 128, 1, 390], [257, 128, 1, 390], page=page, g=2, hkv=2)


@pytest.mark.parametrize("page", [16, 64])
def test_attention_items_of_one_and_two_row_tiles_in_turn(page):
    """A block that goes from an item with few rows (half of a block's softmax warps have none)
    to one with many, over sequences of several units: scales differ from page to page."""
    _attend([1000 + 17 * i for i in range(24)], [90] * 24, page=page, hkv=4, g=4, scales=(-9, -3))


@pytest.mark.parametrize("code,dtype,d", [("e4m3", BF16, 128), ("int8", FP16, 64)])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("window", [1, 17, 100, 333])
def test_attention_windows_that_begin_inside_a_page(code, dtype, d, page, window):
    """Row tiles whose first visible key is anywhere in its page, for single rows and chunks."""
    for nq in ([60, 45, 9], [1, 1, 1], [5, 3, 4]):
        _attend([500, 313, 777], nq, page=page, d=d, hkv=1, g=4, code=code, dtype=dtype, window=window, scales=(-9, -3))


def test_attention_rows_of_no_sequence_and_negative_positions():
    _attend([40, 70], [3, 2], first=2, behind=5)
    _attend([2, 0, 30], [5, 3, 1])                      # rows before a sequence's first token: zeros
    _attend([2, 0, 30], [45, 40, 1], g=8, first=1, behind=1)


def test_attention_bounds_of_max_q_do_not_matter():
    a = _attend([300, 90], [70, 3], max_q=1, g=2)
    b = _attend([300, 90], [70, 3], max_q=500, g=2)
    assert (a.float() - b.float()).abs().max() < 0.05


@pytest.mark.parametrize("nq", [[1, 1, 1], [80, 90, 10]])
def test_attention_bad_pages_count_as_masked(nq):
    _attend([90, 100, 33], nq, break_table={(0, 2): -1}, status=tkv.TKV_ERR_CAPACITY)
    _attend([90, 100, 33], nq, break_table={(1, 0): 10 ** 6, (1, 3): -5}, status=tkv.TKV_ERR_INVALID)
    _attend([90, 100, 16], [min(n, 16) for n in nq], break_table={(2, 0): -1}, status=tkv.TKV_ERR_CAPACITY)


def test_attention_extreme_scales_and_queries():
    _attend([300, 77], [1, 1], scales=(-60, -50), q_mul=1e4)        # logits near zero, tiny values
    _attend([300, 77], [1, 1], scales=(-20, 3))                     # value scales 2^-20 .. 2^2, mixed; sharp logits
    _attend([300, 77], [60, 50], scales=(-20, 3), g=4)
    _attend([300, 77], [1, 1], q_mul=2.0 ** 60, scales=(-70, -64))  # bf16 queries outside fp16's range
    _attend([300, 77], [60, 50], q_mul=2.0 ** 60, scales=(-70, -64))


def test_attention_one_key_takes_all_and_none():
    """A far larger logit (others vanish), and equal logits (zero keys)."""
    page, d, n = 64, 128, 500
    c = TkvPagedCache(1, 1, 1, d, page, 8, 8)
    c.k_scale.fill_(1.0), c.v_scale.fill_(0.5)
    v = torch.randn((8, 1, page, d), generator=_gen(1)).cuda().mul_(50).to(torch.float8_e4m3fn)
    c.v_pool.copy_(v)
    q = torch.ones((1, 1, d), dtype=BF16, device="cuda")
    t = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    out = c.attention(q, t, _i32([n]).cuda(), 1.0)
    want = v.float().double().reshape(-1, d)[:n].mean(0) * 0.5
    assert ((out[0, 0].double() - want).abs() <= want.abs() * 2.0 ** -8 + 50 * 2.0 ** -11).all()
    c.k_pool[3, 0, 7] = torch.full((d,), 448.0, device="cuda").to(torch.float8_e4m3fn)
    out = c.attention(q, t, _i32([n]).cuda(), 1.0)
    want = v[3, 0, 7].float() * 0.5
    assert ((out[0, 0].float() - want).abs() <= want.abs() * 2.0 ** -8).all()


def test_attention_long_sequence_against_blocks():
    """70,000 tokens: the split over the card, joined again, against the 64-bit form."""
    _attend([70000, 3], [1, 1], page=128, hkv=1, g=8, code="int8", poison=True)


# ------------------------------------------------------------------ together
def _step(c, x, table, lens, hkv, g, rope, cu, max_new):
    q = c.append(x[:, hkv * g:hkv * (g + 1)], x[:, hkv * (g + 1):], table, lens, cu=cu, max_new=max_new, rope=rope,
                 q=x[:, :hkv * g])
    return c.attention(q, table, lens, 128 ** -0.5, cu=cu, max_q=max_new)


def test_prompt_then_decode_steps_follow_plain_attention():
    """Prompts appended and attended to, then single tokens: every step's output against the
    64-bit attention over what the pools hold, queries encoded by the plain form."""
    gen = _gen(21)
    hkv, g, d, page, B = 2, 4, 128, 32, 3
    inv, w, rope = _rope(gen, d, 128, BF16, True, False)
    c = TkvPagedCache(B, hkv, g, d, page, 24, 8)
    table = torch.randperm(24, generator=gen).to(torch.int32).view(B, 8)
    lens = [0, 0, 0]
    for new in ([100, 31, 1], [1, 1, 1], [1, 1, 1], [4, 2, 3], [70, 1, 33]):
        lens = [a + n for a, n in zip(lens, new)]
        cu = _cu(new)
        x = torch.randn((cu[-1], hkv * (g + 2), d), generator=gen).to(BF16)
        one = new == [1] * B
        out = _step(c, x.cuda(), table.cuda(), _i32(lens).cuda(), hkv, g, rope, None if one else _i32(cu).cuda(), max(new))
        pos = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)])
        q, _ = po.norm_rope(x[:, :hkv * g], pos, inv, False, w[0])
        want, tol = po.attention(q.to(BF16), c.k_pool.float().cpu().double(), c.v_pool.float().cpu().double(),
                                 c.k_scale.cpu(), c.v_scale.cpu(), table, lens, cu, d ** -0.5, 0, page)
        # the plain form's query may be rounded the other way at a tie: one step of bf16 in a few elements
        lim = want.abs() * 2.0 ** -8 + tol + 2.0 ** -8
        assert ((out.cpu().double() - want).abs() <= lim).all()
    assert c.poll_error() == tkv.TKV_OK
    assert c.launch_count() > 0


def test_encoded_keys_by_either_route_agree():
    """append with rope equals tkv_qk_norm_rope then append without, up to the extra rounding."""
    gen = _gen(5)
    hkv, g, d, page, T = 2, 2, 64, 16, 40
    inv, w, rope = _rope(gen, d, 32, FP16, True, True)
    x = torch.randn((T, hkv * (g + 2), d), generator=gen).to(FP16).cuda()
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    table, lens, cu = _i32([[2, 0, 1]]).cuda(), _i32([T]).cuda(), _i32([0, T]).cuda()
    a, b = (TkvPagedCache(1, hkv, g, d, page, 3, 3, dtype=FP16) for _ in range(2))
    qa = tkv_paged_append(a, k, v, table, lens, cu=cu, max_new=T, rope=rope, q=q)
    qb, kb = tkv_qk_norm_rope(q, k, torch.arange(T, dtype=torch.int32, device="cuda"), rope)
    assert tkv_paged_append(b, kb, v, table, lens, cu=cu, max_new=T) is None
    assert torch.equal(qa, qb) and torch.equal(a.v_pool.view(torch.uint8), b.v_pool.view(torch.uint8))
    oa = tkv_paged_attention(a, qa, table, lens, 0.125, cu=cu, max_q=T)
    ob = tkv_paged_attention(b, qb, table, lens, 0.125, cu=cu, max_q=T)
    assert (oa.float() - ob.float()).abs().max() < 0.25       # codes one E4M3 step apart here and there


def test_results_repeat_bit_for_bit():
    a = _attend([4000, 130, 900], [1, 1, 1], page=64, g=8, calls=1)
    b = _attend([4000, 130, 900], [1, 1, 1], page=64, g=8, calls=3)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    a = _attend([700, 130], [200, 100], page=64, g=4, calls=1)
    b = _attend([700, 130], [200, 100], page=64, g=4, calls=3)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("new", [1, 40])
def test_captured_steps_replay_with_new_lengths(new):
    """A step (append + attention) captured once and replayed with lengths, tables and rows
    changed in place gives what eager calls give; two graphs of one cache replay in turn."""
    gen = _gen(2)
    hkv, g, d, page, B, mp = 2, 4, 128, 16, 2, 40
    inv, w, rope = _rope(gen, d, 128, BF16, True, False)
    eager, graphed = (TkvPagedCache(B, hkv, g, d, page, B * mp, mp) for _ in range(2))
    table = torch.randperm(B * mp, generator=gen).to(torch.int32).view(B, mp).cuda()
    lens, cu = _i32([0, 0]).cuda(), _i32([0, new, 2 * new]).cuda()
    x = torch.zeros((B * new, hkv * (g + 2), d), dtype=BF16, device="cuda")
    s = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        _step(graphed, x, table, lens, hkv, g, rope, cu, new)           # lengths 0: padding, nothing written
    s.synchronize()
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            out = _step(graphed, x, table, lens, hkv, g, rope, cu, new)
        graphs.append((gr, out))
    n = torch.tensor([0, 0], dtype=torch.int32)
    for i in range(6):
        n += new
        x.copy_(torch.randn(x.shape, generator=gen).to(BF16))
        lens.copy_(n)
        gr, out = graphs[i % 2]
        gr.replay()
        want = _step(eager, x, table, lens, hkv, g, rope, cu, new)
        assert torch.equal(out, want)
    assert torch.equal(eager.k_pool.view(torch.uint8), graphed.k_pool.view(torch.uint8))
    assert graphed.poll_error() == tkv.TKV_OK


def test_side_stream_and_two_caches_at_once():
    gen = _gen(8)
    outs, wants = [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        c = TkvPagedCache(2, 2, 4, 128, 64, 40, 20)
        c.k_pool.copy_(torch.randn((40, 2, 64, 128), generator=gen).cuda().mul_(50).to(torch.float8_e4m3fn))
        c.v_pool.copy_(c.k_pool.flip(0))
        c.k_scale.fill_(2.0 ** -6), c.v_scale.fill_(2.0 ** -6)
        q = torch.randn((2, 8, 128), generator=gen).to(BF16).cuda()
        t = torch.randperm(40, generator=gen).to(torch.int32).view(2, 20).cuda()
        n = _i32([1280, 700]).cuda()
        wants.append(c.attention(q, t, n, 0.1))
        torch.cuda.synchronize()
        outs.append((c, q, t, n, s))
    for _ in range(5):
        got = [c.attention(q, t, n, 0.1, stream=s) for c, q, t, n, s in outs]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, wants))


def test_binding_refuses_wrong_tensors():
    c = TkvPagedCache(2, 2, 2, 64, 16, 4, 2)
    k = torch.zeros((2, 2, 64), dtype=BF16, device="cuda")
    q = torch.zeros((2, 4, 64), dtype=BF16, device="cuda")
    t, n = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    cases = [lambda: c.append(k.half(), k, t, n), lambda: c.append(k, k.cpu(), t, n), lambda: c.append(k[:1], k[:1], t, n),
             lambda: c.append(k, k[:1], t, n), lambda: c.append(k, k, t.long(), n), lambda: c.append(k, k, t[:, :1], n),
             lambda: c.append(k, k, t, n, max_new=0), lambda: c.append(k, k, t, n, q=k),
             lambda: c.append(k, k, t, n, q_out=q), lambda: c.append(k, k, t, n, cu=n),
             lambda: c.append(k.transpose(1, 2).contiguous().transpose(1, 2), k, t, n),
             lambda: c.attention(k, t, n, 1.0), lambda: c.attention(q, t, n, math.nan),
             lambda: c.attention(q, t, n, 1.0, window=-1), lambda: c.attention(q, t, n, 1.0, max_q=0),
             lambda: c.attention(q, t, n, 1.0, out=k), lambda: c.attention(q, t, n, 1.0, out=q[:1].expand(2, 4, 64)),
             lambda: c.attention(q.view(-1)[1:1 + 3 * 64].view(1, 3, 64), t, n, 1.0),
             lambda: TkvPagedCache(2, 2, 2, 64, 16, 4, 2, pools=(c.k_pool, c.v_pool, c.k_scale, c.v_scale[:1])),
             lambda: TkvPagedCache(2, 2, 2, 64, 16, 4, 2, code="int8", pools=(c.k_pool, c.v_pool, c.k_scale, c.v_scale)),
             lambda: TkvRope(torch.zeros(4)), lambda: TkvRope(None, False, k[0, 0], None),
             lambda: c.append(k, k, t, n, rope=TkvRope(torch.zeros(33, device="cuda"))),
             lambda: c.append(k, k, t, n, rope=TkvRope(torch.zeros(3, device="cuda"))),
             lambda: c.append(k, k, t, n, rope=TkvRope(None, False, k[0, 0, :32].clone(), k[0, 0, :32].clone())),
             lambda: tkv_qk_norm_rope(q, k, n[:1], TkvRope()), lambda: tkv_qk_norm_rope(q, k.half(), n, TkvRope())]
    for i, f in enumerate(cases):
        with pytest.raises(TkvError):
            f()
            raise AssertionError(i)
    assert c.launch_count() == 0 and c.poll_error() == tkv.TKV_OK


# ------------------------------------------------------------------ the rarer calls
def test_append_one_long_sequence_among_many_short_ones():
    """Far fewer pages than sequences times the longest one's: pages are numbered over the sequences."""
    lens = [1 + (7 * i) % 40 for i in range(300)]
    new = [1] * 300
    lens[211], new[211] = 1000, 700
    lens[17], new[17], lens[255], new[255], lens[256], new[256] = 0, 0, 40, 40, 30, 0
    _check_append("e4m3", 16, lens, new, d=64, hkv=2, g=1)
    _check_append("int8", 128, lens, new, d=128, hkv=3, g=1, with_q=False)


def test_attention_of_many_sequences():
    lens = [1 + (13 * i) % 70 for i in range(300)]
    _attend(lens, [1] * 300, d=64, hkv=2, g=2)
    lens = [3 + (11 * i) % 90 for i in range(600)]
    _attend(lens, [3] * 600, d=64, hkv=1, g=16)


def test_lengths_beyond_the_table_and_bad_rows():
    gen = _gen(4)
    page, hkv, g, d, B = 16, 1, 4, 64, 3
    kp, ks = po.make_pool(gen, 8, hkv, page, d, "int8")
    c = TkvPagedCache(B, hkv, g, d, page, 8, 2, code="int8", pools=(kp.cuda(), kp.cuda(), ks.cuda(), ks.cuda()))
    table = _i32([[0, 1], [2, 3], [4, 5]])
    nums = kp.float().double()
    for nq in ([1, 1, 1], [20, 16, 15]):
        q = torch.randn((sum(nq), g * hkv, d), generator=gen).to(BF16)
        cu = _cu(nq)
        run = lambda lens, cu=cu: c.attention(q.cuda(), table.cuda(), _i32(lens).cuda(), 0.1, cu=_i32(cu).cuda(), max_q=max(nq),
                                              out=torch.full_like(q, 9.0).cuda()).cpu()
        out = run([100, 32, 20])                                  # 100 tokens, room for 32
        assert c.poll_error() == tkv.TKV_ERR_CAPACITY
        want, tol = po.attention(q, nums, nums, ks, ks, table, [100, 32, 20], cu, 0.1, 0, page)
        assert ((out.double() - want).abs() <= want.abs() * 2.0 ** -8 + tol).all()
        out = run([-3, 32, 2 ** 31 - 1])                          # lengths that cannot be: zeros
        assert c.poll_error() == tkv.TKV_ERR_INVALID
        assert (out[:cu[1]] == 0).all() and (out[cu[2]:] == 0).all()
        assert ((out[cu[1]:cu[2]].double() - want[cu[1]:cu[2]]).abs() <= (want.abs() * 2.0 ** -8 + tol)[cu[1]:cu[2]]).all()
        for bad in ([0, -1, cu[2], cu[3]], [0, cu[1], cu[2], cu[3] + 1], [5 * cu[3], cu[1], cu[2], cu[3]]):
            out = run([20, 32, 20], bad)
            assert c.poll_error() == tkv.TKV_ERR_INVALID and not out.isnan().any()
    k = torch.randn((5, hkv, d), generator=gen).to(BF16).cuda()
    before = c.k_pool.clone()
    for lens, cu in (([-1, 0, 0], [0, 1, 1, 1]), ([9, 9, 9], [0, 6, 6, 6]), ([9, 9, 9], [3, 1, 1, 1]), ([2 ** 31 - 1, 0, 0], [0, 1, 1, 1])):
        c.append(k, k, table.cuda(), _i32(lens).cuda(), cu=_i32(cu).cuda(), max_new=5)
        assert c.poll_error() == tkv.TKV_ERR_INVALID and torch.equal(c.k_pool, before)


@pytest.mark.parametrize("nq", [[1, 1], [60, 40]])
@pytest.mark.parametrize("page", [16, 64])
def test_scales_of_zero_and_softmax_scales_of_either_sign(nq, page):
    gen = _gen(6)
    hkv, g, d, lens = 2, 4, 64, [200, 70]
    table, pages = po.make_table(gen, lens, page, 14)
    kp, ks = po.make_pool(gen, pages, hkv, page, d, "e4m3")
    vp, vs = po.make_pool(gen, pages, hkv, page, d, "e4m3")
    ks[int(table[0, 0])] = 0.0                  # keys of zeros in a page, values of zeros in another
    vs[int(table[0, 1])] = 0.0
    vs[int(table[1, 0])] = 0.0
    for all_zero in (False, True):
        if all_zero:
            vs.zero_()
        c = TkvPagedCache(2, hkv, g, d, page, pages, 14, pools=tuple(t.cuda() for t in (kp, vp, ks, vs)))
        q = torch.randn((sum(nq), hkv * g, d), generator=gen).to(BF16)
        cu = _cu(nq)
        for scale in (0.125, -0.125, 0.0):
            out = c.attention(q.cuda(), table.cuda(), _i32(lens).cuda(), scale, cu=_i32(cu).cuda(), max_q=max(nq)).cpu()
            want, tol = po.attention(q, kp.float().double(), vp.float().double(), ks, vs, table, lens, cu, scale, 0, page)
            assert ((out.double() - want).abs() <= want.abs() * 2.0 ** -8 + tol + 1e-38).all()
            assert not all_zero or (out == 0).all()


@pytest.mark.parametrize("nq", [[1, 1], [60, 40]])
def test_output_over_the_queries_and_strided_rows(nq):
    """The output may take the queries' place; rows may lie in a larger array, heads before tokens."""
    gen = _gen(7)
    page, hkv, g, d, lens = 32, 2, 4, 128, [3000, 500]
    table, pages = po.make_table(gen, lens, page, 100)
    kp, ks = po.make_pool(gen, pages, hkv, page, d, "int8")
    c = TkvPagedCache(2, hkv, g, d, page, pages, 100, code="int8", dtype=FP16, pools=tuple(t.cuda() for t in (kp, kp, ks, ks)))
    x = torch.randn((hkv * g, sum(nq), d + 4), generator=gen).to(FP16).cuda()
    q = x[:, :, 4:].transpose(0, 1)
    args = (table.cuda(), _i32(lens).cuda(), 0.08)
    kw = dict(cu=_i32(_cu(nq)).cuda(), max_q=max(nq))
    want = c.attention(q.contiguous(), *args, **kw)
    assert torch.equal(c.attention(q, *args, **kw), want)
    assert c.attention(q, *args, out=q, **kw) is q and torch.equal(q, want)
    assert c.poll_error() == tkv.TKV_OK


def test_layers_share_a_workspace():
    gen = _gen(12)
    page, hkv, g, d, B = 64, 2, 8, 128, 2
    a = TkvPagedCache(B, hkv, g, d, page, 40, 20)
    b = TkvPagedCache(B, hkv, g, d, page, 40, 20, code="int8", share=a)
    small = TkvPagedCache(1, 1, 1, 64, 16, 1, 1)
    assert b.workspace is a.workspace
    with pytest.raises(TkvError):
        TkvPagedCache(B, hkv, g, d, page, 40, 20, share=small)
    alone = TkvPagedCache(B, hkv, g, d, page, 40, 20, code="int8", pools=(b.k_pool, b.v_pool, b.k_scale, b.v_scale))
    table = torch.randperm(40, generator=gen).to(torch.int32).view(B, 20).cuda()
    lens, cu = _i32([1280, 900]).cuda(), _i32([0, 1280, 2180]).cuda()
    x = torch.randn((2180, hkv, d), generator=gen).to(BF16).cuda()
    for c in (a, b):
        c.append(x, x, table, lens, cu=cu, max_new=1280)
    for _ in range(3):
        for rows in (2, 100):
            q = torch.randn((rows, hkv * g, d), generator=gen).to(BF16).cuda()
            kw = dict(cu=_i32([0, rows // 2, rows]).cuda(), max_q=rows // 2)
            oa, ob = a.attention(q, table, lens, 0.1, **kw), b.attention(q, table, lens, 0.1, **kw)
            assert torch.equal(ob, alone.attention(q, table, lens, 0.1, **kw))
            # the same keys and values, in other codes: E4M3 is off by 2^-4 of a value at most
            assert (oa.float() - ob.float()).abs().max() < 0.5
    assert a.poll_error() == tkv.TKV_OK


def test_arguments_that_no_struct_holds():
    c = TkvPagedCache(1, 1, 1, 64, 16, 1, 1)
    q = torch.zeros((1, 1, 64), dtype=BF16, device="cuda")
    t, n = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for kw in (dict(window=1 << 40), dict(max_q=2.5), dict(window=None)):
        with pytest.raises(TkvError):
            c.attention(q, t, n, 0.1, **kw)
    with pytest.raises(TkvError):
        c.attention(q, t, n, "no")
    with pytest.raises(TkvError):
        c.append(q, q, t, n, max_new=1 << 33)
    assert c.launch_count() == 0


@pytest.mark.parametrize("rows", [1, 50])
def test_queries_that_see_nothing_and_calls_without_rows(rows):
    """NaN queries of padded sequences give zeros and reach nobody else; rows of no sequence at all
    are a call that writes nothing, also as the first one in a captured graph."""
    gen = _gen(14)
    page, hkv, g, d = 64, 1, 8, 128
    c = TkvPagedCache(3, hkv, g, d, page, 4, 4)
    c.k_pool.copy_(torch.randn(c.k_pool.shape, generator=gen).cuda().mul_(50).to(torch.float8_e4m3fn))
    c.v_pool.copy_(c.k_pool.flip(0))
    c.k_scale.fill_(2.0 ** -6), c.v_scale.fill_(2.0 ** -6)
    table = _i32([[0, 1, 2, 3]] * 3).cuda()
    q = torch.randn((3 * rows, hkv * g, d), generator=gen).to(BF16).cuda()
    want = c.attention(q, table, _i32([0, 200, 0]).cuda(), 0.1, cu=_i32([0, rows, 2 * rows, 3 * rows]).cuda(), max_q=rows)
    q[:rows] = math.nan
    q[2 * rows:] = math.inf
    got = c.attention(q, table, _i32([0, 200, 0]).cuda(), 0.1, cu=_i32([0, rows, 2 * rows, 3 * rows]).cuda(), max_q=rows)
    assert torch.equal(got, want) and (got[:rows] == 0).all() and (got[2 * rows:] == 0).all()
    fresh = TkvPagedCache(3, hkv, g, d, page, 4, 4, code="int8", dtype=FP16)
    out = torch.full((3 * rows, hkv * g, d), 5.0, dtype=FP16, device="cuda")
    cu, lens, qh = _i32([0, 0, 0, 0]).cuda(), _i32([9, 9, 9]).cuda(), q.half()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        fresh.attention(qh, table, lens, 0.1, cu=cu, max_q=rows, out=out)
        fresh.append(qh[:, :1], qh[:, :1], table, lens, cu=cu, max_new=rows)
    gr.replay()
    gr.replay()
    assert (out == 5.0).all() and (fresh.k_pool == 0).all() and fresh.poll_error() == tkv.TKV_OK
