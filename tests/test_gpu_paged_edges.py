"""The paged 8-bit cache's calls at the edges of what include/tkv.h allows: lengths that the block
table has no room for, windows without an end, value scales far apart, values and queries that
are not finite, other streams than the current one.  Against 64-bit forms, as in
tests/test_gpu_paged.py."""
import math

import pytest
import torch

from reasoning_model_kv_b200 import TkvPagedCache, tkv
from tests import paged_oracle as po
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA device")]

BF16, FP16, F64 = torch.bfloat16, torch.float16, torch.float64


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _cu(n):
    return [0, *torch.tensor(n).cumsum(0).tolist()]


def exact(q, pools, table, lens, nq, scale, window, page, qmax):
    """(out, bound before the last rounding) in 64 bits, from the definition: a row sees what its
    mask and the readable pages leave, nothing else touches it, whatever it is.

    Bound: a weight p_j is rounded to fp16, by 2^-11 of itself or, below fp16's normal numbers,
    by 2^-32 of the row's largest (times 2^7, half a step of 2^-24).  The second kind only meets
    values whose page's scale is at most 2^10 times the smallest one's, so |v| <= qmax 2^10 smin:
    2^-22 qmax smin a token.  A logit is a sum of D products in fp32 with two scales on it, off
    by (D + 8) 2^-23 of the sum of magnitudes (twice the rounding unit, for sums that the matrix
    instructions truncate) and so is p_j, twice: as a summand and in the sum of weights.  2^-15: a
    scale's logarithm beside the logit (up to 128, so 2^-18) and the running sums."""
    kp, vp, ks, vs = (t.cpu() for t in pools)
    T, Hq, D = q.shape
    hkv = kp.shape[1]
    g = Hq // hkv
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
                smin = s[s > 0].min().item() if (s > 0).any() else 0.0
                qq = q[cu[b] + i, h * g:(h + 1) * g].to(F64)
                p = torch.softmax(qq @ k.T * scale, -1)
                d = 2 * (qq.abs() @ k.abs().T) * abs(scale) * (D + 8) * 2.0 ** -23
                o = p @ v
                out[cu[b] + i, h * g:(h + 1) * g] = o
                tol[cu[b] + i, h * g:(h + 1) * g] = ((p * (2.0 ** -11 + 2.0 ** -15 + d)) @ v.abs() +
                                                     (p * d).sum(-1, keepdim=True) * o.abs() +
                                                     len(js) * 2.0 ** -22 * p.amax(-1, keepdim=True) * smin * qmax)
    return out, tol


def check(got, want, tol, dtype):
    """Within the bound and the output's rounding where the formula gives a number, NaN where it
    gives NaN."""
    got = got.cpu().to(F64)
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan), (got.isnan().sum().item(), nan.sum().item())
    lim = want.abs() * (torch.finfo(dtype).eps / 2) + tol + torch.finfo(dtype).tiny
    err = (got - want).abs()
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
        check(out, *exact(q, pools, table, lens, rows, d ** -0.5, window, page, 448.0), BF16)


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
    check(out, *exact(q, pools, table, lens, nq, d ** -0.5, window, page, 127.0), FP16)
