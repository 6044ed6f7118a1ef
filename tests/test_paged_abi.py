"""Host-side checks of the paged 8-bit cache's C ABI that need no GPU: configurations and
arguments are refused on the host and nothing is launched."""
import ctypes

import pytest
import torch

from reasoning_model_kv_b200 import TkvError, TkvPagedCache, TkvRope, paged, tkv, tkv_qk_norm_rope
from tests import paged_oracle as po

INV = tkv.TKV_ERR_INVALID
GOOD = dict(B=2, Hkv=2, G=4, D=128, page=64, pages=8, max_pages=4, code=1, dtype=0)


def _bytes(**kw):
    return tkv.lib().tkv_paged_workspace_bytes(ctypes.byref(paged.TkvPagedConfig(**{**GOOD, **kw})))


def test_config_rules():
    assert _bytes() > 0
    for kw in (dict(D=64), dict(page=16), dict(page=128), dict(G=1), dict(G=16), dict(code=0), dict(dtype=1), dict(G=7),
               dict(B=65535, Hkv=8), dict(max_pages=1 << 20, page=64)):
        assert _bytes(**kw) > 0, kw
    for kw in (dict(B=0), dict(B=65536), dict(Hkv=0), dict(G=0), dict(G=17), dict(D=96), dict(D=256), dict(page=8),
               dict(page=48), dict(page=256), dict(pages=0), dict(max_pages=0), dict(max_pages=1 << 30), dict(code=2),
               dict(dtype=2), dict(code=-1), dict(Hkv=60000, G=2), dict(pages=1 << 30, Hkv=4)):
        assert _bytes(**kw) == 0, kw
    assert tkv.lib().tkv_paged_workspace_bytes(None) == 0


def _create(**kw):
    L = tkv.lib()
    cfg = paged.TkvPagedConfig(**{**GOOD, **kw})
    n, h = _bytes(**kw), ctypes.c_void_p()
    p = 1 << 24
    assert L.tkv_paged_create(ctypes.byref(cfg), p, p, p, p, p, n, ctypes.byref(h)) == 0
    return h


def test_create_refuses_bad_pointers():
    L, cfg, n, h, p = tkv.lib(), paged.TkvPagedConfig(**GOOD), _bytes(), ctypes.c_void_p(), 1 << 24
    ok = [p, p, p, p, p, n]
    for i, v in ((0, None), (1, None), (2, None), (3, None), (4, None), (0, p + 8), (1, p + 4), (2, p + 2), (3, p + 1),
                 (4, p + 128), (5, n - 1)):
        args = list(ok)
        args[i] = v
        assert L.tkv_paged_create(ctypes.byref(cfg), *args, ctypes.byref(h)) == INV, (i, v)
        assert not h.value
    assert L.tkv_paged_create(ctypes.byref(cfg), *ok, None) == INV
    assert L.tkv_paged_create(None, *ok, ctypes.byref(h)) == INV


KEEP = []


def _rope(**kw):
    args = dict(inv_freq=1 << 24, rot=64, interleaved=0, q_weight=1 << 24, k_weight=1 << 24, eps=1e-6)
    r = paged.TkvRopeArgs(**{**args, **kw})
    KEEP.append(r)
    return ctypes.addressof(r)


BAD_ROPES = [dict(rot=-8), dict(rot=136), dict(rot=4), dict(rot=12), dict(inv_freq=None), dict(inv_freq=(1 << 24) + 2),
             dict(interleaved=2), dict(q_weight=None), dict(k_weight=None), dict(q_weight=(1 << 24) + 1),
             dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))]


def test_append_and_attention_refuse_bad_arguments_without_launching():
    L, h, p = tkv.lib(), _create(), 1 << 24
    row = [p, 6 * 128, 128]
    q = [p, 8 * 128, 128]

    def append(rope=0, k=row, v=row, q=q, qo=q, T=2, table=p, lens=p, cu=0, max_new=1, c=h):
        return L.tkv_paged_append(c, paged._APPEND_ARGS.pack(*k, *v, *q, *qo, table, lens, cu, rope, T, max_new), None)

    def attend(q=q, o=q, T=2, table=p, lens=p, cu=0, max_q=1, window=0, scale=0.1, c=h):
        return L.tkv_paged_attention(c, paged._ATTENTION_ARGS.pack(*q, *o, table, lens, cu, T, max_q, window, scale), None)

    bad_rows = ([0, 768, 128], [p + 4, 768, 128], [p, 770, 128], [p, 768, 126], [p, -768, 128], [p, 768, -4])
    overlap = ([p, 0, 128], [p, 8 * 128, 64], [p, 64, 128])
    common = (dict(T=-1), dict(T=3), dict(table=0), dict(lens=0), dict(table=p + 2), dict(lens=p + 1), dict(cu=p + 2),
              dict(c=None))
    for kw in (*common, dict(max_new=0), dict(max_new=-1), dict(max_new=(1 << 30) + 1), *(dict(k=r) for r in bad_rows),
               *(dict(v=r) for r in bad_rows), *(dict(q=r) for r in bad_rows[1:]), *(dict(qo=r) for r in bad_rows),
               *(dict(qo=r) for r in overlap), dict(q=[0, 0, 0]), *(dict(rope=_rope(**r)) for r in BAD_ROPES)):
        assert append(**kw) == INV, kw
    for kw in (*common, dict(max_q=0), dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf")),
               *(dict(q=r) for r in bad_rows), *(dict(o=r) for r in bad_rows), *(dict(o=r) for r in overlap)):
        assert attend(**kw) == INV, kw
    assert L.tkv_paged_append(h, None, None) == INV and L.tkv_paged_attention(h, None, None) == INV
    assert append(T=0, cu=p) == 0 and attend(T=0, cu=p) == 0           # no rows: no-op
    assert L.tkv_paged_launch_count(h) == 0 and L.tkv_paged_launch_count(None) == 0
    assert L.tkv_paged_reset(None, None) == INV and L.tkv_paged_poll_error(None, None) == INV
    assert L.tkv_paged_destroy(h) == 0 and L.tkv_paged_destroy(None) == 0


def test_norm_rope_refuses_bad_arguments_without_launching():
    L, p = tkv.lib(), 1 << 24

    def call(rope=_rope(), q=(p, 1024, 128), k=(p, 256, 128), pos=p, qo=p, ko=p, qs=(1024, 128), ks=(256, 128), T=4, Hq=8,
             Hkv=2, D=128, dtype=0):
        return L.tkv_qk_norm_rope(paged._NORM_ROPE_ARGS.pack(*q, *k, qo, *qs, ko, *ks, pos, rope, T, Hq, Hkv, D, dtype), None)

    assert L.tkv_qk_norm_rope(None, None) == INV
    for kw in (dict(rope=0), dict(pos=0), dict(pos=p + 2), dict(T=-1), dict(Hq=-1), dict(Hkv=-1), dict(Hq=65536),
               dict(D=96), dict(dtype=2), dict(qo=0), dict(ko=0), dict(qo=p + 4), dict(qs=(64, 128)),
               dict(qs=(1024, 64)), dict(ks=(256, 0)), dict(q=(p, 1022, 128)), dict(k=(p + 2, 256, 128)),
               dict(k=(p, 256, -128)), *(dict(rope=_rope(**r)) for r in BAD_ROPES)):
        assert call(**kw) == INV, kw
    assert call(T=0) == 0 and call(Hq=0, Hkv=0) == 0


def test_binding_refuses_host_tensors_and_unknown_types():
    with pytest.raises(TkvError):
        TkvRope(torch.zeros(4))
    with pytest.raises(TkvError):
        tkv_qk_norm_rope(torch.zeros(1, 1, 64), torch.zeros(1, 1, 64), torch.zeros(1, dtype=torch.int32), TkvRope())
    for kw in (dict(code="e5m2"), dict(dtype=torch.float32), dict(D=80)):
        args = dict(B=1, Hkv=1, G=1, D=64, page=16, pages=2, max_pages=2)
        with pytest.raises(TkvError):
            TkvPagedCache(**{**args, **kw})


def test_oracle_scale_and_codes():
    """The oracle's own pins: scales at the borders, ties, and a hand-computed attention row."""
    assert po.pow2_scale(448.0, "e4m3") == 1.0 and po.pow2_scale(448.0 * (1 + 2 ** -20), "e4m3") == 2.0
    assert po.pow2_scale(127.0, "int8") == 1.0 and po.pow2_scale(63.5, "int8") == 0.5 and po.pow2_scale(0.0, "int8") == 2.0 ** -64
    assert po.to_codes(torch.tensor([0.5, 1.5, -2.5, 200.0], dtype=po.F64), "int8").tolist() == [0, 2, -2, 127]
    assert po.to_codes(torch.tensor([17.0, 19.0, 500.0], dtype=po.F64), "e4m3").tolist() == [16, 20, 448]
    k = torch.zeros((1, 1, 16, 64), dtype=po.F64)
    k[0, 0, 1, 0] = 1.0
    v = torch.arange(16, dtype=po.F64).view(1, 1, 16, 1).expand(1, 1, 16, 64).contiguous()
    one = torch.ones((1, 1))
    q = torch.zeros((1, 1, 64))
    q[0, 0, 0] = 8.0
    out, _ = po.attention(q, k, v, one, one, [[0]], [2], [0, 1], 0.125, 0, 16)
    e = 2.718281828459045
    assert abs(out[0, 0, 0].item() - e / (1 + e)) < 1e-12


def test_more_rows_than_positions_are_refused():
    """T up to 2^30, so that a row's position less a window stays within 32 bits."""
    L, h, p = tkv.lib(), _create(), 1 << 24
    row = [p, 0, 128]
    for T in ((1 << 30) + 1, (1 << 31) - 1):
        assert L.tkv_paged_append(h, paged._APPEND_ARGS.pack(*row, *row, 0, 0, 0, 0, 0, 0, p, p, p, 0, T, 1), None) == INV
        assert L.tkv_paged_attention(h, paged._ATTENTION_ARGS.pack(*row, p, 1024, 128, p, p, p, T, 1, 0, 0.1), None) == INV
    assert L.tkv_paged_launch_count(h) == 0 and L.tkv_paged_destroy(h) == 0


def test_output_rows_that_overlap_across_tokens_and_heads_are_refused():
    """Equal strides make (token 0, head 1) and (token 1, head 0) one row, and so on.  (Outputs with
    heads before tokens, which do not overlap, are in the GPU tests.)"""
    L, p = tkv.lib(), 1 << 24
    h, row = _create(B=4), [p, 768, 128]
    for strides in ((128, 128), (256, 128), (7 * 128, 128), (128, 256), (128, 384), (1 << 40, 1 << 38)):
        out = [p, *strides]
        args = [(L.tkv_paged_attention, h, paged._ATTENTION_ARGS.pack(p, 1024, 128, *out, p, p, 0, 4, 1, 0, 0.1)),
                (L.tkv_paged_append, h, paged._APPEND_ARGS.pack(*row, *row, p, 1024, 128, *out, p, p, 0, 0, 4, 1)),
                (L.tkv_qk_norm_rope, paged._NORM_ROPE_ARGS.pack(p, 1024, 128, *row, *out, *row, p, _rope(), 4, 8, 2, 128, 0)),
                (L.tkv_qk_norm_rope, paged._NORM_ROPE_ARGS.pack(*row, p, 1024, 128, *row, *out, p, _rope(), 4, 2, 8, 128, 0))]
        for fn, *a in args:
            assert fn(*a, None) == INV and "overlap" in tkv.lib().tkv_last_error_string().decode(), strides
    assert L.tkv_paged_launch_count(h) == 0 and L.tkv_paged_destroy(h) == 0


def test_softmax_scales_that_leave_fp32_in_log2_units_are_refused():
    L, h, p = tkv.lib(), _create(), 1 << 24
    for scale in (3e38, -3e38, 2.4e38):
        assert L.tkv_paged_attention(h, paged._ATTENTION_ARGS.pack(p, 1024, 128, p, 1024, 128, p, p, 0, 2, 1, 0, scale), None) == INV
    assert L.tkv_paged_launch_count(h) == 0 and L.tkv_paged_destroy(h) == 0
