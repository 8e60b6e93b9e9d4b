"""Checks of include/decode.h that need no GPU: bad arguments are rejected on
the host with the documented status, the group-weight layout is the documented
one, the host rotation table holds the cosines and sines it says."""
import ctypes
import math
import os

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "w4a4_post_quantized_b200", "libw4a4.so")
vp, i32, i64, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t

A = 0x10000  # fake, 16-byte aligned device addresses: never dereferenced on the host
OK, ARG, SHAPE, ALIGN, UNSUPPORTED = range(5)
FP16, PAIRS, GELU_OUT = 0x200, 0x400, 0x10


class GroupT(ctypes.Structure):
    _fields_ = [("N", i32), ("K", i32), ("group", i32), ("flags", u32), ("data", vp)]


class CacheT(ctypes.Structure):
    _fields_ = [("k", vp), ("v", vp), ("n_pages", i64), ("page_size", i32), ("n_heads", i32), ("head_dim", i32),
                ("flags", u32), ("stride_page", i64), ("stride_token", i64), ("stride_head", i64)]


class AppendT(ctypes.Structure):
    _fields_ = [("k", vp), ("v", vp), ("q", vp), ("q_out", vp), ("k_stride", i64), ("v_stride", i64),
                ("q_stride", i64), ("n_tokens", i64), ("pages", vp), ("seq", vp), ("pos", vp), ("table_pos", vp),
                ("table", vp), ("n_seqs", i32), ("max_pages", i32), ("n_q_heads", i32), ("n_table", i32),
                ("rot_dim", i32), ("flags", u32)]


class AttendT(ctypes.Structure):
    _fields_ = [("q", vp), ("out", vp), ("lse", vp), ("workspace", vp), ("pages", vp), ("lens", vp),
                ("q_stride", i64), ("workspace_bytes", sz), ("n_seqs", i32), ("max_pages", i32), ("n_q_heads", i32),
                ("window", i32), ("scale", ctypes.c_float)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from w4a4_post_quantized_b200 import build
        build.build()
    L = ctypes.CDLL(LIB)
    L.w4a4_group_weights_bytes.restype = sz
    L.w4a4_group_weights_bytes.argtypes = [i32, i32, i32]
    L.w4a4_group_bind.argtypes = [vp, sz, i32, i32, i32, u32, ctypes.POINTER(GroupT)]
    L.w4a4_group_quantize.argtypes = [vp, ctypes.POINTER(GroupT), vp]
    L.w4a4_group_pack.argtypes = [vp, vp, ctypes.POINTER(GroupT), vp]
    L.w4a4_group_dequantize.argtypes = [ctypes.POINTER(GroupT), vp, vp]
    L.w4a4_group_gemv.argtypes = [vp, i64, ctypes.POINTER(GroupT), vp, vp, u32, vp]
    L.w4a4_rope_table.argtypes = [i32, i32, ctypes.c_double, vp]
    L.w4a4_kv_append.argtypes = [ctypes.POINTER(CacheT), ctypes.POINTER(AppendT), vp]
    L.w4a4_kv_attend_workspace_bytes.restype = sz
    L.w4a4_kv_attend_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.w4a4_kv_attend.argtypes = [ctypes.POINTER(CacheT), ctypes.POINTER(AttendT), vp]
    return L


def _group(N=256, K=512, group=64, flags=0, data=A):
    return ctypes.byref(GroupT(N, K, group, flags, data))


def test_group_weights_layout(lib):
    bytes_ = lib.w4a4_group_weights_bytes
    for N, K, g in [(256, 512, 64), (1, 32, 32), (17, 160, 32), (1021, 4096, 128), (16, 128, 64)]:
        # per 16 rows and 128 inputs 1024 bytes of codes and 16 rows' steps
        assert bytes_(N, K, g) == -(-N // 16) * -(-K // 128) * (1024 + 16 * (128 // g) * 2)
        out = GroupT()
        assert lib.w4a4_group_bind(A, bytes_(N, K, g), N, K, g, FP16, ctypes.byref(out)) == OK
        assert (out.N, out.K, out.group, out.flags) == (N, K, g, FP16)
        assert out.data == A
        assert lib.w4a4_group_bind(A, bytes_(N, K, g) - 1, N, K, g, 0, ctypes.byref(out)) == SHAPE
    for N, K, g in [(0, 512, 64), (-1, 512, 64), (256, 0, 64), (256, 96, 64), (256, 512, 16), (256, 512, 256),
                    (256, (1 << 20) + 128, 128), (0x7FFFFFFF, 128, 128),
                    ((1 << 24) + 1, 128, 128)]:
        assert bytes_(N, K, g) == 0
    out = GroupT()
    assert lib.w4a4_group_bind(None, 1 << 30, 16, 128, 128, 0, ctypes.byref(out)) == ARG
    assert lib.w4a4_group_bind(A, 1 << 30, 16, 128, 128, 0, None) == ARG
    assert lib.w4a4_group_bind(A + 8, 1 << 30, 16, 128, 128, 0, ctypes.byref(out)) == ALIGN
    assert lib.w4a4_group_bind(A, 1 << 30, 16, 128, 48, 0, ctypes.byref(out)) == UNSUPPORTED
    assert lib.w4a4_group_bind(A, 1 << 30, 16, 128, 128, 1, ctypes.byref(out)) == UNSUPPORTED
    assert lib.w4a4_group_bind(A, 1 << 30, 16, 100, 128, 0, ctypes.byref(out)) == SHAPE


def test_group_argument_checks(lib):
    Q, P, D, G = lib.w4a4_group_quantize, lib.w4a4_group_pack, lib.w4a4_group_dequantize, lib.w4a4_group_gemv
    bad = [(None, ARG), (_group(group=16), UNSUPPORTED), (_group(flags=0x2), UNSUPPORTED), (_group(N=0), SHAPE),
           (_group(K=500), SHAPE), (_group(data=None), ARG), (_group(data=A + 4), ALIGN)]
    for w, want in bad:
        assert Q(A, w, None) == want
        assert P(A, A, w, None) == want
        assert D(w, A, None) == want
        assert G(A, 1, w, None, A, 0, None) == want
    assert Q(None, _group(), None) == ARG and Q(A + 2, _group(), None) == ALIGN
    assert P(None, A, _group(), None) == ARG and P(A, None, _group(), None) == ARG
    assert P(A + 4, A, _group(), None) == ALIGN and P(A, A + 2, _group(), None) == ALIGN
    assert D(_group(), None, None) == ARG and D(_group(), A + 2, None) == ALIGN
    assert G(None, 1, _group(), None, A, 0, None) == ARG and G(A, 1, _group(), None, None, 0, None) == ARG
    assert G(A, 0, _group(), None, A, 0, None) == OK and G(None, 0, _group(), None, None, 0, None) == OK
    assert G(A, 17, _group(), None, A, 0, None) == SHAPE and G(A, -1, _group(), None, A, 0, None) == SHAPE
    assert G(A + 2, 1, _group(), None, A, 0, None) == ALIGN and G(A, 1, _group(), A + 2, A, 0, None) == ALIGN
    assert G(A, 1, _group(), None, A + 2, 0, None) == ALIGN
    assert G(A, 1, _group(), None, A, 0x1, None) == UNSUPPORTED
    assert G(A, 1, _group(flags=FP16), None, A, GELU_OUT, None) == UNSUPPORTED


@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 10000.0), (128, 500000.0)])
def test_rope_table(lib, rot, base):
    n = 200_000  # far positions: an angle in 32 bits would be off by about 1e-2
    t = np.empty((n, rot), np.float32)
    assert lib.w4a4_rope_table(n, rot, base, t.ctypes.data) == OK
    p = np.arange(n, dtype=np.longdouble)[-1000:, None]
    f = np.longdouble(base) ** (-np.arange(0, rot, 2, dtype=np.longdouble) / rot)
    want = np.concatenate([np.cos(p * f), np.sin(p * f)], 1)
    # fp32 rounding of values up to 1, and the angle's own rounding: n * 2^-52
    assert np.max(np.abs(t[-1000:] - want)) <= 2.0 ** -25 + 4 * n * 2.0 ** -53
    assert np.array_equal(t[0], np.r_[np.ones(rot // 2), np.zeros(rot // 2)])


def test_rope_table_argument_checks(lib):
    t = np.empty((4, 64), np.float32)
    R = lib.w4a4_rope_table
    assert R(4, 0, 1e4, t.ctypes.data) == UNSUPPORTED and R(4, 24, 1e4, t.ctypes.data) == UNSUPPORTED
    assert R(4, 144, 1e4, t.ctypes.data) == UNSUPPORTED and R(-1, 64, 1e4, t.ctypes.data) == SHAPE
    assert R(4, 64, 0.0, t.ctypes.data) == ARG and R(4, 64, math.nan, t.ctypes.data) == ARG
    assert R(4, 64, math.inf, t.ctypes.data) == ARG and R(4, 64, 1e4, None) == ARG
    assert R(0, 64, 1e4, None) == OK


def _cache(**kw):
    c = dict(k=A, v=A, n_pages=10, page_size=16, n_heads=4, head_dim=64, flags=0, stride_page=16 * 4 * 64,
             stride_token=4 * 64, stride_head=64)
    c.update(kw)
    return ctypes.byref(CacheT(**c))


BAD_CACHES = [(dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(flags=1), UNSUPPORTED),
              (dict(n_pages=-1), SHAPE), (dict(n_pages=1 << 31), SHAPE), (dict(page_size=0), SHAPE),
              (dict(n_heads=0), SHAPE), (dict(n_heads=1 << 16), SHAPE), (dict(stride_page=-8), SHAPE),
              (dict(stride_token=100), ALIGN), (dict(stride_head=4), ALIGN), (dict(k=None), ARG),
              (dict(v=None), ARG), (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN)]


def test_append_argument_checks(lib):
    def f(cache=None, **kw):
        a = dict(k=A, v=A, q=A, q_out=A + 0x1000, k_stride=256, v_stride=256, q_stride=512, n_tokens=5, pages=A,
                 seq=None, pos=A, table_pos=None, table=A, n_seqs=5, max_pages=3, n_q_heads=8, n_table=100, rot_dim=64,
                 flags=0)
        a.update(kw)
        return lib.w4a4_kv_append(cache if cache is not None else _cache(), ctypes.byref(AppendT(**a)), None)
    assert f(n_tokens=0) == OK and f(n_tokens=0, k=None, v=None, q=None, pos=None) == OK
    assert lib.w4a4_kv_append(None, ctypes.byref(AppendT()), None) == ARG
    assert lib.w4a4_kv_append(_cache(), None, None) == ARG
    for kw, want in BAD_CACHES:
        assert f(_cache(**kw), n_tokens=0) == want, kw
    for kw in (dict(stride_page=0), dict(stride_token=0), dict(stride_head=0)):
        assert f(_cache(**kw)) == SHAPE
    for kw in (dict(n_tokens=-1), dict(n_tokens=1 << 31), dict(n_table=-1), dict(n_q_heads=0), dict(n_seqs=-1), dict(max_pages=-1),
               dict(n_seqs=(1 << 24) + 1, max_pages=1),
               dict(n_seqs=1 << 16, max_pages=1 << 15), dict(k_stride=248), dict(v_stride=0), dict(q_stride=504)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(k=None), dict(v=None), dict(pos=None), dict(q_out=None), dict(table=None), dict(pages=None),
               dict(q_out=A, q_stride=520)):
        assert f(**kw) == ARG, kw
    for kw in (dict(k=A + 2), dict(v=A + 8), dict(q=A + 4), dict(q_out=A + 2), dict(k_stride=260),
               dict(v_stride=257), dict(q_stride=516), dict(table=A + 4), dict(pos=A + 2), dict(seq=A + 1),
               dict(table_pos=A + 3), dict(pages=A + 2)):
        assert f(**kw) == ALIGN, kw
    for kw in (dict(rot_dim=-16), dict(rot_dim=24), dict(rot_dim=80), dict(flags=0x1)):
        assert f(**kw) == UNSUPPORTED, kw


def test_attend_argument_checks(lib):
    need = lib.w4a4_kv_attend_workspace_bytes(5, 8, 4, 64)
    assert need > 0
    for args in [(-1, 8, 4, 64), (5, 0, 4, 64), (5, 8, 0, 64), (5, 9, 4, 64), (5, 8, 4, 80)]:
        assert lib.w4a4_kv_attend_workspace_bytes(*args) == 0

    def f(cache=None, **kw):
        a = dict(q=A, out=A, lse=None, workspace=A, pages=A, lens=A, q_stride=512, workspace_bytes=need, n_seqs=5,
                 max_pages=3, n_q_heads=8, window=0, scale=0.125)
        a.update(kw)
        return lib.w4a4_kv_attend(cache if cache is not None else _cache(), ctypes.byref(AttendT(**a)), None)
    assert f(n_seqs=0) == OK
    assert f(n_seqs=0, q=None, lens=None, out=None, workspace=None, workspace_bytes=0, pages=None) == OK
    assert lib.w4a4_kv_attend(None, ctypes.byref(AttendT()), None) == ARG
    assert lib.w4a4_kv_attend(_cache(), None, None) == ARG
    for kw, want in BAD_CACHES:
        assert f(_cache(**kw), n_seqs=0) == want, kw
    for kw in (dict(n_q_heads=0), dict(n_q_heads=9), dict(n_q_heads=1 << 16), dict(window=-1), dict(n_seqs=-1),
               dict(q_stride=504),
               dict(workspace_bytes=need - 1), dict(cache=_cache(page_size=1 << 29), max_pages=3),
               dict(cache=_cache(page_size=1 << 28), max_pages=4, n_seqs=32), dict(n_seqs=1 << 16, max_pages=1 << 15, workspace_bytes=1 << 40)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(q=None), dict(lens=None), dict(out=None), dict(workspace=None), dict(pages=None),
               dict(scale=math.nan), dict(scale=math.inf)):
        assert f(**kw) == ARG, kw
    for kw in (dict(q=A + 2), dict(q_stride=516), dict(lens=A + 2), dict(out=A + 8), dict(lse=A + 2),
               dict(workspace=A + 4),
               dict(pages=A + 1)):
        assert f(**kw) == ALIGN, kw


def test_outputs_that_overlap_their_inputs_are_refused(lib):
    """Every byte offset of an output around its input that matters, against sets of addresses."""
    G = lib.w4a4_group_gemv
    assert G(A, 2, _group(), None, A, 0, None) == ARG
    assert G(A, 2, _group(), None, A + 2 * 2 * 512 - 16, 0, None) == ARG
    assert G(A, 2, _group(), None, A - 2 * 2 * 256 + 16, 0, None) == ARG

    def append(**kw):
        a = dict(k=A, v=A, q=A, q_out=A, k_stride=256, v_stride=256, n_tokens=3, pages=A, pos=A, n_seqs=5, max_pages=3,
                 n_q_heads=2)
        a.update(kw)
        return lib.w4a4_kv_append(_cache(), ctypes.byref(AppendT(**a)), None)

    def attend(**kw):
        a = dict(q=A, out=A, workspace=A, pages=A, lens=A, workspace_bytes=1 << 40, n_seqs=3, max_pages=3, n_q_heads=4,
                 scale=0.125)
        a.update(kw)
        return lib.w4a4_kv_attend(_cache(), ctypes.byref(AttendT(**a)), None)
    for f, name, width in ((append, "q_out", 2 * 64), (attend, "out", 4 * 64)):
        for stride in (width, width + 8, 5 * width):
            used = {t * stride + i for t in range(3) for i in range(width)}
            for at in range(-3 * width, 3 * stride, 8):
                if used & set(range(at, at + 3 * width)) and (at, stride) != (0, width):
                    assert f(**{"q_stride": stride, name: A + 2 * at}) == ARG, (stride, at)
    assert attend(scale=3e38) == ARG
