"""Outputs of the single-token operators (include/decode.h) that share memory with
another array of the same call are refused on the host, wherever they begin."""
import ctypes

import pytest

from test_abi_decode import A, ARG, SHAPE, AppendT, AttendT, CacheT, GroupT, lib  # noqa: F401  (lib: the library as a fixture)

FAR = 1 << 40  # addresses of arrays that take no part


def cache(**kw):
    c = dict(k=4 * FAR, v=5 * FAR, n_pages=10, page_size=16, n_heads=2, head_dim=64, flags=0, stride_page=16 * 2 * 64,
             stride_token=2 * 64, stride_head=64)
    c.update(kw)
    return ctypes.byref(CacheT(**c))


@pytest.mark.parametrize("name", ["k", "v"])
def test_append_queries_over_keys_or_values(lib, name):  # noqa: F811
    """Rotated queries would overwrite keys or values that another warp has yet to read."""
    T, Hq, width = 3, 2, 2 * 64  # tokens; elements of a token's keys
    for stride in (width, width + 8, 5 * width):
        used = {t * stride + i for t in range(T) for i in range(width)}
        for at in range(-T * width, T * stride, 8):
            if used & set(range(at, at + T * width)):
                a = dict(k=FAR, v=2 * FAR, q=3 * FAR, k_stride=256, v_stride=256, q_stride=width, n_tokens=T, pages=6 * FAR,
                         pos=7 * FAR, n_seqs=5, max_pages=3, n_q_heads=Hq)
                a.update({name: A + (1 << 20), f"{name}_stride": stride, "q_out": A + (1 << 20) + 2 * at})
                assert lib.w4a4_kv_append(cache(), ctypes.byref(AppendT(**a)), None) == ARG, (stride, at)


def append_to(lib, **kw):  # noqa: F811
    a = dict(k=FAR, v=2 * FAR, k_stride=256, v_stride=256, n_tokens=3, pages=6 * FAR, pos=7 * FAR, n_seqs=5, max_pages=3)
    return lib.w4a4_kv_append(cache(**kw), ctypes.byref(AppendT(**a)), None)


@pytest.mark.parametrize("name", ["stride_page", "stride_token", "stride_head"])
def test_append_to_rows_that_share_memory(lib, name):  # noqa: F811
    """Neighbours less than a head apart: what one token writes, another overwrites in part."""
    for stride in range(0, 64, 8):
        assert append_to(lib, **{name: stride}) == SHAPE, stride


def test_append_to_keys_that_are_the_values(lib):  # noqa: F811
    for at in range(-64 + 8, 64, 8):
        assert append_to(lib, k=4 * FAR, v=4 * FAR + 2 * at) == ARG, at


def around(bytes_out, bytes_in, step=16):
    """Aligned offsets at which an output of some bytes still meets an input of others: its ends and about its start."""
    ends = {s * step + o // step * step for s in range(2) for o in (-bytes_out + step, bytes_in - 2 * step)}
    return sorted({o for o in ends | {0, -step, step} if -bytes_out < o < bytes_in})


def test_group_products_over_what_they_read(lib):  # noqa: F811
    """Results over tokens, bias or weights; results of the conversions over their inputs."""
    N, K, group, M = 256, 512, 64, 3
    packed = lib.w4a4_group_weights_bytes(N, K, group)
    w = ctypes.byref(GroupT(N, K, group, 0, 2 * FAR))
    for at in around(2 * M * N, 2 * M * K):
        assert lib.w4a4_group_gemv(FAR, M, w, None, FAR + at, 0, None) == ARG, at
    for at in around(2 * M * N, 2 * N):
        assert lib.w4a4_group_gemv(FAR, M, w, 3 * FAR, 3 * FAR + at, 0, None) == ARG, at
    for at in around(2 * M * N, packed):
        assert lib.w4a4_group_gemv(FAR, M, w, None, 2 * FAR + at, 0, None) == ARG, at
    for at in around(packed, 2 * N * K):
        assert lib.w4a4_group_quantize(2 * FAR - at, w, None) == ARG, at
    for at in around(packed, N * K // 2):
        assert lib.w4a4_group_pack(2 * FAR - at, FAR, w, None) == ARG, at
    for at in around(packed, 2 * N * (K // group)):
        assert lib.w4a4_group_pack(FAR, 2 * FAR - at, w, None) == ARG, at
    for at in around(2 * N * K, packed):
        assert lib.w4a4_group_dequantize(w, 2 * FAR + at, None) == ARG, at


def test_attend_outputs_over_what_it_reads_and_each_other(lib):  # noqa: F811
    B, Hq, H, D, max_pages = 3, 4, 2, 64, 5
    need = lib.w4a4_kv_attend_workspace_bytes(B, Hq, H, D)
    rows, stride = 2 * B * Hq * D, Hq * D + 8
    size = dict(out=rows, lse=4 * B * Hq, workspace=need, pages=4 * B * max_pages, lens=4 * B,
                q=2 * ((B - 1) * stride + Hq * D))
    place = {n: (6 + i) * FAR for i, n in enumerate(size)}

    def f(**kw):
        a = dict(place, q_stride=stride, workspace_bytes=need + 4096, n_seqs=B, max_pages=max_pages, n_q_heads=Hq, scale=0.125)
        a.update(kw)
        return lib.w4a4_kv_attend(cache(), ctypes.byref(AttendT(**a)), None)

    for written in ("out", "lse", "workspace"):
        for other in size:
            if other == written:
                continue
            for at in around(size[written], size[other]):
                gap = other == "q" and any(t * 2 * stride + 2 * Hq * D <= at and at + size[written] <= (t + 1) * 2 * stride
                                           for t in range(B))
                assert gap or f(**{written: place[other] + at}) == ARG, (written, other, at)


def test_append_queries_over_what_is_looked_up(lib):  # noqa: F811
    """Pages, positions, sequences and the rotation's table are read by every warp of a token, whenever it comes."""
    T, Hq, n_seqs, max_pages, n_table, rot = 8, 2, 6, 2, 5, 16
    size = dict(pages=4 * n_seqs * max_pages, pos=4 * T, seq=4 * T, table_pos=4 * T, table=4 * n_table * rot)
    place = {n: (6 + i) * FAR for i, n in enumerate(size)}
    for name, n in size.items():
        for at in around(2 * T * Hq * 64, n):
            a = dict(place, k=FAR, v=2 * FAR, q=3 * FAR, q_out=place[name] + at, k_stride=256, v_stride=256, q_stride=128, n_tokens=T,
                     n_seqs=n_seqs, max_pages=max_pages, n_q_heads=Hq, n_table=n_table, rot_dim=rot)
            assert lib.w4a4_kv_append(cache(), ctypes.byref(AppendT(**a)), None) == ARG, (name, at)
