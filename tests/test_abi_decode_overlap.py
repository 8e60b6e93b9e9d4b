"""Outputs of the single-token operators (include/decode.h) that share memory with
another array of the same call are refused on the host, wherever they begin."""
import ctypes

import pytest

from test_abi_decode import A, ARG, SHAPE, AppendT, CacheT, lib  # noqa: F401  (lib: the library as a fixture)

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
