"""Sizes at the ends of what include/decode.h accepts, on the host."""
import ctypes

import pytest

from test_abi_decode import A, SHAPE, AttendT, CacheT, lib  # noqa: F401  (lib: the library as a fixture)

MOST_SEQS, MOST_HEADS = 1 << 24, 65535


@pytest.mark.parametrize("n_seqs,heads", [(MOST_SEQS + 1, 4), ((1 << 31) - 1, 4), (1, MOST_HEADS + 1), (1, (1 << 31) - 4),
                                          (MOST_SEQS + 1, MOST_HEADS + 1)])
def test_no_workspace_for_what_attend_refuses(lib, n_seqs, heads):  # noqa: F811
    kv = heads // 4 if heads % 4 == 0 else heads
    assert lib.w4a4_kv_attend_workspace_bytes(n_seqs, heads, kv, 64) == 0
    c = ctypes.byref(CacheT(k=A, v=A, n_pages=1, page_size=16, n_heads=min(kv, MOST_HEADS), head_dim=64, stride_page=1 << 30,
                            stride_token=1 << 24, stride_head=64))
    t = AttendT(q=A, out=A, workspace=A, pages=A, lens=A, q_stride=heads * 64, workspace_bytes=1 << 62, n_seqs=n_seqs,
                max_pages=0, n_q_heads=heads, scale=1.0)
    assert lib.w4a4_kv_attend(c, ctypes.byref(t), None) == SHAPE


def test_workspace_at_the_ends(lib):  # noqa: F811
    f = lib.w4a4_kv_attend_workspace_bytes
    assert f(MOST_SEQS, 4, 4, 64) == f(1, 4, 4, 64) == f(0, 4, 4, 64) > 0
    assert f(1, MOST_HEADS, MOST_HEADS, 128) > 0 and f(1, MOST_HEADS, 1, 128) > 0
