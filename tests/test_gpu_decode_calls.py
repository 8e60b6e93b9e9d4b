"""Calls of the single-token operators (include/decode.h) that lie next to a refused
one and are answered: their refused neighbours are in test_abi_decode_overlap.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def w4():
    from w4a4_post_quantized_b200 import w4a4
    return w4a4


def gen(seed):
    return torch.Generator().manual_seed(seed)


def test_append_to_a_cache_without_pages(w4):
    """Keys and values of no page have no addresses: every token is left out and reported."""
    w4.w4a4_clear_device_status()
    none = torch.empty(0, 16, 2, 64, dtype=BF16, device="cuda")
    h = torch.ones(3, 2, 64, dtype=BF16, device="cuda")
    pages, pos = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    w4.w4a4_kv_append(w4.KVCache(none, none.clone()), h, h, pages, pos)
    assert w4.w4a4_get_device_status() == w4.W4A4_DEV_RANGE
    w4.w4a4_clear_device_status()


@pytest.mark.parametrize("D", [64, 128])
def test_append_one_token_in_place_next_to_its_keys_and_values(w4, D):
    """Queries of one token turned where they lie, in a row that goes on with keys and values: the same
    bits as with an output of their own."""
    Hq, H, page = 6, 2, 16
    row = torch.randn(1, Hq + 2 * H, D, generator=gen(D)).to(BF16).cuda()
    table = torch.from_numpy(w4.w4a4_rope_table(8, D)).cuda()
    pages, pos = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.full((1,), 5, dtype=torch.int32, device="cuda")
    got = []
    for in_place in (False, True):
        x = row.clone()
        cache = w4.KVCache(*(torch.zeros(1, page, H, D, dtype=BF16, device="cuda") for _ in range(2)))
        q = w4.w4a4_kv_append(cache, x[:, Hq:Hq + H], x[:, Hq + H:], pages, pos, q=x[:, :Hq], table=table,
                              q_out=x[:, :Hq] if in_place else None)
        got.append((q.clone(), cache.k, cache.v))
        assert torch.equal(x[:, Hq:], row[:, Hq:])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.equal(got[1][2][0, 5], row[0, Hq + H:])
