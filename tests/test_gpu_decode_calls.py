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


class Arena:
    """Arrays that follow one another in one allocation without a gap, each aligned to 16 bytes."""

    def __init__(self, nbytes):
        self.store, self.at = torch.full((nbytes,), 0x7F, dtype=torch.uint8, device="cuda"), 0

    def __call__(self, t):
        n = t.numel() * t.element_size()
        assert n % 16 == 0
        out = self.store[self.at:self.at + n].view(t.dtype).view(t.shape)
        self.at += n
        return out.copy_(t)


def test_arrays_that_touch(w4):
    """Everything a call reads and writes side by side in one allocation: answered as with arrays of their own."""
    g = gen(8)
    M, N, K, S, Hq, H, D, page = 4, 256, 512, 4, 4, 2, 64, 16
    X, W, bias = (torch.randn(*s, generator=g).to(BF16) for s in ((M, K), (N, K), (N,)))
    a = Arena(1 << 26)
    x = a(X)
    w = w4.GroupWeights(N, K, 64)
    w.storage = a(w.storage)
    w.struct.data = w.storage.data_ptr()
    wd = a(W)
    assert w4.w4a4_group_quantize(wd, 64, out=w) is w
    y, b, back = a(torch.zeros(M, N, dtype=BF16)), a(bias), a(torch.zeros(N, K, dtype=BF16))
    w4.w4a4_group_gemv(x, w, b, Y=y)
    w4.w4a4_group_dequantize(w, back)
    own = w4.w4a4_group_quantize(W.cuda(), 64)
    assert torch.equal(w.storage, own.storage) and torch.equal(back, w4.w4a4_group_dequantize(own))
    assert torch.equal(y, w4.w4a4_group_gemv(X.cuda(), own, bias.cuda())) and torch.equal(wd.cpu(), W)

    k, v, q = (torch.randn(S, h, D, generator=g).to(BF16) for h in (H, H, Hq))
    pages, pos = torch.randperm(S, generator=g).int().view(S, 1), torch.tensor([0, 5, 15, 7], dtype=torch.int32)
    got = []
    for place in (lambda t: t.cuda(), a):
        zero = torch.zeros(S, page, H, D, dtype=BF16)
        kd = place(k)
        qo = place(torch.zeros(S, Hq, D, dtype=BF16))
        vd, K_, qd, V_, pg, ps = place(v), place(zero), place(q), place(zero), place(pages), place(pos)
        table = place(torch.from_numpy(w4.w4a4_rope_table(16, D)))
        cache = w4.KVCache(K_, V_)
        w4.w4a4_kv_append(cache, kd, vd, pg, ps, q=qd, q_out=qo, table=table)
        ws = place(torch.zeros(w4.w4a4_kv_attend_workspace_bytes(S, Hq, H, D), dtype=torch.uint8))
        out, n = place(torch.zeros(S, Hq, D, dtype=BF16)), place(pos + 1)
        lse = place(torch.zeros(S, Hq))
        w4.w4a4_kv_attend(qo, cache, pg, n, out=out, lse=lse, workspace=ws)
        got.append((K_, V_, qo, out, lse))
    assert all(torch.equal(s, t) for s, t in zip(*got)) and got[0][3].any()
    assert w4.w4a4_get_device_status() == 0
