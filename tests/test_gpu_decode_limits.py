"""The single-token operators at the ends of their ranges, and in a row without a pause."""
import math

import pytest
import torch

from decode_exact import BF16, FP16, gen, packed_codes

pytestmark = pytest.mark.gpu
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def w4():
    from w4a4_post_quantized_b200 import w4a4
    return w4a4


@pytest.fixture(autouse=True)
def clean_status(w4):
    w4.w4a4_clear_device_status()
    yield
    torch.cuda.synchronize()
    assert w4.w4a4_get_device_status() == 0


# ---------------------------------------------------------------- products
@pytest.mark.parametrize("M", [1, 16])
def test_the_most_rows(w4, M):
    """2^24 rows: every token reads one input, so a result is one weight."""
    N, K = 1 << 24, 128
    w = w4.GroupWeights(N, K, 128)
    w.storage.random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(1))
    w.storage.view(-1, 1024 + 32)[:, 1024:].view(BF16).fill_(0.5)
    at = [(37 * m) % K for m in range(M)]
    X = torch.zeros(M, K, dtype=BF16, device="cuda")
    X[torch.arange(M), at] = 1.0
    Y, W = w4.w4a4_group_gemv(X, w), w4.w4a4_group_dequantize(w)
    for m in range(M):
        assert torch.equal(Y[m], W[:, at[m]])


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("M", [3, 16])
def test_the_most_inputs(w4, M, dt):
    """2^20 inputs of 17 rows: sums of units below 2^24, to the bit."""
    N, K, group = 17, 1 << 20, 32
    g = gen(M)
    codes, X = torch.randint(-8, 8, (N, K), generator=g), torch.zeros(M, K, dtype=torch.float64)
    X[:, ::8] = torch.randint(-1, 2, (M, K // 8), generator=g).double()    # 2^17 inputs of at most 8
    X[:, -1] = 3.0
    w = w4.w4a4_group_pack(packed_codes(codes).cuda(), torch.full((N, K // group), 0.125, dtype=dt).cuda())
    assert torch.equal(w4.w4a4_group_gemv(X.to(dt).cuda(), w).cpu(), (X @ codes.double().T * 0.125).to(dt))
    W = (codes[:, :4096].repeat(1, K // 4096)).to(dt)
    W[:, 7::32] = 7.0                              # every group's step is 8 / 7 or 1, rounded
    back = w4.w4a4_group_dequantize(w4.w4a4_group_quantize(W.cuda(), group)).cpu()
    assert torch.equal(back[:, :4096].repeat(1, K // 4096), back) and (back.double() - W.double()).abs().max() <= 0.58


# --------------------------------------------------------------- attention
def one_page_each(w4, B, H, D, lens, dt, g, page=16):
    """(cache, pages, keys' places [B], values [B, H, D]): of every sequence's tokens one holds all the weight, with a value of
    its own; those of other tokens are large, rows without a token NaN."""
    K, V = torch.zeros(B, page, H, D, dtype=dt), torch.full((B, page, H, D), 1000.0, dtype=dt)
    at = (torch.rand(B, generator=g) * lens.clamp(min=1)).long()
    b = torch.arange(B)
    own = torch.randint(-100, 101, (B, H, D), generator=g).to(dt)
    K[b, at, :, 0], V[b, at] = 16.0, own
    K[torch.arange(page) >= lens[:, None]] = math.nan
    V[torch.arange(page) >= lens[:, None]] = math.nan
    order = torch.randperm(B, generator=g)
    k, v = torch.empty_like(K), torch.empty_like(V)
    k[order], v[order] = K, V
    return w4.KVCache(k.cuda(), v.cuda()), order.int().view(B, 1), torch.where(lens[:, None, None] > 0, own, 0.0)


@pytest.mark.parametrize("wide", [1, 40])
@pytest.mark.parametrize("B,H,G,D", [(70_000, 1, 1, 64), (3000, 4, 2, 128), (1, 65_535, 1, 64), (2, 4095, 16, 64), (1, 1, 65_535, 128),
                                     (33, 7, 40, 64)])
def test_many_sequences_and_heads(w4, B, H, G, D, wide):
    g = gen(B + H)
    lens = torch.randint(0, 17, (B,), generator=g) if B > 1 else torch.tensor([16])
    cache, pages, want = one_page_each(w4, B, H, D, lens, BF16, g)
    q = torch.zeros(B, H * G, D, dtype=BF16)
    q[..., 0] = 16.0
    lse = torch.empty(B, H * G, device="cuda")
    table = torch.nn.functional.pad(pages, (0, wide - 1), value=-1)
    out = w4.w4a4_kv_attend(q.cuda(), cache, table.cuda(), lens.int().cuda(), scale=1.0, lse=lse)
    assert torch.equal(out.cpu(), want.repeat_interleave(G, 1))
    assert torch.all(lse[lens.cuda() == 0] == -math.inf) and torch.all((lse[lens.cuda() > 0] - 256).abs() <= 2.0 ** -14)


def test_lengths_and_windows_at_the_ends_of_32_bits(w4):
    lens = torch.tensor([16, 3, 16, 0])
    cache, pages, want = one_page_each(w4, 4, 2, 64, lens, FP16, gen(5))
    q = torch.zeros(4, 2, 64, dtype=FP16)
    q[..., 0] = 16.0
    for n, bad in ((lens, False), (torch.tensor([INT_MAX, 3, INT_MAX, -INT_MAX - 1]), True)):
        out = w4.w4a4_kv_attend(q.cuda(), cache, pages.cuda(), n.int().cuda(), scale=1.0, window=INT_MAX)
        assert torch.equal(out.cpu(), want)
        assert w4.w4a4_get_device_status() == (w4.W4A4_DEV_RANGE if bad else 0)
    w4.w4a4_clear_device_status()


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("T,Hq,H,D", [(2, 65_535, 65_535, 64), (300_001, 1, 1, 64), (4000, 3, 2, 128)])
def test_append_many_tokens_and_heads(w4, T, Hq, H, D):
    """Copies (no rotation) are exact; a quarter turn swaps halves."""
    page, g = 16, gen(T)
    need = -(-T // page)
    pages = torch.randperm(need, generator=g).int().view(1, -1).cuda()
    pos = torch.randperm(T, generator=g).int().cuda()
    k, v, q = (torch.randn(T, h, D, generator=g).to(BF16).cuda() for h in (H, H, Hq))
    table = torch.cat([torch.zeros(T, 8), torch.ones(T, 8)], 1).cuda()
    cache = w4.KVCache(*(torch.full((need, page, H, D), 7.0, dtype=BF16, device="cuda") for _ in range(2)))
    r = w4.w4a4_kv_append(cache, k, v, pages, pos, q=q, table=table, seq=torch.zeros(T, dtype=torch.int32, device="cuda"))
    at = pages[0, (pos // page).long()].long(), (pos % page).long()
    turned = lambda x: torch.cat([-x[..., 8:16], x[..., :8], x[..., 16:]], -1)
    assert torch.equal(cache.k[at], turned(k)) and torch.equal(cache.v[at], v) and torch.equal(r, turned(q))
    rest = torch.ones(need, page, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.all(cache.k[rest] == 7.0) and torch.all(cache.v[rest] == 7.0)


def test_append_numbers_at_the_ends_of_32_bits(w4):
    """Positions, sequences, table rows and pages as far out as they go: left out, and reported."""
    far = [INT_MAX, -INT_MAX - 1, INT_MAX - 1, 1 << 30]
    h = torch.ones(4, 2, 64, dtype=BF16, device="cuda")
    cache = w4.KVCache(torch.zeros_like(h).view(1, 4, 2, 64), torch.zeros_like(h).view(1, 4, 2, 64))
    zero, out = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.tensor(far, dtype=torch.int32, device="cuda")
    table = torch.ones(4, 64, device="cuda")
    page = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for kw in (dict(pos=out), dict(seq=out), dict(table_pos=out), dict(pages=out.view(4, 1), seq=torch.arange(4, dtype=torch.int32).cuda())):
        w4.w4a4_kv_append(cache, h, h, **{**dict(pages=page, pos=zero, seq=zero, table=table), **kw})
        assert w4.w4a4_get_device_status() == w4.W4A4_DEV_RANGE
        w4.w4a4_clear_device_status()
    assert not cache.k.any() and not cache.v.any()


# ---------------------------------------------- in a row, over the same memory
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_a_row_of_calls_that_read_what_the_one_in_front_wrote(w4, dt):
    """Products, appends and attentions back and forth over three buffers, so that each call's input was another's output
    just before: the same bits with a wait between any two, eager and replayed."""
    S, H, D, steps = 7, 4, 64, 24
    g = gen(11)
    quant = lambda o, i: w4.w4a4_group_quantize((torch.randn(o, i, generator=g) / math.sqrt(i)).to(dt).cuda(), 64)
    up, down = quant(3 * H * D, H * D), quant(H * D, H * D)
    table = torch.from_numpy(w4.w4a4_rope_table(steps, D)).cuda()
    pages = torch.randperm(S * 2, generator=g).int().view(S, 2).cuda()
    x0 = torch.randn(S, H * D, generator=g).to(dt).cuda()
    ats = [torch.full((S,), t, dtype=torch.int32, device="cuda") for t in range(steps)]
    ws = torch.empty(w4.w4a4_kv_attend_workspace_bytes(S, H, H, D), dtype=torch.uint8, device="cuda")
    cache = w4.KVCache(*(torch.zeros(2 * S, 16, H, D, dtype=dt, device="cuda") for _ in range(2)))
    x, big, o = x0.clone(), torch.empty(S, 3, H, D, dtype=dt, device="cuda"), torch.empty(S, H, D, dtype=dt, device="cuda")

    def run(pause):
        x.copy_(x0)
        for t in range(steps):
            w4.w4a4_group_gemv(x, up, Y=big.view(S, -1))
            pause()
            w4.w4a4_kv_append(cache, big[:, 1], big[:, 2], pages, ats[t], q=big[:, 0], q_out=o, table=table)
            pause()
            w4.w4a4_kv_attend(o, cache, pages, ats[t] + 1, out=o, workspace=ws)
            pause()
            w4.w4a4_group_gemv(o.view(S, -1), down, Y=x)
            pause()
        return x.clone(), cache.k.clone(), cache.v.clone()

    want = run(torch.cuda.synchronize)
    assert all(torch.isfinite(t).all() for t in want) and want[0].abs().max() > 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(lambda: None)
    for i in range(30):
        cache.k.zero_(), cache.v.zero_()
        if i % 2:
            graph.replay()
            got = captured
        else:
            got = run(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_conversions_and_appends_on_other_streams(w4):
    """Calls given a stream run there, one stream's after another's, whatever the current one does."""
    g = gen(3)
    W = torch.randn(500, 1024, generator=g).to(BF16).cuda()
    h = torch.randn(9, 2, 64, generator=g).to(BF16).cuda()
    pages, pos = torch.arange(9, dtype=torch.int32).view(9, 1).cuda(), torch.arange(9, dtype=torch.int32).cuda()
    lens = pos + 1
    want = w4.w4a4_group_dequantize(w4.w4a4_group_quantize(W, 64))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got, caches = [], []
    for i in range(20):
        st = streams[i % 2]
        packed = w4.w4a4_group_quantize(W, 64, stream=st)
        got.append(w4.w4a4_group_dequantize(packed, stream=st))
        with torch.cuda.stream(st):
            caches.append(w4.KVCache(torch.zeros(9, 16, 2, 64, dtype=BF16, device="cuda"), torch.zeros(9, 16, 2, 64, dtype=BF16, device="cuda")))
        q = w4.w4a4_kv_append(caches[-1], h, h, pages, pos, q=h, stream=st)
        got.append(w4.w4a4_kv_attend(q, caches[-1], pages, lens, window=1, stream=st))
        torch.randn(1 << 18, device="cuda")
    torch.cuda.synchronize()
    for a, b in zip(got[0::2], got[1::2]):
        assert torch.equal(a, want) and torch.equal(b, h)
