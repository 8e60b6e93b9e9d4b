"""The single-token operators where a lost, doubled or misplaced term cannot hide behind a
tolerance: exact sums at lengths of 10^3 to 10^5, and bounds that follow the kernels' order of
summation (decode_exact.py has both, and how it is known that they see such mistakes)."""
import math

import pytest
import torch

from decode_exact import (BF16, FP16, equal_scores, equal_scores_close, gen, needles, packed_codes, product_bound,
                          product_case, random_scores)

pytestmark = pytest.mark.gpu


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
@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("M", [1, 3, 8, 9, 16])
@pytest.mark.parametrize("N,K,group", [(48, 65536 + 32, 32), (64, 8320, 64), (33, 1024, 128), (2400, 4096, 32), (9600, 2176, 128),
                                       (19000, 1024, 64), (40016, 512, 128)])
def test_products_to_the_bit(w4, M, N, K, group, dt):
    """Up to 16 tiles to a block, in one round or more, and every remainder."""
    X, codes, steps, want = product_case(M, N, K, group, dt, N + M)
    Y = w4.w4a4_group_gemv(X.cuda(), w4.w4a4_group_pack(packed_codes(codes).cuda(), steps.cuda()))
    assert torch.equal(Y.cpu(), want)


@pytest.mark.parametrize("M", [3, 16])
def test_products_to_the_bit_beyond_32_bits(w4, M):
    """More than 2^31 codes; the tokens of one 1 read single weights off everywhere."""
    N, K, group = 70016, 32768, 128
    w = w4.GroupWeights(N, K, group)
    w.storage.random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(5))
    w.storage.view(-1, 1024 + 32)[:, 1024:].view(BF16).fill_(0.0078125)
    X = product_case(M, 1, K, group, BF16, 6)[0].cuda()
    Y, W = w4.w4a4_group_gemv(X, w), w4.w4a4_group_dequantize(w)
    for rows in (slice(0, 64), slice(32752, 32800), slice(N - 64, N)):
        assert torch.equal(Y[:, rows], (X.double() @ W[rows].double().T).to(BF16))


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("M,N,K,group", [(8, 48, 65536 + 32, 32), (16, 48, 65536 + 32, 32), (5, 300, 32768, 128), (16, 2400, 4096, 64),
                                         (8, 9600, 4096, 128), (16, 40016, 1024, 32)])
def test_products_of_random_tokens(w4, M, N, K, group, dt):
    g = gen(N + K)
    codes = torch.randint(-8, 8, (N, K), generator=g)
    steps = (torch.rand(N, K // group, generator=g) * 0.01 + 0.001).to(dt)
    X = torch.randn(M, K, generator=g)
    X[:, :: K // 8] *= 30.0
    X, bias = X.to(dt), torch.randn(N, generator=g).to(dt)
    W = codes.double() * steps.double().repeat_interleave(group, 1)
    want, size = X.double() @ W.T + bias.double(), X.double().abs() @ W.abs().T + bias.double().abs()
    Y = w4.w4a4_group_gemv(X.cuda(), w4.w4a4_group_pack(packed_codes(codes).cuda(), steps.cuda()), bias.cuda())
    h = torch.finfo(dt).eps / 2
    tol = h * want.abs() + (1 + h) * product_bound(size, K, group) + (2.0 ** -25 if dt == FP16 else 0.0)
    assert tol.median() < 0.1 * want.abs().median()
    assert torch.all((Y.double().cpu() - want).abs() <= tol)


@pytest.mark.parametrize("dt", [BF16, FP16])
def test_an_infinite_token_makes_every_result_of_its_row_infinite_or_nan(w4, dt):
    """Each result has the infinity, with the sign of its weight, or NaN where the code is 0; a NaN is in all of them."""
    N, K, group = 1000, 1024, 32
    X, codes, steps, want = product_case(6, N, K, group, dt, 9)
    X[1, 7], X[2, 1000], X[3, 7], X[3, 640], X[4, 100] = math.inf, -math.inf, math.inf, -math.inf, math.nan
    W = codes.double() * steps.double().repeat_interleave(group, 1)
    want = torch.stack([(x.double() * W).sum(1) for x in X])
    Y = w4.w4a4_group_gemv(X.cuda(), w4.w4a4_group_pack(packed_codes(codes).cuda(), steps.cuda())).double().cpu()
    assert (codes[:, [7, 1000, 640]] == 0).any(0).all() and not Y[1:4].isfinite().any() and Y[4].isnan().all()
    assert torch.equal(Y.isnan(), want.isnan())
    assert torch.equal(Y.nan_to_num(0.0, 1e30, -1e30), want.to(dt).double().nan_to_num(0.0, 1e30, -1e30))


# --------------------------------------------------------------- attention
def cache_of(w4, K, V, page, seed, hnd=False):
    """One sequence's keys and values [n, H, D] in shuffled pages; what is left of the last page, and a page more, is NaN."""
    n, H, D = K.shape
    need = -(-n // page)
    order = torch.randperm(need + 1, generator=gen(seed))
    store = []
    for x in (K, V):
        t = torch.full((need + 1, page, H, D), math.nan, dtype=x.dtype)
        rows = torch.full((need * page, H, D), math.nan, dtype=x.dtype)
        rows[:n] = x
        t[order[:need]] = rows.view(need, page, H, D)
        t = t.cuda()
        store.append(t.transpose(1, 2).contiguous().transpose(1, 2) if hnd else t)
    return w4.KVCache(*store), order[:need].int().view(1, -1)


def attend_exact(w4, q, cache, pages, lens, **kw):
    """Out and lse for the table as it is, with room for a longer context, and over a workspace of NaN."""
    B, Hq, D = q.shape
    ws = torch.full((w4.w4a4_kv_attend_workspace_bytes(B, Hq, cache.n_heads, D),), 0xFF, dtype=torch.uint8, device="cuda")
    for more in (0, 4096 // cache.page_size + 300):
        table = torch.nn.functional.pad(pages, (0, more), value=-1).cuda()
        lse = torch.empty(B, Hq, device="cuda")
        yield w4.w4a4_kv_attend(q.cuda(), cache, table, lens.cuda(), lse=lse, workspace=ws, **kw), lse


LONG = [  # tokens, heads, query heads per head, D, page, by head
    (1, 2, 1, 64, 16, False), (16, 4, 3, 128, 16, False), (17, 2, 8, 64, 16, True), (500, 16, 1, 64, 16, False), (1374, 16, 1, 64, 16, False),
    (1374, 2, 9, 128, 24, True), (5003, 8, 4, 128, 7, False), (10_992, 3, 2, 64, 64, True), (87_936, 16, 1, 64, 64, True),
    (100_003, 1, 12, 128, 64, False), (70_001, 2, 17, 64, 16, False), (65_537, 4, 1, 128, 1, False), (200_000, 1, 1, 64, 48, False)]


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("n,H,G,D,page,hnd", LONG)
def test_equal_scores(w4, n, H, G, D, page, hnd, dt):
    """Every token counts once: keys of zero, and the values say which tokens were there."""
    V, want, lse_want = equal_scores(n, H, D, dt)
    cache, pages = cache_of(w4, torch.zeros_like(V), V, page, n, hnd)
    q = torch.randn(1, H * G, D, generator=gen(n)).to(dt)
    for out, lse in attend_exact(w4, q, cache, pages, torch.tensor([n], dtype=torch.int32)):
        assert equal_scores_close(out[0], lse[0], want.repeat_interleave(G, 0), lse_want, dt)


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("n,H,G,D,page,hnd", LONG[3:])
def test_needles_in_long_caches(w4, n, H, G, D, page, hnd, dt):
    """Four tokens hold all the weight, wherever they lie: the others count for nothing, to the bit."""
    for seed in range(3):
        q, K, V, want, _ = needles(n, H, D, dt, seed)
        cache, pages = cache_of(w4, K, V, page, seed, hnd)
        q = q.repeat_interleave(G, 0).unsqueeze(0)
        for out, lse in attend_exact(w4, q, cache, pages, torch.tensor([n], dtype=torch.int32), scale=1.0):
            assert torch.equal(out[0].double().cpu(), want.repeat_interleave(G, 0))
            assert torch.all((lse.double() - (256 + math.log(4))).abs() <= 2.0 ** -14)   # 8 fp32 steps at 256


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("H,G,D,page", [(4, 2, 64, 16), (1, 16, 128, 24), (8, 4, 128, 64), (3, 1, 64, 5)])
def test_batches_where_every_sequence_has_its_own_tokens(w4, H, G, D, page, dt):
    """Sequences of 0 to 9000 tokens, each with one token that holds all the weight, and a window shorter than the
    longest: no part of a sequence reaches another's result."""
    g = gen(H * G + page)
    lens = [0, 1, 15, 16, 9000, 33, 700, 0, 4097, 64, 65, 1374, 2048, 31, 0, 3000, 500, 127, 7, 1000, 0, 2, 128, 6001] * 2
    B = len(lens)
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + 1, generator=g)
    pages, start = torch.full((B, max(need)), -1, dtype=torch.int32), 0
    K = torch.full((len(order) * page, H, D), math.nan, dtype=dt)
    V, window = K.clone(), 2900
    want = torch.zeros(B, H, D, dtype=torch.float64)
    for b, n in enumerate(lens):
        pages[b, :need[b]] = order[start:start + need[b]]
        start += need[b]
        if n == 0:
            continue
        rows = pages[b, torch.arange(n) // page].long() * page + torch.arange(n) % page
        K[rows], V[rows] = 0.0, 1000.0
        first = max(0, n - window)
        at = first + int(torch.randint(0, n - first, (1,), generator=g))
        K[rows[at], :, 0] = 16.0
        K[rows[:first], :, 0] = 32.0               # in front of the window: would win
        V[rows[at]] = torch.randint(-100, 101, (H, D), generator=g).to(dt)
        want[b] = V[rows[at]].double()
    cache = w4.KVCache(K.view(-1, page, H, D).cuda(), V.view(-1, page, H, D).cuda())
    q = torch.zeros(B, H * G, D, dtype=dt)
    q[..., 0] = 16.0
    n = torch.tensor(lens, dtype=torch.int32)
    for out, lse in attend_exact(w4, q, cache, pages, n, scale=1.0, window=window):
        assert torch.equal(out.double().cpu(), want.repeat_interleave(G, 1))
        lse = lse.cpu()
        assert torch.all(lse[n == 0] == -math.inf) and torch.all((lse[n > 0] - 256).abs() <= 2.0 ** -14)


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("B,L,H,G,D", [(1, 100_003, 1, 12, 128), (1, 40_000, 16, 1, 64), (2, 30_000, 1, 8, 128), (3, 9000, 4, 16, 128),
                                       (7, 1374, 4, 4, 64)])
def test_random_scores_over_long_caches(w4, B, L, H, G, D, dt):
    """The pieces are shared evenly by the 4 warps of at least 2 blocks per SM; in the form for little work none has over 12."""
    g = gen(L)
    q = torch.randn(B, H * G, D, generator=g).to(dt)
    K, V = (torch.randn(B, L, H, D, generator=g).to(dt) for _ in range(2))
    page = 32
    need = -(-L // page)
    pool = [torch.nn.functional.pad(x, (0, 0, 0, 0, 0, need * page - L)).view(B * need, page, H, D).cuda() for x in (K, V)]
    pages = torch.arange(B * need, dtype=torch.int32).view(B, need)
    lens = torch.full((B,), L, dtype=torch.int32)
    warps = 2 * 4 * torch.cuda.get_device_properties(0).multi_processor_count
    pieces = max(12, B * H * -(-L // (32 if D == 64 else 16)) // warps + 2)
    want = [random_scores(q[b].view(H, G, D), K[b], V[b], D ** -0.5, pieces) for b in range(B)]
    h = torch.finfo(dt).eps / 2
    for out, lse in attend_exact(w4, q, w4.KVCache(*pool), pages, lens):
        for b, (o, bound, l, l_bound) in enumerate(want):
            tol = h * o.abs() + (1 + h) * bound + (2.0 ** -25 if dt == FP16 else 0.0)
            assert tol.median() < 0.1 * o.abs().median()
            assert torch.all((out[b].double().cpu().view(H, G, D) - o).abs() <= tol)
            assert torch.all((lse[b].double().cpu().view(H, G) - l).abs() <= l_bound)


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("power", [10, 20, 24, 26, 28, 30])
@pytest.mark.parametrize("n,D", [(64, 64), (5000, 128), (40_000, 64)])
def test_weights_far_below_the_largest(w4, n, D, power, dt):
    """Every 16th token has weight 1 and value 0, the others 2^-power 2/3 and value 2^15: all of the result comes from weights
    that are held to 2^-16 of themselves or, in fp16, to 2^-40 of the largest, whichever is more (a step of 2^-24 where
    the largest is 2^15), and that all round the same way."""
    V = torch.full((n, 1, D), 2.0 ** 15, dtype=dt)
    K = torch.zeros(n, 1, D, dtype=dt)
    K[5::16, 0, 0], V[5::16] = 1.0, 0.0
    cache, pages = cache_of(w4, K, V, 64, power)
    q = torch.zeros(1, 1, D, dtype=dt)
    q[..., 0] = float(power)
    exponent = power + math.log2(1.5)
    scale = exponent / power * math.log(2.0)
    tops = len(range(5, n, 16))
    w = 2.0 ** -exponent
    want = (n - tops) * w * 2.0 ** 15 / (tops + (n - tops) * w)
    held = 2.0 ** -16 if dt == BF16 else max(2.0 ** -16, 2.0 ** (exponent - 40))
    # roundings of scale, scale * log2(e), the score and the difference; the power; sums as in random_scores, 12 pieces
    rel = held + 4 * exponent * 2.0 ** -24 + 2.0 ** -21 + (12 * (71 + 11) + 2 * (444 + 128)) * 2.0 ** -23
    h = torch.finfo(dt).eps / 2
    for out, lse in attend_exact(w4, q, cache, pages, torch.tensor([n], dtype=torch.int32), scale=scale):
        assert torch.all((out.double().cpu() / want - 1).abs() <= h + (1 + h) * rel)
        top = exponent * math.log(2.0) + math.log(tops + (n - tops) * w)
        assert abs(float(lse) - top) <= rel - held + 2.0 ** -22 * (17 + 2 * top)
