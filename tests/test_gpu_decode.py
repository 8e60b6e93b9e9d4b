"""The single-token operators (include/decode.h) against plain implementations
in 64 bits.

Tolerances.  h = eps / 2 of the 16-bit type is half a rounding step relative to
the value (2^-8 for bf16, 2^-11 for fp16); an fp16 result below its normal range
is off by at most 2^-25 instead.  An fp32 sum of n terms t_i is off by at most n
2^-23 sum |t_i| whatever its order (2^-23: tensor cores may truncate instead of
rounding).
"""
import math
import subprocess
import sys
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
TINY = {BF16: 0.0, FP16: 2.0 ** -25}
RANGE = 0x2


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


def half_step(dt):
    return torch.finfo(dt).eps / 2


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(got, want, bound, dt):
    """got (16-bit) within one rounding of a value that is within `bound` of want."""
    h = half_step(dt)
    err = (got.double().cpu() - want).abs()
    tol = h * want.abs() + (1 + h) * bound + TINY[dt]
    assert torch.all(err <= tol), f"worst {(err / tol).nan_to_num(math.inf).max():.3g} of the tolerance"


# ------------------------------------------------------------ group weights
def oracle_quantize(W, group):
    """(codes [N, K] int64, steps [N, K/group] in W's type) from the definition, in 64 bits."""
    N, K = W.shape
    w = W.double().view(N, K // group, group)
    steps = (w.abs().amax(2) / 7.0).to(W.dtype)
    d = steps.double()[:, :, None]
    c = torch.where(d > 0, torch.round(w / torch.where(d > 0, d, 1.0)), 0.0).clamp(-8, 7)
    return c.view(N, K).long(), steps


def weights(N, K, group, dt, seed):
    W = torch.randn(N, K, generator=gen(seed)) * 0.02
    W[0, :group] = 0.0                     # a group without a step
    W[-1, -group:] = 0.0
    W[N // 2, 0] = 3.0                     # an outlier: the other codes of its group are 0
    if dt == FP16:
        W[:, :group] *= 2.0 ** -12         # steps below the normal range
    return W.to(dt)


def dense(codes, steps, group):
    return codes.double() * steps.double().repeat_interleave(group, 1)


SHAPES = [(1, 32, 32), (16, 128, 128), (17, 160, 32), (5, 192, 64), (33, 1024, 128), (259, 96, 32), (1021, 4096, 64),
          (64, 8320, 64)]


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("N,K,group", SHAPES)
def test_quantize_and_back(w4, N, K, group, dt):
    W = weights(N, K, group, dt, N + K)
    codes, steps = oracle_quantize(W, group)
    w = w4.w4a4_group_quantize(W.cuda(), group)
    assert torch.equal(w4.w4a4_group_dequantize(w).cpu(), dense(codes, steps, group).to(dt))


@pytest.mark.parametrize("dt,power", [(BF16, -120), (BF16, -128), (BF16, -131), (FP16, -22), (FP16, 10), (BF16, 100)])
def test_quantize_at_the_ends_of_the_range(w4, dt, power):
    """Steps below the normal range, whose own rounding sends codes to the clamp,
    and whose reciprocal would overflow; and large ones."""
    W = (torch.randn(48, 256, generator=gen(7)) * 2.0 ** power).to(dt)
    codes, steps = oracle_quantize(W, 32)
    w = w4.w4a4_group_quantize(W.cuda(), 32)
    assert torch.equal(w4.w4a4_group_dequantize(w).cpu(), dense(codes, steps, 32).to(dt))


def test_quantize_ties(w4):
    """Every quotient that ends in one half, with steps of 1 and of odd numbers, goes to the even code."""
    rows = []
    for step in (1.0, 3.0, 5.0, 0.75, 127.0):
        half = torch.arange(-13, 14, 2) * 0.5 * step
        rows.append(torch.cat([half, torch.tensor([7 * step]), torch.zeros(32 - 15)]))
    W = torch.stack(rows).to(FP16)                 # all exact in 11 bits
    codes, steps = oracle_quantize(W, 32)
    assert (codes[:, :14] % 2 == 0).all()
    w = w4.w4a4_group_quantize(W.cuda(), 32)
    assert torch.equal(w4.w4a4_group_dequantize(w).cpu(), dense(codes, steps, 32).to(FP16))


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("N,K,group", SHAPES)
def test_pack_gives_what_quantize_stores(w4, N, K, group, dt):
    """Every byte of the packed form, the padding's among them, and codes of -8
    (which the quantizer never gives but other tools do)."""
    W = weights(N, K, group, dt, 3)
    codes, steps = oracle_quantize(W, group)
    plain = ((codes[:, 0::2] & 15) | ((codes[:, 1::2] & 15) << 4)).to(torch.uint8)
    a = w4.GroupWeights(N, K, group, dt)
    b = w4.GroupWeights(N, K, group, dt)
    a.storage.fill_(0xA5)
    b.storage.fill_(0xA5)
    w4.w4a4_group_quantize(W.cuda(), group, out=a)
    w4.w4a4_group_pack(plain.cuda(), steps.cuda(), out=b)
    assert torch.equal(a.storage, b.storage)
    full = torch.randint(0, 256, plain.shape, generator=gen(1), dtype=torch.uint8)
    c = torch.stack([full & 15, full >> 4], 2).view(N, K).long()
    c = torch.where(c > 7, c - 16, c)
    w = w4.w4a4_group_pack(full.cuda(), steps.cuda())
    assert torch.equal(w4.w4a4_group_dequantize(w).cpu(), dense(c, steps, group).to(dt))


def gemv_case(w4, M, N, K, group, dt, bias, seed):
    g = gen(seed)
    full = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    steps = (torch.rand(N, K // group, generator=g) * 0.01 + 0.001).to(dt)
    X = torch.randn(M, K, generator=g)
    X[:, :: max(1, K // 8)] *= 30.0
    X = X.to(dt)
    b = (torch.randn(N, generator=g)).to(dt) if bias else None
    c = torch.stack([full & 15, full >> 4], 2).view(N, K).long()
    D = dense(torch.where(c > 7, c - 16, c), steps, group)
    want = X.double() @ D.T
    size = X.double().abs() @ D.abs().T
    if bias:
        want, size = want + b.double(), size + b.double().abs()
    w = w4.w4a4_group_pack(full.cuda(), steps.cuda())
    return X.cuda(), w, None if b is None else b.cuda(), want, (K + 2 * (K // group) + 8) * 2.0 ** -23 * size


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16])
@pytest.mark.parametrize("N,K,group", SHAPES + [(4096, 1024, 128), (48, 65536 + 32, 32)])
def test_gemv(w4, M, N, K, group, dt):
    X, w, b, want, bound = gemv_case(w4, M, N, K, group, dt, (M + N) % 2 == 0, M * N)
    Y = torch.full((M + 1, N), 7.0, dtype=dt, device="cuda")
    w4.w4a4_group_gemv(X, w, b, Y=Y[:M])
    close(Y[:M], want, bound, dt)
    assert torch.all(Y[M] == 7.0)          # the row behind the last token


def test_gemv_large(w4):
    """More than 2^31 codes: offsets pass 32 bits."""
    N, K, group = 70016, 32768, 128
    w = w4.GroupWeights(N, K, group)
    w.storage.random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(5))
    # the steps of every record: one power of two instead of random patterns
    w.storage.view(-1, 1024 + 32)[:, 1024:].view(BF16).fill_(0.0078125)
    X = torch.randn(3, K, generator=gen(6)).to(BF16)
    Y = w4.w4a4_group_gemv(X.cuda(), w)
    W = w4.w4a4_group_dequantize(w)
    for rows in (slice(0, 64), slice(32752, 32800), slice(N - 64, N)):
        D = W[rows].double().cpu()         # codes times a power of two: exact in bf16
        close(Y[:, rows], X.double() @ D.T, K * 2.0 ** -23 * (X.double().abs() @ D.abs().T), BF16)


def test_gemv_gelu_is_the_gelu_of_the_rounded_result(w4):
    X, w, b, _, _ = gemv_case(w4, 5, 1000, 512, 64, BF16, True, 8)
    X = (X.float() / 8).to(BF16)
    y = w4.w4a4_group_gemv(X, w, b)
    z = w4.w4a4_group_gemv(X, w, b, flags=w4.W4A4_FLAG_GELU_OUT)
    yd = y.double().cpu()
    want = (yd * 0.5 * torch.erfc(-yd / math.sqrt(2.0))).to(BF16)
    inside = (yd.abs() >= 1e-30) & (yd >= -5.9375)
    assert inside.float().mean() > 0.5
    assert torch.equal(z.cpu()[inside], want[inside])


def test_gemv_infinities_stay_in_their_row(w4):
    X, w, _, want, bound = gemv_case(w4, 4, 100, 256, 32, BF16, False, 9)
    X[1, 7], X[2, 200] = math.inf, math.nan
    Y = w4.w4a4_group_gemv(X, w)
    close(Y[[0, 3]], want[[0, 3]], bound[[0, 3]], BF16)
    assert not torch.isfinite(Y[1]).any() or torch.isnan(Y[1]).any() or torch.isinf(Y[1]).any()
    assert torch.isnan(Y[2]).all()


# ------------------------------------------------------------ the paged cache
def pool(w4, pages, page, H, D, dt, layout, fill, g=None):
    """A KVCache whose memory order is nhd, hnd, or nhd with gaps between tokens."""
    def one():
        if layout == "hnd":
            t = torch.empty(pages, H, page, D, dtype=dt, device="cuda").transpose(1, 2)
        elif layout == "gaps":
            t = torch.empty(pages, page, H + 1, D + 8, dtype=dt, device="cuda")[:, :, :H, :D]
        else:
            t = torch.empty(pages, page, H, D, dtype=dt, device="cuda")
        t.copy_(fill if fill is not None and not isinstance(fill, float) else
                torch.full_like(t, fill) if fill is not None else torch.randn(t.shape, generator=g).to(dt))
        return t
    return w4.KVCache(one(), one())


def table_for(counts, page, seed, spare=2):
    """Shuffled pages of sequences that hold counts tokens; unused entries -1."""
    need = [-(-n // page) for n in counts]
    order = torch.randperm(sum(need) + spare, generator=gen(seed))
    table = torch.full((len(counts), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def rotate64(x, rows, pairs):
    """x [T, H, D] double, rows [T, rot] fp32 table rows -> (rotated, fp32 error bound)."""
    half = rows.shape[1] // 2
    c, s = rows[:, None, :half].double(), rows[:, None, half:].double()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if pairs else (x[..., :half], x[..., half:2 * half])
    ra, rb = a * c - b * s, b * c + a * s
    bound = 3 * 2.0 ** -24 * torch.stack([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1)
    if pairs:
        r, e = torch.stack([ra, rb], -1).flatten(-2), bound.flatten(-2)
    else:
        r, e = torch.cat([ra, rb], -1), torch.cat([bound[..., 0], bound[..., 1]], -1)
    return (torch.cat([r, x[..., 2 * half:]], -1),
            torch.cat([e, torch.zeros_like(x[..., 2 * half:])], -1))


APPEND = [  # T, sequences, Hq, Hkv, D, rot, pairs, page, layout
    (1, 1, 1, 1, 64, 64, False, 1, "nhd"), (3, 3, 16, 16, 64, 64, False, 16, "hnd"),
    (7, 2, 5, 1, 128, 64, True, 7, "nhd"), (130, 3, 8, 2, 128, 128, True, 64, "gaps"),
    (517, 4, 0, 3, 64, 16, False, 24, "hnd"), (64, 5, 4, 4, 128, 112, False, 16, "gaps"),
    (33, 2, 12, 3, 64, 48, True, 5, "nhd"), (20, 20, 6, 2, 64, 0, False, 16, "nhd"),
    (1500, 2, 20, 20, 128, 128, False, 32, "nhd"), (40, 4, 3, 1, 64, 32, False, 16, "hnd")]


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("T,S,Hq,Hkv,D,rot,pairs,page,layout", APPEND)
def test_append(w4, T, S, Hq, Hkv, D, rot, pairs, page, layout, dt):
    g = gen(T)
    start = [(i * 13) % 29 for i in range(S)]
    seq = torch.sort(torch.randint(0, S, (T,), generator=g)).values if T != S else torch.arange(S)
    pos = torch.tensor([start[s] + int((seq[:t] == s).sum()) for t, s in enumerate(seq.tolist())])
    counts = [start[i] + int((seq == i).sum()) for i in range(S)]
    pages, total = table_for(counts, page, T + 1)
    cache = pool(w4, total, page, Hkv, D, dt, layout, None, g)
    shuffle = torch.randperm(T, generator=g)       # tokens in any order
    seq, pos = seq[shuffle], pos[shuffle]
    padded = torch.rand(T, generator=g) < 0.2 if T > 5 else torch.zeros(T, dtype=torch.bool)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    own_rows = T % 2 == 0                          # table rows of their own, or the positions
    n_table = max(counts) + 3
    tpos = torch.randint(0, n_table, (T,), generator=g) if own_rows else pos
    table = torch.randn(n_table, rot, generator=g) if rot else None
    K0, V0 = cache.k.cpu().clone(), cache.v.cpu().clone()
    live = ~padded
    rows = table[tpos] if rot else torch.zeros(T, 0)
    kw, kb = rotate64(k.double(), rows, pairs)
    qw, qb = rotate64(q.double(), rows, pairs)
    pos_in = torch.where(padded, -1 - pos, pos).int()
    dev = qkv.cuda()
    out = torch.full((T, Hq, D), 5.0, dtype=dt, device="cuda")
    r = w4.w4a4_kv_append(
        cache, dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], pages.cuda(), pos_in.cuda(), q=dev[:, :Hq] if Hq else None,
        q_out=out if Hq else None, table=table.cuda() if rot else None,
        table_pos=tpos.int().cuda() if own_rows and rot else None, seq=seq.int().cuda(),
        flags=w4.W4A4_FLAG_ROPE_PAIRS if pairs else 0)
    assert (r is None) == (Hq == 0)
    at = pages[seq, pos // page].long()[live], (pos % page)[live]
    V0[at] = v[live]
    assert torch.equal(cache.v.cpu(), V0)
    K = cache.k.cpu()
    close(K[at], kw[live], kb[live], dt)
    K[at] = K0[at]
    assert torch.equal(K, K0)                      # every other row as it was
    if Hq:
        close(out[live.cuda()], qw[live], qb[live], dt)
        assert torch.all(out[padded.cuda()] == 5.0)


def test_append_in_place_and_decode_default(w4):
    """q rotated in place, and one token per sequence without seq."""
    S, H, D, page = 9, 4, 64, 16
    g = gen(2)
    pos = torch.tensor([0, 15, 16, 17, 31, 32, 5, 100, 64])
    pages, total = table_for([int(p) + 1 for p in pos], page, 4)
    cache = pool(w4, total, page, H, D, BF16, "nhd", 0.0)
    k, v, q = (torch.randn(S, H, D, generator=g).to(BF16) for _ in range(3))
    table = torch.from_numpy(w4.w4a4_rope_table(128, D))
    qd = q.cuda()
    r = w4.w4a4_kv_append(cache, k.cuda(), v.cuda(), pages.cuda(), pos.int().cuda(), q=qd, q_out=qd,
                          table=table.cuda())
    assert r is qd
    want, bound = rotate64(q.double(), table[pos], False)
    close(qd, want, bound, BF16)
    want, bound = rotate64(k.double(), table[pos], False)
    at = pages[torch.arange(S), pos // page].long(), pos % page
    close(cache.k.cpu()[at], want, bound, BF16)
    assert torch.equal(cache.v.cpu()[at], v)


def test_append_out_of_range_is_left_out_and_reported(w4):
    """A position, sequence, page or table row out of range: the token is left
    out, its neighbours are not, the status says so."""
    H, D, page, n = 2, 64, 16, 6
    pages = torch.tensor([[0, 1], [2, 99], [-1, 3]], dtype=torch.int32)
    cache = pool(w4, 4, page, H, D, BF16, "nhd", 0.0)
    ones = torch.ones(n, H, D, dtype=BF16, device="cuda")
    table = torch.cat([torch.ones(40, 32), torch.zeros(40, 32)], 1).cuda()
    seq = torch.tensor([0, 1, 2, 3, -1, 0], dtype=torch.int32)
    pos = torch.tensor([32, 17, 3, 1, 1, 5], dtype=torch.int32)   # only the last token has a place
    w4.w4a4_kv_append(cache, ones, ones, pages.cuda(), pos.cuda(), table=table, seq=seq.cuda())
    assert w4.w4a4_get_device_status() == RANGE
    w4.w4a4_clear_device_status()
    want = torch.zeros(4, page, H, D, dtype=BF16)
    want[0, 5] = 1.0
    assert torch.equal(cache.k.cpu(), want) and torch.equal(cache.v.cpu(), want)
    w4.w4a4_kv_append(cache, ones[:2], ones[:2], pages.cuda(), pos[4:].cuda(), table=table, seq=seq[5:].repeat(2).cuda(),
                      table_pos=torch.tensor([40, -1], dtype=torch.int32).cuda())
    assert w4.w4a4_get_device_status() == RANGE
    w4.w4a4_clear_device_status()
    assert torch.equal(cache.k.cpu(), want)


# ------------------------------------------------------------ attention
def oracle_attend(q, K, V, pages, lens, scale, window):
    """(out, lse, error bound of out before its rounding, bound of lse) in 64 bits."""
    B, Hq, D = q.shape
    page, H = K.shape[1], K.shape[2]
    G = Hq // H
    out, bound = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    lse, lse_bound = torch.full((B, Hq), -math.inf, dtype=torch.float64), torch.zeros(B, Hq, dtype=torch.float64)
    for b, n in enumerate(lens.tolist()):
        first = max(0, n - window) if window else 0
        if n <= first:
            continue
        at = torch.arange(first, n)
        k, v = K[pages[b, at // page].long(), at % page].double(), V[pages[b, at // page].long(), at % page].double()
        qb = q[b].double().view(H, G, D)
        s = torch.einsum("hgd,thd->hgt", qb, k) * scale
        size = torch.einsum("hgd,thd->hgt", qb.abs(), k.abs()) * abs(scale)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        total = p.sum(-1, keepdim=True)
        p = p / total
        # the score's own sum and scaling, the subtraction of the maximum, exp
        # (argument in units of log 2: one more rounding; the function 2^-22)
        d = (D + 4) * 2.0 ** -23 * size.amax(-1, keepdim=True) + 2.0 ** -22 * (s - m).abs() + 2.0 ** -22
        # every weight once in the sum over v and once in the total; weights held as
        # two 16-bit terms: 2^-16; sums over n terms
        rel = 2 * d.amax(-1, keepdim=True) + 2.0 ** -16 + (n - first + 16) * 2.0 ** -22
        o = torch.einsum("hgt,thd->hgd", p, v)
        e = torch.einsum("hgt,thd->hgd", p, v.abs()) * rel
        out[b], bound[b] = o.reshape(Hq, D), e.reshape(Hq, D)
        lse[b] = (m + torch.log(total)).view(Hq)
        lse_bound[b] = (rel + 2.0 ** -22 * (1 + (m + torch.log(total)).abs() + m.abs())).view(Hq)
    return out, lse, bound, lse_bound


def attend_case(w4, B, lens, Hq, H, D, page, layout, dt, seed, junk=math.nan):
    """Caches whose rows that hold no token are junk."""
    g = gen(seed)
    pages, total = table_for([max(0, n) for n in lens], page, seed)
    cache = pool(w4, total, page, H, D, dt, layout, junk)
    K, V = torch.full((total, page, H, D), junk, dtype=dt), torch.full((total, page, H, D), junk, dtype=dt)
    for b, n in enumerate(lens):
        at = torch.arange(max(0, n))
        where = pages[b, at // page].long(), at % page
        K[where] = torch.randn(len(at), H, D, generator=g).to(dt)
        V[where] = torch.randn(len(at), H, D, generator=g).to(dt)
    cache.k.copy_(K)
    cache.v.copy_(V)
    q = (torch.randn(B, Hq, D, generator=g) * 2).to(dt)
    return q, cache, K, V, pages, torch.tensor(lens, dtype=torch.int32)


def check_attend(w4, q, cache, K, V, pages, lens, window=0, scale=None, **kw):
    dt = q.dtype
    B, Hq, D = q.shape
    want, wl, bound, lb = oracle_attend(q, K, V, pages, lens, D ** -0.5 if scale is None else scale, window)
    empty = wl == -math.inf
    # the width of the table decides how the work is cut: as it is, and with room for 16000 tokens
    more = 16_000 // cache.page_size + 1 - pages.shape[1]
    for table in [pages] if more <= 0 else [pages, torch.nn.functional.pad(pages, (0, more), value=-1)]:
        lse = torch.full((B + 1, Hq), 3.0, device="cuda")
        out = torch.full((B + 1, Hq, D), 3.0, dtype=dt, device="cuda")
        w4.w4a4_kv_attend(q.cuda(), cache, table.cuda(), lens.cuda(), scale=scale, window=window, out=out[:B],
                          lse=lse[:B], **kw)
        close(out[:B], want, bound, dt)
        got = lse[:B].double().cpu()
        assert torch.all(got[empty] == -math.inf)
        assert torch.all((got - wl).abs()[~empty] <= lb[~empty])
        assert torch.all(out[B] == 3.0) and torch.all(lse[B] == 3.0)
        assert torch.all(out[:B].cpu()[empty] == 0.0)


EDGE = [0, 1, 2, 7, 8, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000, -3]


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,H,page,layout", [(1, 3, 16, "nhd"), (2, 2, 1, "hnd"), (4, 1, 7, "gaps"), (5, 2, 24, "nhd"),
                                             (8, 2, 64, "hnd"), (12, 1, 128, "nhd"), (16, 2, 16, "gaps"),
                                             (20, 1, 33, "hnd"), (37, 1, 16, "nhd")])
def test_attend_lengths(w4, G, H, page, layout, D, dt):
    case = attend_case(w4, len(EDGE), EDGE, G * H, H, D, page, layout, dt, G * 1000 + page)
    check_attend(w4, *case)


@pytest.mark.parametrize("junk", [math.inf, -math.inf, 65504.0])
def test_attend_ignores_what_rows_behind_the_length_hold(w4, junk):
    check_attend(w4, *attend_case(w4, 5, [1, 30, 0, 17, 100], 8, 2, 64, 16, "nhd", FP16, 5, junk))


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 1 << 30])
def test_attend_window(w4, window):
    lens = [0, 1, 14, 16, 17, 40, 99, 100, 101, 1000, 2053]
    q, cache, K, V, pages, lens = attend_case(w4, len(lens), lens, 6, 3, 64, 24, "nhd", BF16, window % 1000)
    for b, n in enumerate(lens.tolist()):          # rows in front of the window are never read
        first = max(0, n - window)
        at = torch.arange(first)
        where = pages[b, at // 24].long(), at % 24
        K[where], V[where] = math.nan, math.nan
        pages[b, : first // 24] = -7               # nor are their pages
    cache.k.copy_(K)
    cache.v.copy_(V)
    check_attend(w4, q, cache, K, V, pages, lens, window)


@pytest.mark.parametrize("B,L,Hq,H,D", [(1, 5000, 1, 1, 64), (1, 40000, 16, 16, 64), (2, 30000, 8, 1, 128),
                                        (1, 100_003, 12, 1, 128), (300, 70, 4, 2, 64), (3, 9000, 64, 4, 128)])
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_attend_long_and_many(w4, B, L, Hq, H, D, dt):
    lens = [max(0, L - 37 * i * (L // (B * 40) + 1)) for i in range(B)]
    check_attend(w4, *attend_case(w4, B, lens, Hq, H, D, 64, "hnd", dt, L))


@pytest.mark.parametrize("seed", range(24))
def test_attend_drawn(w4, seed):
    """Drawn batches: the line of pieces is cut at ever other places, into parts of
    single warps and of whole blocks."""
    g = gen(1000 + seed)
    pick = lambda *v: v[int(torch.randint(0, len(v), (1,), generator=g))]
    B, H, G = pick(1, 2, 3, 7, 31, 33, 60), pick(1, 2, 3, 4, 6, 8), pick(1, 2, 3, 8, 9, 17)
    top = pick(3, 40, 700, 4000)
    lens = torch.randint(0, top + 1, (B,), generator=g).tolist()
    lens[int(torch.randint(0, B, (1,), generator=g))] = top * pick(1, 5)
    D, page = pick(64, 128), pick(1, 5, 16, 32, 48, 64)
    case = attend_case(w4, B, lens, G * H, H, D, page, pick("nhd", "hnd", "gaps"), pick(BF16, FP16), seed)
    check_attend(w4, *case, window=pick(0, 0, 13, 64, 1000))


@pytest.mark.parametrize("H,G", [(1, 4), (2, 1), (4, 2), (4, 12), (6, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_with_wide_tables(w4, D, H, G):
    """The table's width is all the host knows of the lengths; results hold for any."""
    q, cache, K, V, pages, lens = attend_case(w4, 8, [1, 700, 33, 0, 2500, 16, 15, 90], H * G, H, D, 16, "nhd", BF16, 26)
    wide = torch.full((8, 1 << 14), -1, dtype=torch.int32)
    wide[:, :pages.shape[1]] = pages
    check_attend(w4, q, cache, K, V, pages, lens)
    check_attend(w4, q, cache, K, V, wide, lens)


def test_attend_very_many(w4):
    """More sequences than threads: every thread adds up a run of them."""
    lens = [(i * i) % 23 if i % 7 else 0 for i in range(1500)]
    lens[1400] = 3000
    check_attend(w4, *attend_case(w4, 1500, lens, 4, 2, 64, 16, "nhd", BF16, 77))


def test_attend_one_long_among_many_short(w4):
    check_attend(w4, *attend_case(w4, 40, [20_011 if i == 17 else i % 3 for i in range(40)], 8, 4, 64, 16, "nhd", BF16, 3))


def test_attend_large_scores(w4):
    """Scores of +-1000s: the running maximum has to move, and weights vanish."""
    q, cache, K, V, pages, lens = attend_case(w4, 4, [1, 300, 77, 2000], 4, 2, 64, 16, "nhd", BF16, 12)
    check_attend(w4, q, cache, K, V, pages, lens, scale=40.0)
    check_attend(w4, q, cache, K, V, pages, lens, scale=-3.0)
    check_attend(w4, q, cache, K, V, pages, lens, scale=0.0)


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("D,Hq", [(64, 1), (128, 12)])
def test_attend_many_weights_far_below_the_largest(w4, D, Hq, dt):
    """One token of score 18 holds value 0, 200000 of score 0 hold 1: weights of 2^-26 that are 2^-8 of
    the sum together, and all of the result."""
    n, page = 200_000, 64
    K, V = torch.zeros(n // page, page, 1, D, dtype=dt), torch.ones(n // page, page, 1, D, dtype=dt)
    K[1000, 7, 0, 0], V[1000, 7] = 4.5, 0.0
    q = torch.zeros(1, Hq, D, dtype=dt)
    q[..., 0] = 4.0
    pages = torch.arange(n // page, dtype=torch.int32).view(1, -1)
    check_attend(w4, q, w4.KVCache(K.cuda(), V.cuda()), K, V, pages, torch.tensor([n], dtype=torch.int32), scale=1.0)


def test_attend_in_place_and_into_the_gaps_of_q(w4):
    """out may be q itself, long sequences split over many warps included, or lie between its rows."""
    q, cache, K, V, pages, lens = attend_case(w4, 4, [5000, 1, 0, 333], 20, 1, 64, 16, "nhd", BF16, 23)
    want = w4.w4a4_kv_attend(q.cuda(), cache, pages.cuda(), lens.cuda())
    qd = q.cuda()
    assert w4.w4a4_kv_attend(qd, cache, pages.cuda(), lens.cuda(), out=qd) is qd
    assert torch.equal(qd, want)
    wide = torch.zeros(4, 5 * 20 * 64, dtype=BF16, device="cuda")
    wide[:, :20 * 64] = q.view(4, -1).cuda()
    out = wide[1, 20 * 64:].view(4, 20, 64)
    w4.w4a4_kv_attend(wide[:, :20 * 64].view(4, 20, 64), cache, pages.cuda(), lens.cuda(), out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("D,H,G", [(64, 16, 1), (128, 2, 4), (128, 8, 1)])
@pytest.mark.parametrize("window", [1, 2, 17, 18, 33, 34, 300])
def test_attend_windows_at_every_place_of_a_piece(w4, window, D, H, G):
    """The most pieces that a window can touch decide how the work is cut."""
    lens = [window - 1, window, window + 1] + [640 + i for i in range(33)]
    q, cache, K, V, pages, lens = attend_case(w4, len(lens), lens, H * G, H, D, 16, "nhd", BF16, 27)
    check_attend(w4, q, cache, K, V, pages, lens, window)
    check_attend(w4, q[:2], cache, K, V, pages[:2], lens[:2], window)


@pytest.mark.parametrize("page", [7, 16, 64])
def test_attend_window_over_freed_pages(w4, page):
    """Pages that lie wholly in front of the window need not be there."""
    q, cache, K, V, pages, lens = attend_case(w4, 3, [500, 321, 90], 4, 2, 64, page, "nhd", BF16, 24)
    want = w4.w4a4_kv_attend(q.cuda(), cache, pages.cuda(), lens.cuda(), window=75)
    freed = pages.clone()
    for b, n in enumerate(lens.tolist()):
        freed[b, :(n - 75) // page] = 1 << 30
    got = w4.w4a4_kv_attend(q.cuda(), cache, freed.cuda(), lens.cuda(), window=75)
    assert torch.equal(got, want)                  # and the status stays clear


@pytest.mark.parametrize("page", [1, 7, 24])
def test_attend_absent_pages_that_end_inside_a_tile(w4, page):
    """Pages out of range among rows that are looked up one by one: left out and reported."""
    n, D = 200, 128
    q, cache, K, V, pages, lens = attend_case(w4, 1, [n], 4, 2, D, page, "nhd", FP16, 25)
    bad = pages.clone()
    gone = [0, 3, (n - 1) // page]
    bad[0, gone] = torch.tensor([-1, 1 << 30, cache.n_pages], dtype=torch.int32)
    out = w4.w4a4_kv_attend(q.cuda(), cache, bad.cuda(), lens.cuda())
    assert w4.w4a4_get_device_status() == RANGE
    w4.w4a4_clear_device_status()
    keep = torch.tensor([t for t in range(n) if t // page not in gone])
    row = pages[0, keep // page].long(), keep % page
    want, _, bound, _ = oracle_attend(q, K[row][:, None], V[row][:, None], torch.arange(len(keep)).view(1, -1),
                                      torch.tensor([len(keep)]), D ** -0.5, 0)
    close(out, want, bound, FP16)


def test_attend_lowest_scores(w4):
    """All scores are huge and negative: the softmax still sums to one."""
    q, cache, K, V, pages, lens = attend_case(w4, 2, [50, 1], 2, 1, 64, 16, "nhd", BF16, 13)
    q = torch.full_like(q, 1e18)
    K = torch.where(K.isnan(), K, torch.full_like(K, -1e18))
    cache.k.copy_(K)
    check_attend(w4, q, cache, K, V, pages, lens)


def test_attend_shared_pages_and_strided_q(w4):
    """Sequences that share a prefix's pages; q as a view of a larger tensor."""
    q, cache, K, V, pages, lens = attend_case(w4, 1, [200], 8, 2, 128, 16, "nhd", BF16, 21)
    pages, lens = pages.repeat(6, 1), torch.tensor([200, 199, 150, 16, 1, 0], dtype=torch.int32)
    wide = torch.randn(6, 12, 128, generator=gen(22)).to(BF16).cuda()
    out = w4.w4a4_kv_attend(wide[:, 2:10], cache, pages.cuda(), lens.cuda())
    want, _, bound, _ = oracle_attend(wide[:, 2:10].cpu(), K, V, pages, lens, 128 ** -0.5, 0)
    close(out, want, bound, BF16)


def test_attend_out_of_range_is_left_out_and_reported(w4):
    q, cache, K, V, pages, lens = attend_case(w4, 3, [100, 64, 5], 4, 2, 64, 16, "nhd", BF16, 31)
    bad = pages.clone()
    bad[0, 3], bad[0, 5] = 9999, -2                # rows 48..63 and 80..95 are absent
    out = w4.w4a4_kv_attend(q.cuda(), cache, bad.cuda(), lens.cuda())
    assert w4.w4a4_get_device_status() == RANGE
    w4.w4a4_clear_device_status()
    want, _, bound, _ = oracle_attend(q, K, V, pages, lens, 0.125, 0)
    close(out[1:], want[1:], bound[1:], BF16)
    keep = torch.tensor([t for t in range(100) if not (48 <= t < 64 or 80 <= t < 96)])
    row = pages[0, keep // 16].long(), keep % 16
    K1, V1 = torch.zeros(5, 16, 2, 64, dtype=BF16), torch.zeros(5, 16, 2, 64, dtype=BF16)
    K1.view(80, 2, 64)[:68], V1.view(80, 2, 64)[:68] = K[row], V[row]
    want, _, bound, _ = oracle_attend(q[:1], K1, V1, torch.arange(5).view(1, 5), torch.tensor([68]), 0.125, 0)
    close(out[:1], want, bound, BF16)
    # a length above what the table holds counts as that many
    full = torch.tensor([112, 500, 5], dtype=torch.int32)
    a = w4.w4a4_kv_attend(q[1:2].cuda(), cache, pages[1:2, :4].contiguous().cuda(), full[1:2].cuda())
    assert w4.w4a4_get_device_status() == RANGE
    w4.w4a4_clear_device_status()
    b = w4.w4a4_kv_attend(q[1:2].cuda(), cache, pages[1:2, :4].contiguous().cuda(), lens[1:2].cuda())
    assert torch.equal(a, b)


def test_attend_without_pages_or_sequences(w4):
    cache = w4.KVCache(torch.empty(0, 16, 2, 64, dtype=BF16, device="cuda"),
                       torch.empty(0, 16, 2, 64, dtype=BF16, device="cuda"))
    q = torch.ones(2, 4, 64, dtype=BF16, device="cuda")
    none = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert torch.all(w4.w4a4_kv_attend(q, cache, none, zero) == 0)
    assert w4.w4a4_kv_attend(q[:0], cache, none[:0], zero[:0]).shape == (0, 4, 64)
    assert w4.w4a4_kv_append(cache, q[:0, :2], q[:0, :2], none, zero[:0]) is None
    x = torch.empty(0, 128, dtype=BF16, device="cuda")
    assert w4.w4a4_group_gemv(x, w4.GroupWeights(32, 128, 128)).shape == (0, 32)


def test_offsets_beyond_32_bits(w4):
    """Pages 2^31 + 2^20 elements apart: appended to and attended over."""
    H, D, page, far = 2, 64, 16, (1 << 31) + (1 << 20)
    store = torch.empty(2 * far + page * H * D * 2, dtype=BF16, device="cuda")
    k = torch.as_strided(store, (3, page, H, D), (far, H * D, D, 1), 0)
    v = torch.as_strided(store, (3, page, H, D), (far, H * D, D, 1), page * H * D)
    cache = w4.KVCache(k, v)
    pages, n = torch.tensor([[2, 0, 1]], dtype=torch.int32), 41
    x = torch.randn(2, n, H, D, generator=gen(41)).to(BF16)
    pos = torch.arange(n, dtype=torch.int32)
    w4.w4a4_kv_append(cache, x[0].cuda(), x[1].cuda(), pages.cuda(), pos.cuda(), seq=torch.zeros_like(pos).cuda())
    at = pages[0, pos // page].long(), (pos % page).long()
    assert torch.equal(k.cpu()[at], x[0]) and torch.equal(v.cpu()[at], x[1])
    q = torch.randn(1, 4, D, generator=gen(42)).to(BF16)
    check_attend(w4, q, cache, k.cpu(), v.cpu(), pages, torch.tensor([n], dtype=torch.int32))


def test_same_inputs_same_bits(w4):
    q, cache, _, _, pages, lens = attend_case(w4, 5, [3000, 17, 0, 900, 64], 16, 4, 128, 16, "nhd", BF16, 55)
    args = q.cuda(), cache, pages.cuda(), lens.cuda()
    first = w4.w4a4_kv_attend(*args)
    X, w, b, _, _ = gemv_case(w4, 3, 1021, 4096, 32, BF16, True, 56)
    y = w4.w4a4_group_gemv(X, w, b)
    for _ in range(20):
        assert torch.equal(w4.w4a4_kv_attend(*args), first)
        assert torch.equal(w4.w4a4_group_gemv(X, w, b), y)


# ------------------------------------------------- a block's step, as it is used
class Block:
    """One decoder block on the operators: 4-bit linears, cache, attention."""

    def __init__(self, w4, S, Hq, H, D, group, dt, seed, page=16, room=256):
        self.w4, self.Hq, self.H, self.D, self.dt = w4, Hq, H, D, dt
        g, width = gen(seed), Hq * D
        self.W = {n: (torch.randn(o, i, generator=g) / math.sqrt(i)).to(dt) for n, o, i in [
            ("qkv", (Hq + 2 * H) * D, width), ("proj", width, width), ("fc1", 4 * width, width), ("fc2", width, 4 * width)]}
        self.w = {n: w4.w4a4_group_quantize(W.cuda(), group) for n, W in self.W.items()}
        per = room // page
        self.pages = torch.randperm(S * per, generator=g).view(S, per).int()
        self.cache = pool(w4, S * per, page, H, D, dt, "nhd", math.nan)
        self.table = torch.from_numpy(w4.w4a4_rope_table(room, D))
        self.pages_d, self.table_d = self.pages.cuda(), self.table.cuda()
        self.ws = torch.empty(w4.w4a4_kv_attend_workspace_bytes(S, Hq, H, D), dtype=torch.uint8, device="cuda")

    def step(self, x, pos, lens):
        w4, S = self.w4, x.shape[0]
        h = w4.w4a4_group_gemv(x, self.w["qkv"]).view(S, self.Hq + 2 * self.H, self.D)
        q = w4.w4a4_kv_append(self.cache, h[:, self.Hq:self.Hq + self.H], h[:, self.Hq + self.H:], self.pages_d, pos,
                              q=h[:, :self.Hq], table=self.table_d)
        o = w4.w4a4_kv_attend(q, self.cache, self.pages_d, lens, workspace=self.ws)
        y = w4.w4a4_group_gemv(o.view(S, -1), self.w["proj"])
        z = w4.w4a4_group_gemv(y, self.w["fc1"], flags=0 if self.dt == FP16 else w4.W4A4_FLAG_GELU_OUT)
        return w4.w4a4_group_gemv(z, self.w["fc2"])

    def plain(self, xs):
        """All steps of one sequence list in 64 bits: xs [steps][S, width]."""
        W = {n: dense(*oracle_quantize(w, self.w[n].group), self.w[n].group) for n, w in self.W.items()}
        S = xs[0].shape[0]
        G, ks, vs, outs = self.Hq // self.H, [], [], []
        for t, x in enumerate(xs):
            h = (x.double() @ W["qkv"].T).view(S, -1, self.D)
            rows = self.table[torch.full((S,), t)]
            q, _ = rotate64(h[:, :self.Hq], rows, False)
            k, _ = rotate64(h[:, self.Hq:self.Hq + self.H], rows, False)
            ks.append(k)
            vs.append(h[:, self.Hq + self.H:])
            K, V = torch.stack(ks, 1), torch.stack(vs, 1)
            s = torch.einsum("shgd,sthd->shgt", q.view(S, self.H, G, self.D), K) / math.sqrt(self.D)
            o = torch.einsum("shgt,sthd->shgd", torch.softmax(s, -1), V).reshape(S, -1)
            z = (o @ W["proj"].T) @ W["fc1"].T
            if self.dt == BF16:
                z = z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
            outs.append(z @ W["fc2"].T)
        return outs


@pytest.mark.parametrize("dt,Hq,H,D,group", [(BF16, 4, 4, 64, 64), (FP16, 4, 2, 128, 32), (BF16, 8, 1, 64, 128)])
def test_a_block_step_by_step(w4, dt, Hq, H, D, group):
    """33 tokens of 3 sequences, one by one.  Every step rounds six times in a
    row (qkv, rotation, attention, proj, fc1, fc2), each a relative error of at most h
    of its operator's result; random signs keep each operator's relative (norm)
    error from growing, and the softmax doubles what the scores (of a few
    units) pass on: 6 * 2 * h in the norm, with room for the GELU's slope of 1.13."""
    S, steps = 3, 33
    b = Block(w4, S, Hq, H, D, group, dt, Hq + D)
    xs = [torch.randn(S, Hq * D, generator=gen(100 + t)).to(dt) for t in range(steps)]
    want = b.plain(xs)
    for t, x in enumerate(xs):
        pos = torch.full((S,), t, dtype=torch.int32, device="cuda")
        got = b.step(x.cuda(), pos, pos + 1)
        err = (got.double().cpu() - want[t]).norm() / want[t].norm()
        assert err <= 12 * 1.13 * half_step(dt), (t, err)


def test_a_step_captured_and_replayed(w4):
    """The whole step in a CUDA graph, positions advanced on the device: the
    same bits as eager calls; a second graph over the same buffers interleaved."""
    S = 3
    a, b = (Block(w4, S, 4, 2, 64, 64, BF16, 9) for _ in range(2))
    xs = [torch.randn(S, 256, generator=gen(200 + t)).to(BF16).cuda() for t in range(20)]
    want = []
    for t, x in enumerate(xs):
        pos = torch.full((S,), t, dtype=torch.int32, device="cuda")
        want.append(a.step(x, pos, pos + 1))
    x, pos, lens = xs[0].clone(), torch.zeros(S, dtype=torch.int32, device="cuda"), torch.ones(S, dtype=torch.int32, device="cuda")
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.step(x, pos, lens))
        graphs.append(g)
    for t in range(20):
        x.copy_(xs[t])
        pos.fill_(t)
        lens.fill_(t + 1)
        graphs[t % 2].replay()
        assert torch.equal(outs[t % 2], want[t]), t


def test_graphs_that_share_a_workspace(w4):
    """Two captured calls of different shapes over one workspace, and an eager one between them."""
    cases = [attend_case(w4, 2, [9000, 4000], 8, 4, 64, 16, "nhd", BF16, 81),
             attend_case(w4, 3, [100, 7000, 3], 16, 1, 128, 64, "hnd", BF16, 82)]
    args = [(c[0].cuda(), c[1], c[4].cuda(), c[5].cuda()) for c in cases]
    want = [w4.w4a4_kv_attend(*a) for a in args]
    need = max(w4.w4a4_kv_attend_workspace_bytes(a[0].shape[0], a[0].shape[1], a[1].n_heads, a[0].shape[2])
               for a in args)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w4.w4a4_kv_attend(*a, workspace=ws))
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o.fill_(7.0)
        graphs[0].replay()
        eager = w4.w4a4_kv_attend(*args[1], workspace=ws)
        graphs[1].replay()
        graphs[0].replay()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(eager, want[1])


@pytest.mark.parametrize("dt", [BF16, FP16])
def test_a_padded_batch(w4, dt):
    """Rows without a sequence (position -1, length 0, tokens of NaN) change nothing of the others, and
    leave the attention's zeros behind."""
    S, Hq, H, D = 5, 4, 2, 64
    full, padded = (Block(w4, S, Hq, H, D, 64, dt, 91) for _ in range(2))
    x = torch.randn(S, Hq * D, generator=gen(92)).to(dt).cuda()
    pos = torch.zeros(S, dtype=torch.int32, device="cuda")
    want = full.step(x, pos, pos + 1)
    x, pos = x.clone(), pos.clone()
    x[1], x[4], pos[1], pos[4] = math.nan, math.inf, -1, -1
    got = padded.step(x, pos, pos + 1)             # one token each, so no item is split differently
    live = [0, 2, 3]
    assert torch.equal(got[live], want[live]) and torch.all(got[[1, 4]] == 0)
    for a, b in ((full.cache.k, padded.cache.k), (full.cache.v, padded.cache.v)):
        rows = full.pages_d[live, 0].long()
        assert torch.equal(a[rows, 0], b[rows, 0])
        assert b.isnan().flatten(1).any(1).all() and b[padded.pages_d[[1, 4], 0].long()].isnan().all()


def test_first_calls_in_a_capture():
    """The first use of every operator in a process may be a captured one."""
    code = (
        "import torch\n"
        "from w4a4_post_quantized_b200 import w4a4 as w\n"
        "B = torch.bfloat16\n"
        "W = torch.randn(64, 128, device='cuda').to(B); x = torch.randn(2, 128, device='cuda').to(B)\n"
        "c = w.KVCache(torch.zeros(4, 16, 1, 64, device='cuda', dtype=B), torch.zeros(4, 16, 1, 64, device='cuda', dtype=B))\n"
        "pg = torch.arange(4, device='cuda', dtype=torch.int32).view(2, 2)\n"
        "pos = torch.zeros(2, dtype=torch.int32, device='cuda'); lens = pos + 1\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    gw = w.w4a4_group_quantize(W)\n"
        "    h = w.w4a4_group_gemv(x, gw).view(2, 1, 64)\n"
        "    w.w4a4_kv_append(c, h, h, pg, pos)\n"
        "    o = w.w4a4_kv_attend(h, c, pg, lens)\n"
        "g.replay(); torch.cuda.synchronize()\n"
        "assert torch.equal(o, h) and w.w4a4_get_device_status() == 0\n"
        "print('captured')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_on_another_stream(w4):
    """Work that waits on a side stream: nothing leaks to the current one."""
    q, cache, K, V, pages, lens = attend_case(w4, 3, [500, 20, 0], 8, 2, 64, 16, "nhd", BF16, 61)
    X, w, b, want, bound = gemv_case(w4, 4, 300, 1024, 64, BF16, True, 62)
    args = q.cuda(), cache, pages.cuda(), lens.cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        outs = [w4.w4a4_kv_attend(*args, stream=side) for _ in range(4)]
        ys = [w4.w4a4_group_gemv(X, w, b, stream=side) for _ in range(4)]
        torch.randn(1 << 20, device="cuda")        # the current stream allocates meanwhile
        side.synchronize()
        o, _, ob, _ = oracle_attend(q, K, V, pages, lens, 0.125, 0)
        for got in outs:
            close(got, o, ob, BF16)
        for y in ys:
            close(y, want, bound, BF16)


def test_two_calls_at_once(w4):
    """Calls on two streams, each with a workspace of its own, while a third appends elsewhere."""
    cases = [attend_case(w4, 2, [9000, 4000], 8, 4, 64, 16, "nhd", BF16, 71),
             attend_case(w4, 3, [100, 7000, 3], 16, 1, 128, 64, "hnd", BF16, 72)]
    args = [(c[0].cuda(), c[1], c[4].cuda(), c[5].cuda()) for c in cases]
    want = [w4.w4a4_kv_attend(*a) for a in args]
    X, w, b, _, _ = gemv_case(w4, 16, 700, 4096, 64, BF16, True, 73)
    y = w4.w4a4_group_gemv(X, w, b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[], [], []]
    for _ in range(20):
        for i in range(2):
            outs[i].append(w4.w4a4_kv_attend(*args[i], stream=streams[i]))
        outs[2].append(w4.w4a4_group_gemv(X, w, b, stream=streams[2]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])
    assert all(torch.equal(o, y) for o in outs[2])


def test_refusals_of_the_binding(w4):
    dev = "cuda"
    x = torch.zeros(2, 128, dtype=BF16, device=dev)
    w = w4.w4a4_group_quantize(torch.zeros(16, 128, dtype=BF16, device=dev))
    for bad in (x.half(), x.float(), x[:, ::2], x.cpu(), torch.zeros(2, 256, dtype=BF16, device=dev),
                torch.zeros(128, 2, dtype=BF16, device=dev).t()):
        with pytest.raises(ValueError):
            w4.w4a4_group_gemv(bad, w)
    with pytest.raises(ValueError):
        w4.w4a4_group_gemv(x, w, bias=torch.zeros(15, dtype=BF16, device=dev))
    with pytest.raises(ValueError):
        w4.w4a4_group_gemv(x, w, Y=torch.zeros(2, 17, dtype=BF16, device=dev))
    square = w4.w4a4_group_quantize(torch.zeros(128, 128, dtype=BF16, device=dev))
    with pytest.raises(w4.W4A4Error):
        w4.w4a4_group_gemv(x, square, Y=x)
    with pytest.raises(w4.W4A4Error):
        w4.w4a4_group_gemv(torch.zeros(17, 128, dtype=BF16, device=dev), w)
    with pytest.raises(w4.W4A4Error):
        w4.GroupWeights(16, 100, 128)
    with pytest.raises(w4.W4A4Error):
        w4.w4a4_group_quantize(x, group=16)
    with pytest.raises(ValueError):
        w4.w4a4_group_quantize(x.float())
    with pytest.raises(ValueError):
        w4.w4a4_group_pack(torch.zeros(16, 64, dtype=torch.uint8, device=dev), torch.zeros(16, 3, dtype=BF16, device=dev))
    k = torch.zeros(4, 16, 2, 64, dtype=BF16, device=dev)
    for bad in ((k, k.half()), (k, k[:2]), (k.cpu(), k.cpu()), (k.transpose(2, 3), k.transpose(2, 3)),
                (k, k.transpose(1, 2).contiguous().transpose(1, 2)), (k.float(), k.float())):
        with pytest.raises(ValueError):
            w4.KVCache(*bad)
    cache = w4.KVCache(k, k.clone())
    pages = torch.arange(4, dtype=torch.int32, device=dev).view(2, 2)
    ints = torch.ones(2, dtype=torch.int32, device=dev)
    h = torch.zeros(2, 2, 64, dtype=BF16, device=dev)
    good = dict(k=h, v=h, pages=pages, pos=ints)
    for bad in (dict(k=h.half()), dict(v=h[:1]), dict(pages=pages.long()), dict(pos=ints.long()), dict(pos=ints[:1]),
                dict(k=torch.zeros(2, 64, 2, dtype=BF16, device=dev).transpose(1, 2)), dict(seq=ints.long()),
                dict(table=torch.zeros(9, 64, device=dev).double()), dict(pages=pages[:1]), dict(pos=ints.cpu()),
                dict(q=h, q_out=h.half())):
        with pytest.raises(ValueError):
            w4.w4a4_kv_append(cache, **{**good, **bad})
    with pytest.raises(w4.W4A4Error):
        w4.w4a4_kv_append(cache, **good, table=torch.zeros(9, 24, device=dev))
    wide = w4.KVCache(k[:1].expand(4, 16, 2, 64), k[:1].expand(4, 16, 2, 64))
    with pytest.raises(w4.W4A4Error):
        w4.w4a4_kv_append(wide, **good)
    good = dict(q=h, pages=pages, lens=ints)
    for bad in (dict(q=h.half()), dict(lens=ints.long()), dict(lens=ints[:1]), dict(pages=pages[:1]),
                dict(out=h.half()), dict(lse=torch.zeros(2, 2, device=dev).double()), dict(q=h[:, :, :32])):
        with pytest.raises(ValueError):
            w4.w4a4_kv_attend(cache=cache, **{**good, **bad})
    with pytest.raises(w4.W4A4Error):
        w4.w4a4_kv_attend(cache=cache, q=torch.zeros(2, 3, 64, dtype=BF16, device=dev), pages=pages, lens=ints)
    with pytest.raises(w4.W4A4Error):
        w4.w4a4_kv_attend(cache=cache, **good, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
