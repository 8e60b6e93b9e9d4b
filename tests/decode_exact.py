"""Inputs of the single-token operators whose results are known exactly or within bounds
far below the results, for lengths at which a bound on sums in any order says nothing.

Both kinds are shown on the CPU to reject a result from which a run of terms is missing
(test_decode_exact.py), and are put to the kernels in test_gpu_decode_exact.py.

Sums.  Integers (times a common power of two) whose sums stay below 2^24 are added in fp32
without any rounding, in whatever order and by whichever instruction.  So with integer tokens
and steps that are powers of two, a product is the 64-bit result rounded once; with equal
scores, an attention's sums are, and the quotient is off by a division's and a product's rounding.
"""
import math

import torch

FP16, BF16 = torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- products
def product_case(M, N, K, group, dt, seed):
    """(X [M, K], codes [N, K], steps [N, K / group], Y): Y is the result, rounded once.

    Token 0 is dense, small integers of either sign and never 0, so that a lost run of inputs changes its
    sums by about the root of the run's share.  Every other token holds a single 1, at places that
    run from the first input to the last: its result is one weight, exactly.  Steps differ from
    group to group by powers of two up to 4."""
    g = gen(seed)
    codes = torch.randint(-8, 8, (N, K), generator=g)
    steps = 2.0 ** torch.randint(-6, -3, (N, K // group), generator=g).double()
    # |x| |c| / least step <= 3 * 8 * 4 = 96 units: sums below 2^24 up to 174762 inputs
    X = torch.zeros(M, K, dtype=torch.float64)
    X[0] = (torch.randint(1, 4, (K,), generator=g) * (2 * torch.randint(0, 2, (K,), generator=g) - 1)).double()
    assert 96 * K < 2 ** 24
    for m in range(1, M):
        X[m, (K - 1) * (m - 1) // max(1, M - 2) if M > 2 else K - 1] = 1.0
    W = codes.double() * steps.repeat_interleave(group, 1)
    return X.to(dt), codes, steps.to(dt), (X @ W.T).to(dt)


def packed_codes(codes):
    return ((codes[:, 0::2] & 15) | ((codes[:, 1::2] & 15) << 4)).to(torch.uint8)


def product_bound(size, K, group, sums=16):
    """Error of a product in fp32 by how it is summed: a group of inputs by the tensor core, a warp's groups one after
    the other (at least `sums` / 2 warps share the inputs of a tile evenly, up to one block of 128), then the
    warps' sums and the bias.  size: sum of the magnitudes.  2^-23: tensor cores may truncate."""
    per = 128 // group
    chain = group + (-(-K // 128) // (sums // 2) + 2) * per + sums + 2
    return chain * 2.0 ** -23 * size


# --------------------------------------------------------------- attention
def equal_scores(n, H, D, dt):
    """(V [n, H, D], out [H, D], lse) for keys of zero: token t counts in dimension (t // 8) % D of every head, twice as
    much in odd heads, so that the result is the number of tokens of each dimension over n."""
    t = torch.arange(n)
    V = torch.zeros(n, H, D, dtype=dt)
    V[t, :, (t // 8) % D] = 1.0 + (torch.arange(H) % 2).to(dt)
    return V, V.double().sum(0) / n, math.log(n)


def equal_scores_close(out, lse, want, want_lse, dt):
    """The sums are exact; 1 / sum and the product with it are rounded to fp32, the result once more.  lse: log2 off by one
    step of a value that may be 15 above the result's, then a product, whose constant is off by half a step."""
    err = (out.double().cpu() - want).abs()
    ok = torch.all(err <= want * (torch.finfo(dt).eps / 2 * (1 + 2.0 ** -11) + 3 * 2.0 ** -24))
    step = 2.0 ** (math.floor(math.log2(15 + want_lse / math.log(2.0))) - 23)
    return bool(ok) and bool(torch.all((lse.double().cpu() - want_lse).abs() <= math.log(2.0) * step + 2.0 ** -23 * want_lse + 2.0 ** -24))


def needles(n, H, D, dt, seed, tops=4):
    """(q [H, D], K, V [n, H, D], out [H, D], places [tops]): all weight lies on `tops` tokens, equally, the others
    are 2^-100 and less.  The values there are integers, the sum of `tops` a multiple of it: the result
    is exact.  Everywhere else values are large."""
    g = gen(seed)
    K, V = torch.zeros(n, H, D, dtype=dt), torch.full((n, H, D), 1000.0, dtype=dt)
    places = torch.sort(torch.randperm(n, generator=g)[:tops]).values
    tops = len(places)
    q = torch.zeros(H, D, dtype=dt)
    q[:, 0] = 16.0
    K[places, :, 0] = 16.0                         # a score of 256 against 0, in powers of two 369 (scale 1)
    part = torch.randint(-3, 4, (tops, H, D), generator=g)
    part[-1] -= part.sum(0) % tops
    V[places] = part.to(dt)
    return q, K, V, part.sum(0).double() / tops, places


def random_scores(q, k, v, scale, pieces):
    """(out, its bound, lse, its bound) in 64 bits of queries q [H, G, D] over k, v [n, H, D]; pieces: the most pieces of P
    tokens that one warp takes.  First order in w_t = p_t (1 + d_t): the error of out is sum p_t |v_t| (d_t + what the sum
    loses) + |out| (sum p_t d_t + what the total loses)."""
    H, G, D = q.shape
    P = 32 if D == 64 else 16
    q, k, v = q.double(), k.double(), v.double()
    s, size = torch.einsum("hgd,thd->hgt", q, k) * scale, torch.einsum("hgd,thd->hgt", q.abs(), k.abs()) * abs(scale)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    p = p / total
    # a score: products by 16 in the tensor core (17 terms with the sum so far, each may lose 2^-23 of it), its scaling by a
    # rounded constant, the subtraction of the reference, the power (2^-22)
    d = (D // 16 * 17 + 2) * 2.0 ** -23 * size + 2.0 ** -22 * (s.abs() + (s - m).abs() + 1)
    # a piece: P / 16 products with two terms of a weight each, or P / 4 additions; the maximum may move (a factor off
    # by 2^-22, a rounding).  Joined: at most 1776 parts, by 8 warps, 8 at a time.  Weights are held to 2^-16.
    join = 1776 // 8 * 2 + 128
    sums = (pieces * (2 * (P // 16) * 17 + 3) + join) * 2.0 ** -23 + 2.0 ** -16
    adds = (pieces * (P // 4 + 3) + join) * 2.0 ** -23
    out = torch.einsum("hgt,thd->hgd", p, v)
    mean = (p * d).sum(-1, keepdim=True)
    bound = torch.einsum("hgt,thd->hgd", p * (d + sums), v.abs()) + out.abs() * (mean + adds)
    lse = (m + torch.log(total)).squeeze(-1)
    return out, 1.01 * bound, lse, 1.01 * (mean.squeeze(-1) + adds) + 2.0 ** -22 * (17 + lse.abs() + m.squeeze(-1).abs())
