"""The exact cases of decode_exact.py see a result from which terms are missing, or counted
twice; mistakes are planted in the 64-bit results."""
import math

import pytest
import torch

from decode_exact import (BF16, FP16, equal_scores, equal_scores_close, needles, packed_codes, product_bound,
                          product_case, random_scores)


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("N,K,group", [(48, 65536 + 32, 32), (64, 8320, 64), (33, 1024, 128)])
def test_products_see_lost_inputs(N, K, group, dt):
    X, codes, steps, Y = product_case(8, N, K, group, dt, 1)
    W = codes.double() * steps.double().repeat_interleave(group, 1)
    for lost in (slice(K - 32, K), slice(0, 32), slice(K // 256 * 128, K // 256 * 128 + 128), slice(K // 2, K // 2 + 1)):
        part = W.clone()
        part[:, lost] = 0.0
        assert not torch.equal((X.double() @ part.T).to(dt), Y), lost
        assert not torch.equal((X.double() @ (2 * W - part).T).to(dt), Y), lost


def test_packed_codes():
    c = torch.tensor([[-8, 7, -1, 0]])
    assert packed_codes(c).tolist() == [[0x78, 0x0F]]


@pytest.mark.parametrize("K,group", [(65536 + 32, 32), (32768, 128), (4096, 64)])
def test_product_bound_is_far_below_the_result(K, group):
    """Random tokens with outliers: a lost record of 128 inputs shows in most results."""
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(K, generator=g).double(), torch.randint(-8, 8, (200, K), generator=g).double()
    x[:: K // 8] *= 30.0
    y, size = w @ x, w.abs() @ x.abs()
    tol = product_bound(size, K, group) + y.abs() * 2.0 ** -8
    lost = (w[:, 256:384] @ x[256:384]).abs()
    assert (lost > tol).double().mean() > 0.5
    assert tol.median() < 0.1 * y.abs().median()


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("n,D", [(100_003, 128), (87_936, 64), (5000, 64), (1374, 64)])
def test_equal_scores_see_lost_tokens(n, D, dt):
    V, out, lse = equal_scores(n, 2, D, dt)
    o = out.to(dt)
    assert equal_scores_close(o, torch.full((2,), lse).float(), out, lse, dt)
    for lost in (slice(0, 16), slice(n - 3, n), slice(n // 2, n // 2 + 16), slice(n // 3, n // 3 + 1)):
        for sign in (1, -1):
            left = n - sign * len(range(*lost.indices(n)))
            part = (V.double().sum(0) - sign * V[lost].double().sum(0)) / left
            assert not equal_scores_close(part.to(dt), torch.full((2,), math.log(left)).float(), out, lse, dt), lost
            if lost.stop - lost.start >= 16:       # and without the logarithm
                assert not equal_scores_close(part.to(dt), torch.full((2,), lse).float(), out, lse, dt), lost


@pytest.mark.parametrize("dt", [BF16, FP16])
def test_needles(dt):
    q, K, V, out, at = needles(4096, 2, 64, dt, 5)
    s = torch.einsum("hd,thd->ht", q.double(), K.double())
    p = torch.softmax(s, -1)
    assert torch.equal(torch.einsum("ht,thd->hd", p, V.double()).round(), out)
    assert torch.equal(out.to(dt).double(), out) and (s.sort(-1).values[:, -5] == 0).all() and len(at) == 4


@pytest.mark.parametrize("n,G,D", [(100_003, 12, 128), (40_000, 1, 64)])
def test_random_scores_bound_is_far_below_the_result(n, G, D):
    """A run of 1024 tokens missing from 10^5 shows in many elements, one of 100 in a few and in the logarithm."""
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(*s, generator=g) for s in ((1, G, D), (n, 1, D), (n, 1, D)))
    out, bound, lse, lse_bound = random_scores(q, k, v, D ** -0.5, 20)
    tol = bound + out.abs() * 2.0 ** -11
    assert tol.median() < 0.1 * out.abs().median()
    for lost, share in ((1024, 0.4), (100, 0.0)):
        left = torch.ones(n, dtype=torch.bool)
        left[5000:5000 + lost] = False
        part, _, part_lse, _ = random_scores(q, k[left], v[left], D ** -0.5, 20)
        assert ((part - out).abs() > tol).double().mean() > share
        assert ((part_lse - lse).abs() > lse_bound).all()
