"""wc12_linear_adapters and wc12_moe with infinite values, one input at a time:
infinities and NaN come out where the definition in 64 bits has them, with its
sign, and everything else is as near as ever.  Definitions and tolerances are
those of test_gpu_split12_ops.py."""
import numpy as np
import pytest
import torch

from test_gpu_split12_ops import adapters_case, adapters_exact, f64, wc  # noqa: F401

pytestmark = pytest.mark.gpu

INF = float("inf")


def check_like(got, want, bound):
    """NaN and infinities in the same places, the rest within the bound."""
    got = f64(got.cpu())
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.where(torch.isinf(got), got, 0.0), torch.where(torch.isinf(want), want, 0.0))
    ok = torch.isfinite(want)
    assert bool(((got - want).abs()[ok] <= bound[ok]).all())
    return want


def adapters(wc, w, x, ad, a, b, s):  # noqa: F811
    N, K = w.shape
    got = wc.split12_linear_adapters(wc.split12_encode(w.cuda()), N, K, x.cuda(), ad.cuda(), a.cuda(), b.cuda(), s.cuda())
    return check_like(got, *adapters_exact(w, x, ad, a, b, s))


@pytest.mark.parametrize("M", [4, 16, 17, 40])
@pytest.mark.parametrize("r", [8, 16])
def test_infinite_a(wc, M, r):  # noqa: F811
    """An infinite value of A makes its adapter's sums infinite, and so the
    rows of the tokens that have it."""
    w, x, ad, a, b, s = adapters_case(np.random.default_rng(M + r), M, 128, 256, 3, r)
    ad = torch.from_numpy((np.arange(M) % 4 - 1).astype(np.int32))
    a[1, 3, 5], a[2, 7, 100] = INF, -INF
    assert bool((b != 0).all()) and bool((x != 0).all())
    want = adapters(wc, w, x, ad, a, b, s)
    assert torch.equal(torch.isinf(want), (ad >= 1).unsqueeze(1).expand(M, 128))


@pytest.mark.parametrize("M", [4, 40])
def test_infinite_scale(wc, M):  # noqa: F811
    w, x, ad, a, b, s = adapters_case(np.random.default_rng(M), M, 128, 128, 2, 8)
    s[1] = INF
    ad = torch.from_numpy((np.arange(M) % 3 - 1).astype(np.int32))
    b[1] = b[1].abs() + 0.01
    # one sign for each token's sums, so that infinite parts agree
    a[1] = a[1][0]
    assert bool(torch.isinf(adapters(wc, w, x, ad, a, b, s)[ad == 1]).all())


@pytest.mark.parametrize("M", [4, 16, 17, 40])
@pytest.mark.parametrize("r", [8, 24])
def test_infinite_b(wc, M, r):  # noqa: F811
    """An infinite value of B makes its row's outputs infinite, with the sign
    of the sum that it meets, though that is held in parts of which some are
    zero and some have the other sign; so with a sum of a power of two."""
    w, x, ad, a, b, s = adapters_case(np.random.default_rng(M + r), M, 128, 256, 3, r)
    ad = torch.from_numpy((np.arange(M) % 4 - 1).astype(np.int32))
    b[1, 77, 2], b[2, 0, r - 1], b[2, 127, 0] = INF, -INF, INF
    s[2], x[:, 9] = 1.0, 2.0
    a[2, 0], a[2, 0, 9] = 0.0, 0.5  # the first sum of adapter 2 is 1 exactly
    want = adapters(wc, w, x, ad, a, b, s)
    assert torch.equal(torch.isinf(want[:, 77]), ad == 1)
    assert torch.equal(want[:, 127] == INF, ad == 2) and torch.equal(torch.isinf(want[:, 0]), ad == 2)
    b[1, 77, 2] = float("nan")
    want = adapters(wc, w, x, ad, a, b, s)
    assert torch.equal(torch.isnan(want[:, 77]), ad == 1)
