"""wc12_linear_adapters and wc12_moe with infinite values, one input at a time:
infinities and NaN come out where the definition in 64 bits has them, with its
sign, and everything else is as near as ever.  Definitions and tolerances are
those of test_gpu_split12_ops.py."""
import numpy as np
import pytest
import torch

from test_gpu_split12_ops import adapters_case, adapters_exact, f64, moe_case, moe_exact, wc  # noqa: F401

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


def moe(wc, gu, dn, x, logits, k, dtype=torch.float32):  # noqa: F811
    E, H, F = dn.shape
    cg, cd = wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda())
    got = wc.split12_moe(cg, cd, E, H, F, x.cuda(), logits.cuda(), k, dtype=dtype)
    return check_like(got, *moe_exact(gu, dn, x, logits, k, True, dtype))


def chose(logits, k, e):
    return (torch.topk(logits, k, dim=1).indices == e).any(1)


@pytest.mark.parametrize("T", [1, 3, 12, 33])
@pytest.mark.parametrize("outliers", [0.0, 0.3])
def test_infinite_down(wc, T, outliers):  # noqa: F811
    """An infinite weight of an expert's down product makes its output
    infinite for the tokens that chose the expert, with the gated value's
    sign, though that enters in two parts; few exceptions, and so many that
    they are looked up."""
    E, H, F, k = 5, 128, 192, 2
    for dtype in (torch.float32, torch.bfloat16):
        gu, dn, x, logits = moe_case(np.random.default_rng(T + int(10 * outliers)), T, E, H, F, outliers)
        dn[1, 7, 9], dn[2, 100, 191], dn[3, 5, 0] = INF, -INF, float("nan")
        want = moe(wc, gu, dn, x, logits, k, dtype)
        assert torch.equal(torch.isinf(want[:, 7]), chose(logits, k, 1))
        assert torch.equal(torch.isinf(want[:, 100]), chose(logits, k, 2))
        assert torch.equal(torch.isnan(want[:, 5]), chose(logits, k, 3))


def test_infinite_down_in_the_codebook(wc):  # noqa: F811
    """The same where infinity's high byte is one of the codebook's: no
    exception says where they are."""
    T, E, H, F, k = 9, 3, 128, 64, 1
    gu, dn, x, logits = moe_case(np.random.default_rng(5), T, E, H, F)
    dn[:, :, 9] = INF
    dn[1, :, 9] = -INF
    head = wc.split12_encode(dn.cuda())[:80].cpu().numpy()
    assert {0x7F, 0xFF} & set(head[64:64 + int(head[7])].tolist())
    assert bool(torch.isinf(moe(wc, gu, dn, x, logits, k)).all())


@pytest.mark.parametrize("T", [2, 20])
def test_infinite_gate_and_up(wc, T):  # noqa: F811
    """Infinite weights of G and U: infinite gated values, and NaN where the
    gate is minus infinity, for the tokens that chose the expert."""
    E, H, F, k = 4, 64, 64, 2
    gu, dn, x, logits = moe_case(np.random.default_rng(T), T, E, H, F)
    gu[1, 3, 11] = INF       # G
    gu[2, F + 60, 0] = -INF  # U
    assert bool((dn != 0).all()) and bool((x != 0).all())
    want = moe(wc, gu, dn, x, logits, k)
    some = chose(logits, k, 1) | chose(logits, k, 2)
    assert torch.equal(~torch.isfinite(want), some.unsqueeze(1).expand(T, H))


@pytest.mark.parametrize("T", [1, 9])
def test_largest_gated_values(wc, T):  # noqa: F811
    """A gated value just below the largest fp32 number, which bf16 would
    round to infinity: (2 - 2^-9) 2^127 = 2^64 * (2 - 2^-9) 2^63, one expert.
    The outputs, 2^-20 times that, are finite."""
    E, H, F = 1, 64, 64
    gu, dn = torch.zeros(E, 2 * F, H, dtype=torch.bfloat16), torch.zeros(E, H, F, dtype=torch.bfloat16)
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = 1.0, 1.0
    gu[0, 5, 0] = 2.0 ** 64
    gu[0, F + 5, 0], gu[0, F + 5, 1] = (2 - 2.0 ** -7) * 2.0 ** 63, (2.0 ** -7 - 2.0 ** -9) * 2.0 ** 63
    dn[0, :, 5] = 2.0 ** -20
    dn[0, 1::2, 5] = -1.5 * 2.0 ** -20
    want = moe(wc, gu, dn, x, torch.zeros(T, E), 1)
    assert float(want.abs().min()) == (2 - 2.0 ** -9) * 2.0 ** 107
