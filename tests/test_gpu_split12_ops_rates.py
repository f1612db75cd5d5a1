"""wc12_linear_adapters and wc12_moe with so many exceptions that the lanes'
queues are filled more than once on the way, or do not hold those of two units.
Definitions and tolerances are those of test_gpu_split12_ops.py."""
import numpy as np
import pytest
import torch

from test_gpu_split12_ops import adapters_exact, bf16, f64, moe_exact, wc  # noqa: F401

pytestmark = pytest.mark.gpu


def weights(rng, *shape, rate, scale):
    """bf16 normal weights, a share of them with a high byte of one of 90 binades"""
    w = (scale * rng.standard_normal(shape)).astype(np.float32)
    rare = rng.random(shape) < rate
    w[rare] = np.exp2(-20 - 90 * rng.random(int(rare.sum()))).astype(np.float32)
    return torch.from_numpy(w).bfloat16()


@pytest.mark.parametrize("rate", [0.005, 0.02, 0.08, 0.3])
@pytest.mark.parametrize("M,K", [(5, 4096), (16, 4032), (1, 16448)])
def test_adapters_rates(wc, M, K, rate):  # noqa: F811
    N, L, r = 128, 2, 8
    rng = np.random.default_rng(int(1000 * rate) + M)
    w = weights(rng, N, K, rate=rate, scale=0.02)
    x, a, b = bf16(rng, M, K), bf16(rng, L, r, K, scale=K ** -0.5), bf16(rng, L, N, r, scale=0.1)
    s, ad = torch.tensor([0.75, 1.5]), torch.arange(M, dtype=torch.int32) % 3 - 1
    cont = wc.split12_encode(w.cuda())
    args = [t.cuda() for t in (x, ad, a, b, s)]
    y = wc.split12_linear_adapters(cont, N, K, *args)
    assert torch.equal(y.view(torch.int32), wc.split12_linear_adapters(cont, N, K, *args).view(torch.int32))
    want, bound = adapters_exact(w, x, ad, a, b, s)
    assert bool(((f64(y.cpu()) - want).abs() <= bound).all())


def test_adapters_crowded_places(wc):  # noqa: F811
    """Ranges of K with nothing but exceptions in rows with none elsewhere: a
    filling that ends before, in and after them."""
    N, K, M, L, r = 128, 4096, 9, 1, 8
    rng = np.random.default_rng(11)
    w = weights(rng, N, K, rate=0.0, scale=0.02)
    dense = weights(rng, N, K, rate=1.0, scale=0.02)
    for row, k0, k1 in ((0, 0, 64), (3, 100, 400), (15, 4000, 4096), (16, 0, 4096), (40, 63, 65), (40, 1024, 1152), (77, 2048, 2049),
                        (100, 640, 768), (127, 4095, 4096)):
        w[row, k0:k1] = dense[row, k0:k1]
    x, a, b = bf16(rng, M, K), bf16(rng, L, r, K, scale=K ** -0.5), bf16(rng, L, N, r, scale=0.1)
    s, ad = torch.tensor([0.5]), torch.zeros(M, dtype=torch.int32)
    y = wc.split12_linear_adapters(wc.split12_encode(w.cuda()), N, K, *[t.cuda() for t in (x, ad, a, b, s)])
    want, bound = adapters_exact(w, x, ad, a, b, s)
    assert bool(((f64(y.cpu()) - want).abs() <= bound).all())


@pytest.mark.parametrize("rate", [0.005, 0.03, 0.3])
def test_moe_rates(wc, rate):  # noqa: F811
    T, E, H, F, k = 5, 3, 2048, 192, 2
    rng = np.random.default_rng(int(1000 * rate))
    gu, dn = weights(rng, E, 2 * F, H, rate=rate, scale=0.06), weights(rng, E, H, F, rate=rate, scale=0.06)
    x, logits = bf16(rng, T, H), torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    got = wc.split12_moe(wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda()), E, H, F, x.cuda(), logits.cuda(), k,
                         dtype=torch.float32)
    want, bound = moe_exact(gu, dn, x, logits, k, True, torch.float32)
    assert bool(((f64(got.cpu()) - want).abs() <= bound).all())
