"""The operators on Split12 weights with containers of more than 2^32 values:
rows, lists of exceptions and planes past every 32-bit offset.  Definitions and
tolerances are those of test_gpu_split12_ops.py, on some of the rows."""
import numpy as np
import pytest
import torch

from test_gpu_split12_ops import adapters_exact, bf16, f64, moe_exact, wc  # noqa: F401

pytestmark = pytest.mark.gpu


def normal(scale, *shape):
    """bf16 weights on the device, one in 5,000 of them with a high byte that no codebook has"""
    w = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, scale)
    flat = w.view(-1)
    flat[::5003] = 2.0 ** -40
    return w


def test_embed_large(wc):  # noqa: F811
    V, K = (1 << 20) + 37, 4104
    assert V * K > 1 << 32
    torch.manual_seed(1)
    w = normal(1.0, V, K)
    cont = wc.split12_encode(w)
    first = (1 << 32) // K
    ids = torch.tensor([0, 1, first - 1, first, first + 1, (1 << 31) // K, V - 2, V - 1, V // 3], device="cuda")
    for i in (ids, ids.int()):
        got = wc.split12_embed(cont, V, K, i)
        assert torch.equal(got.view(torch.int16), w[ids].view(torch.int16))
    got = wc.split12_embed(cont, V, K, ids, scale=3.0, dtype=torch.float32)
    assert torch.equal(got, w[ids].float() * 3.0)


@pytest.mark.parametrize("M", [5, 20])
def test_adapters_large(wc, M):  # noqa: F811
    N, K, L, r = 65536 + 128, 65536, 2, 8
    assert N * K > 1 << 32
    rng = np.random.default_rng(M)
    torch.manual_seed(2)
    w = normal(0.02, N, K)
    cont = wc.split12_encode(w)
    x, a, b = bf16(rng, M, K), bf16(rng, L, r, K), bf16(rng, L, N, r)
    s = torch.tensor([0.25, -1.5])
    ad = torch.arange(M, dtype=torch.int32) % 3 - 1
    y = wc.split12_linear_adapters(cont, N, K, x.cuda(), ad.cuda(), a.cuda(), b.cuda(), s.cuda()).cpu()
    rows = torch.cat([torch.arange(0, 20), torch.arange(32760, 32780), torch.arange(65530, 65545), torch.arange(N - 20, N)])
    some = (w[rows.cuda()].cpu(), x, ad, a, b[:, rows].contiguous())
    want, _ = adapters_exact(*some, s)
    # the bound is gamma times the sum of the terms' sizes |s x A B|, which the
    # helper adds up as s |x| |A| |B|: the same where s is not negative
    _, bound = adapters_exact(*some, s.abs())
    assert bool(((f64(y[:, rows]) - want).abs() <= bound).all())


def test_moe_large(wc):  # noqa: F811
    E, H, F, T, k = 512, 2112, 2048, 3, 2
    assert E * 2 * F * H > 1 << 32
    rng = np.random.default_rng(3)
    torch.manual_seed(3)
    gu, dn = normal(0.05, E, 2 * F, H), normal(0.05, E, H, F)
    cg, cd = wc.split12_encode(gu), wc.split12_encode(dn)
    x = bf16(rng, T, H)
    logits = torch.full((T, E), -float("inf"))
    for t, chosen in enumerate(([511, 495], [0, 511], [496, 250])):
        logits[t, chosen[0]], logits[t, chosen[1]] = 1.5, 0.75
    got = wc.split12_moe(cg, cd, E, H, F, x.cuda(), logits.cuda(), k, dtype=torch.float32).cpu()
    used = torch.tensor([0, 250, 495, 496, 511])
    want, bound = moe_exact(gu[used.cuda()].cpu(), dn[used.cuda()].cpu(), x, logits[:, used], k, True, torch.float32)
    assert bool(((f64(got) - want).abs() <= bound).all())
