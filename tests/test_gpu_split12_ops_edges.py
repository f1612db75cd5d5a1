"""wc12_linear_adapters and wc12_moe where their kernels change their way: each
kind of codebook, exceptions that crowd one lane's values, rows of nothing but
exceptions, infinite weights, long rows, many experts.  Definitions and
tolerances are those of test_gpu_split12_ops.py."""
import numpy as np
import pytest
import torch

from test_gpu_split12_ops import adapters_case, adapters_exact, bf16, f64, gamma, moe_exact, wc  # noqa: F401

pytestmark = pytest.mark.gpu


def with_highs(rng, highs, n):
    """n bf16 values (bits) whose high bytes are drawn from `highs`."""
    return (rng.choice(np.asarray(highs, np.uint16), n) << 8 | rng.integers(0, 256, n).astype(np.uint16)).astype(np.uint16)


def tensor(bits, *shape):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).view(*shape)


def book_of(cont):
    head = cont[:80].cpu().numpy()
    return int(head[7]), list(head[64:80])


RUN = list(range(0x38, 0x40))
BOOKS = {
    "runs": RUN + [h | 0x80 for h in RUN],                                       # two runs of 8: put together by arithmetic
    "runs_from_zero": list(range(8)) + [h | 0x80 for h in range(8)],             # zeros and subnormals among them
    "one_sign": RUN,                                                             # fewer than 16 entries
    "uneven": RUN + [0x37] + [h | 0x80 for h in RUN[:7]],                        # 9 and 7
    "gaps": [0x30, 0x32, 0x34, 0x36, 0x38, 0x39, 0x3A, 0x3B] + [h | 0x80 for h in RUN],
}


@pytest.mark.parametrize("book", BOOKS)
@pytest.mark.parametrize("rare", [0, 3])
def test_codebooks(wc, book, rare):  # noqa: F811
    """Every kind of codebook, without exceptions and with a few."""
    rng = np.random.default_rng(len(book) + rare)
    N, K, M = 128, 512, 5
    bits = with_highs(rng, BOOKS[book], N * K)
    if rare:
        at = rng.choice(N * K, rare, replace=False)
        bits[at] = with_highs(rng, [0x41, 0xC1, 0x20], rare)
    w = tensor(bits, N, K)
    cont = wc.split12_encode(w.cuda())
    kk, entries = book_of(cont)
    if not rare:
        assert sorted(entries[:kk]) == sorted(BOOKS[book])
    _w, x, ad, a, b, s = adapters_case(rng, M, N, K, 2, 8)
    y, bound = adapters_exact(w, x, ad, a, b, s)
    got = wc.split12_linear_adapters(cont, N, K, x.cuda(), ad.cuda(), a.cuda(), b.cuda(), s.cuda())
    assert bool(((f64(got.cpu()) - y).abs() <= bound).all())
    gu, dn = tensor(bits[:2 * 128 * 64 * 2], 2, 128, 128), tensor(bits[:2 * 128 * 64], 2, 128, 64)
    x, l = bf16(rng, 3, 128), torch.from_numpy(rng.standard_normal((3, 2)).astype(np.float32))
    got = wc.split12_moe(wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda()), 2, 128, 64, x.cuda(), l.cuda(), 2, dtype=torch.float32)
    want, bound = moe_exact(gu, dn, x, l, 2, True, torch.float32)
    # a result below fp32's smallest number (2^-149) is lost whole: with highs
    # from 0 on |g|, |u| and |D| are under 2^-104 (128 values under 2^-111), so
    # that g u is; what is lost of h reaches the output times 2 * 64 * |D| < 1
    bound = bound + 2.0 ** -149
    assert bool(((f64(got.cpu()) - want).abs() <= bound).all())


@pytest.mark.parametrize("run", [1, 2, 3, 4, 5, 16, 17, 64, 1000])
@pytest.mark.parametrize("M", [3, 12])
def test_exceptions_in_a_row(wc, M, run):  # noqa: F811
    """A run of exceptions in successive values: one, two and more for the
    same lane, as many as its queue holds and more; at the ends of units and
    chunks too."""
    rng = np.random.default_rng(run + M)
    N, K = 256, 1088
    bits = with_highs(rng, BOOKS["runs"], N * K)
    for at in (0, 5, 63, 64, 127, K - 3, 65536 - 2, 100 * K + 200, N * K - run):
        bits[at:at + run] = with_highs(rng, [0x40, 0xC0, 0x10, 0x90], len(bits[at:at + run]))
    w = tensor(bits, N, K)
    cont = wc.split12_encode(w.cuda())
    _w, x, ad, a, b, s = adapters_case(rng, M, N, K, 3, 16)
    y, bound = adapters_exact(w, x, ad, a, b, s)
    got = wc.split12_linear_adapters(cont, N, K, x.cuda(), ad.cuda(), a.cuda(), b.cuda(), s.cuda())
    assert bool(((f64(got.cpu()) - y).abs() <= bound).all())
    E, H, F = 2, 64, 320
    gu, dn = tensor(bits[:E * 2 * F * H], E, 2 * F, H), tensor(bits[7:7 + E * H * F], E, H, F)
    x, l = bf16(rng, M, H), torch.from_numpy(rng.standard_normal((M, E)).astype(np.float32))
    got = wc.split12_moe(wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda()), E, H, F, x.cuda(), l.cuda(), 2, dtype=torch.float32)
    want, bound = moe_exact(gu, dn, x, l, 2, True, torch.float32)
    assert bool(((f64(got.cpu()) - want).abs() <= bound).all())


@pytest.mark.parametrize("M", [2, 16, 20])
def test_rows_of_exceptions_and_infinite_weights(wc, M):  # noqa: F811
    """Rows of zeros that the codebook does not hold give zeros exactly; an
    infinite weight reaches its row only."""
    rng = np.random.default_rng(M)
    N, K = 128, 512
    bits = with_highs(rng, BOOKS["runs"], N * K).reshape(N, K)
    bits[5] = 0
    bits[77, ::2] = 0x8000
    bits[77, 1::2] = 0
    bits[30, 100] = 0x7F80
    bits[31, 100] = 0x7FC1
    w = tensor(bits.reshape(-1), N, K)
    cont = wc.split12_encode(w.cuda())
    x, ad = bf16(rng, M, K), torch.full((M,), -1, dtype=torch.int32)
    x[:, 100] = 1.0
    _w, _x, _ad, a, b, s = adapters_case(rng, M, N, K, 2, 8)
    got = wc.split12_linear_adapters(cont, N, K, x.cuda(), ad.cuda(), a.cuda(), b.cuda(), s.cuda()).cpu()
    assert bool((got[:, 5] == 0).all()) and bool((got[:, 77] == 0).all())
    assert bool(torch.isinf(got[:, 30]).all()) and bool(torch.isnan(got[:, 31]).all())
    rest = [i for i in range(N) if i not in (30, 31)]
    xd, wd = f64(x), f64(w[rest])
    assert bool(((f64(got[:, rest]) - xd @ wd.T).abs() <= gamma(K + 2) * (xd.abs() @ wd.abs().T)).all())


@pytest.mark.parametrize("M,N,K,r", [(1, 1024, 14336, 16), (7, 128, 65536, 8), (16, 2048, 2048, 64), (513, 256, 512, 16), (1100, 128, 192, 24)])
def test_adapters_long(wc, M, N, K, r):  # noqa: F811
    """Long rows, more row blocks than run at once, several slices of tokens;
    the definition computed on the device in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    w = (0.02 * torch.randn(N, K, generator=g, device="cuda")).bfloat16()
    w[0, :3] = 100.0
    x, a = torch.randn(M, K, generator=g, device="cuda").bfloat16(), (torch.randn(5, r, K, generator=g, device="cuda") * K ** -0.5).bfloat16()
    b, s = (0.1 * torch.randn(5, N, r, generator=g, device="cuda")).bfloat16(), torch.rand(5, generator=g, device="cuda") + 0.5
    ad = torch.randint(-1, 5, (M,), generator=g, device="cuda").int()
    cont = wc.split12_encode(w)
    got = f64(wc.split12_linear_adapters(cont, N, K, x, ad, a, b, s))
    xd = f64(x)
    y, size = xd @ f64(w).T, xd.abs() @ f64(w).abs().T
    for l in range(5):
        m = ad == l
        y[m] += f64(s[l]) * ((xd[m] @ f64(a[l]).T) @ f64(b[l]).T)
        size[m] += f64(s[l]) * ((xd[m].abs() @ f64(a[l]).abs().T) @ f64(b[l]).abs().T)
    assert bool(((got - y).abs() <= gamma(K + K // 64 + 3 * r + 2) * size).all())


@pytest.mark.parametrize("T,E,H,F,k", [(20, 40, 2048, 768, 4), (32, 40, 64, 1024, 8), (3, 6, 4096, 192, 2), (1, 64, 1024, 640, 8)])
def test_moe_many_jobs(wc, T, E, H, F, k):  # noqa: F811
    """More (expert, rows) jobs than CTAs that run at once, and few that are
    split; long and short rows of H; every row of the experts its own scale."""
    g = torch.Generator(device="cuda").manual_seed(T + E)
    gu = (0.02 * torch.randn(E, 2 * F, H, generator=g, device="cuda")).bfloat16()
    dn = (0.02 * torch.randn(E, H, F, generator=g, device="cuda")).bfloat16()
    x, l = torch.randn(T, H, generator=g, device="cuda").bfloat16(), torch.randn(T, E, generator=g, device="cuda")
    cg, cd = wc.split12_encode(gu), wc.split12_encode(dn)
    got = wc.split12_moe(cg, cd, E, H, F, x, l, k, dtype=torch.float32)
    used = torch.unique(torch.topk(l, k, dim=1).indices)
    remap = torch.full((E,), -1)
    remap[used.cpu()] = torch.arange(used.numel())
    want, bound = moe_exact(gu[used].cpu(), dn[used].cpu(), x.cpu(), l[:, used].cpu(), k, True, torch.float32)
    assert bool(((f64(got.cpu()) - want).abs() <= bound).all())
