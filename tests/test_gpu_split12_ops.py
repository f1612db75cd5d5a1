"""The operators on Split12 weights beside the linear layer, on the GPU:
wc12_embed, wc12_linear_adapters and wc12_moe through the binding, against
their definitions in 64 bits (numpy and torch on the CPU, from the bf16
weights themselves).

Tolerances, from the arithmetic.  A product of two bf16 values is exact in
fp32.  A sum of n terms added in fp32 in any order, each addition off by at
most one unit in the last place of its result (2^-23 of it, which also covers
the tensor cores' rounding toward zero), is within gamma_n sum|terms| of the
exact one, gamma_n = n u / (1 - n u), u = 2^-23.  What else is rounded is
said at each test.
"""
import numpy as np
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.fixture(scope="module")
def wc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp32_weight_compression_b200 import build
    build.build()
    from fp32_weight_compression_b200 import wc as w
    return w


def gamma(n):
    return n * U / (1 - n * U)


def weights(rng, *shape, outliers=0.0, scale=0.02):
    """bf16 weights (CPU): N(0, scale), with a fraction of values whose high
    bytes are spread over many rare ones (exceptions of the container)."""
    n = int(np.prod(shape))
    w = workloads.rne_bf16(rng.standard_normal(n).astype(np.float32) * np.float32(scale))
    if outliers:
        m = rng.random(n) < outliers
        mag = np.float32(2.0) ** rng.integers(-24, 4, int(m.sum())).astype(np.float32)
        w[m] = workloads.rne_bf16(mag * np.where(rng.random(int(m.sum())) < 0.5, -1.5, 1.5).astype(np.float32))
    return torch.from_numpy(w.view(np.int16)).view(torch.bfloat16).view(*shape)


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16()


def f64(t):
    return t.to(torch.float64)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# embedding lookup

def embed_bits(w, ids, scale, dtype):
    """The definition: the table's bits with scale 1, else the fp32 product,
    rounded to bf16 by nearest even."""
    rows = w[ids]
    if dtype == torch.float32:
        return (rows.float() * np.float32(scale)).view(torch.int32)
    if scale == 1.0:
        return rows.view(torch.int16)
    return (rows.float() * np.float32(scale)).bfloat16().view(torch.int16)


@pytest.mark.parametrize("V,K", [(5, 8), (100, 64), (77, 1000), (40, 4096), (3, 200000)])
@pytest.mark.parametrize("outliers", [0.0, 0.002, 0.3])
def test_embed(wc, V, K, outliers):
    rng = np.random.default_rng(V + K)
    w = weights(rng, V, K, outliers=outliers)
    cont = wc.split12_encode(w.cuda())
    for T, idt in ((1, torch.int64), (37, torch.int32), (64, torch.int64)):
        ids = torch.from_numpy(rng.integers(0, V, T)).to(idt)
        ids[0] = V - 1
        for scale in (1.0, 0.37, 64.0):
            for dtype in (torch.bfloat16, torch.float32):
                got = wc.split12_embed(cont, V, K, ids.cuda(), scale=scale, dtype=dtype).cpu()
                assert got.shape == (T, K) and got.dtype == dtype
                want = embed_bits(w, ids.long(), scale, dtype)
                assert torch.equal(got.view(want.dtype), want)


def test_embed_any_bits_and_shapes(wc):
    """Every kind of bit pattern (NaN payloads, infinities, subnormals) comes
    back with scale 1; ids of any shape, none, repeated, strided."""
    bits = workloads._adversarial_chunks(np.random.default_rng(3), 4)
    w = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).view(-1, 512)
    cont = wc.split12_encode(w.cuda())
    V = w.shape[0]
    ids = torch.arange(V).flip(0).repeat(2)
    got = wc.split12_embed(cont, V, 512, ids.cuda()).cpu()
    assert torch.equal(got.view(torch.int16), w[ids].view(torch.int16))
    two = ids.view(8, -1).cuda()
    got = wc.split12_embed(cont, V, 512, two.t()).cpu()
    assert torch.equal(got.view(torch.int16), w[two.t().cpu()].view(torch.int16))
    assert wc.split12_embed(cont, V, 512, ids[:0].cuda()).shape == (0, 512)


def test_embed_bad_ids(wc):
    rng = np.random.default_rng(8)
    w = weights(rng, 50, 128, outliers=0.01)
    cont = wc.split12_encode(w.cuda())
    for idt in (torch.int64, torch.int32):
        ids = torch.tensor([3, -1, 49, 50, 2 ** 31 - 1, 0], dtype=idt, device="cuda")
        with pytest.raises(wc.WCError) as ei:
            wc.split12_embed(cont, 50, 128, ids)
        assert ei.value.code == wc.ERR_INVALID_ARG
        st = status_word()
        got = wc.split12_embed(cont, 50, 128, ids, status=st).cpu()
        assert int(st) == wc.ERR_INVALID_ARG
        want = torch.zeros(6, 128, dtype=torch.bfloat16)
        for i, r in ((0, 3), (2, 49), (5, 0)):
            want[i] = w[r]
        assert torch.equal(got, want)
        with pytest.raises(wc.WCError):
            wc.check_status(st)


def damaged(wc, cont):
    """Containers that a kernel must report: header fields, exception offsets
    out of order, an exception position past its chunk."""
    n, ne, _k = wc.split12_read_header(cont[:64].cpu().numpy(), cont.numel())
    off_exc = int(cont[48:56].cpu().numpy().view("<u8")[0])
    assert ne > 0 and n < 65536
    for off, val in ((0, 0), (4, 9), (8, 1), (16, 1), (24, 0x55), (40, 1)):
        bad = cont.clone()
        bad[off] ^= val | 0x40
        yield bad
    bad = cont.clone()
    bad[88:96] = torch.from_numpy(np.array([ne + 1], "<u8").view(np.uint8)).cuda()  # exc_off[1] past the list
    yield bad
    bad = cont.clone()
    bad[off_exc:off_exc + 2] = 0xFF
    yield bad


def test_embed_corrupt(wc):
    w = weights(np.random.default_rng(4), 50, 128, outliers=0.02)
    cont = wc.split12_encode(w.cuda())
    ids = torch.arange(50, device="cuda")
    for bad in damaged(wc, cont):
        with pytest.raises(wc.WCError) as ei:
            wc.split12_embed(bad, 50, 128, ids)
        assert ei.value.code == wc.ERR_CORRUPT
    assert torch.equal(wc.split12_embed(cont, 50, 128, ids).cpu(), w)


# ---------------------------------------------------------------------------
# linear layer with adapters

def adapters_case(rng, M, N, K, L, r, outliers=0.0):
    w = weights(rng, N, K, outliers=outliers)
    x = bf16(rng, M, K)
    a, b = bf16(rng, L, r, K, scale=K ** -0.5), bf16(rng, L, N, r, scale=0.1)
    s = torch.from_numpy((0.5 + rng.random(L)).astype(np.float32))
    ad = torch.from_numpy(rng.integers(-1, L, M).astype(np.int32))
    return w, x, ad, a, b, s


def adapters_exact(w, x, ad, a, b, s):
    """(y, bound): K products and the additions of parts of K for the shared
    product; t has K products and one rounding of the scaling, the second
    product r terms (three bf16 parts each, exact together), one addition
    joins the two."""
    M, K = x.shape
    r = a.shape[1]
    xd = f64(x)
    y, size = xd @ f64(w).T, xd.abs() @ f64(w).abs().T
    for m in range(M):
        if int(ad[m]) >= 0:
            A, B, sc = f64(a[ad[m]]), f64(b[ad[m]]), float(s[ad[m]])
            y[m] += sc * (B @ (A @ xd[m]))
            size[m] += sc * (B.abs() @ (A.abs() @ xd[m].abs()))
    return y, gamma(K + K // 64 + 3 * r + 2) * size


def check_adapters(wc, rng, M, N, K, L, r, outliers=0.0, plan=False):
    w, x, ad, a, b, s = adapters_case(rng, M, N, K, L, r, outliers)
    cont = wc.split12_encode(w.cuda())
    pl = wc.split12_plan(cont, N, K) if plan else None
    got = wc.split12_linear_adapters(cont, N, K, x.cuda(), ad.cuda(), a.cuda(), b.cuda(), s.cuda(), plan=pl)
    y, bound = adapters_exact(w, x, ad, a, b, s)
    err = (f64(got.cpu()) - y).abs()
    assert bool((err <= bound).all()), (int((err > bound).sum()), float((err / bound.clamp_min(1e-300)).max()))


def test_adapters_one_small_shape_first(wc):
    check_adapters(wc, np.random.default_rng(0), 1, 128, 64, 1, 8)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 33, 64, 130, 256, 300])
@pytest.mark.parametrize("N,K,L,r", [(128, 64, 1, 8), (256, 192, 3, 16), (128, 4096, 20, 24), (384, 1088, 2, 256)])
def test_adapters(wc, M, N, K, L, r):
    check_adapters(wc, np.random.default_rng(M + N + K + r), M, N, K, L, r, plan=M % 2 == 1)


@pytest.mark.parametrize("outliers", [0.002, 0.05, 0.3])
@pytest.mark.parametrize("M", [1, 12, 40])
def test_adapters_exceptions(wc, M, outliers):
    """A few exceptions a warp, a full list, and more than a list holds."""
    for N, K in ((128, 128), (256, 4096), (128, 1088)):
        check_adapters(wc, np.random.default_rng(M + N + K), M, N, K, 4, 16, outliers=outliers)


@pytest.mark.parametrize("M", [5, 16, 90])
def test_adapters_none_and_one(wc, M):
    """No token with an adapter: the shared product alone; all with the same."""
    rng = np.random.default_rng(M)
    w, x, ad, a, b, s = adapters_case(rng, M, 256, 512, 4, 16)
    cont = wc.split12_encode(w.cuda())
    for fill in (-1, 3):
        ad = torch.full((M,), fill, dtype=torch.int32)
        got = wc.split12_linear_adapters(cont, 256, 512, x.cuda(), ad.cuda(), a.cuda(), b.cuda(), s.cuda())
        y, bound = adapters_exact(w, x, ad, a, b, s)
        assert bool(((f64(got.cpu()) - y).abs() <= bound).all())


@pytest.mark.parametrize("M", [4, 16, 40, 70])
def test_adapters_of_others_do_not_matter(wc, M):
    """Infinities and NaN in one adapter, or in one token, stay with the
    tokens that have it."""
    rng = np.random.default_rng(M + 1)
    w, x, ad, a, b, s = adapters_case(rng, M, 128, 256, 3, 16)
    ad = torch.from_numpy((np.arange(M) % 3).astype(np.int32))
    a[1, 3, 5] = float("inf")
    b[1, :, 2] = float("nan")
    x[2, 7] = float("nan")
    cont = wc.split12_encode(w.cuda())
    got = wc.split12_linear_adapters(cont, 128, 256, x.cuda(), ad.cuda(), a.cuda(), b.cuda(), s.cuda()).cpu()
    x[2, 7] = 0
    keep = (ad == 1) | (torch.arange(M) == 2)
    assert torch.isnan(got[keep]).all()
    ad2 = torch.where(keep, -1, ad)
    y, bound = adapters_exact(w, x, ad2.int(), a, b, s)
    ok = (f64(got) - y).abs() <= bound
    assert bool(ok[~keep].all())


def test_adapters_same_bits_twice(wc):
    rng = np.random.default_rng(5)
    for M in (1, 16):
        w, x, ad, a, b, s = adapters_case(rng, M, 256, 4096, 4, 16, 0.01)
        cont = wc.split12_encode(w.cuda())
        args = [t.cuda() for t in (x, ad, a, b, s)]
        one = wc.split12_linear_adapters(cont, 256, 4096, *args)
        for _ in range(5):
            assert torch.equal(wc.split12_linear_adapters(cont, 256, 4096, *args), one)


@pytest.mark.parametrize("M", [3, 50])
def test_adapters_bad_adapter(wc, M):
    rng = np.random.default_rng(6)
    w, x, ad, a, b, s = adapters_case(rng, M, 128, 128, 2, 8)
    ad[0], ad[1], ad[2] = 2, -2, 2 ** 31 - 1
    cont = wc.split12_encode(w.cuda())
    args = [t.cuda() for t in (x, ad, a, b, s)]
    with pytest.raises(wc.WCError) as ei:
        wc.split12_linear_adapters(cont, 128, 128, *args)
    assert ei.value.code == wc.ERR_INVALID_ARG
    st = status_word()
    got = wc.split12_linear_adapters(cont, 128, 128, *args, status=st)
    assert int(st) == wc.ERR_INVALID_ARG
    ad[:3] = -1
    y, bound = adapters_exact(w, x, ad, a, b, s)
    assert bool(((f64(got.cpu()) - y).abs() <= bound).all())


def test_adapters_corrupt(wc):
    rng = np.random.default_rng(7)
    for M in (2, 20):
        w, x, ad, a, b, s = adapters_case(rng, M, 128, 64, 2, 8, 0.02)
        cont = wc.split12_encode(w.cuda())
        args = [t.cuda() for t in (x, ad, a, b, s)]
        for bad in damaged(wc, cont):
            with pytest.raises(wc.WCError) as ei:
                wc.split12_linear_adapters(bad, 128, 64, *args)
            assert ei.value.code == wc.ERR_CORRUPT
        y, bound = adapters_exact(w, x, ad, a, b, s)
        got = wc.split12_linear_adapters(cont, 128, 64, *args)
        assert bool(((f64(got.cpu()) - y).abs() <= bound).all())


# ---------------------------------------------------------------------------
# mixture of experts

def moe_case(rng, T, E, H, F, outliers=0.0):
    gu = weights(rng, E, 2 * F, H, outliers=outliers, scale=0.06)
    dn = weights(rng, E, H, F, outliers=outliers, scale=0.06)
    x = bf16(rng, T, H)
    logits = torch.from_numpy((1.5 * rng.standard_normal((T, E))).astype(np.float32))
    return gu, dn, x, logits


def moe_exact(gu, dn, x, logits, k, renormalize, dtype):
    """(out, bound).  g and u: sums of H exact products.  silu has a slope of
    at most 1.1; expf is off by 2 ulp (2^-22), the rest of silu, its product
    with u and p by 6 roundings (2^-24 each), p by two expf of arguments that
    were rounded (2^-24 of the logits' distance to the largest), a sum of at
    most E terms and a division.  The gated value enters with 2^-18, the
    second sum has F terms in two parts from each expert."""
    T, H = x.shape
    E, F = dn.shape[0], dn.shape[2]
    out = torch.zeros(T, H, dtype=torch.float64)
    bound = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        l = f64(logits[t])
        order = sorted((e for e in range(E) if l[e] != -float("inf")), key=lambda e: (-float(l[e]), e))[:k]
        if not order:
            continue
        ex = torch.exp(l - l[order[0]])
        p = ex / (ex[order].sum() if renormalize else ex[ex == ex].sum())
        far = float((l[order[0]] - l[order]).abs().max())
        d_p = 2 * (2.0 ** -22 + far * 2.0 ** -24) + (E + 2) * 2.0 ** -24
        xd = f64(x[t])
        for e in order:
            w = f64(gu[e])
            s, size = w @ xd, w.abs() @ xd.abs()
            g, u = s[:F], s[F:]
            dg, du = gamma(H + H // 64 + 4) * size[:F], gamma(H + H // 64 + 4) * size[F:]
            si = g * torch.sigmoid(g)
            h = si * u
            dh = 1.1 * dg * (u.abs() + du) + si.abs() * du + h.abs() * (2.0 ** -22 + 6 * 2.0 ** -24 + d_p + 2.0 ** -18)
            dd = f64(dn[e])
            out[t] += float(p[e]) * (dd @ h)
            bound[t] += float(p[e]) * (dd.abs() @ dh + gamma(2 * k * F + k * F // 64 + 8) * (dd.abs() @ (h.abs() + dh)))
    if dtype == torch.bfloat16:
        bound += (out.abs() + bound) * 2.0 ** -8
    return out, bound


def check_moe(wc, rng, T, E, H, F, k, renormalize=True, outliers=0.0, dtype=torch.float32, logits=None):
    gu, dn, x, l = moe_case(rng, T, E, H, F, outliers)
    if logits is not None:
        l = logits
    cg, cd = wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda())
    got = wc.split12_moe(cg, cd, E, H, F, x.cuda(), l.cuda(), k, renormalize=renormalize, dtype=dtype)
    assert got.dtype == dtype and got.shape == (T, H)
    want, bound = moe_exact(gu, dn, x, l, k, renormalize, dtype)
    err = (f64(got.cpu()) - want).abs()
    assert bool((err <= bound).all()), (int((err > bound).sum()), float((err / bound.clamp_min(1e-300)).max()))


def test_moe_one_small_shape_first(wc):
    check_moe(wc, np.random.default_rng(0), 1, 2, 64, 64, 1)


@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 16, 17, 32, 33, 70])
@pytest.mark.parametrize("E,H,F,k", [(1, 64, 64, 1), (4, 192, 128, 2), (40, 128, 192, 8), (7, 1088, 320, 3)])
def test_moe(wc, T, E, H, F, k):
    check_moe(wc, np.random.default_rng(T + E + H), T, E, H, F, k, renormalize=T % 3 != 0,
              dtype=torch.bfloat16 if T % 2 else torch.float32)


@pytest.mark.parametrize("E,k", [(130, 16), (512, 5), (16, 16)])
def test_moe_many_experts(wc, E, k):
    for T in (1, 31):
        check_moe(wc, np.random.default_rng(E + T), T, E, 64, 64, k, renormalize=False)


@pytest.mark.parametrize("outliers", [0.002, 0.05, 0.3])
def test_moe_exceptions(wc, outliers):
    for T, E, H, F, k in ((1, 4, 256, 128, 2), (12, 6, 2048, 192, 2), (20, 3, 128, 1088, 2)):
        check_moe(wc, np.random.default_rng(T), T, E, H, F, k, outliers=outliers)


def test_moe_ties_and_masks(wc):
    """Equal logits go to the lower expert (+0 and -0 are equal); experts at
    -inf are never chosen, though fewer than k are left; the type's lowest
    value is an ordinary logit; a row of -inf gives zeros."""
    rng = np.random.default_rng(2)
    T, E = 9, 8
    l = torch.from_numpy(rng.integers(-2, 3, (T, E)).astype(np.float32))
    l[1] = 0.0
    l[1, ::2] = -0.0
    l[2, 1:] = -float("inf")
    l[3] = -float("inf")
    l[4] = torch.finfo(torch.float32).min
    l[5, 0] = torch.finfo(torch.float32).max / 4
    l[6] = torch.finfo(torch.float32).min
    l[6, 5] = -float("inf")
    for renormalize in (True, False):
        check_moe(wc, rng, T, E, 128, 128, 3, renormalize=renormalize, logits=l)


def test_moe_bad_values_stay_with_their_tokens(wc):
    """A row with a NaN or +inf logit is NaN; infinite weights of an expert
    reach the tokens that chose it only."""
    rng = np.random.default_rng(3)
    T, E, H, F = 12, 6, 128, 128
    gu, dn, x, l = moe_case(rng, T, E, H, F)
    l[:, 5] = -20.0
    l[3, 5] = 20.0       # token 3 alone chooses expert 5
    dn[5, :, 7] = float("inf")
    gu[5, 9] = float("nan")
    l[4, 1] = float("nan")
    l[6, 2] = float("inf")
    cg, cd = wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda())
    got = wc.split12_moe(cg, cd, E, H, F, x.cuda(), l.cuda(), 2, dtype=torch.float32).cpu()
    for t in (3, 4, 6):
        assert torch.isnan(got[t]).all()
    rest = [t for t in range(T) if t not in (3, 4, 6)]
    want, bound = moe_exact(gu, dn, x[rest], l[rest], 2, True, torch.float32)
    assert bool(((f64(got[rest]) - want).abs() <= bound).all())


def test_moe_same_bits_twice_and_alone(wc):
    """The same bits every time; a token's expert sums do not depend on the
    batch beyond the order of its experts' parts."""
    rng = np.random.default_rng(4)
    gu, dn, x, l = moe_case(rng, 16, 8, 512, 256, 0.01)
    cg, cd = wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda())
    one = wc.split12_moe(cg, cd, 8, 512, 256, x.cuda(), l.cuda(), 2)
    for _ in range(5):
        assert torch.equal(wc.split12_moe(cg, cd, 8, 512, 256, x.cuda(), l.cuda(), 2), one)


def test_moe_corrupt(wc):
    rng = np.random.default_rng(5)
    gu, dn, x, l = moe_case(rng, 3, 2, 64, 64, 0.02)
    cg, cd = wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda())
    for which in (0, 1):
        for bad in damaged(wc, (cg, cd)[which]):
            pair = (bad, cd) if which == 0 else (cg, bad)
            with pytest.raises(wc.WCError) as ei:
                wc.split12_moe(*pair, 2, 64, 64, x.cuda(), l.cuda(), 2)
            assert ei.value.code == wc.ERR_CORRUPT
    assert torch.isfinite(wc.split12_moe(cg, cd, 2, 64, 64, x.cuda(), l.cuda(), 2)).all()


# ---------------------------------------------------------------------------
# streams, graphs, a run of all of them

def small_model(wc, rng):
    """An embedding, a projection with adapters, experts and a head."""
    V, H, N, E, F, L, r = 300, 256, 256, 6, 192, 3, 16
    m = {"V": V, "H": H, "N": N, "E": E, "F": F}
    m["emb"], m["proj"] = weights(rng, V, H, outliers=0.002, scale=1.0), weights(rng, N, H, outliers=0.002, scale=0.06)
    m["gu"], m["dn"] = weights(rng, E, 2 * F, N, scale=0.06), weights(rng, E, N, F, scale=0.06)
    m["head"] = weights(rng, 384, N, scale=0.06)
    m["a"], m["b"] = bf16(rng, L, r, H, scale=0.06), bf16(rng, L, N, r, scale=0.1)
    m["s"] = torch.tensor([0.5, 1.0, 2.0])
    m["router"] = torch.from_numpy((0.1 * rng.standard_normal((E, N))).astype(np.float32))
    m["c"] = {n: wc.split12_encode(m[n].cuda()) for n in ("emb", "proj", "gu", "dn", "head")}
    m["d"] = {n: m[n].cuda() for n in ("a", "b", "s", "router")}
    return m


def forward(wc, m, ids, ad, st, head=True):
    c, d = m["c"], m["d"]
    h = wc.split12_embed(c["emb"], m["V"], m["H"], ids, scale=2.0, status=st)
    y = wc.split12_linear_adapters(c["proj"], m["N"], m["H"], h, ad, d["a"], d["b"], d["s"], status=st)
    z = y.bfloat16()
    logits = y @ d["router"].T
    o = wc.split12_moe(c["gu"], c["dn"], m["E"], m["N"], m["F"], z, logits, 2, status=st)
    # the head's call waits, so that a captured run leaves it out
    return h, y, logits, o, wc.split12_linear(c["head"], 384, m["N"], o) if head else None


def test_a_run_of_them(wc):
    """Each operator of a forward pass against its definition on the values
    that the one before it gave."""
    rng = np.random.default_rng(11)
    m = small_model(wc, rng)
    for T in (1, 6, 16, 45):
        ids, ad = torch.from_numpy(rng.integers(0, m["V"], T)), torch.from_numpy(rng.integers(-1, 3, T).astype(np.int32))
        st = status_word()
        h, y, logits, o, out = forward(wc, m, ids.cuda(), ad.cuda(), st)
        wc.check_status(st)
        assert torch.equal(h.cpu().view(torch.int16), embed_bits(m["emb"], ids, 2.0, torch.bfloat16))
        want, bound = adapters_exact(m["proj"], h.cpu(), ad, m["a"], m["b"], m["s"])
        assert bool(((f64(y.cpu()) - want).abs() <= bound).all())
        want, bound = moe_exact(m["gu"], m["dn"], y.bfloat16().cpu(), logits.cpu(), 2, True, torch.bfloat16)
        assert bool(((f64(o.cpu()) - want).abs() <= bound).all())
        od = f64(o.cpu())
        want, size = od @ f64(m["head"]).T, od.abs() @ f64(m["head"]).abs().T
        assert bool(((f64(out.cpu()) - want).abs() <= gamma(m["N"] + m["N"] // 64) * size).all())


@pytest.mark.parametrize("T", [4, 40])
def test_captured_and_replayed(wc, T):
    """One graph of the run, replayed with other inputs, and two graphs in
    turn; a captured call without a status word is refused."""
    rng = np.random.default_rng(12)
    m = small_model(wc, rng)
    st = status_word()
    ids, ad = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    graphs = []
    forward(wc, m, ids, ad, st, head=False)
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = forward(wc, m, ids, ad, st, head=False)
        graphs.append((g, out))
    for i in range(4):
        ids.copy_(torch.from_numpy(rng.integers(0, m["V"], T)))
        ad.copy_(torch.from_numpy(rng.integers(-1, 3, T).astype(np.int32)))
        g, out = graphs[i % 2]
        g.replay()
        torch.cuda.synchronize()
        wc.check_status(st)
        h, y, _l, o, _ = forward(wc, m, ids, ad, st, head=False)
        assert torch.equal(out[0], h)
        want, bound = adapters_exact(m["proj"], h.cpu(), ad.cpu(), m["a"], m["b"], m["s"])
        assert bool(((f64(out[1].cpu()) - want).abs() <= bound).all())
        want, bound = moe_exact(m["gu"], m["dn"], out[1].bfloat16().cpu(), out[2].cpu(), 2, True, torch.bfloat16)
        assert bool(((f64(out[3].cpu()) - want).abs() <= bound).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(ValueError):
            wc.split12_embed(m["c"]["emb"], m["V"], m["H"], ids)
        keep = wc.split12_embed(m["c"]["emb"], m["V"], m["H"], ids, status=st)
    del keep


def test_side_streams(wc):
    """Several calls at once on streams of their own, given and current."""
    rng = np.random.default_rng(13)
    m = small_model(wc, rng)
    streams = [torch.cuda.Stream() for _ in range(3)]
    work = []
    for T in (1, 16, 30):
        work.append((torch.from_numpy(rng.integers(0, m["V"], T)).cuda(),
                     torch.from_numpy(rng.integers(-1, 3, T).astype(np.int32)).cuda()))
    want = [forward(wc, m, *w, status_word(), head=False) for w in work]
    torch.cuda.synchronize()
    got, sts = [], [status_word() for _ in work]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, w, st in zip(streams, work, sts):
            with torch.cuda.stream(s):
                got.append(forward(wc, m, *w, st, head=False))
    h2 = wc.split12_embed(m["c"]["emb"], m["V"], m["H"], work[1][0], scale=2.0, status=sts[0], stream=streams[2])
    torch.cuda.synchronize()
    assert torch.equal(h2, want[1][0])
    for st in sts:
        wc.check_status(st)
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a[0], b[0])
        if i < 2:  # up to 16 tokens: the same bits
            assert torch.equal(a[1], b[1]) and torch.equal(a[3], b[3])


def test_strided_inputs_and_given_outputs(wc):
    rng = np.random.default_rng(14)
    m = small_model(wc, rng)
    T = 6
    ad = torch.from_numpy(rng.integers(-1, 3, 2 * T).astype(np.int32)).cuda()[::2]
    wide = bf16(rng, T, 2 * m["H"]).cuda()
    x = wide[:, ::2]
    out = torch.full((T + 2, m["N"]), 7.0, device="cuda")
    y = wc.split12_linear_adapters(m["c"]["proj"], m["N"], m["H"], x, ad, m["d"]["a"], m["d"]["b"], m["d"]["s"],
                                   out=out[:T])
    assert y.data_ptr() == out.data_ptr() and bool((out[T:] == 7.0).all())
    want, bound = adapters_exact(m["proj"], x.cpu(), ad.cpu(), m["a"], m["b"], m["s"])
    assert bool(((f64(y.cpu()) - want).abs() <= bound).all())
    e = torch.full((5, m["H"]), 9.0, dtype=torch.bfloat16, device="cuda")
    wc.split12_embed(m["c"]["emb"], m["V"], m["H"], torch.arange(3, device="cuda"), out=e[:3])
    assert torch.equal(e[:3].cpu(), m["emb"][:3]) and bool((e[3:] == 9.0).all())
    o = torch.full((T + 1, m["N"]), 5.0, dtype=torch.bfloat16, device="cuda")
    l = torch.from_numpy(rng.standard_normal((T, 2 * m["E"])).astype(np.float32)).cuda()[:, ::2]
    z = y.bfloat16()
    wc.split12_moe(m["c"]["gu"], m["c"]["dn"], m["E"], m["N"], m["F"], z, l, 2, out=o[:T])
    want, bound = moe_exact(m["gu"], m["dn"], z.cpu(), l.cpu(), 2, True, torch.bfloat16)
    assert bool(((f64(o[:T].cpu()) - want).abs() <= bound).all()) and bool((o[T:] == 5.0).all())
