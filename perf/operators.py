"""Cases of the operators that work on Split12 weights next to the linear
layer: the embedding lookup, the linear layer with low-rank adapters, and the
mixture-of-experts layer.

A case is a dict of plain values; prepare() makes its inputs on the GPU from
a seed, run() makes one pass (in elementary torch operations, or with `own`
through the library) and exact() gives the same outputs in 64 bits.  The
weights are drawn as the 8B-shaped workload draws them (0.015 x Student-t
with 4 degrees of freedom, bf16) and are given both as bf16 tensors, which
the plain form works on, and as the Split12 container of the same bits.
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one request decoding: the first operation of a step, latency counts
        {"name": "embed_one_token", "op": "embed", "tokens": 1, "V": 151936, "K": 1024, "scale": 1.0},
        # a decode batch of an odd number of requests
        {"name": "embed_decode_batch", "op": "embed", "tokens": 61, "V": 151936, "K": 1024, "scale": 1.0},
        # a prefill of many tokens, rows scaled by sqrt(K)
        {"name": "embed_prefill", "op": "embed", "tokens": 8192, "V": 32000, "K": 4096, "scale": 64.0},
        # one request with an adapter, an attention projection
        {"name": "adapters_one_token", "op": "adapters", "tokens": 1, "requests": 1, "N": 4096, "K": 4096, "rank": 16, "adapters": 4},
        # down projection, a few requests of a small rank
        {"name": "adapters_7_down", "op": "adapters", "tokens": 7, "requests": 7, "N": 4096, "K": 14336, "rank": 8, "adapters": 8},
        # gate projection, a decode batch whose requests all have their own adapters
        {"name": "adapters_16_gate", "op": "adapters", "tokens": 16, "requests": 16, "N": 14336, "K": 4096, "rank": 16, "adapters": 32},
        # a few short prompts together, a large rank, an odd number of tokens
        {"name": "adapters_203_ragged", "op": "adapters", "tokens": 203, "requests": 5, "N": 4096, "K": 4096, "rank": 64, "adapters": 8},
        # a prefill batch of ragged prompts
        {"name": "adapters_2048_prefill", "op": "adapters", "tokens": 2048, "requests": 9, "N": 14336, "K": 4096, "rank": 32, "adapters": 16},
        # one request decoding through many small experts
        {"name": "moe_one_token", "op": "moe", "tokens": 1, "experts": 64, "k": 8, "H": 2048, "F": 768, "renormalize": True},
        # few large experts, an odd number of requests
        {"name": "moe_5_large", "op": "moe", "tokens": 5, "experts": 8, "k": 2, "H": 4096, "F": 1792, "renormalize": True},
        # weights of the softmax over all experts, not renormalised
        {"name": "moe_16_narrow", "op": "moe", "tokens": 16, "experts": 32, "k": 4, "H": 1024, "F": 1408, "renormalize": False},
        # a decode batch that reaches most of many experts
        {"name": "moe_32_wide", "op": "moe", "tokens": 32, "experts": 128, "k": 8, "H": 2048, "F": 768, "renormalize": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "adapters", "adapters", "moe", "moe"])
    if op == "embed":
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "V": _log_int(rng, 1000, 32000), "K": 8 * _log_int(rng, 8, 512),
                "scale": rng.choice([1.0, rng.uniform(0.1, 64.0)])}
    if op == "adapters":
        tokens = _log_int(rng, 1, 2048)
        # a decode batch has a token of each request, a prefill batch many
        requests = tokens if tokens <= 32 and rng.random() < 0.7 else rng.randint(1, min(tokens, 16))
        return {"op": op, "tokens": tokens, "requests": requests, "N": 128 * _log_int(rng, 1, 104), "K": 64 * _log_int(rng, 2, 64),
                "rank": 8 * rng.randint(1, 8), "adapters": rng.randint(1, 16)}
    experts = rng.choice([4, 8, 16, 24, 32, 48, 64, 96, 128])
    H, F = 64 * _log_int(rng, 4, 32), 64 * _log_int(rng, 2, 12)
    return {"op": op, "tokens": _log_int(rng, 1, 32), "experts": experts, "k": rng.randint(1, min(8, experts)), "H": H, "F": F,
            "renormalize": rng.random() < 0.7}


# ---------------------------------------------------------------------------
# inputs

_SLICE = 1 << 26  # values handled at a time


def _weights(gen, *shape):
    """0.015 x Student-t with 4 degrees of freedom, in bf16: Z / sqrt(G / 2),
    G ~ Gamma(2, 1) as the sum of two exponentials."""
    n = math.prod(shape)
    w = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    for i in range(0, n, _SLICE):
        m = min(_SLICE, n - i)
        z = torch.randn(m, generator=gen, device="cuda")
        u = torch.rand(m, generator=gen, device="cuda") * torch.rand(m, generator=gen, device="cuda")
        w[i:i + m] = 0.015 * z * torch.rsqrt(-0.5 * torch.log(u.clamp_min(1e-30)).clamp_max(-1e-6))
    return w.view(shape)


def _container(w):
    """The Split12 container of a bf16 tensor (an even number of values)."""
    b = w.reshape(-1).view(torch.uint8).view(-1, 2)
    n = b.shape[0]
    hist = torch.zeros(256, dtype=torch.int64, device="cuda")
    for i in range(0, n, _SLICE):
        hist += torch.bincount(b[i:i + _SLICE, 1].int(), minlength=256)
    kk = min(16, int((hist > 0).sum()))
    # the most frequent high bytes, ties to the smaller byte, ascending
    rank = hist * 256 + (255 - torch.arange(256, device="cuda"))
    book = torch.sort(torch.topk(rank, kk).indices).values
    lut = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    lut[book] = torch.arange(kk, dtype=torch.uint8, device="cuda")
    nc = -(-n // 65536)
    r16 = lambda v: -(-v // 16) * 16  # noqa: E731
    off_idx = r16(80 + 8 * (nc + 1))
    off_lo = r16(off_idx + (n + 1) // 2)
    off_exc = r16(off_lo + n)
    idx, where = torch.empty(n // 2, dtype=torch.uint8, device="cuda"), []
    for i in range(0, n, _SLICE):
        q = lut[b[i:i + _SLICE, 1].int()]
        miss = q == 255
        where.append(miss.nonzero().view(-1) + i)
        q = q.masked_fill(miss, 0).view(-1, 2)
        idx[i // 2:i // 2 + q.shape[0]] = q[:, 0] | (q[:, 1] << 4)
    pos = torch.cat(where)
    ne = pos.numel()
    total = off_exc + r16(2 * ne) + r16(ne)
    out = torch.zeros(total, dtype=torch.uint8, device="cuda")

    def put(at, t):
        raw = t.contiguous().view(torch.uint8).view(-1)
        out[at:at + raw.numel()] = raw

    put(0, torch.tensor([0x43323157, 1 | (1 << 16) | (kk << 24)], dtype=torch.int64, device="cuda").int())
    put(8, torch.tensor([n, 65536 | (nc << 32), ne, off_idx, off_lo, off_exc, total], dtype=torch.int64, device="cuda"))
    put(64, book.to(torch.uint8))
    put(80, torch.searchsorted(pos, torch.arange(nc + 1, device="cuda") * 65536))
    put(off_idx, idx)
    put(off_lo, b[:, 0])
    if ne:
        put(off_exc, ((pos << 48) >> 48).to(torch.int16))  # the low 16 bits
        put(off_exc + r16(2 * ne), b[pos, 1])
    return out


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    T = case["tokens"]
    s = {"case": case}
    if case["op"] == "embed":
        s["w"] = _weights(gen, case["V"], case["K"])
        s["ids"] = torch.randint(0, case["V"], (T,), generator=gen, device="cuda")
    elif case["op"] == "adapters":
        N, K, r, L = case["N"], case["K"], case["rank"], case["adapters"]
        s["w"] = _weights(gen, N, K)
        s["x"] = normal(T, K).bfloat16()
        s["a"] = (normal(L, r, K) / math.sqrt(K)).bfloat16()
        s["b"] = (0.02 * normal(L, N, r)).bfloat16()
        s["scales"] = 0.5 + 1.5 * torch.rand(L, generator=gen, device="cuda")
        # ragged requests one after another; one in eight has no adapter
        cuts = torch.sort(torch.randperm(T - 1, generator=gen, device="cuda")[:case["requests"] - 1] + 1).values if T > 1 else \
            torch.zeros(0, dtype=torch.int64, device="cuda")
        of = torch.randint(0, L, (case["requests"],), generator=gen, device="cuda")
        of = torch.where(torch.rand(case["requests"], generator=gen, device="cuda") < 0.125, -1, of)
        s["adapter"] = of[torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)].int()
    else:
        E, H, F = case["experts"], case["H"], case["F"]
        s["gate_up"] = _weights(gen, E, 2 * F, H)
        s["down"] = _weights(gen, E, H, F)
        s["x"] = normal(T, H).bfloat16()
        s["logits"] = 1.5 * normal(T, E)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    for name in ("w", "gate_up", "down"):
        if name in s:
            s[name + "12"] = _container(s[name])
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        from fp32_weight_compression_b200 import wc
        if case["op"] == "adapters":  # built once per weight, kept beside the container
            s["plan"] = wc.split12_plan(s["w12"], case["N"], case["K"])
    return s


# ---------------------------------------------------------------------------
# one pass

def _embed(s):
    return (s["w"][s["ids"]].float() * s["case"]["scale"]).bfloat16()


def _adapters(s):
    c = s["case"]
    x = s["x"].float()
    y = x @ s["w"].float().T
    # every adapter's products, those of a token's own adapter kept and scaled
    t = (x @ s["a"].float().view(-1, c["K"]).T).view(c["tokens"], c["adapters"], c["rank"])
    mine = s["adapter"].view(-1, 1) == torch.arange(c["adapters"], device="cuda")
    t = torch.where(mine.unsqueeze(2), t * s["scales"].view(1, -1, 1), 0.0)
    return y + t.reshape(c["tokens"], -1) @ s["b"].float().permute(0, 2, 1).reshape(-1, c["N"])


def _moe(s):
    c = s["case"]
    order = torch.sort(s["logits"], dim=1, descending=True, stable=True)  # ties to the lower expert
    top, ids = order.values[:, :c["k"]], order.indices[:, :c["k"]]
    p = torch.softmax(top if c["renormalize"] else s["logits"], dim=1)
    weight = torch.zeros_like(s["logits"]).scatter_(1, ids, p if c["renormalize"] else p.gather(1, ids))
    # the experts that some token chose
    act = torch.unique(ids)
    x = s["x"].float()
    gu = x @ s["gate_up"][act].float().view(-1, c["H"]).T
    g, u = gu.view(c["tokens"], act.numel(), 2, c["F"]).unbind(2)
    h = g / (1.0 + torch.exp(-g)) * u * weight[:, act].unsqueeze(2)
    return torch.bmm(h.transpose(0, 1), s["down"][act].float().transpose(1, 2)).sum(0).bfloat16()


def run(s):
    c = s["case"]
    if not own:
        return {"embed": _embed, "adapters": _adapters, "moe": _moe}[c["op"]](s)
    from fp32_weight_compression_b200 import wc
    if c["op"] == "embed":
        return wc.split12_embed(s["w12"], c["V"], c["K"], s["ids"], scale=c["scale"], status=s["status"])
    if c["op"] == "adapters":
        return wc.split12_linear_adapters(s["w12"], c["N"], c["K"], s["x"], s["adapter"], s["a"], s["b"], s["scales"],
                                          plan=s["plan"], status=s["status"])
    return wc.split12_moe(s["gate_up12"], s["down12"], c["experts"], c["H"], c["F"], s["x"], s["logits"], c["k"],
                          renormalize=c["renormalize"], status=s["status"])


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    T = case["tokens"]
    if case["op"] == "embed":
        return {"bytes": T * (8 + 3.5 * case["K"]), "flops": T * case["K"]}
    if case["op"] == "adapters":
        N, K, r = case["N"], case["K"], case["rank"]
        used = min(case["adapters"], case["requests"])  # at most; requests may share one
        return {"bytes": 1.5 * N * K + 2 * T * K + 4 * T * N + 2 * used * r * (N + K),
                "flops": 2.0 * T * N * K + 2.0 * T * r * (N + K)}
    E, H, F, k = case["experts"], case["H"], case["F"], case["k"]
    active = E * (1 - (1 - k / E) ** T)  # experts that some token chooses, on average
    return {"bytes": 1.5 * 3 * active * F * H + 4 * T * H + 4 * T * E, "flops": 2.0 * T * k * 3 * F * H}


# ---------------------------------------------------------------------------
# the definition in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "embed":
        # from the container: codebook entry by nibble, exceptions by position
        c, V, K = _container(s["w"]), case["V"], case["K"]
        n, chunks, ne, off_idx, off_lo, off_exc, _ = c[8:64].view(torch.int64).tolist()
        nc = chunks >> 32
        f = s["ids"].view(-1, 1) * K + torch.arange(K, device="cuda")
        nib = (c[off_idx + f // 2].long() >> (4 * (f % 2))) & 15
        high = c[64:80].long()[nib]
        if ne:
            counts = c[80:80 + 8 * (nc + 1)].view(torch.int64).diff()
            at = torch.repeat_interleave(torch.arange(nc, device="cuda"), counts) * 65536 + \
                (c[off_exc:off_exc + 2 * ne].view(torch.int16).long() & 0xFFFF)
            place = torch.searchsorted(at, f).clamp_max(ne - 1)
            high = torch.where(at[place] == f, c[off_exc + -(-2 * ne // 16) * 16 + place].long(), high)
        bits = (high << 8) | c[off_lo + f].long()
        sign, e, m = bits >> 15, (bits >> 7) & 255, bits & 127
        mag = torch.where(e > 0, torch.ldexp((128 + m).double(), (e - 134).double()), torch.ldexp(m.double(), torch.full_like(m, -133).double()))
        return torch.where(sign > 0, -mag, mag) * case["scale"]
    x = s["x"].double()
    if case["op"] == "adapters":
        y = x @ s["w"].double().T
        for l in range(case["adapters"]):
            rows = (s["adapter"] == l).nonzero().view(-1)
            if rows.numel():
                y[rows] += s["scales"][l].double() * ((x[rows] @ s["a"][l].double().T) @ s["b"][l].double().T)
        return y
    out = torch.zeros(case["tokens"], case["H"], dtype=torch.float64, device="cuda")
    F = case["F"]
    for t in range(case["tokens"]):
        l = s["logits"][t].double()
        chosen = torch.sort(l, descending=True, stable=True).indices[:case["k"]]
        p = torch.exp(l - l.max())
        p = p / (p[chosen].sum() if case["renormalize"] else p.sum())
        gu = (s["gate_up"][chosen].double() @ x[t])
        g, u = gu[:, :F], gu[:, F:]
        h = g * torch.sigmoid(g) * u * p[chosen].unsqueeze(1)
        out[t] = (s["down"][chosen].double() @ h.unsqueeze(2)).sum(0).view(-1)
    return out
