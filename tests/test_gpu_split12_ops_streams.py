"""Calls of the operators on a stream that is given, with a status word of the
caller's: inputs and outputs that the caller lets go of keep their memory until
the work that uses them is done."""
import numpy as np
import pytest
import torch

from test_gpu_split12_ops import bf16, status_word, weights, wc  # noqa: F401

pytestmark = pytest.mark.gpu

SLEEP = 200_000_000  # cycles: a tenth of a second


def calls(wc):  # noqa: F811
    """Of each operator: the input of 4 MiB that is let go of, the call on it,
    and what another of its size is filled with (valid for the call, so that a
    reuse of its memory would change the answer and nothing else)."""
    rng = np.random.default_rng(3)
    out = {}
    V, K = 16, 8
    table = wc.split12_encode(weights(rng, V, K).cuda())
    out["embed"] = (torch.full((1 << 19,), 3), 7, lambda t, **kw: wc.split12_embed(table, V, K, t, **kw))
    N, K2, M, r, L = 128, 4096, 512, 8, 2
    cont = wc.split12_encode(weights(rng, N, K2).cuda())
    ad, s = torch.zeros(M, dtype=torch.int32, device="cuda"), torch.ones(L, device="cuda")
    a, b = bf16(rng, L, r, K2).cuda(), bf16(rng, L, N, r).cuda()
    out["adapters"] = (bf16(rng, M, K2), 2.0, lambda t, **kw: wc.split12_linear_adapters(cont, N, K2, t, ad, a, b, s, **kw))
    E, H, F, T, k = 2, 65536, 64, 32, 1
    gu, dn = wc.split12_encode(weights(rng, E, 2 * F, H).cuda()), wc.split12_encode(weights(rng, E, H, F).cuda())
    logits = torch.zeros(T, E, device="cuda")
    out["moe"] = (bf16(rng, T, H), 2.0, lambda t, **kw: wc.split12_moe(gu, dn, E, H, F, t, logits, k, **kw))
    return out


@pytest.mark.parametrize("op", ["embed", "adapters", "moe"])
def test_inputs_are_held(wc, op):  # noqa: F811
    value, fill, call = calls(wc)[op]
    want = call(value.cuda())
    side, st = torch.cuda.Stream(), status_word()
    t = value.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    y = call(t, status=st, stream=side)
    del t
    again = [torch.full_like(value, fill, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    wc.check_status(st)
    size = want.abs().max()  # sums beyond 16 tokens are added in any order
    assert bool(((y - want).abs() <= 1e-5 * size).all())
    del again


@pytest.mark.parametrize("op", ["embed", "adapters", "moe"])
def test_outputs_are_held(wc, op):  # noqa: F811
    value, _fill, call = calls(wc)[op]
    t = value.cuda()
    want = call(t)
    side, st = torch.cuda.Stream(), status_word()
    torch.cuda.synchronize()
    y = call(t, status=st, stream=side)
    side.synchronize()
    torch.cuda._sleep(SLEEP)
    copy = y.clone()
    with torch.cuda.stream(side):
        empty = torch.empty_like(y)  # before y goes: what has to be made new is
        del y
        again = [torch.full_like(empty, 5.0) for _ in range(16)]
    torch.cuda.synchronize()
    wc.check_status(st)
    assert bool(((copy - want).abs() <= 1e-5 * want.abs().max()).all())
    del again, empty
