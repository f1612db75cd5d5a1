"""Batches of no tokens, which a serving loop meets: every operator's call on
them gives an empty output and leaves the status word as it was."""
import numpy as np
import pytest
import torch

from test_gpu_split12_ops import adapters_case, moe_case, status_word, weights, wc  # noqa: F401

pytestmark = pytest.mark.gpu


def test_no_tokens(wc):  # noqa: F811
    rng, st = np.random.default_rng(0), status_word()
    V, N, K, L, r, E, F = 9, 128, 64, 2, 8, 3, 64
    table = wc.split12_encode(weights(rng, V, K).cuda())
    w, x, ad, a, b, s = adapters_case(rng, 4, N, K, L, r)
    cont = wc.split12_encode(w.cuda())
    gu, dn, xe, logits = moe_case(rng, 4, E, K, F)
    cg, cd = wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda())
    x, ad, a, b, s, xe, logits = [t.cuda() for t in (x, ad, a, b, s, xe, logits)]
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    for n in (0, 4, 0):
        for kw in ({}, {"status": st}):
            assert wc.split12_embed(table, V, K, ids[:n], **kw).shape == (n, K)
            y = wc.split12_linear_adapters(cont, N, K, x[:n], ad[:n], a, b, s, **kw)
            assert y.shape == (n, N) and y.dtype == torch.float32
            out = torch.full((5, N), 3.0, device="cuda")
            assert wc.split12_linear_adapters(cont, N, K, x[:n], ad[:n], a, b, s, plan=wc.split12_plan(cont, N, K), out=out[:n],
                                              **kw).data_ptr() == out[:n].data_ptr()
            assert bool((out[n:] == 3.0).all())
            assert wc.split12_moe(cg, cd, E, K, F, xe[:n], logits[:n], 2, **kw).shape == (n, K)
    wc.check_status(st)
