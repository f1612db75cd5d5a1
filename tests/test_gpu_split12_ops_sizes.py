"""Sizes that the C calls' types do not hold are refused by the binding, not
taken as what is left of them in 32 or 64 bits; a k that no experts have is
refused before a workspace of that size is made."""
import numpy as np
import pytest
import torch

from test_gpu_split12_ops import moe_case, weights, wc  # noqa: F401

pytestmark = pytest.mark.gpu


def refused(wc, call, *args):  # noqa: F811
    with pytest.raises(wc.WCError) as ei:
        call(*args)
    assert ei.value.code == wc.ERR_INVALID_ARG


@pytest.mark.parametrize("V,K", [(9 + (1 << 64), 64), (-9, 64), (0, 64), (9, 64 + (1 << 32)), (9, 0), (9, -64)])
def test_embed(wc, V, K):  # noqa: F811
    table = wc.split12_encode(weights(np.random.default_rng(0), 9, 64).cuda())
    ids = torch.zeros(0 if K > 64 else 2, dtype=torch.int64, device="cuda")
    refused(wc, lambda: wc.split12_embed(table, V, K, ids))


@pytest.mark.parametrize("k,F", [(-1, 64), (0, 64), (4, 64), (1 << 31, 64), (2 + (1 << 32), 64), (2, 64 + (1 << 32)), (2, 0), (2, -64)])
def test_moe(wc, k, F):  # noqa: F811
    E, H, T = 3, 64, 5
    gu, dn, x, logits = moe_case(np.random.default_rng(1), T, E, H, 64)
    cg, cd = wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda())
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    refused(wc, lambda: wc.split12_moe(cg, cd, E, H, F, x.cuda(), logits.cuda(), k))
    assert torch.cuda.max_memory_allocated() - before < 1 << 20
