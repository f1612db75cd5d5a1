"""The operators on Split12 weights have no backward pass: a call whose inputs
ask for a gradient is refused rather than answered without a graph, and the
same call without gradients gives what it always gives."""
import numpy as np
import pytest
import torch

from test_gpu_split12_ops import adapters_case, moe_case, wc  # noqa: F401

pytestmark = pytest.mark.gpu


def refused_then_same(call, tensors, which):
    want = call(*tensors)
    for i in which:
        asked = list(tensors)
        asked[i] = tensors[i].clone().requires_grad_()
        with pytest.raises(ValueError, match="no backward"):
            call(*asked)
        with torch.no_grad():
            got = call(*asked)
        assert torch.equal(got, want) and not got.requires_grad
        with torch.inference_mode():
            assert torch.equal(call(*asked), want)


def test_adapters(wc):  # noqa: F811
    N, K, M, L, r = 128, 128, 5, 2, 8
    w, *rest = adapters_case(np.random.default_rng(0), M, N, K, L, r)
    cont = wc.split12_encode(w.cuda())
    refused_then_same(lambda *t: wc.split12_linear_adapters(cont, N, K, *t), [t.cuda() for t in rest], (0, 2, 3, 4))


def test_moe(wc):  # noqa: F811
    E, H, F, T = 3, 64, 128, 5
    gu, dn, x, logits = moe_case(np.random.default_rng(1), T, E, H, F)
    cg, cd = wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda())
    refused_then_same(lambda *t: wc.split12_moe(cg, cd, E, H, F, *t, 2), [x.cuda(), logits.cuda()], (0, 1))
