"""wc12_moe: what the other tokens of a batch change in a token's row is its
rounding and nothing else.  Definitions and tolerances are those of
test_gpu_split12_ops.py."""
import numpy as np
import pytest
import torch

from test_gpu_split12_ops import f64, moe_case, moe_exact, wc  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,H,F,k", [(16, 8, 512, 256, 2), (33, 20, 128, 192, 4)])
def test_alone_and_among_others(wc, T, E, H, F, k):  # noqa: F811
    """Each token in the batch, alone, and among others that were changed (other
    choices, values that are not finite): always within the definition's
    bound."""
    rng = np.random.default_rng(T)
    gu, dn, x, logits = moe_case(rng, T, E, H, F, 0.002)
    cg, cd = wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda())

    def run(x, logits):
        return f64(wc.split12_moe(cg, cd, E, H, F, x.cuda(), logits.cuda(), k, dtype=torch.float32).cpu())

    want, bound = moe_exact(gu, dn, x, logits, k, True, torch.float32)
    whole = run(x, logits)
    assert bool(((whole - want).abs() <= bound).all())
    for t in range(T):
        alone = run(x[t:t + 1], logits[t:t + 1])[0]
        assert bool(((alone - want[t]).abs() <= bound[t]).all())
        _gu, _dn, x2, logits2 = moe_case(rng, T, E, H, F)
        x2[(t + 1) % T, 3], x2[(t + 2) % T, 5], logits2[(t + 3) % T, 0] = float("inf"), float("nan"), float("nan")
        logits2[(t + 4) % T] = -float("inf")
        x2[t], logits2[t] = x[t], logits[t]
        among = run(x2, logits2)[t]
        assert bool(((among - want[t]).abs() <= bound[t]).all())
