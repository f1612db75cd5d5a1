"""wc12_moe with rows that its kernels take in several parts, a filling of the
exceptions' queues each; and that ordinary exceptions in such rows cost little.
Definitions and tolerances are those of test_gpu_split12_ops.py."""
import numpy as np
import pytest
import torch

from test_gpu_split12_ops import check_moe, wc  # noqa: F401
from test_gpu_split12_ops_rates import weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("outliers", [0.0, 0.002, 0.02])
@pytest.mark.parametrize("T,E,H,F,k", [(32, 2, 16448, 320, 2), (4, 8, 64, 65536, 2), (3, 2, 8256, 8320, 1)])
def test_parts_of_rows(wc, T, E, H, F, k, outliers):  # noqa: F811
    """More jobs than CTAs that split one, so that a CTA has whole rows of H;
    items whose part of F is more than a filling; ends inside a part."""
    check_moe(wc, np.random.default_rng(H), T, E, H, F, k, outliers=outliers)


def replay_time(call):
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = float("inf")
    for _ in range(6):
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("H,F,rate", [(32768, 2048, 0.0004), (4096, 4096, 0.004)])
def test_exceptions_cost_little(wc, H, F, rate):  # noqa: F811
    """Rows whose lanes have more exceptions in all than a queue holds take at
    most three times as long as rows without any: 1.1 and 2 where they are
    taken in parts, 9 and 7 where their values are looked up."""
    T, E, k = 8, 2, 2
    rng, times = np.random.default_rng(H), []
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16().cuda()
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    for r in (0.0, rate):
        part = weights(rng, 2 * F, H, rate=r, scale=0.02).cuda()
        gu, dn = torch.stack([part, part.flip(0)]), part.view(2, H, F)
        cg, cd = wc.split12_encode(gu), wc.split12_encode(dn)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        times.append(replay_time(lambda: wc.split12_moe(cg, cd, E, H, F, x, logits, k, status=st)))
        wc.check_status(st)
    assert times[1] < 3 * times[0], times
