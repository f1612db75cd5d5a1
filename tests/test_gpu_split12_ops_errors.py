"""A launch that fails is reported once, by the call that made it: the calls
after it work.  The failure is the host's alone: while a stream that waits for
the default stream is being captured, nothing may be launched into that one."""
import ctypes

import numpy as np
import pytest
import torch

from test_gpu_split12_ops import adapters_case, moe_case, status_word, wc  # noqa: F401

pytestmark = pytest.mark.gpu


class Capture:
    """A capture under way on a blocking stream of the driver's."""

    def __enter__(self):
        self.cu, self.stream = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p()
        assert self.cu.cuStreamCreate(ctypes.byref(self.stream), 0) == 0
        assert self.cu.cuStreamBeginCapture_v2(self.stream, 0) == 0

    def __exit__(self, *_):
        graph = ctypes.c_void_p()
        self.cu.cuStreamEndCapture(self.stream, ctypes.byref(graph))
        assert self.cu.cuStreamDestroy_v2(self.stream) == 0


def calls(wc):  # noqa: F811
    """Each operator's call on the stream given (0: the default stream), and
    what it holds."""
    lib, rng = wc.load(), np.random.default_rng(1)
    keep, made = [], {}

    def dev(*tensors):
        keep.extend(t.cuda() for t in tensors)
        return [t.data_ptr() for t in keep[-len(tensors):]]

    N, K, r, L = 128, 128, 8, 2
    for M in (3, 20):
        w, x, ad, a, b, s = adapters_case(rng, M, N, K, L, r)
        cont = wc.split12_encode(w.cuda())
        size = lib.wc12_linear_adapters_work_bytes(M, r)
        y, work, st = torch.empty(M, N, device="cuda"), torch.empty(size, dtype=torch.uint8, device="cuda"), status_word()
        keep += [cont, y, work, st]
        args = dev(x, ad, a, b, s)
        made[f"adapters {M}"] = lambda q, c=cont, y=y, wk=work, st=st, M=M, g=args, size=size: lib.wc12_linear_adapters(
            c.data_ptr(), c.numel(), None, 0, N, K, g[0], M, *g[1:], L, r, y.data_ptr(), wk.data_ptr(), size, st.data_ptr(), q)
        made[f"linear {M}"] = lambda q, c=cont, y=y, st=st, M=M, g=args: lib.wc12_linear(
            c.data_ptr(), c.numel(), N, K, g[0], M, y.data_ptr(), st.data_ptr(), q)
    E, H, F, T, k = 2, 64, 64, 3, 1
    gu, dn, x, logits = moe_case(rng, T, E, H, F)
    cg, cd, size = wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda()), lib.wc12_moe_work_bytes(T, k, F)
    out, work, st = torch.empty(T, H, device="cuda"), torch.empty(size, dtype=torch.uint8, device="cuda"), status_word()
    xd, ld = dev(x, logits)
    keep += [cg, cd, out, work, st]
    made["moe"] = lambda q: lib.wc12_moe(cg.data_ptr(), cg.numel(), cd.data_ptr(), cd.numel(), E, H, F, xd, ld, T, k, 1,
                                         out.data_ptr(), wc.FP32, work.data_ptr(), size, st.data_ptr(), q)
    ids = torch.zeros(2, dtype=torch.int64, device="cuda")
    rows = torch.empty(2, H, dtype=torch.bfloat16, device="cuda")
    keep += [ids, rows]
    made["embed"] = lambda q: lib.wc12_embed(cd.data_ptr(), cd.numel(), E * F, H, ids.data_ptr(), 8, 2, 1.0, rows.data_ptr(), wc.BF16,
                                             st.data_ptr(), q)
    return made, keep


def test_a_failed_launch_is_reported_once(wc):  # noqa: F811
    made, keep = calls(wc)
    stream = torch.cuda.current_stream().cuda_stream
    for call in made.values():
        assert call(stream) == wc.OK  # set up, outside of any capture
    torch.cuda.synchronize()
    for name, call in made.items():
        with Capture():
            assert call(None) == wc.ERR_CUDA, name
        for after, other in made.items():
            assert other(stream) == wc.OK, (name, after)
        torch.cuda.synchronize()
    del keep
