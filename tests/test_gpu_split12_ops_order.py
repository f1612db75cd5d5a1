"""What may run beside what in wc12_moe: the edges of a captured call's graph.
The down product reads the route before it waits for the up product, so that
the up product must not begin before the route is finished."""
import ctypes

import numpy as np
import pytest
import torch

from test_gpu_split12_ops import moe_case, status_word, wc  # noqa: F401

pytestmark = pytest.mark.gpu

FULL, PROGRAMMATIC = 0, 1  # CUgraphDependencyType


class EdgeData(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte), ("reserved", ctypes.c_ubyte * 5)]


def edges(graph):
    """(from, to, type) of the edges of a captured graph."""
    cu = ctypes.CDLL("libcuda.so.1")
    g, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetEdges_v2(g, None, None, None, ctypes.byref(n)) == 0
    a, b, d = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (EdgeData * n.value)()
    assert cu.cuGraphGetEdges_v2(g, a, b, d, ctypes.byref(n)) == 0
    return [(a[i], b[i], d[i].type) for i in range(n.value)]


def chain(edge_list):
    """The types of the edges of a graph that is one chain, in order."""
    after = {a: (b, t) for a, b, t in edge_list}
    assert len(after) == len(edge_list)
    at, types = (set(after) - {b for b, _t in after.values()}).pop(), []
    while at in after:
        at, t = after[at]
        types.append(t)
    return types


@pytest.mark.parametrize("T,slices", [(3, 1), (40, 2)])
def test_up_product_begins_after_the_route(wc, T, slices):  # noqa: F811
    E, H, F, k = 4, 128, 64, 2
    gu, dn, x, logits = moe_case(np.random.default_rng(T), T, E, H, F)
    cg, cd, x, logits, st = wc.split12_encode(gu.cuda()), wc.split12_encode(dn.cuda()), x.cuda(), logits.cuda(), status_word()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        out = wc.split12_moe(cg, cd, E, H, F, x, logits, k, status=st)
    types = chain(edges(g))
    # route, up, down of each slice of 32 tokens
    assert len(types) == 3 * slices - 1
    for i in range(slices):
        assert types[3 * i:3 * i + 2] == [FULL, PROGRAMMATIC]
        if i:
            assert types[3 * i - 1] == FULL
    del out
