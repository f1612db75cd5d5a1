"""The operators on Split12 weights without a GPU: every refusal of their C
entry points comes before the device is touched, empty calls do nothing, and
the workspace sizes are what the header says; the binding's own checks."""
import pytest
import torch

W, PLAN, X, AD, A, B, S, Y, WORK, ST = (0x10000 * (i + 1) for i in range(10))  # aligned addresses, never read


@pytest.fixture(scope="module")
def wcm():
    from fp32_weight_compression_b200 import build, wc
    build.build()
    wc.load()
    return wc


def container_bytes(n):
    """Up to the end of the low plane of a container of n values."""
    r16 = lambda v: -(-v // 16) * 16  # noqa: E731
    return r16(r16(80 + 8 * (-(-n // 65536) + 1)) + (n + 1) // 2) + n


# --- wc12_embed -------------------------------------------------------------

EMBED = dict(w=W, w_bytes=container_bytes(100 * 64), V=100, K=64, ids=X, id_bytes=8, T=5, scale=1.0, out=Y, dtype=1, status=ST)


@pytest.mark.parametrize("change", [
    dict(w=None), dict(w=W + 8), dict(status=None), dict(status=ST + 2), dict(V=0), dict(K=0), dict(K=63), dict(K=60),
    dict(w_bytes=95), dict(w_bytes=EMBED["w_bytes"] - 1), dict(V=101), dict(V=1 << 45), dict(id_bytes=2), dict(id_bytes=16),
    dict(dtype=3), dict(dtype=0), dict(ids=None), dict(ids=X + 4), dict(out=None), dict(out=Y + 8), dict(T=1 << 31),
])
def test_embed_refuses(wcm, change):
    assert wcm.load().wc12_embed(*{**EMBED, **change}.values(), None) == wcm.ERR_INVALID_ARG


def test_embed_of_nothing(wcm):
    assert wcm.load().wc12_embed(*{**EMBED, "T": 0, "ids": None, "out": None}.values(), None) == wcm.OK


# --- wc12_linear_adapters ---------------------------------------------------

LINEAR = dict(w=W, w_bytes=container_bytes(256 * 128), plan=None, plan_bytes=0, N=256, K=128, x=X, M=3, adapter=AD, a=A, b=B, scale=S,
              L=2, r=16, y=Y, work=WORK, work_bytes=1 << 20, status=ST)


@pytest.mark.parametrize("change", [
    dict(w=None), dict(x=None), dict(y=None), dict(status=None), dict(w=W + 8), dict(x=X + 8), dict(y=Y + 2), dict(status=ST + 1),
    dict(N=0), dict(K=0), dict(N=192), dict(K=96), dict(M=0), dict(w_bytes=95), dict(w_bytes=LINEAR["w_bytes"] - 1),
    dict(plan=PLAN + 8, plan_bytes=1 << 20), dict(plan=PLAN, plan_bytes=32),
    dict(adapter=None), dict(a=None), dict(b=None), dict(scale=None), dict(work=None),
    dict(adapter=AD + 2), dict(a=A + 8), dict(b=B + 8), dict(scale=S + 2), dict(work=WORK + 8),
    dict(L=0), dict(L=1 << 31), dict(r=0), dict(r=4), dict(r=12), dict(r=264), dict(M=1 << 31),
    dict(K=65536 + 64, w_bytes=1 << 40), dict(N=1 << 22, w_bytes=1 << 40),
])
def test_adapters_refuse(wcm, change):
    assert wcm.load().wc12_linear_adapters(*{**LINEAR, **change}.values(), None) == wcm.ERR_INVALID_ARG


@pytest.mark.parametrize("M,r", [(1, 8), (16, 256), (17, 8), (4096, 64)])
def test_adapters_workspace(wcm, M, r):
    need = wcm.load().wc12_linear_adapters_work_bytes(M, r)
    assert need == M * r * (4 if M <= 16 else 6)
    assert wcm.load().wc12_linear_adapters(*{**LINEAR, "M": M, "r": r, "work_bytes": need - 1}.values(), None) == wcm.ERR_CAPACITY


# --- wc12_moe ----------------------------------------------------------------

E, H, F, T, K_ = 4, 128, 192, 3, 2
MOE = dict(gate_up=W, gate_up_bytes=container_bytes(E * 2 * F * H), down=PLAN, down_bytes=container_bytes(E * H * F), E=E, H=H, F=F,
           x=X, logits=A, T=T, k=K_, renormalize=1, out=Y, dtype=1, work=WORK, work_bytes=1 << 20, status=ST)


@pytest.mark.parametrize("change", [
    dict(gate_up=None), dict(down=None), dict(status=None), dict(gate_up=W + 8), dict(down=PLAN + 4), dict(status=ST + 2),
    dict(E=0), dict(E=513), dict(k=0), dict(k=17, E=32, gate_up_bytes=1 << 40, down_bytes=1 << 40), dict(k=5),
    dict(H=0), dict(F=0), dict(H=96), dict(F=96), dict(H=65536 + 64, gate_up_bytes=1 << 45, down_bytes=1 << 45),
    dict(F=65536 + 64, gate_up_bytes=1 << 45, down_bytes=1 << 45), dict(dtype=3), dict(gate_up_bytes=95), dict(down_bytes=95),
    dict(gate_up_bytes=MOE["gate_up_bytes"] - 1), dict(down_bytes=MOE["down_bytes"] - 1),
    dict(x=None), dict(logits=None), dict(out=None), dict(work=None), dict(x=X + 8), dict(logits=A + 2), dict(out=Y + 2),
    dict(work=WORK + 8),
])
def test_moe_refuses(wcm, change):
    assert wcm.load().wc12_moe(*{**MOE, **change}.values(), None) == wcm.ERR_INVALID_ARG


def test_moe_of_nothing_and_workspace(wcm):
    lib = wcm.load()
    assert lib.wc12_moe(*{**MOE, "T": 0, "x": None, "logits": None, "out": None, "work": None}.values(), None) == wcm.OK
    need = lib.wc12_moe_work_bytes(T, K_, F)
    assert need >= T * K_ * F * 4
    assert lib.wc12_moe(*{**MOE, "work_bytes": need - 1}.values(), None) == wcm.ERR_CAPACITY
    # a slice of 32 tokens at a time
    assert lib.wc12_moe_work_bytes(32, 8, 768) == lib.wc12_moe_work_bytes(1000, 8, 768)


# --- the binding's checks ----------------------------------------------------

def test_binding_checks_its_tensors(wcm):
    c = torch.zeros(4096, dtype=torch.uint8)
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a CUDA device
        wcm.split12_embed(c, 10, 64, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        wcm.split12_embed(c.float(), 10, 64, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        wcm.split12_linear_adapters(None, 128, 64, x, None, None, None, None)
    with pytest.raises(TypeError):
        wcm.split12_moe(c.view(64, 64), c, 2, 64, 64, x, torch.zeros(2, 2), 1)
