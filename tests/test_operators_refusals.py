"""CPU checks of what the router, row sort, few-token expert layer and adapter calls refuse: every case returns its
status before any CUDA call."""
import pytest
import torch

import w4a4_mxfp4_quantized_b200 as mq
from w4a4_mxfp4_quantized_b200 import build as mq_build

P = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    mq_build.build()
    return mq.lib()


def caller(fn, **defaults):
    return lambda **kw: fn(*{**defaults, **kw}.values())


def test_moe_route(lib):
    f = caller(lib.macaq_moe_route, logits=P, dt=0, ld=64, T=4, E=64, k=4, scoring=0, renorm=1, scale=1.0, w=P, ids=P, off=P, row=P,
               pos=P, st=None)
    assert f(E=0) == 2 and f(E=1025, ld=1025) == 2 and f(k=0) == 2 and f(k=33) == 2 and f(E=3, k=4) == 2
    assert f(T=-1) == 2 and f(T=1 << 28) == 2 and f(ld=63) == 2
    assert f(dt=2) == 1 and f(scoring=2) == 1
    for name in ("logits", "w", "ids", "off", "row", "pos"):
        assert f(**{name: None}) == 1, name
    for name in ("w", "ids", "off", "row", "pos"):
        assert f(**{name: P + 4}) == 3, name
    assert f(logits=P + 1) == 3 and f(logits=P + 2, dt=1) == 3


def test_row_groups(lib):
    f = caller(lib.macaq_row_groups, ids=P, T=4, k=2, E=8, off=P, row=P, pos=P, st=None)
    assert f(E=0) == 2 and f(E=1025) == 2 and f(k=0) == 2 and f(T=-1) == 2 and f(T=1 << 29) == 2
    for name in ("ids", "off", "row", "pos"):
        assert f(**{name: None}) == 1, name
        assert f(**{name: P + 8}) == 3, name


def test_moe_w4a16(lib):
    f = caller(lib.macaq_moe_w4a16, X=P, T=4, K=256, w=P, k=2, off=P, E=8, row=P, pos=P, qg=P, sg=P, ig=None, b=32, I=128, qd=P, sd=P,
               idn=None, bd=32, N=256, out=P, ws=P, wsb=1 << 30, st=None)
    assert f(T=65) == 2 and f(T=-1) == 2 and f(K=192) == 2 and f(K=16512) == 2 and f(I=64) == 2 and f(I=16512) == 2 and f(N=64) == 2
    assert f(k=0) == 2 and f(k=33) == 2 and f(E=0) == 2 and f(E=1025) == 2
    assert f(b=8) == 4 and f(bd=256) == 4
    for name in ("X", "w", "off", "row", "pos", "qg", "sg", "qd", "sd", "out"):
        assert f(**{name: None}) == 1, name
    for name in ("X", "w", "off", "row", "pos", "qg", "sg", "ig", "qd", "sd", "idn", "out", "ws"):
        assert f(**{name: P + 8}) == 3, name
    need = mq.moe_w4a16_workspace_bytes(4, 2, 8, 256, 128, 256)
    assert need > 0 and f(wsb=need - 1) == 7 and f(ws=None) == 7
    assert f(T=0) == 0
    assert mq.moe_w4a16_workspace_bytes(65, 2, 8, 256, 128, 256) == 0


def test_lora_add(lib):
    f = caller(lib.macaq_lora_add, Y=P, ldy=256, out=P + 4096, ldo=256, dt=0, X=P, ldx=128, M=4, K=128, N=256, A=P, B=P, r=16, L=3,
               scale=None, off=P, row=P, ws=None, wsb=0, st=None)
    assert f(K=100) == 2 and f(N=100) == 2 and f(r=12) == 2 and f(r=0) == 2 and f(r=136) == 2 and f(L=0) == 2 and f(L=1025) == 2
    assert f(K=(1 << 24) + 8, ldx=1 << 25) == 2 and f(N=(1 << 24) + 8, ldy=1 << 25, ldo=1 << 25) == 2
    assert f(M=-1) == 2 and f(ldx=120) == 2 and f(ldx=132) == 2 and f(ldy=248) == 2 and f(ldy=260) == 2 and f(ldo=252) == 2
    assert f(out=P, ldo=512) == 2                       # in place with another stride
    assert f(dt=2) == 1
    for name in ("Y", "out", "X", "A", "B", "off"):
        assert f(**{name: None}) == 1, name
    for name in ("Y", "out", "X", "A", "B", "off", "row"):
        assert f(**{name: P + 8}) == 3, name
    assert f(scale=P + 2) == 3 and f(ws=P + 8) == 3
    assert f(M=0) == 0
    need = mq.lora_workspace_bytes(5000, 16, 3)      # many rows take a workspace
    assert need > 0 and f(M=5000) == 7 and f(M=5000, ws=P, wsb=need - 1) == 7
    assert mq.lora_workspace_bytes(5, 12, 3) == 0


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        mq.moe_route(x, 2)
    with pytest.raises(ValueError, match="CUDA"):
        mq.row_groups(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="CUDA"):
        mq.lora_add(x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        mq.moe_w4a16(x, x, x, x, x, x, x, x, x)
