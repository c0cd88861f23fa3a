"""CPU checks of the entry points of include/moe_balance.h and
include/moe_lora.h: every declared function is exported, and bad arguments
return the documented status before anything is launched (no GPU is touched:
every call below fails validation or is a documented no-op)."""
import ctypes as C
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F32, BF16, E4M3 = 0, 1, 2
P, P2, P3 = C.c_void_p(0x10000), C.c_void_p(0x20000), C.c_void_p(0x30000)
MIS, NUL = C.c_void_p(0x10002), C.c_void_p(0)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from grouped_gemm_router_amd import api
    return api.lib


@pytest.mark.parametrize("header", ["moe_balance.h", "moe_lora.h"])
def test_every_declared_function_is_exported_and_bound(lib, header):
    from grouped_gemm_router_amd import api
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text))
    assert len(names) in (3, 4)
    for n in names:
        assert hasattr(lib, n) and n in api.EXPORTS and hasattr(api, n), n


def test_balance_loss_validation(lib):
    def f(T=16, E=8, k=2, S=1, off=NUL, mask=NUL, lg=P, idx=P, c=P, p=P, t=P, l=P, ws=P2, wsb=BIG):
        return lib.moe_balance_loss(lg, idx, off, mask, T, E, k, S, 0.01, c, p, t, l, ws, wsb, NUL)
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(S=0), dict(S=2),
                dict(lg=MIS), dict(lg=NUL), dict(idx=MIS), dict(c=NUL), dict(p=MIS), dict(t=NUL),
                dict(l=MIS), dict(off=MIS), dict(ws=NUL), dict(ws=MIS)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(E=1025), dict(E=64, k=33), dict(S=65537, off=P), dict(T=(1 << 26) + 1)):
        assert f(**bad) == UNSUPPORTED, bad
    need = lib.moe_balance_loss_workspace_size(4096, 256, 4)
    assert need > 0
    assert f(T=4096, E=256, S=4, off=P, wsb=need - 1) == WORKSPACE
    assert lib.moe_balance_loss_workspace_size(-1, 8, 1) == 0
    assert lib.moe_balance_loss_workspace_size(8, 2000, 1) == 0


def test_route_backward_validation(lib):
    def f(T=16, E=8, k=2, S=1, off=NUL, lg=P, idx=P, dw=P, flags=0, c=P, t=P, dl=P, out=P2):
        return lib.moe_route_backward(lg, idx, dw, flags, c, t, 0.01, dl, off, NUL, T, E, k, S, out,
                                      NUL)
    assert f(T=0) == OK
    assert f(T=0, dw=NUL) == OK and f(T=0, c=NUL, t=NUL, dl=NUL) == OK
    for bad in (dict(flags=2), dict(flags=4), dict(dw=NUL, flags=1),    # renorm without a gate term
                dict(dw=NUL, c=NUL, t=NUL, dl=NUL),                     # nothing to do
                dict(c=NUL), dict(t=NUL), dict(c=NUL, t=NUL),           # d_loss without the loss
                dict(out=P), dict(out=NUL), dict(out=MIS), dict(lg=MIS), dict(dw=MIS),
                dict(dl=MIS), dict(S=3), dict(k=9), dict(T=-1)):
        assert f(**bad) == INVALID, bad
    assert f(E=2000) == UNSUPPORTED


def test_lora_linear_validation(lib):
    def f(T=16, N=64, K=64, r=8, n=2, dt=BF16, ydt=BF16, x=P, W=P, ldw=0, A=P, B=P, sc=P, ad=P, y=P2,
          v=P3, ws=NUL, wsb=0):
        return lib.moe_lora_linear(x, W, ldw, A, B, dt, sc, ad, T, N, K, r, n, y, ydt, v, ws, wsb,
                                   NUL)
    assert f(T=0) == OK and f(T=0, W=NUL) == OK and f(T=0, N=7, ydt=F32) == OK
    assert f(T=0, ldw=72) == OK and f(T=0, dt=F32, ydt=F32, ldw=68) == OK
    for bad in (dict(T=-1), dict(N=0), dict(K=0), dict(r=0), dict(n=0), dict(x=NUL), dict(x=MIS),
                dict(W=MIS), dict(A=NUL), dict(B=MIS), dict(sc=NUL), dict(ad=MIS), dict(y=NUL),
                dict(v=MIS), dict(ldw=56), dict(ldw=68), dict(W=NUL, ldw=64), dict(wsb=8)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(K=60), dict(r=12), dict(r=136), dict(n=1025), dict(dt=E4M3), dict(ydt=E4M3),
                dict(dt=F32), dict(T=(1 << 24) + 1), dict(N=(1 << 20) + 1),
                dict(T=1 << 24, N=1 << 13)):
        assert f(**bad) == UNSUPPORTED, bad
    big = dict(T=4000, N=4096, K=4096)
    need = lib.moe_lora_linear_workspace_size(4000, 4096, 4096, 8, 2, BF16)
    assert need > 0 and f(**big, ws=P, wsb=need - 1) == WORKSPACE
    assert f(**big, ws=MIS, wsb=need) == INVALID


def test_lora_backward_validation(lib):
    def f(T=16, N=64, K=64, r=8, n=2, dt=BF16, dy=P, x=P, W=P, ldw=0, A=P, B=P, sc=P, ad=P, v=P, u=P,
          dx=P, dA=P, dB=P, ws=P, wsb=BIG):
        return lib.moe_lora_linear_backward(dy, x, W, ldw, A, B, dt, sc, ad, v, T, N, K, r, n, u, dx,
                                            dA, dB, ws, wsb, NUL)
    assert f(T=0, dA=NUL, dB=NUL, x=NUL, v=NUL) == OK
    for bad in (dict(dA=NUL), dict(dB=NUL), dict(dx=NUL), dict(dx=NUL, W=NUL, dA=NUL, dB=NUL),
                dict(dy=MIS), dict(x=NUL), dict(v=NUL), dict(u=NUL), dict(dx=MIS), dict(ws=NUL),
                dict(ws=MIS), dict(ldw=56), dict(W=NUL, ldw=64), dict(r=-8)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(N=60), dict(K=60), dict(r=4), dict(dt=E4M3)):
        assert f(**bad) == UNSUPPORTED, bad
    need = lib.moe_lora_backward_workspace_size(1000, 64, 64, 8, 2, BF16)
    assert need > 0 and f(T=1000, wsb=need - 1) == WORKSPACE
    assert lib.moe_lora_backward_workspace_size(1000, 60, 64, 8, 2, BF16) == 0
    assert lib.moe_lora_linear_workspace_size(-1, 64, 64, 8, 2, BF16) == 0


def test_binding_refuses_host_tensors():
    """No call reaches the library with memory that a GPU cannot read."""
    from grouped_gemm_router_amd import api
    z = torch.zeros
    with pytest.raises(ValueError, match="GPU"):
        api.moe_balance_loss(z(4, 8), z(4, 2, dtype=torch.int32), z(1, 8), z(1, 8), z(2), z(1))
    with pytest.raises(ValueError, match="GPU"):
        api.moe_route_backward(z(4, 8), z(4, 2, dtype=torch.int32), z(4, 8))
    with pytest.raises(ValueError, match="GPU"):
        api.moe_lora_linear(z(4, 8), z(2, 8, 8), z(2, 8, 16), z(2), z(4, dtype=torch.int32),
                            z(4, 16), z(4, 8))
    with pytest.raises(ValueError, match="GPU"):
        api.moe_lora_linear_backward(z(4, 16), z(4, 8), z(2, 8, 8), z(2, 8, 16), z(2),
                                     z(4, dtype=torch.int32), z(4, 8), z(4, 8))


def test_lora_outputs_on_inputs_are_refused(lib):
    """y over x is allowed only where the projection is not computed here, dx
    never over dy or x."""
    def f(x, y, W):
        return lib.moe_lora_linear(x, W, 0, P, P, BF16, P, P, 16, 64, 64, 8, 2, y, BF16, P3, NUL, 0,
                                   NUL)
    assert f(P, P, P) == INVALID

    def b(dy, x, dx):
        return lib.moe_lora_linear_backward(dy, x, P, 0, P, P, BF16, P, P, P, 16, 64, 64, 8, 2, P, dx,
                                            NUL, NUL, P, BIG, NUL)
    assert b(P, P2, P) == INVALID and b(P, P2, P2) == INVALID
