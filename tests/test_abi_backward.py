"""CPU checks of the entry points of include/moe_backward.h: every declared
function is exported, and bad arguments return the documented status before
anything is launched (no GPU is touched: every call below fails validation or
is a documented no-op)."""
import ctypes as C
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F32, BF16, E4M3 = 0, 1, 2
P, P2, P3, P4, P5, P6 = (C.c_void_p(0x10000 * i) for i in range(1, 7))
MIS, NUL = C.c_void_p(0x10002), C.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    from grouped_gemm_router_amd import api
    return api.lib


def test_every_declared_function_is_exported_and_bound(lib):
    from grouped_gemm_router_amd import api
    text = open(os.path.join(ROOT, "include", "moe_backward.h")).read()
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert len(names) == 10
    for n in names:
        assert hasattr(lib, n) and n in api.EXPORTS and hasattr(api, n), n


def test_combine_backward_validation(lib):
    def f(T=4, k=2, d=64, ns=0, g=P, dt=BF16, y=P2, ydt=F32, f2r=P3, w=P4, dY=P5, dw=P6):
        return lib.moe_combine_backward(g, dt, y, ydt, f2r, w, T, k, d, ns, dY, dw, NUL)
    assert f(T=0) == OK and f(T=0, g=NUL, y=NUL) == OK
    for bad in (dict(T=-1), dict(k=0), dict(d=0), dict(ns=-1), dict(g=NUL), dict(g=MIS),
                dict(y=NUL), dict(y=MIS), dict(f2r=NUL), dict(w=MIS), dict(dY=MIS), dict(dw=MIS),
                dict(dY=NUL, dw=NUL, y=NUL), dict(dw=NUL), dict(dY=P), dict(dY=P2)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(k=33), dict(ns=9), dict(d=60), dict(dt=E4M3), dict(ydt=E4M3),
                dict(T=1 << 24)):
        assert f(**bad) == UNSUPPORTED, bad


def test_permute_backward_validation(lib):
    def f(T=4, k=2, d=64, ns=0, p=P, pdt=F32, f2r=P2, add=NUL, dx=P3, dt=BF16):
        return lib.moe_permute_backward(p, pdt, f2r, T, k, d, ns, add, dx, dt, NUL)
    assert f(T=0) == OK
    for bad in (dict(T=-1), dict(k=0), dict(ns=-1), dict(p=NUL), dict(p=MIS), dict(f2r=MIS),
                dict(add=MIS), dict(dx=NUL), dict(dx=MIS), dict(dx=P)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(k=33), dict(ns=9), dict(d=12), dict(dt=E4M3), dict(pdt=E4M3)):
        assert f(**bad) == UNSUPPORTED, bad


def test_dgrad_validation(lib):
    def f(G=2, rows=16, N=64, K=64, ldb=0, dC=P, B=P2, dC2=NUL, B2=NUL, dt=BF16, dA=P3, adt=BF16,
          off=P4, ws=NUL, wsb=0):
        return lib.moe_grouped_gemm_dgrad(dC, B, dC2, B2, dt, dA, adt, off, G, rows, N, K, ldb, ws,
                                          wsb, NUL)
    assert f(rows=0) == OK and f(rows=0, ldb=72) == OK and f(rows=0, adt=F32) == OK
    for bad in (dict(G=0), dict(rows=-1), dict(N=0), dict(K=0), dict(ldb=56), dict(ldb=68),
                dict(dC=NUL), dict(B=MIS), dict(dC2=P5), dict(B2=P5), dict(dC2=MIS, B2=P5),
                dict(dA=NUL), dict(dA=P), dict(dA=P5, dC2=P5, B2=P6), dict(off=MIS),
                dict(ws=NUL, wsb=16), dict(ws=MIS, wsb=1 << 40)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(G=1041), dict(N=60), dict(K=60), dict(dt=E4M3), dict(adt=E4M3),
                dict(dt=F32, adt=BF16), dict(N=1 << 24, K=1 << 20),
                dict(rows=1 << 30, K=1 << 16), dict(N=1 << 23, K=8), dict(K=8, ldb=1 << 23)):
        assert f(**bad) == UNSUPPORTED, bad
    size = lib.moe_grouped_gemm_dgrad_workspace_size  # few tiles, long sums: slices
    need = size(2, 16, 4096, 64, BF16)
    assert need >= 2 * 16 * 64 * 4 and size(2, 16, 4096, 64, F32) > 0
    assert size(8, 8192, 4096, 14336, BF16) == 0 == size(0, 16, 4096, 64, BF16)
    assert size(2, 16, 4096, 60, BF16) == 0
    assert f(N=4096, ws=P5, wsb=need - 1) == WORKSPACE and f(N=4096) == WORKSPACE
    assert f(N=4096, ws=MIS, wsb=need) == INVALID


def test_dgrad_swiglu_validation(lib):
    def f(rows=16, N=64, K=64, dC=P, B=P2, dt=BF16, gate=P3, up=P4, dg=P5, du=P6, h=NUL, off=P2):
        return lib.moe_grouped_gemm_dgrad_swiglu(dC, B, dt, gate, up, dg, du, h, off, 2, rows, N, K,
                                                 0, NUL, 0, NUL)
    assert f(rows=0) == OK
    for bad in (dict(dC=NUL), dict(B=NUL), dict(gate=MIS), dict(up=NUL), dict(dg=MIS), dict(du=NUL),
                dict(h=MIS), dict(off=NUL), dict(dg=P), dict(du=P), dict(dg=P6), dict(dg=P4),
                dict(du=P3), dict(h=P), dict(h=P3), dict(h=P4), dict(h=P5), dict(h=P6)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(dt=E4M3), dict(N=4), dict(K=4)):
        assert f(**bad) == UNSUPPORTED, bad


def test_wgrad_validation(lib):
    def f(G=2, rows=16, N=64, K=64, dC=P, A=P2, dt=BF16, dB=P3, bdt=BF16, off=P4, acc=0, ws=None,
          wsb=None):
        need = lib.moe_grouped_gemm_wgrad_workspace_size(G, rows, N, K, dt)
        ws = (P5 if need else NUL) if ws is None else ws
        return lib.moe_grouped_gemm_wgrad(dC, A, dt, dB, bdt, off, G, rows, N, K, acc, ws,
                                          need if wsb is None else wsb, NUL)
    assert f(rows=0, acc=1) == OK and f(rows=0, acc=1, dC=NUL, A=NUL) == OK
    for bad in (dict(G=0), dict(rows=-1), dict(N=0), dict(K=-8), dict(dC=NUL), dict(A=MIS),
                dict(dB=NUL), dict(dB=P), dict(dB=P2), dict(off=NUL)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(G=2000), dict(N=60), dict(K=60), dict(dt=E4M3), dict(bdt=E4M3),
                dict(dt=F32, bdt=BF16), dict(N=1 << 20, K=1 << 20), dict(N=1 << 23, K=8)):
        assert f(**bad) == UNSUPPORTED, bad
    need = lib.moe_grouped_gemm_wgrad_workspace_size(1, 4096, 64, 64, BF16)
    assert need >= 2 * 64 * 64 * 4
    assert f(G=1, rows=4096, ws=P5, wsb=need - 1) == WORKSPACE
    assert lib.moe_grouped_gemm_wgrad_workspace_size(8, 8192, 14336, 4096, BF16) == 0
    assert lib.moe_grouped_gemm_wgrad_workspace_size(0, 1, 8, 8, BF16) == 0
    assert lib.moe_grouped_gemm_wgrad_workspace_size(1, 1, 9, 8, BF16) == 0


def lists(*tensors):
    n = len(tensors)
    return ((C.c_void_p * n)(*[t[0] for t in tensors]), (C.c_int64 * n)(*[t[1] for t in tensors]),
            (C.c_int * n)(*[t[2] for t in tensors]), n)


def test_grad_norm_and_clip_validation(lib):
    def norm(*t, out=P, ws=P2, wsb=1 << 30):
        return lib.moe_grad_norm(*lists(*t), out, ws, wsb, NUL)

    def clip(*t, nrm=P, top=1.0, out=None):
        o = None if out is None else (C.c_void_p * len(out))(*out)
        return lib.moe_grad_clip(*lists(*t), nrm, top, o, NUL)

    good = (0x10000, 8, F32)
    for f in (norm, clip):
        for t, want in (((0, 8, F32), INVALID), ((0x10002, 8, F32), INVALID),
                        ((0x10001, 8, BF16), INVALID), ((0x10000, -1, F32), INVALID),
                        ((0x10000, 8, E4M3), UNSUPPORTED), ((0x10000, 1 << 40, F32), UNSUPPORTED)):
            assert f(good, t) == want, t
    assert norm(good, out=MIS) == INVALID and norm(good, out=NUL) == INVALID
    assert norm(good, ws=C.c_void_p(0x10004)) == INVALID and norm(good, ws=NUL) == INVALID
    need = lib.moe_grad_norm_workspace_size(1)
    assert need > 0 and norm(good, wsb=need - 1) == WORKSPACE
    assert lib.moe_grad_norm_workspace_size(-1) == 0 == lib.moe_grad_norm_workspace_size(1 << 20)
    assert lib.moe_grad_norm_workspace_size(0) == 0
    assert lib.moe_grad_norm(None, None, None, 1, P, P2, 1 << 30, NUL) == INVALID
    assert lib.moe_grad_norm(None, None, None, -1, P, P2, 1 << 30, NUL) == INVALID
    assert lib.moe_grad_norm(None, None, None, 1 << 17, P, P2, 1 << 30, NUL) == UNSUPPORTED
    for bad in (dict(nrm=NUL), dict(nrm=MIS), dict(top=-1.0), dict(top=float("nan")),
                dict(top=float("inf")), dict(out=[0]), dict(out=[0x10002])):
        assert clip(good, **bad) == INVALID, bad
    assert clip() == OK and clip((0, 0, F32)) == OK  # nothing to scale


@pytest.mark.parametrize("n", [0, 300])  # the ranges of few and of many tensors
def test_grad_clip_refuses_outputs_that_overlap(lib, n):
    """Refused before anything is launched: each call here overlaps once."""
    rest = [(0x100000 + 64 * ((i * 7) % 300), 16, F32) for i in range(n)]
    norm = 0x9000

    def clip(t, out=None, nrm=norm):
        t = rest + t
        o = None if out is None else (C.c_void_p * len(t))(*([r[0] for r in rest] + out))
        return lib.moe_grad_clip(*lists(*t), C.c_void_p(nrm), 1.0, o, NUL)

    a, b = (0x10000, 8, F32), (0x20000, 8, F32)
    assert clip([a, b, a]) == INVALID                       # the same one twice
    assert clip([a, (0x1001C, 8, F32)]) == INVALID          # its last value
    assert clip([(0x1001C, 8, F32), a]) == INVALID
    assert clip([(0x10000, 64, F32), (0x10010, 2, BF16), b]) == INVALID  # one inside another
    assert clip([a, b], nrm=0x1001C) == INVALID             # the norm
    assert clip([a, b], [0x30000, 0x30010]) == INVALID      # two outputs
    assert clip([a, b], [0x10004, 0x20000]) == INVALID      # its own gradient in part
    assert clip([a, b], [0x20000, 0x10000]) == INVALID      # each other's gradient
    assert clip([a, b], [0x30000, 0x10010]) == INVALID
    assert clip([a, a], [0x30000, 0x10000]) == INVALID      # read for one, written by the other


def test_binding_refuses_host_tensors():
    """No call reaches the library with memory that a GPU cannot read."""
    from grouped_gemm_router_amd import api
    z, i32 = torch.zeros, torch.int32
    for call in (lambda: api.moe_combine_backward(z(2, 8), z(2, 8), z(2, dtype=i32), z(2, 1),
                                                  z(2, 8), z(2, 1)),
                 lambda: api.moe_permute_backward(z(2, 8), z(2, dtype=i32), z(2, 8), 1),
                 lambda: api.moe_grouped_gemm_dgrad(z(2, 8), z(1, 8, 8), z(2, 8), z(2, dtype=i32)),
                 lambda: api.moe_grouped_gemm_dgrad_swiglu(z(2, 8), z(1, 8, 8), z(2, 8), z(2, 8),
                                                           z(2, 8), z(2, 8), z(2, dtype=i32)),
                 lambda: api.moe_grouped_gemm_wgrad(z(2, 8), z(2, 8), z(1, 8, 8), z(2, dtype=i32)),
                 lambda: api.moe_grad_norm([z(3)], z(1)),
                 lambda: api.moe_grad_clip([z(3)], z(1), 1.0)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_the_binding_checks_what_it_passes_on(monkeypatch):
    """Shapes, types and devices, with the library's calls left out."""
    from grouped_gemm_router_amd import api
    monkeypatch.setattr(api, "_gpu", lambda t, name: -1)  # (host tensors report -1)
    monkeypatch.setattr(api, "_raw_stream", lambda s, d: 0)
    z, bf, i32 = torch.zeros, torch.bfloat16, torch.int32
    off = z(3, dtype=i32)
    with pytest.raises(ValueError, match="together"):
        api.moe_combine_backward(z(2, 8), None, z(2, dtype=i32), z(2, 1), z(2, 8), z(2, 1))
    with pytest.raises(ValueError, match="dY"):
        api.moe_combine_backward(z(2, 8), z(2, 8), z(2, dtype=i32), z(2, 1), z(3, 8), z(2, 1))
    with pytest.raises(TypeError, match="addend"):
        api.moe_permute_backward(z(2, 8), z(2, dtype=i32), z(2, 8), 1, addend=z(2, 8, dtype=bf))
    with pytest.raises(ValueError, match="B must have 8 rows"):
        api.moe_grouped_gemm_dgrad(z(4, 8), z(2, 16, 8), z(4, 8), off)
    with pytest.raises(TypeError, match="B must be"):
        api.moe_grouped_gemm_dgrad(z(4, 8), z(2, 8, 8, dtype=bf), z(4, 8), off)
    with pytest.raises(ValueError, match="B2"):
        api.moe_grouped_gemm_dgrad(z(4, 8), z(2, 8, 8), z(4, 8), off, dC2=z(4, 8), B2=z(2, 8, 16))
    with pytest.raises(TypeError, match="dA"):
        api.moe_grouped_gemm_dgrad(z(4, 8), z(2, 8, 8), z(4, 8, dtype=bf), off)
    with pytest.raises(ValueError, match="offsets"):
        api.moe_grouped_gemm_dgrad(z(4, 8), z(2, 8, 8), z(4, 8), z(2, dtype=i32))
    with pytest.raises(TypeError, match="h must"):
        api.moe_grouped_gemm_dgrad_swiglu(z(4, 8), z(2, 8, 8), *[z(4, 8)] * 4, off,
                                          h=z(4, 8, dtype=bf))
    with pytest.raises(ValueError, match="A must"):
        api.moe_grouped_gemm_wgrad(z(4, 8), z(5, 8), z(2, 8, 8), off)
    with pytest.raises(ValueError, match="contiguous"):
        api.moe_grad_norm([z(4, 8).t()], z(1), ws=z(1 << 20))
    with pytest.raises(TypeError, match="grads"):
        api.moe_grad_norm([z(4, dtype=torch.float16)], z(1), ws=z(1 << 20))
    with pytest.raises(ValueError, match="out must"):
        api.moe_grad_clip([z(4)], z(1), 1.0, out=[z(5)])


def test_an_fp8_layer_has_no_backward():
    from grouped_gemm_router_amd.layer import MoELayer
    m = MoELayer.__new__(MoELayer)
    m.fp8, m._T = True, 4
    with pytest.raises(RuntimeError, match="bf16 or fp32"):
        m.backward(torch.zeros(4, 8))
    m.fp8, m._T = False, None
    with pytest.raises(RuntimeError, match="forward pass"):
        m.backward(torch.zeros(4, 8))
    m._T, m.d, m.dff, m.G, m.n_shared, m.act_dtype = 4, 8, 8, 1, 0, torch.float32
    for bad in (torch.zeros(3, 8), torch.zeros(4, 8, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="d_out"):
            m.backward(bad)
