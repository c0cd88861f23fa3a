"""GPU tests that the backward calls take arrays that only touch, and outputs
that may be an operand, and give the same bits as with arrays far apart."""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def api():
    from grouped_gemm_router_amd import api as a
    return a


def touching(*tensors):
    """Copies of the tensors, one right behind the other in one buffer (each a
    multiple of 16 bytes)."""
    bytes_ = [t.numel() * t.element_size() for t in tensors]
    assert all(b % 16 == 0 for b in bytes_)
    store = torch.empty((sum(bytes_),), dtype=torch.uint8, device=DEV)
    out, at = [], 0
    for t, b in zip(tensors, bytes_):
        v = store[at:at + b].view(t.dtype).view(t.shape)
        v.copy_(t)
        out.append(v)
        at += b
    return out


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_combine_and_permute():
    T, k, d = 8, 2, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    d_out, Y, w = rnd(T, d).to(BF), rnd(T * k, d), rnd(T, k)
    f2r = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32)
    dY, dw = torch.empty((T * k, d), dtype=BF, device=DEV), torch.empty_like(w)
    api().moe_combine_backward(d_out, Y, f2r, w, dY, dw)
    order = touching(w, dY, Y, dw, d_out, f2r)
    w2, dY2, Y2, dw2, d_out2, f2r2 = order
    api().moe_combine_backward(d_out2, Y2, f2r2, w2, dY2, dw2)
    assert same((w2, dY2, Y2, dw2, d_out2, f2r2), (w, dY, Y, dw, d_out, f2r))
    for wide in (k, 11):  # (more entries than are summed at a time)
        f2r = torch.randperm(T * wide, generator=g, device=DEV).to(torch.int32)
        Y, w = rnd(T * wide, d), rnd(T, wide)
        dY, dw = torch.empty((T * wide, d), dtype=BF, device=DEV), torch.empty_like(w)
        api().moe_combine_backward(d_out, Y, f2r, w, dY, dw)
        dY2, into = torch.empty_like(dY), w.clone()
        api().moe_combine_backward(d_out, Y, f2r, into, dY2, into)
        assert same((dY2, into), (dY, dw))
    add, dx = rnd(T, d).to(BF), torch.empty((T, d), dtype=BF, device=DEV)
    api().moe_permute_backward(Y, f2r, dx, 11, addend=add)
    Y2, dx2, add2 = touching(Y, dx, add)
    api().moe_permute_backward(Y2, f2r, dx2, 11, addend=add2)
    api().moe_permute_backward(Y, f2r, add, 11, addend=add)
    assert same((dx2, add), (dx, dx))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N", [64, 2048])  # the latter's sums are cut: a workspace
def test_products(dt, N):
    G, rows, K = 2, 48, 64
    g = torch.Generator(device=DEV).manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(dt)  # noqa: E731
    dC, B, gate, up = rnd(rows, N), rnd(G, N, K), rnd(rows, K), rnd(rows, K)
    off = torch.tensor([0, 20, 44, 44], dtype=torch.int32, device=DEV)  # (one too many, for 16 bytes)
    a = api()
    ws = torch.empty((max(16, a.moe_grouped_gemm_dgrad_workspace_size(G, rows, N, K, dt)),),
                     dtype=torch.uint8, device=DEV)
    ws2 = torch.empty((max(16, a.moe_grouped_gemm_wgrad_workspace_size(G, rows, N, K, dt)),),
                      dtype=torch.uint8, device=DEV)
    z = torch.zeros_like
    dA, dg, du, h, dB = z(gate), z(gate), z(gate), z(gate), z(B)
    a.moe_grouped_gemm_dgrad(dC, B, dA, off[:3], dC2=dC, B2=B)
    a.moe_grouped_gemm_dgrad_swiglu(dC, B, gate, up, dg, du, off[:3], h=h)
    a.moe_grouped_gemm_wgrad(dC, gate, dB, off[:3])
    p = touching(dC, z(dA), B, ws, z(dg), gate, z(du), up, z(h), z(dB), ws2, off)
    dC2, dA2, B2, w, dg2, gate2, du2, up2, h2, dB2, w2, off2 = p
    a.moe_grouped_gemm_dgrad(dC2, B2, dA2, off2[:3], dC2=dC2, B2=B2, ws=w)
    a.moe_grouped_gemm_dgrad_swiglu(dC2, B2, gate2, up2, dg2, du2, off2[:3], h=h2, ws=w)
    a.moe_grouped_gemm_wgrad(dC2, gate2, dB2, off2[:3], ws=w2)
    assert same((dC2, dA2, B2, dg2, gate2, du2, up2, h2, dB2, off2),
                (dC, dA, B, dg, gate, du, up, h, dB, off))
    a.moe_grouped_gemm_dgrad_swiglu(dC2, B2, gate2, up2, gate2, up2, off2[:3], ws=w)
    assert same((gate2[:44], up2[:44], gate2[44:], up2[44:]),
                (dg[:44], du[:44], gate[44:], up[44:]))


def test_a_list_of_gradients():
    grads = list(torch.randn((3, 1024), device=DEV))
    a = api()
    norm = torch.empty((1,), device=DEV)
    a.moe_grad_norm(grads, norm)
    ws = torch.zeros((a.moe_grad_norm_workspace_size(3),), dtype=torch.uint8, device=DEV)
    g0, w, g1, g2 = touching(grads[0], ws, grads[1], grads[2])
    again = torch.empty((1,), device=DEV)
    a.moe_grad_norm([g0, g1, g2], again, ws=w)
    assert same((again, g0, g1, g2), (norm, *grads))
    with pytest.raises(a.MoEError):
        a.moe_grad_norm([g0, g1, w.view(F32)[5:9]], again, ws=w)
