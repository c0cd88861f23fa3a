"""GPU tests of MoELayer.backward: a training step's run of operators against
autograd in 64 bits at the layer's own selection, and against differences.

Tolerances, in the 2-norm relative to the gradient's.  An fp32 layer: sums of
at most 1000 products, each within 1002 u (u = 2^-24) of the terms' sizes,
through at most four products: 1e-3 of what an elementwise bound allows is
seen in the norm, and 1e-5 is asked for.  A bf16 layer: between the loss and a
weight's gradient dY, gate, up, d_gate (or h) and the result are rounded, each
by at most 2^-8 relative; gate's error goes through SwiGLU's slope, whose
relative change is at most twice gate's: 6 x 2^-8.  x, Y and the weights are
the layer's own values.
"""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TOL = {F32: 1e-5, BF: 6 * 2.0 ** -8}


def build(T, d, dff, E, k, ns, dt, **kw):
    from grouped_gemm_router_amd.layer import MoELayer
    g = torch.Generator(device=DEV).manual_seed(T + d)
    rnd = lambda *s, std=1.0: (torch.randn(s, generator=g, device=DEV) * std).to(dt)  # noqa: E731
    G = E + ns
    w = dict(w_gate=rnd(G, dff, d, std=d ** -0.5), w_up=rnd(G, dff, d, std=d ** -0.5),
             w_down=rnd(G, d, dff, std=dff ** -0.5))
    m = MoELayer(rnd(E, d, std=0.02 * (128 / d) ** 0.5 * 4), *w.values(), k, n_shared=ns, **kw)
    return m, w, rnd(T, d), rnd(T, d, std=0.1)


def reference(m, x, p, w, idx, keep):
    """The layer's output in 64 bits at the given selection and gates."""
    y = torch.zeros(x.shape, dtype=F64, device=DEV)
    for e in range(m.G):
        if e < m.E:
            t, j = torch.nonzero((idx == e) & keep, as_tuple=True)
            gate = p[t, j][:, None]
        else:
            t, gate = torch.arange(len(x), device=DEV), 1.0
        if len(t) == 0:
            continue
        g, u = x[t] @ w["w_gate"][e].t(), x[t] @ w["w_up"][e].t()
        y = y.index_add(0, t, gate * ((g * torch.sigmoid(g) * u) @ w["w_down"][e].t()))
    return y


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


LAYERS = [(64, 128, 256, 8, 2, 0, F32, {}), (33, 64, 40, 5, 3, 1, F32, dict(capacity_factor=0.7)),
          (256, 512, 256, 16, 4, 1, BF, {}), (131, 264, 200, 6, 2, 2, BF, dict(renorm=True)),
          (96, 256, 512, 4, 2, 0, BF, dict(capacity_factor=0.5)), (1, 128, 64, 8, 2, 0, BF, {})]


@pytest.mark.parametrize("T,d,dff,E,k,ns,dt,kw", LAYERS)
def test_a_training_step(T, d, dff, E, k, ns, dt, kw):
    from grouped_gemm_router_amd import api
    m, w, x, d_out = build(T, d, dff, E, k, ns, dt, **kw)
    m(x)
    out = m.backward(d_out, grad_dtype=F32)
    keep = (m.flat_to_row[:T * k] >= 0).reshape(T, k)
    leaf = {n: t.double().requires_grad_() for n, t in w.items()}
    leaf["dx"] = x.double().requires_grad_()
    leaf["d_topk_w"] = m.topk_w.double().requires_grad_()
    y = reference(m, leaf["dx"], leaf["d_topk_w"], leaf, m.topk_idx, keep)
    grads = torch.autograd.grad((y * d_out.double()).sum(), list(leaf.values()))
    want = dict(zip(leaf, grads))
    assert set(out) == set(want)
    for n in want:
        assert out[n].shape == want[n].shape
        assert rel(out[n], want[n]) <= TOL[dt], (n, rel(out[n], want[n]))
    # the router's gradient from d_topk_w, and the norm over all of them
    d_logits = m.route_backward(out["d_topk_w"])
    lg = m.logits.double().requires_grad_()
    pr = torch.softmax(lg, 1).gather(1, m.topk_idx.long())
    if kw.get("renorm"):
        pr = pr / pr.sum(1, keepdim=True)
    r, = torch.autograd.grad((pr * out["d_topk_w"].double()).sum(), lg)
    assert rel(d_logits, r) <= 1e-5
    every = [out[n] for n in ("w_gate", "w_up", "w_down")] + [d_logits]
    norm = torch.empty((1,), device=DEV)
    api.moe_grad_norm(every, norm)
    total = torch.stack([t.double().norm() for t in every]).norm()
    assert abs(float(norm) - float(total)) <= 1e-6 * float(total)
    api.moe_grad_clip(every, norm, float(total) / 2)
    assert rel(out["w_up"], want["w_up"] / 2) <= TOL[dt] + 1e-6


def test_gradients_against_differences():
    """Central differences of the 64-bit layer along a random direction of
    each input: h^2 = 1e-6 of a smooth function's third derivative, next to
    the fp32 layer's 1e-5."""
    m, w, x, d_out = build(48, 64, 96, 4, 2, 1, F32)
    m(x)
    out = m.backward(d_out)
    vals = {n: t.double() for n, t in w.items()}
    vals["dx"], vals["d_topk_w"] = x.double(), m.topk_w.double()
    keep = torch.ones_like(m.topk_idx, dtype=torch.bool)
    g = torch.Generator(device=DEV).manual_seed(1)

    def loss(v):
        y = reference(m, v["dx"], v["d_topk_w"], v, m.topk_idx, keep)
        return float((y * d_out.double()).sum())

    for n in vals:
        v = torch.randn(vals[n].shape, generator=g, device=DEV, dtype=F64)
        v = out[n].double() / out[n].double().norm() + 0.1 * v / v.norm()
        h = 1e-3
        up, down = dict(vals), dict(vals)
        up[n], down[n] = vals[n] + h * v, vals[n] - h * v
        diff = (loss(up) - loss(down)) / (2 * h)
        assert abs(float((out[n].double() * v).sum()) - diff) <= 1e-4 * abs(diff), n


def test_micro_batches_add_up():
    """grads adds to what is there; addend reaches dx; weights=False leaves
    the weights out."""
    m, w, x, d_out = build(64, 128, 256, 8, 2, 1, BF)
    m(x)
    one = m.backward(d_out, grad_dtype=F32)
    grads = {n: one[n].clone() for n in w}
    add = torch.randn_like(x)
    two = m.backward(d_out, grads=grads, addend=add)
    for n in w:
        assert two[n] is grads[n] and torch.equal(two[n], 2 * one[n])
    assert rel(two["dx"], one["dx"].double() + add.double()) <= 2.0 ** -7
    only = m.backward(d_out, weights=False)
    assert set(only) == {"dx", "d_topk_w"} and torch.equal(only["dx"], one["dx"])


def test_a_captured_backward_pass():
    """Replays between eager steps give the eager gradients' bits."""
    m, w, x, d_out = build(128, 256, 256, 8, 2, 1, BF)
    m(x)
    want = m.backward(d_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.backward(d_out)
    for _ in range(3):
        for t in got.values():
            t.zero_()
        graph.replay()
        eager = m.backward(d_out)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]) and torch.equal(eager[n], want[n]), n


def test_another_batch_size():
    """A forward of other tokens replaces what backward works on."""
    m, w, x, d_out = build(40, 64, 128, 4, 2, 1, BF)
    m(x)
    first = {n: t.clone() for n, t in m.backward(d_out).items()}
    m(x[:7].contiguous())
    small = m.backward(d_out[:7].contiguous())
    assert small["dx"].shape == (7, 64)
    with pytest.raises(ValueError, match="d_out"):
        m.backward(d_out)
    m(x)
    again = m.backward(d_out)
    assert all(torch.equal(first[n], again[n]) for n in first)


def test_no_tokens():
    """The operators of a step take a batch of no tokens (the layer's forward
    pass refuses one)."""
    from grouped_gemm_router_amd import api
    e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
    i32 = torch.int32
    api.moe_combine_backward(e(0, 64), e(0, 64, dt=F32), e(0, dt=i32), e(0, 2, dt=F32), e(0, 64),
                             e(0, 2, dt=F32), n_shared=1)
    api.moe_permute_backward(e(0, 64), e(0, dt=i32), e(0, 64), 2, addend=e(0, 64))
    off = torch.zeros((4,), dtype=i32, device=DEV)
    W, dW = e(3, 128, 64), torch.full((3, 128, 64), 7.0, dtype=BF, device=DEV)
    api.moe_grouped_gemm_dgrad(e(0, 128), W, e(0, 64), off, dC2=e(0, 128), B2=W)
    api.moe_grouped_gemm_dgrad_swiglu(e(0, 128), W, *(e(0, 64) for _ in range(4)), off)
    api.moe_grouped_gemm_wgrad(e(0, 128), e(0, 64), dW, off)
    assert (dW == 0).all()


def test_on_another_stream():
    m, w, x, d_out = build(64, 128, 256, 8, 2, 1, BF)
    m(x)
    want = m.backward(d_out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m(x)
        got = m.backward(d_out)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[n], want[n]) for n in want)
