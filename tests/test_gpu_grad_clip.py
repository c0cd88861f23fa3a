"""GPU tests of moe_grad_norm and moe_grad_clip against 64-bit references.

Tolerances (u = 2^-24): the squares of fp32 and bf16 values are exact in 64
bits, their sum of n errs by at most n 2^-53 relative, its root is rounded once
to fp32: u (1 + n 2^-28).  The factor is a sum, a quotient and, against 64
bits, the norm's own error: 4 u; its product is rounded (u) and stored.
"""
import math

import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
STORE = {BF: 2.0 ** -8, F32: U}


def api():
    from grouped_gemm_router_amd import api as a
    return a


def norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def norm_of(grads, **kw):
    norm = torch.empty((1,), device=DEV)
    api().moe_grad_norm(grads, norm, **kw)
    return norm


def close(norm, want, n):
    assert abs(float(norm) - want) <= U * (1 + n * 2.0 ** -28) * want, (float(norm), want)


def make(sizes, dts, shift=0, seed=0):
    """Gradients as views of one buffer a type, each `shift` elements further
    off a 16-byte boundary than the one before; guards between them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    out, at = [], {F32: 0, BF: 0}
    store = {t: torch.full((sum(sizes) + 64 * len(sizes) + 64,), 1e30, dtype=t, device=DEV)
             for t in (F32, BF)}
    for i, n in enumerate(sizes):
        t = dts[i % len(dts)]
        pos = (at[t] + 15) // 16 * 16 + (i * shift) % 16
        v = store[t][pos:pos + n]
        v.copy_(torch.randn((n,), generator=g, device=DEV) * 10.0 ** (i % 3 - 1))
        out.append(v)
        at[t] = pos + n + 1
    return out, store


CASES = [([1], [F32], 0), ([7, 1, 0, 9], [F32, BF], 1), ([16384] * 3, [BF], 0),
         ([16384 * 5 + 3, 40000, 5], [F32], 3), ([16377, 16385, 8, 15, 100003], [BF], 5),
         ([33] * 127 + [5000] * 130, [F32, BF, BF], 7), ([3 << 20, 77, (1 << 21) + 9], [BF, F32], 2)]


@pytest.mark.parametrize("sizes,dts,shift", CASES)
def test_norm_and_clip(sizes, dts, shift):
    grads, store = make(sizes, dts, shift)
    want = norm64(grads)
    norm = norm_of(grads)
    close(norm, want, sum(sizes))
    before = [g.clone() for g in grads]
    guard = {t: s.clone() for t, s in store.items()}
    for limit in (want / 3, want * 2):
        f = min(1.0, limit / (want + 1e-6))
        out = [torch.full((g.numel() + 2,), 5.0, dtype=g.dtype, device=DEV) for g in grads]
        # outputs of other alignments than the gradients' (every third one)
        put = [o[1:-1] if i % 3 == 0 else o[:-2] for i, o in enumerate(out)]
        api().moe_grad_clip(grads, norm, limit, out=put)
        for i, (g, o, full) in enumerate(zip(before, put, out)):
            ref = g.double() * f
            bound = (6 * U + STORE[g.dtype]) * ref.abs() + 1e-40
            assert ((o.double() - ref).abs() <= bound).all()
            rest = [full[0], full[-1]] if i % 3 == 0 else [full[-2], full[-1]]
            assert all(float(r) == 5.0 for r in rest)
            if f == 1.0:
                assert torch.equal(o, g)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    # in place: the same bits, and nothing beside the gradients
    api().moe_grad_clip(grads, norm, want / 3)
    api().moe_grad_clip(before, norm, want / 3, out=before)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    for t in store:
        rest = torch.ones_like(store[t], dtype=torch.bool)
        first = store[t].data_ptr()
        for g in grads:
            if g.dtype == t:
                at = (g.data_ptr() - first) // g.element_size()
                rest[at:at + g.numel()] = False
        assert rest.any() and torch.equal(store[t][rest], guard[t][rest])
    assert float(norm_of(grads)) == pytest.approx(want / 3, rel=0.01)


def test_nothing_to_sum():
    assert float(norm_of([])) == 0
    e = torch.empty((0,), device=DEV)
    assert float(norm_of([e, e.to(BF)])) == 0
    api().moe_grad_clip([], norm_of([]), 1.0)
    z = torch.zeros((5, 3), device=DEV)
    n = norm_of([z])
    api().moe_grad_clip([z], n, 0.0)
    assert float(n) == 0 and (z == 0).all()


def test_large_and_small_values():
    """No finite gradient overflows or vanishes in the sum."""
    big = torch.full((1000,), 1e30, device=DEV)
    close(norm_of([big]), norm64([big]), 1000)
    small = torch.full((1000,), 1e-30, device=DEV)
    close(norm_of([small]), norm64([small]), 1000)
    n = norm_of([big])
    api().moe_grad_clip([big], n, 1.0)
    assert float(big[3]) == pytest.approx(1000 ** -0.5, rel=1e-6)
    top = torch.full((1000,), 3e38, device=DEV)
    assert math.isinf(float(norm_of([top])))  # past fp32


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dt", [BF, F32])
def test_nan_and_infinity(bad, dt):
    a = torch.ones((40000,), dtype=dt, device=DEV)
    b = torch.ones((17,), dtype=dt, device=DEV)
    a[39999] = bad
    n = norm_of([b, a])
    assert math.isnan(float(n)) if math.isnan(bad) else math.isinf(float(n))
    api().moe_grad_clip([a, b], n, 1.0)
    if math.isnan(bad):
        assert a.isnan().all() and b.isnan().all()
    else:
        assert (b == 0).all() and (a[:-1] == 0).all() and a[-1].isnan()


def test_where_nothing_is_clipped_nothing_is_written():
    """A factor of 1 leaves even payloads of NaN alone."""
    t = torch.arange(100000, dtype=torch.int32, device=DEV).view(F32)
    t2 = t.clone()
    api().moe_grad_clip([t], torch.zeros((1,), device=DEV), 1.0)
    assert torch.equal(t.view(torch.int32), t2.view(torch.int32))


def test_more_than_2_to_the_31_values():
    g = torch.zeros(((1 << 31) + 5,), dtype=BF, device=DEV)
    g[-1], g[1 << 31], g[0] = 3.0, 4.0, 12.0
    n = norm_of([g])
    assert float(n) == 13.0
    api().moe_grad_clip([g], n, 6.5)
    assert [float(g[i]) for i in (-1, 1 << 31, 0)] == [1.5, 2.0, 6.0]


def test_the_same_bits_again_on_a_stream_and_in_a_graph():
    grads, _ = make([100003, 5, 70000], [F32, BF], 3)
    a = api()
    out = [torch.empty_like(g) for g in grads]
    norm, ws = torch.empty((1,), device=DEV), torch.empty(
        (a.moe_grad_norm_workspace_size(3),), dtype=torch.uint8, device=DEV)

    def step():
        a.moe_grad_norm(grads, norm, ws=ws)
        a.moe_grad_clip(grads, norm, 1.0, out=out)

    step()
    want = [norm.clone()] + [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(want, [norm] + out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        for g in grads:
            g.mul_(2.0)
        graph.replay()
        eager = torch.empty((1,), device=DEV)
        a.moe_grad_norm(grads, eager)
        torch.cuda.synchronize()
        assert torch.equal(norm, eager) and float(norm) == float(want[0]) * 2 ** (k + 1)


def test_a_deferred_step():
    """Calls marshalled once: their host arrays live as long as the thunk, and
    they read what the gradients hold then."""
    import gc
    grads, _ = make([4000, 9, 70001], [F32, BF], 1)
    a = api()
    norm = torch.empty((1,), device=DEV)
    ws = torch.empty((a.moe_grad_norm_workspace_size(3),), dtype=torch.uint8, device=DEV)
    out = [torch.empty_like(g) for g in grads]
    calls = [a.deferred(a.moe_grad_norm, grads, norm, ws=ws),
             a.deferred(a.moe_grad_clip, grads, norm, 0.5, out=out)]
    gc.collect()
    for _ in range(2):
        for g in grads:
            g.mul_(3.0)
        for c in calls:
            c()
        want = norm64(grads)
        close(norm, want, 1)
        assert norm64(out) == pytest.approx(0.5, rel=0.01)


def test_any_iterable_of_gradients():
    grads, _ = make([500, 70], [F32, BF], 1)
    want = norm64(grads)
    n = norm_of(g for g in grads)
    close(n, want, 600)
    api().moe_grad_clip((g for g in grads), n, want / 2)
    assert norm64(grads) == pytest.approx(want / 2, rel=0.01)


@pytest.mark.parametrize("n", [1, 200])  # the ranges of few and of many tensors
def test_neighbours_and_shared_sources_are_no_overlap(n):
    """Outputs that touch, in any order, and one gradient read for several."""
    store = torch.randn((n * 70 + 1,), device=DEV)
    parts = [store[70 * i:70 * i + 70] for i in range(n)][::-1]
    norm = torch.full((1,), 4.0, device=DEV)
    scale = 2.0 / (torch.tensor(4.0) + 1e-6)
    want = [p * scale.to(DEV) for p in parts]
    empty = store[3:3]
    out = [torch.empty_like(p) for p in parts]
    first = torch.empty_like(parts[0])
    api().moe_grad_clip(parts + [parts[0], empty, empty], norm, 2.0, out=out + [first, empty, empty])
    api().moe_grad_clip(parts + [empty, empty], norm, 2.0)
    for w, o, p in zip(want, out, parts):
        assert torch.allclose(o, w, rtol=4 * U, atol=0) and torch.equal(o, p)
    assert torch.equal(first, out[0])
    with pytest.raises(api().MoEError):
        api().moe_grad_clip(parts + parts[:1], norm, 2.0)
    for w, p in zip(out, parts):
        assert torch.equal(w, p)
