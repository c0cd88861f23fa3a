"""GPU parity of products' gradients whose few, long sums are cut into slices
(dgrad along N, wgrad along the rows), which a second launch adds in order.
Tolerances as in test_gpu_backward.py: a sum of m products, whatever its
order, errs by at most (m + 2) u times its terms' sizes; the slices' partial
sums are among its additions."""
import pytest
import torch

from gpu_util import DEV
from test_gpu_backward import BF, F32, STORE, U, Groups, api, rowbuf, within

pytestmark = pytest.mark.gpu


def ws_of(kind, o):
    a = api()
    size = getattr(a, "moe_grouped_gemm_%s_workspace_size" % kind)(o.G, o.rows, o.N, o.K, o.dt)
    assert size > 0, "this shape is not cut"
    return torch.full((size,), 255, dtype=torch.uint8, device=DEV)  # NaN


@pytest.mark.parametrize("sizes", [[1], [3, 0, 40], [0, 257, 64], [5, 5, 5, 5, 5]])
@pytest.mark.parametrize("N,K", [(512, 8), (4104, 72), (2048, 264), (1000, 128)])
@pytest.mark.parametrize("dt,out", [(BF, BF), (BF, F32), (F32, F32)])
def test_dgrad(sizes, N, K, dt, out):
    o = Groups(sizes, N, K, dt, pad=8)
    for pair in (False, True):
        dA = rowbuf(o, out)
        api().moe_grouped_gemm_dgrad(o.g_dC, o.g_B, dA, o.g_off, dC2=o.g_dC2 if pair else None,
                                     B2=o.g_B2 if pair else None, ws=ws_of("dgrad", o))
        ref, e = o.dgrad(pair)
        within(dA[:o.live], ref, e + STORE[out] * (ref.abs() + e), "dA")
        assert (dA[o.live:] == 7).all()


@pytest.mark.parametrize("sizes", [[2], [3, 0, 40]])
@pytest.mark.parametrize("N,K", [(4104, 72), (2048, 264)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_dgrad_swiglu(sizes, N, K, dt):
    o = Groups(sizes, N, K, dt)
    dg, du, h = (rowbuf(o, dt) for _ in range(3))
    api().moe_grouped_gemm_dgrad_swiglu(o.g_dC, o.g_B, o.g_gate, o.g_up, dg, du, o.g_off, h=h,
                                        ws=ws_of("dgrad", o))
    a, ea = o.dgrad(False)
    z, up = o.gate[:o.live].double(), o.up[:o.live].double()
    s = torch.sigmoid(z)
    es = (4 + 2 * z.abs()) * U
    slope = s * (1 + z * (1 - s))
    eslope = es * slope.abs() + s * (8 + 4 * z.abs()) * U * (1 + z.abs())
    for got, ref, e in ((dg, a * up * slope, ea * (up * slope).abs() + (a * up).abs() * eslope),
                        (du, a * z * s, ea * (z * s).abs() + (a * z * s).abs() * es),
                        (h, z * s * up, (z * s * up).abs() * es)):
        e = 1.01 * e + 4 * U * ref.abs()
        within(got[:o.live], ref, e + STORE[dt] * (ref.abs() + e), "swiglu")
        assert (got[o.live:] == 7).all()
    gate, up = o.g_gate.clone(), o.g_up.clone()
    api().moe_grouped_gemm_dgrad_swiglu(o.g_dC, o.g_B, gate, up, gate, up, o.g_off)
    assert torch.equal(gate[:o.live], dg[:o.live]) and torch.equal(up[:o.live], du[:o.live])


@pytest.mark.parametrize("sizes", [[900], [1500, 0, 700], [300, 301, 0, 1, 1007]])
@pytest.mark.parametrize("N,K", [(8, 8), (40, 264), (136, 72)])
@pytest.mark.parametrize("dt,out", [(BF, BF), (BF, F32), (F32, F32)])
def test_wgrad(sizes, N, K, dt, out):
    o = Groups(sizes, N, K, dt)
    dB = torch.full((o.G + 1, N, K), 7.0, dtype=out, device=DEV)
    api().moe_grouped_gemm_wgrad(o.g_dC, o.g_A, dB[:o.G], o.g_off, ws=ws_of("wgrad", o))
    ref, e = o.wgrad()
    within(dB[:o.G], ref, e + STORE[out] * (ref.abs() + e), "dB")
    assert (dB[o.G:] == 7).all()
    base = torch.randn((o.G, N, K), generator=torch.Generator().manual_seed(3)).to(out)
    acc = base.to(DEV)
    api().moe_grouped_gemm_wgrad(o.g_dC, o.g_A, acc, o.g_off, accumulate=True,
                                 ws=ws_of("wgrad", o))
    ref = ref + base.double()
    e = e + U * (ref.abs() + e)
    within(acc, ref, e + STORE[out] * (ref.abs() + e), "dB + dB")


@pytest.mark.parametrize("off", [[0, 90, 40, 120], [-7, 20, 60, 10], [50, 50, 50, 50],
                                 [5, 20, 100, 1 << 30]])
@pytest.mark.parametrize("dt", [BF, F32])
def test_offsets_that_are_not_offsets(off, dt):
    o = Groups([40, 40, 40], 1032, 40, dt, spare=0)
    bad = torch.tensor(off, dtype=torch.int32, device=DEV)
    run, at = 0, []
    for v in off:
        run = max(run, min(max(v, 0), 120))
        at.append(run)
    o.off, o.live = torch.tensor(at), 120
    dA = torch.full((120, 40), 7.0, dtype=F32, device=DEV)
    api().moe_grouped_gemm_dgrad(o.g_dC, o.g_B, dA, bad, ws=ws_of("dgrad", o))
    ref, e = o.dgrad(False)
    inside = torch.zeros(120, dtype=torch.bool)
    inside[at[0]:at[-1]] = True
    within(dA[inside.to(DEV)], ref[inside], (e + U * (ref.abs() + e))[inside], "dA")
    assert (dA[~inside.to(DEV)] == 7).all()


def test_the_router_weights_gradient():
    """One group: d_logits^T x and d_logits W, as the layer's router needs
    them, through the same calls."""
    T, E, d = 3000, 8, 256
    g = torch.Generator().manual_seed(5)
    dl, x = torch.randn((T, E), generator=g), torch.randn((T, d), generator=g)
    w = torch.randn((E, d), generator=g)
    off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    dW, dx = torch.empty((1, E, d), device=DEV), torch.empty((T, d), device=DEV)
    api().moe_grouped_gemm_wgrad(dl.to(DEV), x.to(DEV), dW, off)
    api().moe_grouped_gemm_dgrad(dl.to(DEV), w[None].to(DEV), dx, off)
    ref, e = dl.double().t() @ x.double(), (T + 3) * U * (dl.double().abs().t() @ x.double().abs())
    within(dW[0], ref, e, "dW")
    ref, e = dl.double() @ w.double(), (E + 3) * U * (dl.double().abs() @ w.double().abs())
    within(dx, ref, e, "dx")


def test_captured_slices():
    """A captured call of cut sums, replayed between eager ones."""
    o = Groups([30, 7], 2056, 136, BF)
    ws = ws_of("dgrad", o)
    dA, want = rowbuf(o, F32), rowbuf(o, F32)
    api().moe_grouped_gemm_dgrad(o.g_dC, o.g_B, want, o.g_off)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api().moe_grouped_gemm_dgrad(o.g_dC, o.g_B, dA, o.g_off, ws=ws)
    for _ in range(3):
        dA.fill_(9.0)
        graph.replay()
        api().moe_grouped_gemm_dgrad(o.g_dC, o.g_B, want, o.g_off)
        torch.cuda.synchronize()
        assert torch.equal(dA[:o.live], want[:o.live]) and (dA[o.live:] == 9).all()
