"""GPU parity of moe_lora_linear and its backward against 64-bit references.

Tolerances from the arithmetic (u = 2^-24 for fp32; a rounding to bf16 is off
by at most 2^-8 relative).  A sum of m products in fp32 errs by at most
(m + 2) u sum |terms| (bf16 products are exact, fp32 ones rounded once).
  v, u      (K + 4) u scale sum |A x|: the sum, the scaling, the partial sums
  y, dx     the sum over K; the error of v through B; the sum over r; v enters
            the bf16 matrix cores as two terms for a bf16 y (2^-16 of v is
            lost) or three (2^-24), or as fp32; one rounding of the output
  dA, dB    the error of u; the sum over the rows; u and v enter as three
            bf16 terms (2^-24)
"""
import numpy as np
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def api():
    from grouped_gemm_router_amd import api as a
    return a


def rows_of(kind, T, n, g):
    if kind == "none":
        return torch.full((T,), -1, dtype=torch.int32)
    if kind == "one":
        return torch.full((T,), n - 1, dtype=torch.int32)
    if kind == "mixed":  # outside [0, n): no adapter
        a = torch.randint(-2, n + 1, (T,), generator=g)
        return torch.where(torch.rand((T,), generator=g) < 0.02, torch.full_like(a, 2 ** 30),
                           a).to(torch.int32)
    cut = torch.randint(0, T + 1, (n,), generator=g)
    run = (torch.arange(T)[:, None] >= cut[None, :]).sum(1)
    return (torch.randperm(n + 1, generator=g) - 1)[run].to(torch.int32)


class Case:
    def __init__(self, T, N, K, r, n, dt, kind, seed):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda shape, std: (torch.randn(shape, generator=g) * std).to(dt)  # noqa: E731
        self.T, self.N, self.K, self.r, self.n, self.dt = T, N, K, r, n, dt
        self.x = rnd((T, K), 1.0)
        self.W = rnd((N, K), K ** -0.5)
        self.A = rnd((n, r, K), K ** -0.5)
        self.B = rnd((n, r, N), r ** -0.5)
        self.scale = 0.5 + torch.rand((n,), generator=g)
        self.adapter = rows_of(kind, T, n, g)
        self.dy = rnd((T, N), 0.1)

    def gpu(self):
        for k, t in list(self.__dict__.items()):
            if isinstance(t, torch.Tensor):
                setattr(self, "g_" + k, t.to(DEV))
        return self


def shrink_ref(x, F, scale, adapter, n):
    """(value, bound of its error) of scale[a] F[a] x[t] in 64 bits."""
    T, K = x.shape
    v = torch.zeros((T, F.shape[1]), dtype=torch.float64)
    e = torch.zeros_like(v)
    for a in range(n):
        rows = torch.nonzero(adapter == a).flatten()
        if len(rows):
            v[rows] = float(scale[a]) * (x[rows].double() @ F[a].double().t())
            e[rows] = (K + 4) * U * float(scale[a]) * (x[rows].double().abs()
                                                       @ F[a].double().abs().t())
    return v, e


def expand_ref(x, W, base, v, ev, F, adapter, n, out_dt, dt):
    """(value, bound) of W x + v F (base: what y holds instead of W x)."""
    T, r = v.shape
    if W is not None:
        K = x.shape[1]
        y = x.double() @ W.double().t()
        e = (K + 2) * U * (x.double().abs() @ W.double().abs().t())
    else:
        y, e = base.double().clone(), torch.zeros(base.shape, dtype=torch.float64)
    lost = 0.0 if dt == F32 else 2.0 ** -16 if out_dt == BF else U
    for a in range(n):
        rows = torch.nonzero(adapter == a).flatten()
        if len(rows):
            d = v[rows].double() @ F[a].double()
            size = v[rows].double().abs() @ F[a].double().abs()
            y[rows] += d
            e[rows] += ev[rows] @ F[a].double().abs() + ((3 * r + 8) * U + lost) * size
    e = e + 4 * U * y.abs()
    return y, e + (2.0 ** -8 if out_dt == BF else U) * (y.abs() + e)


def within(got, ref, bound, what):
    got = got.cpu().double()
    assert got.shape == ref.shape
    assert torch.isfinite(got).all(), what
    err = (got - ref).abs()
    assert (err <= bound + 1e-37).all(), "%s: %d of %d outside, worst %.3g of the bound" % (
        what, int((err > bound + 1e-37).sum()), err.numel(), float((err / (bound + 1e-37)).max()))


def guarded(T, N, dt):
    """A [T][N] buffer with sentinel rows behind it."""
    store = torch.full((T + 3, N), 123.0, dtype=dt, device=DEV)
    return store, store[:T]


def forward(c, out_dt, with_w=True, base=None, ldw_pad=0):
    a = api()
    store, y = guarded(c.T, c.N, out_dt)
    vstore, v = guarded(c.T, c.r, F32)
    if base is not None:
        y.copy_(base)
    W = None
    if with_w:
        W = c.g_W
        if ldw_pad:
            W = torch.full((c.N, c.K + ldw_pad), float("nan"), dtype=c.dt, device=DEV)
            W[:, :c.K] = c.g_W
            W = W[:, :c.K]
    a.moe_lora_linear(c.g_x, c.g_A, c.g_B, c.g_scale, c.g_adapter, y, v, W=W)
    torch.cuda.synchronize()
    assert (store[c.T:] == 123).all() and (vstore[c.T:] == 123).all()
    return y, v


def check_forward(c, out_dt, with_w=True, ldw_pad=0):
    base = None if with_w else c.dy.to(out_dt)
    y, v = forward(c, out_dt, with_w, base, ldw_pad)
    rv, ev = shrink_ref(c.x, c.A, c.scale, c.adapter, c.n)
    within(v, rv, ev, "v")
    ry, ey = expand_ref(c.x, c.W if with_w else None, base, rv, ev, c.B, c.adapter, c.n, out_dt,
                        c.dt)
    within(y, ry, ey, "y")
    return y, v


# (T, N, K, r, n): row counts at every switch between the kernels (16 and 32
# rows of the few-row kernel), column counts that choose every tile shape, odd N, K that ends inside a 128-byte piece
SIZES = [
    (1, 1, 8, 8, 1), (1, 256, 128, 8, 3), (1, 100, 4096, 16, 2), (2, 33, 72, 8, 2),
    (15, 64, 256, 16, 5), (16, 17, 200, 24, 16), (17, 130, 264, 32, 4), (32, 512, 512, 64, 3),
    (33, 48, 520, 16, 7), (64, 1000, 384, 128, 2), (65, 1000, 384, 16, 9), (127, 96, 136, 8, 64),
    (128, 2049, 320, 16, 33), (129, 256, 640, 48, 6), (200, 8, 1024, 8, 2), (300, 300, 328, 40, 5),
    (513, 256, 256, 16, 4), (1000, 65, 88, 120, 3), (777, 520, 200, 16, 100),
    (1500, 1111, 192, 32, 8), (2300, 2048, 256, 16, 5), (31, 4096, 64, 8, 1024)]


@pytest.mark.parametrize("kind", ["requests", "mixed"])
@pytest.mark.parametrize("out_dt", [BF, F32])
@pytest.mark.parametrize("T,N,K,r,n", SIZES)
def test_forward_bf16(T, N, K, r, n, out_dt, kind):
    print("lora bf16", T, N, K, r, n, out_dt, kind, flush=True)
    check_forward(Case(T, N, K, r, n, BF, kind, T + N).gpu(), out_dt)


@pytest.mark.parametrize("kind", ["requests", "mixed"])
@pytest.mark.parametrize("T,N,K,r,n", [s for s in SIZES if s[0] * s[1] * s[2] < 2e8])
def test_forward_f32(T, N, K, r, n, kind):
    print("lora f32", T, N, K, r, n, kind, flush=True)
    check_forward(Case(T, N, K, r, n, F32, kind, T + K).gpu(), F32)


@pytest.mark.parametrize("dt,out_dt", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("T,N,K,r,n", [(1, 7, 64, 8, 2), (30, 96, 128, 16, 4), (70, 33, 256, 8, 3),
                                       (400, 512, 128, 32, 6), (1000, 300, 72, 16, 3)])
def test_added_to_a_projection_computed_elsewhere(T, N, K, r, n, dt, out_dt):
    for kind in ("requests", "mixed", "none"):
        print("lora in place", T, N, K, r, n, dt, out_dt, kind, flush=True)
        c = Case(T, N, K, r, n, dt, kind, T).gpu()
        y, _ = check_forward(c, out_dt, with_w=False)
        if kind == "none":
            assert torch.equal(y.cpu(), c.dy.to(out_dt))


@pytest.mark.parametrize("kind", ["none", "one"])
@pytest.mark.parametrize("T", [1, 40, 90, 700])
def test_no_adapter_and_one_adapter(T, kind):
    check_forward(Case(T, 264, 256, 16, 3, BF, kind, T).gpu(), BF)


@pytest.mark.parametrize("T", [3, 200])
def test_padded_weight_rows(T):
    for dt in (BF, F32):
        check_forward(Case(T, 140, 128, 8, 2, dt, "mixed", T).gpu(), dt, ldw_pad=24)


def test_low_rank_padded_with_zero_rows():
    """An adapter of rank 3 in a table of rank 16."""
    c = Case(50, 64, 128, 16, 2, BF, "mixed", 1)
    c.A[:, 3:] = 0
    c.B[:, 3:] = 0
    check_forward(c.gpu(), BF)


@pytest.mark.parametrize("T", [5, 60, 130, 600])
@pytest.mark.parametrize("dt", [BF, F32])
def test_one_request_never_meets_another(T, dt):
    """An adapter full of infinities and NaN, and rows of NaN, change nothing
    in the rows of other requests: bit for bit."""
    for kind in ("requests", "mixed"):
        c = Case(T, 200, 256, 16, 4, dt, kind, T).gpu()
        y0, v0 = forward(c, dt)
        c.g_A[2], c.g_B[2] = float("nan"), float("inf")
        y1, v1 = forward(c, dt)
        keep = c.adapter != 2
        assert torch.equal(y0.cpu()[keep], y1.cpu()[keep])
        assert torch.equal(v0.cpu()[keep], v1.cpu()[keep])
        c = Case(T, 200, 256, 16, 4, dt, kind, T).gpu()
        c.g_x[T // 2] = float("nan")
        y1, v1 = forward(c, dt)
        keep = torch.arange(T) != T // 2
        assert torch.equal(y0.cpu()[keep], y1.cpu()[keep])
        assert torch.equal(v0.cpu()[keep], v1.cpu()[keep])


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------

def backward(c, v, with_w=True, base=None, what="xw"):
    a = api()
    ustore, u = guarded(c.T, c.r, F32)
    dx = dA = dB = None
    if "x" in what:
        xstore, dx = guarded(c.T, c.K, c.dt)
        if base is not None:
            dx.copy_(base)
    if "w" in what:
        dA = torch.full((c.n, c.r, c.K), float("nan"), device=DEV)
        dB = torch.full((c.n, c.r, c.N), float("nan"), device=DEV)
    W_t = c.g_W.t().contiguous() if with_w and "x" in what else None
    a.moe_lora_linear_backward(c.g_dy, c.g_x, c.g_A, c.g_B, c.g_scale, c.g_adapter, v, u, W_t=W_t,
                               dx=dx, dA=dA, dB=dB)
    torch.cuda.synchronize()
    assert (ustore[c.T:] == 123).all()
    if "x" in what:
        assert (xstore[c.T:] == 123).all()
    return u, dx, dA, dB


def check_backward(c, with_w=True):
    v = shrink_ref(c.x, c.A, c.scale, c.adapter, c.n)[0].float()
    base = None if with_w else c.x.clone()
    u, dx, dA, dB = backward(c, v.to(DEV), with_w, base)
    ru, eu = shrink_ref(c.dy, c.B, c.scale, c.adapter, c.n)
    within(u, ru, eu, "u")
    rx, ex = expand_ref(c.dy, c.W.t() if with_w else None, base, ru, eu, c.A, c.adapter, c.n, c.dt,
                        c.dt)
    within(dx, rx, ex, "dx")
    for a in range(c.n):
        rows = torch.nonzero(c.adapter == a).flatten()
        m = len(rows)
        x, dy, vv = c.x[rows].double(), c.dy[rows].double(), v[rows].double()
        k = (3 * m + 8) * U
        within(dA[a], ru[rows].t() @ x, (eu[rows].t() + k * ru[rows].abs().t()) @ x.abs(), "dA")
        within(dB[a], vv.t() @ dy, k * (vv.abs().t() @ dy.abs()), "dB")


BACK = [(1, 8, 8, 8, 1), (2, 64, 128, 16, 3), (17, 136, 72, 24, 4), (64, 256, 200, 8, 2),
        (100, 40, 264, 128, 5), (130, 512, 136, 16, 60), (256, 128, 128, 16, 1),
        (257, 128, 256, 32, 1), (700, 72, 520, 40, 3), (1000, 264, 128, 64, 7),
        (3000, 64, 136, 16, 2), (9000, 8, 64, 8, 3), (300, 16, 24, 8, 1024)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("kind", ["requests", "mixed"])
@pytest.mark.parametrize("T,N,K,r,n", BACK)
def test_backward(T, N, K, r, n, kind, dt):
    print("lora backward", T, N, K, r, n, kind, dt, flush=True)
    check_backward(Case(T, N, K, r, n, dt, kind, T + N).gpu())


@pytest.mark.parametrize("dt", [BF, F32])
def test_backward_of_parts(dt):
    c = Case(300, 64, 136, 16, 5, dt, "mixed", 2).gpu()
    check_backward(c, with_w=False)  # added to a dx computed elsewhere
    v = torch.randn((300, 16), device=DEV)
    u, dx, dA, dB = backward(c, v)
    assert torch.equal(backward(c, v, what="x")[1], dx)
    _, _, a2, b2 = backward(c, v, what="w")
    assert torch.equal(a2, dA) and torch.equal(b2, dB)
    none = Case(40, 64, 136, 16, 5, dt, "none", 2).gpu()
    _, _, dA, dB = backward(none, torch.zeros((40, 16), device=DEV))
    assert not dA.any() and not dB.any()


def test_backward_never_meets_another_request():
    for kind in ("requests", "mixed"):
        c = Case(500, 64, 128, 16, 4, BF, kind, 3).gpu()
        v = torch.randn((500, 16), device=DEV)
        want = backward(c, v)
        bad = c.adapter == 2
        c.g_x[bad.to(DEV)] = float("inf")
        c.g_dy[bad.to(DEV)] = float("nan")
        c.g_A[2], c.g_B[2] = float("nan"), float("inf")
        got = backward(c, v)
        for i in (0, 1):
            assert torch.equal(want[i].cpu()[~bad], got[i].cpu()[~bad])
        for i in (2, 3):
            for a in (0, 1, 3):
                assert torch.equal(want[i][a], got[i][a])


def test_gradients_against_differences():
    """The 64-bit forward's central differences along random directions (it
    is bilinear in (A, B) and linear in x, so they are exact up to 64-bit
    rounding): the kernels' dx (bf16, 2^-8 of each element and the errors
    above, together below 2^-7 of the sum of |terms|), dA and dB (fp32)."""
    c = Case(150, 72, 136, 16, 3, BF, "mixed", 9).gpu()
    v = shrink_ref(c.x, c.A, c.scale, c.adapter, c.n)[0].float()
    _, dx, dA, dB = backward(c, v.to(DEV))

    def loss(x, A, B):
        y = x @ c.W.double().t()
        for a in range(c.n):
            rows = torch.nonzero(c.adapter == a).flatten()
            y[rows] += float(c.scale[a]) * (x[rows] @ A[a].t()) @ B[a]
        return float((y * c.dy.double()).sum())

    g = torch.Generator().manual_seed(1)
    at = [c.x.double(), c.A.double(), c.B.double()]
    for i, (grad, tol) in enumerate(((dx, 2.0 ** -7), (dA, 1e-5), (dB, 1e-5))):
        d = torch.randn(at[i].shape, generator=g, dtype=torch.float64)
        e = 1e-2
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + e * d, at[i] - e * d
        slope = (loss(*hi) - loss(*lo)) / (2 * e)
        terms = grad.cpu().double() * d
        assert abs(slope - float(terms.sum())) <= tol * float(terms.abs().sum())


# ---------------------------------------------------------------------------
# as they are used
# ---------------------------------------------------------------------------

def test_deterministic_other_stream_and_graph():
    """Twice the same bits; a side stream; a captured step replayed four times
    on new inputs with eager work in between, workspaces shared by neither."""
    a = api()
    T, N, K, r, n = 300, 256, 384, 16, 6
    sets = [Case(T, N, K, r, n, BF, k, i).gpu()
            for i, k in enumerate(("requests", "mixed", "one", "requests", "mixed"))]
    names = ("x", "A", "B", "scale", "adapter", "dy", "W")
    st = {k: getattr(sets[0], "g_" + k).clone() for k in names}
    st["W_t"] = st["W"].t().contiguous()
    size = a.moe_lora_backward_workspace_size(T, N, K, r, n, BF)

    def buffers():
        f = lambda *s, dt=F32: torch.full(s, float("nan"), dtype=dt, device=DEV)  # noqa: E731
        return {"y": f(T, N, dt=BF), "v": f(T, r), "u": f(T, r), "dx": f(T, K, dt=BF),
                "dA": f(n, r, K), "dB": f(n, r, N),
                "ws": torch.empty(size, dtype=torch.uint8, device=DEV)}

    def step(b, o):
        a.moe_lora_linear(b["x"], b["A"], b["B"], b["scale"], b["adapter"], o["y"], o["v"],
                          W=b["W"], ws=o["ws"])
        a.moe_lora_linear_backward(b["dy"], b["x"], b["A"], b["B"], b["scale"], b["adapter"],
                                   o["v"], o["u"], W_t=b["W_t"], dx=o["dx"], dA=o["dA"],
                                   dB=o["dB"], ws=o["ws"])

    def eager(c):
        b = {k: getattr(c, "g_" + k) for k in names}
        b["W_t"] = b["W"].t().contiguous()
        o = buffers()
        step(b, o)
        torch.cuda.synchronize()
        return o

    def same(p, q):
        for k in ("y", "v", "u", "dx", "dA", "dB"):
            assert torch.equal(p[k], q[k]), k

    want = [eager(c) for c in sets]
    same(want[0], eager(sets[0]))
    out = buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(st, out)
    side.synchronize()
    same(want[0], out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(st, out)
    for i in (1, 2, 3, 4):
        for k in names:
            st[k].copy_(getattr(sets[i], "g_" + k))
        st["W_t"].copy_(st["W"].t())
        graph.replay()
        torch.cuda.synchronize()
        same(want[i], out)
        same(want[0], eager(sets[0]))


def test_adapted_router_fine_tuning_step():
    """The operators together as a fine-tuning step of adapted routers uses
    them: the adapted projection gives the logits, the layer routes from them,
    the balance loss and the gate's gradient come back to the logits, and the
    adapters get their gradients -- against 64-bit autograd of the whole step
    at the step's own selection."""
    from grouped_gemm_router_amd.adapters import AdaptedLinear
    a = api()
    T, K, E, k, r, n, alpha = 500, 256, 24, 4, 16, 5, 0.02
    c = Case(T, E, K, r, n, BF, "requests", 4).gpu()
    router = AdaptedLinear(c.g_W, c.g_A, c.g_B, c.g_scale, grad=True)
    logits, v = router(c.g_x, c.g_adapter, out_dtype=F32)
    idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    a.moe_route(None, None, idx, w, logits=logits, flags=a.MOE_ROUTE_FROM_LOGITS)
    counts = torch.empty((1, E), dtype=torch.int32, device=DEV)
    probs, loss = torch.empty((1, E), device=DEV), torch.empty((1,), device=DEV)
    tokens = torch.empty((2,), dtype=torch.int32, device=DEV)
    a.moe_balance_loss(logits, idx, counts, probs, tokens, loss, alpha=alpha)
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(3)) / T
    d_logits = torch.empty_like(logits)
    a.moe_route_backward(logits, idx, d_logits, d_topk_w=dw.to(DEV), counts=counts, tokens=tokens,
                         alpha=alpha)
    dy = d_logits.to(BF)
    dx, dA, dB = router.backward(dy, c.g_x, c.g_adapter, v)
    torch.cuda.synchronize()

    x = c.x.double().requires_grad_(True)
    A, B = c.A.double().requires_grad_(True), c.B.double().requires_grad_(True)
    hot = torch.nn.functional.one_hot(c.adapter.clamp_min(-1).long() + 1, n + 1)[:, 1:].double()
    low = torch.einsum("tn,nrk,tk->tr", hot * c.scale.double(), A, x)
    lg = x @ c.W.double().t() + torch.einsum("tn,tr,nre->te", hot, low, B)
    p = torch.softmax(lg, 1)
    sel = idx.cpu().long()
    f = torch.bincount(sel.flatten(), minlength=E).double() / (T * k)
    ref_loss = alpha * E * (f * p.mean(0)).sum()
    ((dw.double() * p.gather(1, sel)).sum() + ref_loss).backward()
    # fp32 logits of K terms and the softmax: relative errors of a few hundred u
    assert abs(float(loss) - float(ref_loss)) <= 1e-4 * float(ref_loss)
    # the logits' gradient is rounded to bf16 once (2^-8 of each element), and
    # dx once more; as norms these stay below 2^-8 + 2^-8
    for got, ref, tol in ((dx, x.grad, 2.0 ** -7), (dA, A.grad, 2.0 ** -8), (dB, B.grad, 2.0 ** -8)):
        got = got.cpu().double()
        assert float((got - ref).norm()) <= tol * float(ref.norm())


@pytest.mark.parametrize("dt", [BF, F32])
def test_empty_batch(dt):
    """No rows: nothing to write forward, zero gradients backward."""
    c = Case(0, 64, 128, 8, 2, dt, "none", 0).gpu()
    y, v = forward(c, dt)
    _, _, dA, dB = backward(c, v)
    assert not dA.any() and not dB.any()


def test_offsets_past_32_bits():
    """y of more than 2^32 bytes: the last rows against their own batch."""
    T, N, K, r, n = 1 << 17, 16392, 64, 8, 2
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((T, K), generator=g, device=DEV).to(BF)
    W = (torch.randn((N, K), generator=g, device=DEV) / 8).to(BF)
    A = (torch.randn((n, r, K), generator=g, device=DEV) / 8).to(BF)
    B = torch.randn((n, r, N), generator=g, device=DEV).to(BF)
    scale = torch.ones(n, device=DEV)
    adapter = torch.randint(-1, n, (T,), generator=g, device=DEV, dtype=torch.int32)
    y, v = torch.empty((T, N), dtype=BF, device=DEV), torch.empty((T, r), device=DEV)
    api().moe_lora_linear(x, A, B, scale, adapter, y, v, W=W)
    m = 1000
    y2, v2 = torch.empty((m, N), dtype=BF, device=DEV), torch.empty((m, r), device=DEV)
    api().moe_lora_linear(x[-m:].contiguous(), A, B, scale, adapter[-m:].contiguous(), y2, v2, W=W)
    torch.cuda.synchronize()
    # the same sums in another tile: fp32 sums of 64 + 24 terms, one rounding
    size = x[-m:].float().abs() @ W.float().abs().t() + v2.abs().sum(1, keepdim=True) * 6
    assert ((y[-m:].float() - y2.float()).abs() <= 2.0 ** -7 * y2.float().abs() + 2.0 ** -14 * size).all()


def test_refusals_on_the_gpu():
    a = api()
    c = Case(20, 64, 128, 8, 2, BF, "mixed", 0).gpu()
    y, v = torch.empty((20, 64), dtype=BF, device=DEV), torch.empty((20, 8), device=DEV)
    call = lambda **k: a.moe_lora_linear(**{**dict(  # noqa: E731
        x=c.g_x, A=c.g_A, B=c.g_B, scale=c.g_scale, adapter=c.g_adapter, y=y, v=v, W=c.g_W), **k})
    with pytest.raises(ValueError):
        call(adapter=c.adapter)                      # on the host
    with pytest.raises(TypeError):
        call(adapter=c.g_adapter.long())
    with pytest.raises(ValueError):
        call(v=torch.empty((20, 16), device=DEV))
    with pytest.raises(ValueError):
        call(x=c.g_x.t().contiguous().t())           # not contiguous
    with pytest.raises(ValueError):
        call(W=c.g_W.t())
    with pytest.raises(TypeError):
        call(y=y.half())
    torch.cuda.synchronize()
    assert np.isfinite(float(c.g_x.float().sum()))


# sorted batches whose 32-row blocks hold one to six adapters: ranks behind one
# staged chunk (72, 128), an odd rank of eights, odd N, more adapters in a tile
# than are staged at once, tiles of every size
@pytest.mark.parametrize("out_dt", [BF, F32])
@pytest.mark.parametrize("T,N,K,r,n", [
    (600, 1000, 2048, 72, 40), (700, 1200, 256, 128, 12), (1500, 1111, 256, 64, 100),
    (2100, 3000, 256, 40, 200), (5000, 4096, 128, 128, 400), (330, 2050, 1024, 128, 30),
    (6000, 2048, 256, 16, 5), (4100, 1600, 640, 24, 900), (8000, 1500, 512, 8, 300)])
def test_blocks_of_a_few_adapters(T, N, K, r, n, out_dt):
    print("lora few", T, N, K, r, n, out_dt, flush=True)
    c = Case(T, N, K, r, n, BF, "mixed", T).gpu()
    y0, v0 = check_forward(c, out_dt)
    # an adapter that is not finite shares blocks and tiles with others, and
    # changes no bit of them
    c.g_A[n // 2], c.g_B[n // 2] = float("nan"), float("inf")
    y1, v1 = forward(c, out_dt)
    keep = (c.adapter != n // 2).to(DEV)
    assert not keep.all()
    assert torch.equal(y0[keep], y1[keep]) and torch.equal(v0[keep], v1[keep])
    assert not torch.isfinite(y1[~keep].float()).any()


def test_adapted_linear_graph_beside_larger_calls():
    """A captured call keeps what it needs: eager calls of other, larger
    batches of the same object between its replays, on two streams, change
    nothing of it, nor it of them."""
    from grouped_gemm_router_amd.adapters import AdaptedLinear
    small = [Case(200, 512, 2048, 32, 9, BF, "mixed", i).gpu() for i in range(4)]
    large = Case(1600, 512, 2048, 32, 9, BF, "mixed", 9).gpu()
    s0 = small[0]
    lin = AdaptedLinear(s0.g_W, s0.g_A, s0.g_B, s0.g_scale, grad=True)

    def step(c):
        y, v = lin(c.g_x, c.g_adapter)
        return (y, v, *lin.backward(c.g_dy, c.g_x, c.g_adapter, v))

    def same(p, q):
        assert all(torch.equal(a, b) for a, b in zip(p, q))

    want = [step(c) for c in small]
    want_large = step(large)
    st = Case(200, 512, 2048, 32, 9, BF, "mixed", 0).gpu()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(st)
    side = torch.cuda.Stream()
    for i in (1, 2, 3, 0):
        for k in ("x", "adapter", "dy"):
            getattr(st, "g_" + k).copy_(getattr(small[i], "g_" + k))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            beside = step(large)
        again = step(large)
        torch.cuda.synchronize()
        same(want[i], out)
        same(want_large, beside)
        same(want_large, again)


def test_workspace_grows_with_the_rows():
    """The sums' slices take T r floats each, however many adapters there are."""
    a = api()
    for T, n in ((1024, 1024), (128, 1024), (4096, 16)):
        size = a.moe_lora_linear_workspace_size(T, 14336, 4096, 64, n, BF)
        assert size <= 8 * T * 64 * 4 + 8 * T + 16 * n + 4096, (T, n, size)


def test_refuses_another_devices_stream():
    class Other:
        device_index, cuda_stream = 1, 0
    a = api()
    c = Case(20, 64, 128, 8, 2, BF, "mixed", 0).gpu()
    y, v = torch.empty((20, 64), dtype=BF, device=DEV), torch.empty((20, 8), device=DEV)
    with pytest.raises(ValueError, match="stream"):
        a.moe_lora_linear(c.g_x, c.g_A, c.g_B, c.g_scale, c.g_adapter, y, v, W=c.g_W,
                          ws=torch.empty(16, dtype=torch.uint8, device=DEV), stream=Other())


def test_workspace_comes_from_the_calls_stream():
    """A workspace made for a call on a side stream is that stream's memory:
    the current stream's may still be in use by work that is pending there."""
    a = api()
    side = torch.cuda.Stream()
    for stream in (None, side):
        ws, size = a._workspace(None, 3 << 20, 0, stream)
        assert size == 3 << 20
        owner = [seg["stream"] for seg in torch.cuda.memory_snapshot()
                 if seg["address"] <= ws.data_ptr() < seg["address"] + seg["total_size"]]
        want = torch.cuda.current_stream() if stream is None else stream
        assert owner == [want.cuda_stream]
    # and such a call gives what the current stream's gives
    c = Case(1600, 512, 2048, 32, 9, BF, "mixed", 1).gpu()
    y0, v0 = forward(c, BF)
    y1, v1 = torch.empty_like(y0), torch.empty_like(v0)
    side.wait_stream(torch.cuda.current_stream())
    a.moe_lora_linear(c.g_x, c.g_A, c.g_B, c.g_scale, c.g_adapter, y1, v1, W=c.g_W, stream=side)
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(v0, v1)
