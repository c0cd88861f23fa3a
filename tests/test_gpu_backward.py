"""GPU parity of the expert layer's backward pass (include/moe_backward.h)
against 64-bit references.

Tolerances from the arithmetic (u = 2^-24; a rounding to bf16 is off by at most
2^-8 relative).  A sum of m products in fp32 errs by at most (m + 2) u
sum |terms| (bf16 products are exact, fp32 ones rounded once).
  combine     dY: one product; d_topk_w: a sum of d products
  permute     a sum of k + n_shared + 1 values
  dgrad       a sum of N (2 N) products; with SwiGLU that error through the
              two derivatives, and theirs: the sigmoid errs by at most
              (4 + 2 |gate|) u relative (the exponent's product, the hardware's
              exp2 and reciprocal), 1 + gate (1 - s) by (8 + 4 |gate|) u (1 +
              |gate|) absolute
  wgrad       a sum over the group's rows, and one addition to what was there
and one rounding of what is stored.
"""
import numpy as np
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
STORE = {BF: 2.0 ** -8, F32: U}


def api():
    from grouped_gemm_router_amd import api as a
    return a


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(got, ref, bound, what):
    got = got.cpu().double()
    assert got.shape == ref.shape
    assert torch.isfinite(got).all(), what
    err = (got - ref).abs()
    assert (err <= bound + 1e-37).all(), "%s: %d of %d outside, worst %.3g of the bound" % (
        what, int((err > bound + 1e-37).sum()), err.numel(), float((err / (bound + 1e-37)).max()))


# ---------------------------------------------------------------------------
# combine and permute
# ---------------------------------------------------------------------------

def rows_of(T, E, k, ns, cap, g):
    """flat_to_row of a random routing with at most cap rows an expert."""
    e = torch.rand((T, E), generator=g).topk(k, dim=1).indices.reshape(-1).numpy()
    order = np.argsort(e, kind="stable")
    row, used, at = np.full(T * k, -1, np.int32), {}, 0
    for f in order:
        used[e[f]] = used.get(e[f], 0) + 1
        if used[e[f]] <= cap:
            row[f] = at
            at += 1
    return torch.from_numpy(np.concatenate([row, at + np.arange(ns * T, dtype=np.int32)]))


SORT = [  # T, d, E, k, ns, cap, dt, other
    (1, 8, 2, 1, 0, 99, F32, F32),
    (1, 64, 8, 8, 0, 99, BF, F32),
    (5, 72, 4, 3, 2, 2, BF, BF),
    (33, 1024, 16, 5, 1, 99, F32, BF),
    (40, 2056, 40, 32, 0, 20, BF, F32),
    (7, 7168, 32, 9, 8, 99, BF, F32),
    (300, 4096, 8, 2, 0, 50, BF, BF),
    (64, 2048, 12, 12, 1, 99, F32, F32),
]


@pytest.mark.parametrize("T,d,E,k,ns,cap,dt,other", SORT)
def test_combine_backward(T, d, E, k, ns, cap, dt, other):
    g = gen(T * 31 + d + k)
    R = T * (k + ns)
    f2r = rows_of(T, E, k, ns, cap, g)
    d_out = torch.randn((T, d), generator=g).to(dt)
    w = torch.rand((T, k), generator=g)
    Y = torch.full((R, d), float("nan"), dtype=other)  # rows that no entry names hold anything
    named = f2r[f2r >= 0].long()
    Y[named] = torch.randn((len(named), d), generator=g).to(other)
    args = [t.to(DEV) for t in (d_out, Y, f2r, w)]
    dY = torch.full((R + 2, d), 7.0, dtype=dt, device=DEV)
    dw = torch.full((T, k), 7.0, device=DEV)
    api().moe_combine_backward(*args, dY[:R], dw, n_shared=ns)
    ref = torch.full((R + 2, d), 7.0, dtype=F64)
    rdw, bdw = torch.zeros((T, k), dtype=F64), torch.zeros((T, k), dtype=F64)
    for t in range(T):
        for j in range(k):
            r = int(f2r[t * k + j])
            if r >= 0:
                ref[r] = w[t, j].double() * d_out[t].double()
                terms = Y[r].double() * d_out[t].double()
                rdw[t, j], bdw[t, j] = terms.sum(), (d + 2) * U * terms.abs().sum()
        for s in range(ns):
            ref[f2r[T * k + s * T + t].long()] = d_out[t].double()
    within(dY, ref, (U + STORE[dt]) * ref.abs(), "dY")
    within(dw, rdw, bdw, "d_topk_w")
    # either part alone
    dY1, dw1 = torch.full_like(dY, 7.0), torch.empty_like(dw)
    api().moe_combine_backward(args[0], None, args[2], args[3], dY1[:R], None, n_shared=ns)
    api().moe_combine_backward(*args, None, dw1, n_shared=ns)
    assert torch.equal(dY1, dY) and torch.equal(dw1, dw)


@pytest.mark.parametrize("T,d,E,k,ns,cap,dt,other", SORT)
def test_permute_backward(T, d, E, k, ns, cap, dt, other):
    g = gen(T * 37 + d + k)
    R = T * (k + ns)
    f2r = rows_of(T, E, k, ns, cap, g)
    part = torch.full((R, d), float("nan"), dtype=other)
    named = f2r[f2r >= 0].long()
    part[named] = torch.randn((len(named), d), generator=g).to(other)
    add = torch.randn((T, d), generator=g).to(dt)
    ref, size = torch.zeros((T, d), dtype=F64), torch.zeros((T, d), dtype=F64)
    for t in range(T):
        at = [f2r[t * k + j] for j in range(k)] + [f2r[T * k + s * T + t] for s in range(ns)]
        for r in at:
            if r >= 0:
                ref[t] += part[r.long()].double()
                size[t] += part[r.long()].double().abs()
    p, f = part.to(DEV), f2r.to(DEV)
    dx = torch.full((T + 1, d), 7.0, dtype=dt, device=DEV)
    api().moe_permute_backward(p, f, dx[:T], k, n_shared=ns)
    n = k + ns + 1
    within(dx[:T], ref, n * U * size + STORE[dt] * ref.abs() * (1 + n * U), "dx")
    assert (dx[T:] == 7).all()
    ref, size = ref + add.double(), size + add.double().abs()
    into = add.to(DEV)
    api().moe_permute_backward(p, f, into, k, n_shared=ns, addend=into)
    within(into, ref, n * U * size + STORE[dt] * (ref.abs() + n * U * size), "dx + addend")


def test_entries_out_of_range_are_dropped():
    """Rows past the buffers are read and written nowhere."""
    T, k, d = 4, 2, 16
    f2r = torch.tensor([0, 8, 2 ** 31 - 1, -5, 1, 2, 3, 100], dtype=torch.int32, device=DEV)
    d_out = torch.ones((T, d), device=DEV)
    Y = torch.ones((T * k, d), device=DEV)
    dY, dw = torch.zeros((T * k, d), device=DEV), torch.empty((T, k), device=DEV)
    api().moe_combine_backward(d_out, Y, f2r, torch.ones((T, k), device=DEV), dY, dw)
    assert dw.flatten().tolist() == [d, 0, 0, 0, d, d, d, 0]
    assert dY.sum(1).tolist() == [d] * 4 + [0] * 4
    dx = torch.empty((T, d), device=DEV)
    api().moe_permute_backward(Y, f2r, dx, k)
    assert dx[:, 0].tolist() == [1, 0, 2, 1]


def test_rows_past_32_bits():
    T, k, d = 33000, 8, 8192  # 2.2e9 values in the rows
    f2r = torch.arange(T * k, dtype=torch.int32, device=DEV).flip(0).contiguous()
    d_out = torch.randn((T, d), device=DEV).to(BF)
    w = torch.rand((T, k), device=DEV)
    dY = torch.empty((T * k, d), dtype=BF, device=DEV)
    dw = torch.empty((T, k), device=DEV)
    api().moe_combine_backward(d_out, None, f2r, w, dY, None)
    for t in (0, 5, T // 2, T - 1):
        rows = f2r[t * k:t * k + k].long()
        want = (w[t][:, None] * d_out[t].float()).to(BF)
        assert torch.equal(dY[rows], want)
    api().moe_combine_backward(d_out, dY, f2r, w, None, dw)
    dx = torch.empty((T, d), dtype=F32, device=DEV)
    api().moe_permute_backward(dY, f2r, dx, k)
    for t in (0, 5, T // 2, T - 1):
        rows = dY[f2r[t * k:t * k + k].long()].double()
        within(dw[t], (rows * d_out[t].double()).sum(1).cpu(),
               ((d + 2) * U * (rows * d_out[t].double()).abs().sum(1)).cpu(), "d_topk_w")
        within(dx[t], rows.sum(0).cpu(), (10 * U * rows.abs().sum(0)).cpu(), "dx")


# ---------------------------------------------------------------------------
# the products
# ---------------------------------------------------------------------------

class Groups:
    """Operands of groups of `sizes` rows, with `spare` rows of none behind
    them, which hold NaN."""

    def __init__(self, sizes, N, K, dt, spare=3, pad=0, seed=0):
        g = gen(seed + N * 7 + K)
        self.G, self.N, self.K, self.dt = len(sizes), N, K, dt
        self.off = torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32)
        self.live = int(self.off[-1])
        self.rows = self.live + spare

        def rows(width, std=1.0):
            x = (torch.randn((self.rows, width), generator=g) * std).to(dt)
            x[self.live:] = float("nan")
            return x

        def weights():
            store = (torch.randn((self.G, N, K + pad), generator=g) * K ** -0.5).to(dt)
            store[:, :, K:] = float("nan")
            return store

        self.dC, self.dC2 = rows(N, 0.1), rows(N, 0.1)
        self.A, self.gate, self.up = rows(K), rows(K, 2.0), rows(K)
        self.B, self.B2 = weights(), weights()
        for k, t in list(self.__dict__.items()):
            if isinstance(t, torch.Tensor):
                setattr(self, "g_" + k, t.to(DEV))
        self.B, self.B2 = self.B[:, :, :K], self.B2[:, :, :K]
        self.g_B, self.g_B2 = self.g_B[:, :, :K], self.g_B2[:, :, :K]

    def groups(self):
        return [(i, int(a), int(b)) for i, (a, b) in enumerate(zip(self.off[:-1], self.off[1:]))]

    def dgrad(self, pair):
        """(dA of the live rows, bound of the sum's error)"""
        v, size = torch.zeros((self.live, self.K), dtype=F64), torch.zeros((self.live, self.K),
                                                                          dtype=F64)
        for i, a, b in self.groups():
            for dC, B in ((self.dC, self.B), (self.dC2, self.B2))[:2 if pair else 1]:
                v[a:b] += dC[a:b].double() @ B[i].double()
                size[a:b] += dC[a:b].double().abs() @ B[i].double().abs()
        return v, ((2 if pair else 1) * self.N + 2) * U * size

    def wgrad(self):
        v = torch.zeros((self.G, self.N, self.K), dtype=F64)
        e = torch.zeros_like(v)
        for i, a, b in self.groups():
            v[i] = self.dC[a:b].double().t() @ self.A[a:b].double()
            e[i] = (b - a + 2) * U * (self.dC[a:b].double().abs().t() @ self.A[a:b].double().abs())
        return v, e


SIZES = [
    [1],
    [0, 5, 0],
    [64, 1, 63, 65],
    [0, 0, 300, 127, 0, 129],
    [256, 31, 33, 257, 2],
]
WIDTHS = [(8, 8), (32, 256), (40, 264), (128, 64), (256, 512), (200, 1000), (520, 136)]


def rowbuf(o, dt):
    return torch.full((o.rows, o.K), 7.0, dtype=dt, device=DEV)


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("N,K", WIDTHS)
@pytest.mark.parametrize("dt,out", [(BF, BF), (BF, F32), (F32, F32)])
def test_dgrad(sizes, N, K, dt, out):
    o = Groups(sizes, N, K, dt, pad=16)
    for pair in (False, True):
        dA = rowbuf(o, out)
        api().moe_grouped_gemm_dgrad(o.g_dC, o.g_B, dA, o.g_off, dC2=o.g_dC2 if pair else None,
                                     B2=o.g_B2 if pair else None)
        ref, e = o.dgrad(pair)
        within(dA[:o.live], ref, e + STORE[out] * (ref.abs() + e), "dA")
        assert (dA[o.live:] == 7).all()


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("N,K", WIDTHS)
@pytest.mark.parametrize("dt", [BF, F32])
def test_dgrad_swiglu(sizes, N, K, dt):
    o = Groups(sizes, N, K, dt)
    dg, du, h = (rowbuf(o, dt) for _ in range(3))
    api().moe_grouped_gemm_dgrad_swiglu(o.g_dC, o.g_B, o.g_gate, o.g_up, dg, du, o.g_off, h=h)
    a, ea = o.dgrad(False)
    z, up = o.gate[:o.live].double(), o.up[:o.live].double()
    s = torch.sigmoid(z)
    es = (4 + 2 * z.abs()) * U
    slope = s * (1 + z * (1 - s))
    eslope = es * slope.abs() + s * (8 + 4 * z.abs()) * U * (1 + z.abs())
    st = STORE[dt]
    for got, ref, e in ((dg, a * up * slope, ea * (up * slope).abs() + (a * up).abs() * eslope),
                        (du, a * z * s, ea * (z * s).abs() + (a * z * s).abs() * es),
                        (h, z * s * up, (z * s * up).abs() * es)):
        e = 1.01 * e + 4 * U * ref.abs()
        within(got[:o.live], ref, e + st * (ref.abs() + e), "swiglu")
        assert (got[o.live:] == 7).all()
    # in place, without h
    gate, up = o.g_gate.clone(), o.g_up.clone()
    api().moe_grouped_gemm_dgrad_swiglu(o.g_dC, o.g_B, gate, up, gate, up, o.g_off)
    assert torch.equal(gate[:o.live], dg[:o.live]) and torch.equal(up[:o.live], du[:o.live])
    assert gate[o.live:].isnan().all() and up[o.live:].isnan().all()


@pytest.mark.parametrize("sizes", SIZES + [[0, 0], [700, 3]])
@pytest.mark.parametrize("N,K", WIDTHS)
@pytest.mark.parametrize("dt,out", [(BF, BF), (BF, F32), (F32, F32)])
def test_wgrad(sizes, N, K, dt, out):
    o = Groups(sizes, N, K, dt)
    dB = torch.full((o.G + 1, N, K), 7.0, dtype=out, device=DEV)
    api().moe_grouped_gemm_wgrad(o.g_dC, o.g_A, dB[:o.G], o.g_off)
    ref, e = o.wgrad()
    within(dB[:o.G], ref, e + STORE[out] * (ref.abs() + e), "dB")
    assert (dB[o.G:] == 7).all()
    base = torch.randn((o.G, N, K), generator=gen(3)).to(out)
    acc = base.to(DEV)
    api().moe_grouped_gemm_wgrad(o.g_dC, o.g_A, acc, o.g_off, accumulate=True)
    ref = ref + base.double()
    e = e + U * (ref.abs() + e)
    within(acc, ref, e + STORE[out] * (ref.abs() + e), "dB + dB")


@pytest.mark.parametrize("dt", [BF, F32])
def test_no_rows(dt):
    o = Groups([0, 0, 0], 64, 128, dt, spare=0)
    e = torch.empty
    api().moe_grouped_gemm_dgrad(o.g_dC, o.g_B, e((0, 128), dtype=dt, device=DEV), o.g_off)
    dB = torch.full((3, 64, 128), 7.0, dtype=dt, device=DEV)
    api().moe_grouped_gemm_wgrad(o.g_dC, o.g_A, dB, o.g_off, accumulate=True)
    assert (dB == 7).all()
    api().moe_grouped_gemm_wgrad(o.g_dC, o.g_A, dB, o.g_off)
    assert (dB == 0).all()


@pytest.mark.parametrize("off", [[0, 90, 40, 120], [0, 30, 1 << 30, 60], [-7, 20, 60, 10],
                                 [50, 50, 50, 50], [5, 20, 100, 119]])
@pytest.mark.parametrize("dt", [BF, F32])
def test_offsets_that_are_not_offsets(off, dt):
    """Clamped to the rows and read as their running maximum, as in the
    forward product."""
    o = Groups([40, 40, 40], 64, 256, dt, spare=0)
    bad = torch.tensor(off, dtype=torch.int32, device=DEV)
    run, at = 0, []
    for v in off:
        run = max(run, min(max(v, 0), 120))
        at.append(run)
    o.off = torch.tensor(at)
    o.live = 120
    dA = torch.full((120, 256), 7.0, dtype=F32, device=DEV)
    api().moe_grouped_gemm_dgrad(o.g_dC, o.g_B, dA, bad)
    ref, e = o.dgrad(False)
    in_group = torch.zeros(120, dtype=torch.bool)
    in_group[at[0]:at[-1]] = True
    within(dA[in_group.to(DEV)], ref[in_group], (e + U * (ref.abs() + e))[in_group], "dA")
    assert (dA[~in_group.to(DEV)] == 7).all()
    dB = torch.empty((3, 64, 256), dtype=F32, device=DEV)
    api().moe_grouped_gemm_wgrad(o.g_dC, o.g_A, dB, bad)
    ref, e = o.wgrad()
    within(dB, ref, e + U * (ref.abs() + e), "dB")


@pytest.mark.parametrize("dt", [BF, F32])
def test_a_group_never_meets_anothers_values(dt):
    """An infinity or NaN in one group's rows or weights changes no bit of
    another group's gradients."""
    o = Groups([70, 50, 90], 136, 264, dt, spare=0)

    def all_of():
        dA, dB = rowbuf(o, dt), torch.empty((3, o.N, o.K), dtype=dt, device=DEV)
        api().moe_grouped_gemm_dgrad(o.g_dC, o.g_B, dA, o.g_off)
        api().moe_grouped_gemm_wgrad(o.g_dC, o.g_A, dB, o.g_off)
        return dA, dB

    dA, dB = all_of()
    o.g_dC[70], o.g_A[119], o.g_dC[119, 3] = float("nan"), float("inf"), float("inf")
    o.g_B[1, 5] = float("nan")
    dA2, dB2 = all_of()
    for a, b in ((0, 70), (120, 210)):
        assert torch.equal(dA[a:b], dA2[a:b])
    assert torch.equal(dB[0], dB2[0]) and torch.equal(dB[2], dB2[2])
    assert dB2[1].isnan().all()


@pytest.mark.parametrize("dt", [BF, F32])
def test_infinities_in_the_last_terms(dt):
    """The sums' padding behind their last term is zero for both operands: an
    infinity in the last row or column gives an infinity, not NaN."""
    o = Groups([5], 40, 72, dt, spare=0)
    dC = torch.ones((5, 40), dtype=dt, device=DEV)
    dC[4, 39] = float("inf")
    B = torch.ones((1, 40, 72), dtype=dt, device=DEV)
    B[0, 39, 71] = float("inf")
    A = torch.ones((5, 72), dtype=dt, device=DEV)
    A[4, 71] = float("inf")
    dA, dB = rowbuf(o, dt), torch.empty((1, 40, 72), dtype=dt, device=DEV)
    api().moe_grouped_gemm_dgrad(dC, B, dA, o.g_off)
    assert dA[:4, :71].eq(40).all() and dA[4].eq(float("inf")).all() and dA[:, 71].isinf().all()
    api().moe_grouped_gemm_wgrad(dC, A, dB, o.g_off)
    assert dB[0, :39, :71].eq(5).all() and dB[0, 39].isinf().all() and dB[0, :, 71].isinf().all()


def test_products_past_32_bits():
    """Rows, gradients and weights of more than 2^31 values."""
    rows, N, K = 270000, 8, 8192
    dC = torch.zeros((rows, N), dtype=BF, device=DEV)
    dC[-1], dC[7] = 1.0, 2.0
    B = torch.ones((2, N, K), dtype=BF, device=DEV)
    off = torch.tensor([0, 100, rows], dtype=torch.int32, device=DEV)
    dA = torch.full((rows, K), 7.0, dtype=BF, device=DEV)
    api().moe_grouped_gemm_dgrad(dC, B, dA, off)
    assert (dA[-1] == 8).all() and (dA[7] == 16).all() and (dA[-2] == 0).all()
    A = dA
    A.fill_(0.5)
    dB = torch.empty((2, N, K), dtype=F32, device=DEV)
    api().moe_grouped_gemm_wgrad(dC, A, dB, off)
    assert (dB[0] == 1).all() and (dB[1] == 0.5).all()
    del dA, A
    G, N, K = 40, 8192, 8192
    dC, A = torch.ones((3, N), dtype=BF, device=DEV), torch.ones((3, K), dtype=BF, device=DEV)
    off = torch.full((G + 1,), 3, dtype=torch.int32, device=DEV)
    off[:G] = 0
    W = torch.full((G, N, K), 7.0, dtype=BF, device=DEV)
    api().moe_grouped_gemm_wgrad(dC, A, W, off)
    assert (W[G - 1] == 3).all() and (W[G - 2] == 0).all() and (W[0] == 0).all()
    dA = torch.empty((3, K), dtype=F32, device=DEV)
    api().moe_grouped_gemm_dgrad(dC, W, dA, off)
    assert (dA == 3.0 * N).all()


def test_many_groups():
    G = 1040
    sizes = [(i * 7) % 5 for i in range(G)]
    o = Groups(sizes, 16, 24, BF, spare=1)
    dA = rowbuf(o, F32)
    api().moe_grouped_gemm_dgrad(o.g_dC, o.g_B, dA, o.g_off)
    ref, e = o.dgrad(False)
    within(dA[:o.live], ref, e + U * (ref.abs() + e), "dA")
    dB = torch.empty((G, 16, 24), dtype=F32, device=DEV)
    api().moe_grouped_gemm_wgrad(o.g_dC, o.g_A, dB, o.g_off)
    ref, e = o.wgrad()
    within(dB, ref, e + U * (ref.abs() + e), "dB")


@pytest.mark.parametrize("dt", [BF, F32])
def test_another_stream_and_a_captured_graph(dt):
    """Calls on a side stream, and replays of a captured run of them between
    eager work, give the eager call's bits."""
    o = Groups([130, 0, 77, 300], 256, 512, dt)

    def step(dg, du, dA, dB, stream=None):
        a = api()
        a.moe_grouped_gemm_dgrad_swiglu(o.g_dC, o.g_B, o.g_gate, o.g_up, dg, du, o.g_off,
                                        stream=stream)
        a.moe_grouped_gemm_dgrad(o.g_dC, o.g_B, dA, o.g_off, dC2=o.g_dC2, B2=o.g_B2, stream=stream)
        a.moe_grouped_gemm_wgrad(o.g_dC, dA, dB, o.g_off, stream=stream)

    def new():
        return [rowbuf(o, dt) for _ in range(3)] + [torch.empty((o.G, o.N, o.K), dtype=dt,
                                                                 device=DEV)]

    def same(x, y):
        return all(torch.equal(a[:o.live], b[:o.live]) for a, b in zip(x[:3], y[:3])) and \
            torch.equal(x[3], y[3])

    want = new()
    step(*want)
    side, got = torch.cuda.Stream(), new()
    side.wait_stream(torch.cuda.current_stream())
    step(*got, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert same(got, want)
    got = new()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*got)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*got)
    for _ in range(3):
        for t in got:
            t.fill_(9.0)
        graph.replay()
        again = new()
        step(*again)
        torch.cuda.synchronize()
        assert same(got, want) and same(again, want)
