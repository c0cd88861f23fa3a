"""GPU parity of the products' gradients where they have tiles enough to fill
the chip, random values throughout: the tile orders over the XCDs, the rings'
unrolled loops with a last stage that ends inside, whole tiles of 256, 192, 128
and 64 rows, and outputs of more than 256 MB, which are stored past the caches.
References in 64 bits on the device, group by group.

Tolerances as in test_gpu_backward.py: a sum of m products errs by at most
(m + 2) u times its terms' sizes (u = 2^-24), and is rounded once when stored."""
import pytest
import torch

from gpu_util import DEV
from test_gpu_backward import BF, F32, STORE, U, api

pytestmark = pytest.mark.gpu

# groups whose last tiles have 192, 128 and 64 rows, a row less and more, none
FEW = [192, 448, 128, 384, 64, 320, 0, 1, 31, 257, 511, 256, 200, 450, 129, 193, 65, 400, 300, 500,
       512, 96]
MANY = [2100, 905, 0, 1728, 449]


class Operands:
    """Of groups of `sizes` rows, with five rows of none behind them (NaN)."""

    def __init__(self, sizes, dt, seed):
        self.sizes, self.dt, self.G = sizes, dt, len(sizes)
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        ends = torch.tensor(sizes).cumsum(0)
        self.off = torch.cat([ends.new_zeros(1), ends]).to(torch.int32).to(DEV)
        self.live = int(ends[-1])
        self.rows = self.live + 5
        self.spans = list(zip([0] + ends.tolist()[:-1], ends.tolist()))

    def of_rows(self, width, std=1.0):
        x = (torch.randn((self.rows, width), generator=self.g, device=DEV) * std).to(self.dt)
        x[self.live:] = float("nan")
        return x

    def weights(self, N, K, pad):
        w = (torch.randn((self.G, N, K + pad), generator=self.g, device=DEV) * K ** -0.5).to(self.dt)
        w[:, :, K:] = float("nan")
        return w[:, :, :K]

    def filled(self, width, dt):
        return torch.full((self.rows, width), 7.0, dtype=dt, device=DEV)


def within(got, ref, bound, what):
    err = (got.double() - ref).abs_()
    ok = err <= bound.add_(1e-37)  # (NaN is not)
    assert ok.all(), "%s: %d of %d outside" % (what, int((~ok).sum()), ok.numel())


def sums(parts, m):
    """A sum of products of 64-bit operands, and the bound of its fp32 error."""
    ref = sum(x @ y for x, y in parts)
    return ref, sum(x.abs() @ y.abs() for x, y in parts).mul_((m + 2) * U)


def stored(ref, e, dt):
    return e + STORE[dt] * (ref.abs() + e)


def check_dgrad(sizes, N, K, dt, out, form, pad, seed):
    o = Operands(sizes, dt, seed)
    a = api()
    assert a.moe_grouped_gemm_dgrad_workspace_size(o.G, o.rows, N, K, dt) == 0, "this shape is cut"
    dC, B = o.of_rows(N, 0.1), o.weights(N, K, pad)
    if form.startswith("swiglu"):
        gate, up = o.of_rows(K, 2.0), o.of_rows(K)
        dg, du = o.filled(K, dt), o.filled(K, dt)
        h = o.filled(K, dt) if form == "swiglu with h" else None
        a.moe_grouped_gemm_dgrad_swiglu(dC, B, gate, up, dg, du, o.off, h=h)
        results = [dg, du] + ([h] if h is not None else [])
    else:
        pair = form == "pair"
        dC2, B2 = (o.of_rows(N, 0.1), o.weights(N, K, pad)) if pair else (None, None)
        dA = o.filled(K, out)
        a.moe_grouped_gemm_dgrad(dC, B, dA, o.off, dC2=dC2, B2=B2)
        results = [dA]
    for i, (r0, r1) in enumerate(o.spans):
        parts = [(dC[r0:r1].double(), B[i].double())]
        if form == "pair":
            parts.append((dC2[r0:r1].double(), B2[i].double()))
        ref, e = sums(parts, N * len(parts))
        if not form.startswith("swiglu"):
            within(dA[r0:r1], ref, stored(ref, e, out), "dA of group %d" % i)
            continue
        z, u = gate[r0:r1].double(), up[r0:r1].double()
        s = torch.sigmoid(z)
        es = (4 + 2 * z.abs()) * U
        slope = s * (1 + z * (1 - s))
        eslope = es * slope.abs() + s * (8 + 4 * z.abs()) * U * (1 + z.abs())
        wanted = [(dg, ref * u * slope, e * (u * slope).abs() + (ref * u).abs() * eslope),
                  (du, ref * z * s, e * (z * s).abs() + (ref * z * s).abs() * es)]
        if h is not None:
            wanted.append((h, z * s * u, (z * s * u).abs() * es))
        for n, (got, want, err) in enumerate(wanted):
            err = 1.01 * err + 4 * U * want.abs()
            within(got[r0:r1], want, stored(want, err, dt), "output %d of group %d" % (n, i))
    assert all((r[o.live:] == 7).all() for r in results)


@pytest.mark.parametrize("sizes", [FEW, MANY], ids=["few rows a group", "many"])
@pytest.mark.parametrize("N", [520, 576, 1032])
@pytest.mark.parametrize("form,out", [("one", BF), ("pair", F32), ("swiglu with h", BF)])
def test_dgrad_of_many_tiles(sizes, N, form, out):
    K = 4104  # 17 tiles, the last of 8 columns
    assert sum(-(-n // 256) for n in sizes) * 17 >= 256
    check_dgrad(sizes, N, K, BF, out, form, 16, N)


@pytest.mark.parametrize("sizes,K,form,out", [
    ([4100, 12301], 8256, "one", BF), ([4100, 12301], 8256, "pair", BF),
    ([3000, 0, 5201], 8256, "one", F32), (FEW + FEW, 8224, "pair", F32),
    ([5000, 3201], 5568, "swiglu with h", BF), (FEW + FEW, 6592, "swiglu", BF)])
@pytest.mark.parametrize("N", [136, 520])
def test_dgrad_to_more_than_the_last_level_cache(sizes, K, form, out, N):
    size = 2 if out == BF else 4
    arrays = {"one": 1, "pair": 1, "swiglu": 2, "swiglu with h": 3}[form]
    assert sum(sizes) * K * size * arrays > 256 << 20 and K * size % 128 == 0
    check_dgrad(sizes, N, K, BF, out, form, 0, N + K)


@pytest.mark.parametrize("form", ["one", "pair", "swiglu with h"])
@pytest.mark.parametrize("N", [264, 1032])
def test_dgrad_of_many_fp32_tiles(form, N):
    check_dgrad([700, 0, 301, 64], N, 2056, F32, F32, form, 16, N)


def check_wgrad(sizes, N, K, dt, out, accumulate, seed):
    o = Operands(sizes, dt, seed)
    a = api()
    assert a.moe_grouped_gemm_wgrad_workspace_size(o.G, o.rows, N, K, dt) == 0, "this shape is cut"
    dC, A = o.of_rows(N, 0.1), o.of_rows(K)
    dB = torch.randn((o.G, N, K), generator=o.g, device=DEV).to(out)
    base = dB.clone() if accumulate else None
    a.moe_grouped_gemm_wgrad(dC, A, dB, o.off, accumulate=accumulate)
    for i, (r0, r1) in enumerate(o.spans):
        x, y = dC[r0:r1].double().t().contiguous(), A[r0:r1].double()
        ref, e = sums([(x, y)], r1 - r0)
        if accumulate:
            ref = ref + base[i].double()
            e = e + U * (ref.abs() + e)
        within(dB[i], ref, stored(ref, e, out), "dB of group %d" % i)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("sizes,N,K", [([33, 100, 0, 161, 700, 31, 1505, 352], 1416, 2056),
                                       ([2049, 159], 1032, 4096), ([700], 2048, 2304)])
def test_wgrad_of_many_tiles(sizes, N, K, out, accumulate):
    check_wgrad(sizes, N, K, BF, out, accumulate, N)


@pytest.mark.parametrize("sizes,N,K,out", [([33, 100, 0, 161, 700, 31, 1505, 352, 64], 3000, 4992, BF),
                                           ([290, 97, 450], 4096, 5504, F32)])
def test_wgrad_to_more_than_the_last_level_cache(sizes, N, K, out):
    size = 2 if out == BF else 4
    assert len(sizes) * N * K * size > 256 << 20 and K * size % 128 == 0
    check_wgrad(sizes, N, K, BF, out, False, N)


def test_wgrad_of_one_long_sum():
    """32768 rows in one accumulator."""
    check_wgrad([32768], 2048, 2304, BF, F32, False, 1)


@pytest.mark.parametrize("accumulate", [False, True])
def test_wgrad_of_many_fp32_tiles(accumulate):
    check_wgrad([1000, 0, 37, 257], 712, 1032, F32, F32, accumulate, 2)
