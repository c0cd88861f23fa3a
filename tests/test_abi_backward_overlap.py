"""CPU checks that the backward calls refuse an output that overlaps an operand,
another output or the workspace, in part too, before anything is launched.  No
GPU is touched: every call here is refused."""
import ctypes as C

import pytest

INVALID = 1
F32, BF16 = 0, 1
NUL = None
BASE = 0x10000000  # the operands' places, far apart
FAR = 0x1000000


@pytest.fixture(scope="module")
def lib():
    from grouped_gemm_router_amd import api
    return api.lib


def refused(fn, sizes, args, apart, may_equal=()):
    """Every pair of `apart` (an output, anything) refused with the output
    beginning in the other's last 16 bytes or inside it, ending in its first
    16, and in the same place unless the pair may be the same."""
    home = {n: BASE + i * FAR for i, n in enumerate(sizes)}
    for out, other in apart:
        first, size = home[other], sizes[other]
        spots = {first + (size - 1) // 16 * 16, first - (sizes[out] - 1) // 16 * 16,
                 first + size // 32 * 16, first} - ({first} if (out, other) in may_equal else set())
        assert len(spots) > 1
        for at in spots:
            got = fn(*args({n: C.c_void_p(v) for n, v in {**home, out: at}.items()}))
            assert got == INVALID, (out, other, hex(at))


def pairs(outs, ins):
    return [(o, i) for o in outs for i in ins] + [(a, b) for a in outs for b in outs if a != b]


@pytest.mark.parametrize("dt,ydt", [(BF16, F32), (F32, BF16), (F32, F32)])
def test_combine(lib, dt, ydt):
    T, k, d, ns = 6, 3, 64, 1
    es, ys, R = 4 if dt == F32 else 2, 4 if ydt == F32 else 2, T * (k + ns)
    sizes = dict(d_out=T * d * es, Y=R * d * ys, f2r=R * 4, w=T * k * 4, dY=R * d * es,
                 dw=T * k * 4)

    def args(p):
        return (p["d_out"], dt, p["Y"], ydt, p["f2r"], p["w"], T, k, d, ns, p["dY"], p["dw"], NUL)

    refused(lib.moe_combine_backward, sizes, args,
            pairs(["dY", "dw"], ["d_out", "Y", "f2r", "w"]), may_equal=[("dw", "w")])


@pytest.mark.parametrize("pdt,dt", [(BF16, F32), (F32, BF16)])
def test_permute(lib, pdt, dt):
    T, k, d, ns = 6, 3, 64, 1
    ps, es, R = 4 if pdt == F32 else 2, 4 if dt == F32 else 2, T * (k + ns)
    sizes = dict(p=R * d * ps, f2r=R * 4, add=T * d * es, dx=T * d * es)

    def args(p):
        return (p["p"], pdt, p["f2r"], T, k, d, ns, p["add"], p["dx"], dt, NUL)

    refused(lib.moe_permute_backward, sizes, args,
            pairs(["dx"], ["p", "f2r", "add"]), may_equal=[("dx", "add")])


G, ROWS = 2, 48


def product_sizes(N, K, ldb, es, os, ws):
    return dict(dC=ROWS * N * es, B=((G * N - 1) * ldb + K) * es, off=(G + 1) * 4,
                dA=ROWS * K * os, ws=ws)


@pytest.mark.parametrize("N,ldb", [(64, 0), (64, 80), (2048, 0)])  # the last is cut: a workspace
@pytest.mark.parametrize("dt,out,pair", [(BF16, BF16, False), (BF16, F32, True), (F32, F32, True)])
def test_dgrad(lib, N, ldb, dt, out, pair):
    K = 64
    need = lib.moe_grouped_gemm_dgrad_workspace_size(G, ROWS, N, K, dt)
    assert (need > 0) == (N > 64)
    sizes = product_sizes(N, K, ldb or K, 2 if dt == BF16 else 4, 2 if out == BF16 else 4, need)
    if pair:
        sizes["dC2"], sizes["B2"] = sizes["dC"], sizes["B"]

    def args(p):
        return (p["dC"], p["B"], p.get("dC2"), p.get("B2"), dt, p["dA"], out, p["off"], G, ROWS, N,
                K, ldb, p["ws"] if need else NUL, need, NUL)

    ins = ["dC", "B", "off"] + (["dC2", "B2"] if pair else [])
    refused(lib.moe_grouped_gemm_dgrad, sizes, args,
            pairs(["dA"] + (["ws"] if need else []), ins))


@pytest.mark.parametrize("N", [64, 2048])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("with_h", [True, False])
def test_dgrad_swiglu(lib, N, dt, with_h):
    K, es = 64, 2 if dt == BF16 else 4
    need = lib.moe_grouped_gemm_dgrad_workspace_size(G, ROWS, N, K, dt)
    sizes = product_sizes(N, K, K, es, es, need)
    of = sizes.pop("dA")
    sizes.update({n: of for n in ("gate", "up", "dg", "du", "h")})

    def args(p):
        return (p["dC"], p["B"], dt, p["gate"], p["up"], p["dg"], p["du"], p["h"] if with_h else NUL,
                p["off"], G, ROWS, N, K, 0, p["ws"] if need else NUL, need, NUL)

    outs = ["dg", "du"] + (["h"] if with_h else []) + (["ws"] if need else [])
    refused(lib.moe_grouped_gemm_dgrad_swiglu, sizes, args,
            pairs(outs, ["dC", "B", "off", "gate", "up"]),
            may_equal=[("dg", "gate"), ("du", "up")])


@pytest.mark.parametrize("rows", [48, 4096])
@pytest.mark.parametrize("dt,out", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_wgrad(lib, rows, dt, out):
    N, K, es = 64, 72, 2 if dt == BF16 else 4
    need = lib.moe_grouped_gemm_wgrad_workspace_size(G, rows, N, K, dt)
    assert (need > 0) == (rows > 48)
    sizes = dict(dC=rows * N * es, A=rows * K * es, dB=G * N * K * (2 if out == BF16 else 4),
                 off=(G + 1) * 4, ws=need)

    def args(p):
        return (p["dC"], p["A"], dt, p["dB"], out, p["off"], G, rows, N, K, 0,
                p["ws"] if need else NUL, need, NUL)

    refused(lib.moe_grouped_gemm_wgrad, sizes, args,
            pairs(["dB"] + (["ws"] if need else []), ["dC", "A", "off"]))


def test_norm(lib):
    need = lib.moe_grad_norm_workspace_size(3)
    grads = [(BASE, 100), (BASE + FAR, 8), (BASE + 2 * FAR, 4096)]
    ptrs = (C.c_void_p * 3)(*[g[0] for g in grads])
    n = (C.c_int64 * 3)(*[g[1] for g in grads])
    dts = (C.c_int * 3)(F32, BF16, F32)
    for at, size in zip([g[0] for g in grads], [400, 16, 4 * 4096]):
        for ws in (at, at + (size - 1) // 8 * 8, at - need + 8):
            assert lib.moe_grad_norm(ptrs, n, dts, 3, C.c_void_p(BASE - FAR), C.c_void_p(ws), need,
                                     NUL) == INVALID
        for norm in (at, at + (size - 1) // 4 * 4):  # (the norm itself, on a gradient)
            assert lib.moe_grad_norm(ptrs, n, dts, 3, C.c_void_p(norm), C.c_void_p(BASE - FAR), need,
                                     NUL) == INVALID
    for norm in (BASE - FAR, BASE - FAR + need - 4):  # on the workspace
        assert lib.moe_grad_norm(ptrs, n, dts, 3, C.c_void_p(norm), C.c_void_p(BASE - FAR), need,
                                 NUL) == INVALID
