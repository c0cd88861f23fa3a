"""CPU checks of the size limits that include/moe_backward.h states: the first
size past each is refused as unsupported, and the last one before it gets as
far as the next check (a missing pointer).  Nothing is launched."""
import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from grouped_gemm_router_amd import api
    return api.lib


def past(lib, T=4, k=2, d=64, ns=0):
    """Status of both with no arrays: INVALID once the sizes are taken."""
    a = lib.moe_combine_backward(None, BF16, None, F32, None, None, T, k, d, ns, None, None, None)
    b = lib.moe_permute_backward(None, F32, None, T, k, d, ns, None, None, BF16, None)
    assert a == b
    return a


def test_combine_and_permute(lib):
    assert past(lib) == INVALID and past(lib, T=0) == OK
    for last, first in ((dict(T=(1 << 24) - 1), dict(T=1 << 24)),
                        (dict(T=(1 << 24) - 1, k=32, ns=8), dict(T=1 << 24, k=1)),
                        (dict(k=32), dict(k=33)), (dict(ns=8), dict(ns=9)),
                        (dict(d=72), dict(d=76))):
        assert past(lib, **last) == INVALID and past(lib, **first) == UNSUPPORTED, first


def products(lib, G=2, rows=16, N=64, K=64, ldb=0, dt=BF16):
    a = lib.moe_grouped_gemm_dgrad(None, None, None, None, dt, None, dt, None, G, rows, N, K, ldb,
                                   None, 0, None)
    b = lib.moe_grouped_gemm_dgrad_swiglu(None, None, dt, None, None, None, None, None, None, G,
                                          rows, N, K, ldb, None, 0, None)
    assert a == b
    if ldb == 0:
        assert lib.moe_grouped_gemm_wgrad(None, None, dt, None, dt, None, G, rows, N, K, 0, None, 0,
                                          None) == a
    return a


def test_products(lib):
    assert products(lib) == INVALID
    wide = 1 << 23
    for last, first in ((dict(N=wide - 8, K=8), dict(N=wide, K=8)),
                        (dict(N=8, K=wide - 8), dict(N=8, K=wide)),
                        (dict(N=8, K=64, ldb=wide - 8), dict(N=8, K=64, ldb=wide)),
                        # G N ldb < 2^40, with narrow weights in wide rows
                        (dict(G=2, N=(1 << 17) - 8, K=8, ldb=1 << 22),
                         dict(G=2, N=1 << 17, K=8, ldb=1 << 22)),
                        # (rows / 64 + G) K / 64 and G N K / 4096, in whole tiles
                        (dict(G=1, rows=(1 << 29) - 128, N=8, K=128),
                         dict(G=1, rows=(1 << 29) - 64, N=8, K=128)),
                        (dict(G=16, rows=1, N=65536, K=65472), dict(G=16, rows=1, N=65536, K=65536)),
                        (dict(N=72, K=72), dict(N=76)), (dict(), dict(K=76))):
        assert products(lib, **last) == INVALID, last
        assert products(lib, **first) == UNSUPPORTED, first
