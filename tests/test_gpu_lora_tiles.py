"""GPU parity of the adapters' kernels that the size lists of test_gpu_lora.py
do not choose: fp32 tiles of 64 x 64, which run from as many tiles as the GPU
has compute units on, and fp32 batches whose rows the forward pass sorts
(more than 250 MB of factors to read row by row); and the row pitches of W
that bf16 tiles treat apart.  References and tolerances are those of
test_gpu_lora.py."""
import pytest
import torch

from gpu_util import DEV
from test_gpu_lora import BF, F32, Case, check_backward, check_forward, forward

pytestmark = pytest.mark.gpu


def full(T, N):
    """Whether the fp32 outputs [T][N] fill the chip with 64 x 64 tiles."""
    cus = torch.cuda.get_device_properties(DEV).multi_processor_count
    return -(-T // 64) * -(-N // 64) >= cus


# (T, N, K, r, n): K that ends inside a step of 64 and K of several steps, odd
# N, T that ends inside a tile; the last two are sorted
WIDE = [(1100, 1025, 72, 8, 3), (1025, 1090, 264, 24, 5), (2111, 577, 128, 16, 40),
        (16385, 8, 8, 8, 2), (1, 16400, 136, 8, 2), (1300, 1000, 200, 64, 9),
        (1100, 1031, 328, 128, 70)]


@pytest.mark.parametrize("kind", ["requests", "mixed"])
@pytest.mark.parametrize("with_w", [True, False])
@pytest.mark.parametrize("T,N,K,r,n", WIDE)
def test_forward_f32_wide(T, N, K, r, n, with_w, kind):
    print("lora f32 wide", T, N, K, r, n, with_w, kind, flush=True)
    assert full(T, N)
    check_forward(Case(T, N, K, r, n, F32, kind, T + N).gpu(), F32, with_w=with_w)


@pytest.mark.parametrize("kind", ["requests", "mixed"])
def test_forward_f32_sorted_small_tiles(kind):
    """463 MB of factors, 187 tiles of 64 x 64: sorted rows in tiles of 32 x 32."""
    assert not full(700, 1030)
    check_forward(Case(700, 1030, 264, 128, 12, F32, kind, 3).gpu(), F32)


def test_forward_f32_wide_padded_rows_of_w():
    check_forward(Case(1100, 1025, 136, 16, 4, F32, "mixed", 4).gpu(), F32, ldw_pad=12)


@pytest.mark.parametrize("kind", ["requests", "mixed"])
@pytest.mark.parametrize("with_w", [True, False])
@pytest.mark.parametrize("T,N,K,r,n", [(1100, 72, 1032, 8, 3), (1090, 136, 1000, 40, 20),
                                       (4100, 64, 264, 16, 5)])
def test_backward_f32_wide(T, N, K, r, n, with_w, kind):
    print("lora f32 backward wide", T, N, K, r, n, with_w, kind, flush=True)
    assert full(T, K)
    check_backward(Case(T, N, K, r, n, F32, kind, T).gpu(), with_w=with_w)


@pytest.mark.parametrize("r", [16, 64])
def test_one_request_never_meets_another_wide(r):
    """As in test_gpu_lora.py, on 64 x 64 tiles of rows as they come and
    sorted: what is not finite in one request changes no bit of the others."""
    c = Case(1300, 1000, 200, r, 4, F32, "mixed", 7).gpu()
    assert full(1300, 1000)
    y0, v0 = forward(c, F32)
    c.g_A[2], c.g_B[2] = float("nan"), float("inf")
    c.g_x[650] = float("nan")
    y1, v1 = forward(c, F32)
    keep = (c.adapter != 2) & (torch.arange(1300) != 650)
    assert torch.equal(y0.cpu()[keep], y1.cpu()[keep])
    assert torch.equal(v0.cpu()[keep], v1.cpu()[keep])


@pytest.mark.parametrize("T,N,K,pad", [
    # rows of W a multiple of 4 KB apart, where workgroups begin at different K:
    # dense, and behind 1984 columns of 2048 (and 2040, which end inside a step)
    (40, 264, 2048, 0), (128, 1000, 4096, 0), (100, 520, 1984, 64), (64, 300, 2040, 8),
    # other pitches, and rows one too many
    (40, 264, 2048, 128), (128, 1000, 4096, 128), (129, 264, 2048, 0)])
def test_forward_bf16_row_pitches(T, N, K, pad):
    print("lora pitch", T, N, K, pad, flush=True)
    check_forward(Case(T, N, K, 16, 5, BF, "mixed", T + N).gpu(), BF, ldw_pad=pad)


@pytest.mark.parametrize("kind", ["requests", "mixed"])
@pytest.mark.parametrize("dt,T,N,K,r,n", [
    (BF, 2049, 40, 64, 128, 8), (BF, 8200, 8, 8, 8, 3), (BF, 300, 65, 72, 56, 700),
    (BF, 128, 33, 16, 128, 2), (F32, 2049, 40, 64, 128, 8), (F32, 4100, 17, 8, 8, 90)])
def test_many_rows_of_short_factors(dt, T, N, K, r, n, kind):
    """Batches that are sorted for their number of rows and ranks alone."""
    print("lora short", dt, T, N, K, r, n, kind, flush=True)
    c = Case(T, N, K, r, n, dt, kind, T).gpu()
    check_forward(c, dt)
    check_forward(c, F32, with_w=False)
