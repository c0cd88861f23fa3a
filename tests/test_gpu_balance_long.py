"""moe_balance_loss over long sequences: the error of probs does not grow with
their length.

Tolerances (u = 2^-24): a softmax term as in test_gpu_balance.py, (E + 60) u.
The sum of a block's tokens adds at most 8 tokens a lane, 5 exchanges and 8
waves, 20 roundings; four blocks are added in 32 bits and the rest of a wave's
in 64, 4 more with their rounding; 16 waves, the count's rounding and the
division are 18.  The loss adds E products (two roundings each), sums of E terms
and of the sequences, and the factors: 2 E + S + 30."""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ALPHA = 0.02


def run(logits, idx, off):
    from grouped_gemm_router_amd import api
    T, E = logits.shape
    S = 1 if off is None else off.numel() - 1
    out = (torch.full((S, E), -7, dtype=torch.int32, device=DEV),
           torch.full((S, E), float("nan"), device=DEV),
           torch.full((S + 1,), -7, dtype=torch.int32, device=DEV),
           torch.full((1,), float("nan"), device=DEV))
    api.moe_balance_loss(logits, idx, *out, alpha=ALPHA, seq_offsets=off)
    torch.cuda.synchronize()
    return [t.cpu() for t in out]


def check(got, counts, probs, lengths, k):
    """counts, probs [S][E] in 64 bits against what the call wrote."""
    S, E = probs.shape
    assert torch.equal(got[0].long(), counts)
    assert got[2].tolist() == lengths + [S]
    tol = (E + 60 + 42) * U
    err = ((got[1].double() - probs).abs() / probs).max()
    assert float(err) <= tol, float(err) / U
    n = torch.tensor(lengths, dtype=torch.float64)[:, None]
    loss = ALPHA * E * float((counts.double() / (n * k) * probs).sum()) / S
    assert abs(float(got[3]) - loss) <= (tol + (2 * E + S + 30) * U) * loss


@pytest.mark.parametrize("T", [(1 << 22) + 77, (1 << 24) + 12345])
def test_equal_tokens(T):
    """Every block's sum is the same number: roundings of a running 32-bit sum
    would all fall on one side."""
    print("balance long", T, flush=True)
    row = torch.tensor([0.0, 1.7])
    logits = row.to(DEV).repeat(T, 1)
    idx = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    check(run(logits, idx, None), torch.tensor([[T, 0]]),
          torch.softmax(row.double(), 0)[None], [T], 1)


@pytest.mark.parametrize("T,E,k,ends", [(131071, 64, 6, []), (300001, 60, 4, [7, 200000])])
def test_one_long_sequence_and_several(T, E, k, ends):
    print("balance long", T, E, k, ends, flush=True)
    g = torch.Generator(device=DEV).manual_seed(T)
    logits = 1.5 * torch.randn((T, E), generator=g, device=DEV)
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    cut = [0] + ends + [T]
    off = torch.tensor(cut, dtype=torch.int32, device=DEV) if ends else None
    p = torch.softmax(logits.double(), 1)
    parts = list(zip(cut[:-1], cut[1:]))
    probs = torch.stack([p[a:b].mean(0) for a, b in parts]).cpu()
    counts = torch.stack([torch.bincount(idx[a:b].flatten().long(), minlength=E)
                          for a, b in parts]).cpu()
    check(run(logits, idx, off), counts, probs, [b - a for a, b in parts], k)
