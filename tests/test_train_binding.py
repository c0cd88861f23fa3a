"""CPU checks of the layer's training methods and of the adapters' binding:
what they pass on and what they refuse, with the library's calls recorded
instead of made."""
import ctypes as C

import pytest
import torch

from grouped_gemm_router_amd import api
from grouped_gemm_router_amd.layer import MoELayer

T, E, K = 6, 8, 2


@pytest.fixture
def calls(monkeypatch):
    """The library's training calls, recorded as (name, positional, keywords)."""
    seen = []
    for name in ("moe_balance_loss", "moe_route_backward"):
        monkeypatch.setattr(api, name,
                            lambda *a, _n=name, **k: seen.append((_n, a, k)))
    return seen


def layer():
    """A layer after a forward pass, without weights."""
    m = MoELayer.__new__(MoELayer)
    m.E, m.k, m.flags, m.device = E, K, api.MOE_ROUTE_RENORM, torch.device("cpu")
    m.logits = torch.zeros((T, E))
    m.topk_idx = torch.zeros((T, K), dtype=torch.int32)
    return m


def test_the_gradient_takes_the_losss_alpha_sequences_and_mask(calls):
    m = layer()
    off = torch.tensor([0, 2, 5], dtype=torch.int32)
    mask = torch.ones(T, dtype=torch.bool)
    bal = m.balance_loss(0.25, seq_offsets=off, token_mask=mask)
    dw = torch.zeros((T, K))
    m.route_backward(dw, balance=bal)
    m.route_backward(dw, balance=bal, alpha=0.25, seq_offsets=off.clone(), token_mask=mask.clone())
    for name, _, kw in calls[1:]:
        assert name == "moe_route_backward" and kw["alpha"] == 0.25
        assert kw["counts"] is bal["counts"] and kw["tokens"] is bal["tokens"]
        assert torch.equal(kw["seq_offsets"], off) and torch.equal(kw["token_mask"], mask)


def test_a_gradient_that_disagrees_with_its_loss_is_refused(calls):
    m = layer()
    off = torch.tensor([0, T], dtype=torch.int32)
    mask = torch.ones(T, dtype=torch.bool)
    bal = m.balance_loss(0.25)
    for bad in (dict(alpha=0.01), dict(seq_offsets=off), dict(token_mask=mask)):
        with pytest.raises(ValueError, match=next(iter(bad))):
            m.route_backward(balance=bal, **bad)
    assert [c[0] for c in calls] == ["moe_balance_loss"]


def test_a_gradient_without_the_layers_loss(calls):
    """The gate's part alone, and counts and tokens from elsewhere: as given,
    alpha 0.01 by default."""
    m = layer()
    mask = torch.ones(T, dtype=torch.bool)
    m.route_backward(torch.zeros((T, K)), token_mask=mask)
    own = {"counts": torch.zeros((1, E), dtype=torch.int32),
           "tokens": torch.zeros(2, dtype=torch.int32)}
    m.route_backward(balance=own, token_mask=mask)
    m.route_backward(balance=own, alpha=0.5)
    (_, _, a), (_, _, b), (_, _, c) = calls
    assert a["alpha"] == b["alpha"] == 0.01 and c["alpha"] == 0.5
    assert a["counts"] is None and b["counts"] is own["counts"]
    assert a["token_mask"] is mask and b["token_mask"] is mask and c["token_mask"] is None
    assert a["flags"] == api.MOE_ROUTE_RENORM and b["flags"] == 0


# ---------------------------------------------------------------------------
# adapters
# ---------------------------------------------------------------------------

def adapted(N, grad, dt=torch.bfloat16):
    from grouped_gemm_router_amd.adapters import AdaptedLinear
    z = lambda *s: torch.zeros(s, dtype=dt)  # noqa: E731
    return AdaptedLinear(z(N, 16), z(2, 8, 16), z(2, 8, N), torch.ones(2), grad=grad)


def test_adapted_linear_refuses_a_backward_it_cannot_run():
    """When it is built, not at the first backward pass."""
    adapted(60, False)
    adapted(64, True)
    with pytest.raises(ValueError, match="N % 8"):
        adapted(60, True)


def test_a_gradient_of_another_type_is_refused_by_its_name():
    """An fp32 gradient of fp32 outputs of bf16 weights."""
    lin = adapted(64, True)
    x, a, v = torch.zeros((T, 16), dtype=torch.bfloat16), torch.zeros(T, dtype=torch.int32), None
    with pytest.raises(TypeError, match="dy"):
        lin.backward(torch.zeros((T, 64)), x, a, v)


def test_the_binding_names_a_dy_of_another_type(monkeypatch):
    monkeypatch.setattr(api, "_gpu", lambda t, name: 0)
    z = torch.zeros
    A, B = (z(2, 8, n, dtype=torch.bfloat16) for n in (16, 64))
    with pytest.raises(TypeError, match="dy"):
        api.moe_lora_linear_backward(z(T, 64), z(T, 16, dtype=torch.bfloat16), A, B, z(2),
                                     z(T, dtype=torch.int32), z(T, 8), z(T, 8))


def test_u_over_v_is_refused():
    """u is written before dB is summed from v."""
    P, P2, P3, NUL = (C.c_void_p(a) for a in (0x10000, 0x20000, 0x30000, 0))
    assert api.lib.moe_lora_linear_backward(P, P, P, 0, P, P, api.MOE_BF16, P, P, P3, 16, 64, 64, 8, 2,
                                            P3, P2, P, P, P, 1 << 40, NUL) == api.MOE_ERR_INVALID


def test_many_rows_of_short_factors_are_sorted():
    """Rows that are sorted have a plan, in the workspace: large batches
    whatever N and K are, not small ones."""
    size = api.moe_lora_linear_workspace_size
    bf, f32 = torch.bfloat16, torch.float32
    assert size(8192, 40, 64, 128, 8, bf) > 0 and size(8192, 8, 8, 8, 8, bf) > 0
    assert size(4096, 40, 64, 128, 8, f32) > 0
    assert size(256, 256, 128, 8, 4, f32) == 0 and size(128, 512, 512, 16, 64, bf) == 0
