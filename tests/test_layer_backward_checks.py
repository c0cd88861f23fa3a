"""CPU checks of what MoELayer.backward refuses before it calls anything: the
layer's buffers stand in as host tensors, and the library's calls are recorded
instead of made."""
import pytest
import torch

from grouped_gemm_router_amd import api
from grouped_gemm_router_amd.layer import MoELayer

T, E, K, D, DFF = 6, 3, 2, 16, 24
BF, F32 = torch.bfloat16, torch.float32
SHAPES = dict(w_down=(E, D, DFF), w_gate=(E, DFF, D), w_up=(E, DFF, D))


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, recorded as (name, positional, keywords)."""
    seen = []
    for name in ("moe_combine_backward", "moe_permute_backward", "moe_grouped_gemm",
                 "moe_grouped_gemm_dgrad", "moe_grouped_gemm_dgrad_swiglu",
                 "moe_grouped_gemm_wgrad"):
        monkeypatch.setattr(api, name, lambda *a, _n=name, **k: seen.append((_n, a, k)))
    return seen


def layer(dt=BF):
    """A layer on the host; alloc() and steps() as they are."""
    rnd = lambda *s: torch.randn(s).to(dt)  # noqa: E731
    m = MoELayer(rnd(E, D), rnd(E, DFF, D), rnd(E, DFF, D), rnd(E, D, DFF), K)
    m.alloc(T)
    return m


def forward(m, monkeypatch):
    """A forward pass whose five calls do nothing."""
    monkeypatch.setattr(api, "deferred", lambda entry, *a, **k: lambda: None)
    x = torch.zeros((m._T, D), dtype=m.act_dtype)
    for _, fn in m.steps(x, torch.empty_like(x)):
        fn()


def sums(**other):
    return {**{n: torch.zeros(s, dtype=F32) for n, s in SHAPES.items()}, **other}


def test_sums_that_do_not_fit_are_refused_before_anything_is_added(calls, monkeypatch):
    m = layer()
    forward(m, monkeypatch)
    d_out = torch.zeros((T, D), dtype=BF)
    for name, shape in SHAPES.items():
        lacking = sums()
        del lacking[name]
        for bad in (lacking, sums(**{name: None}),
                    sums(**{name: torch.zeros(shape[::-1])}),
                    sums(**{name: torch.zeros(shape, dtype=torch.float16)}),
                    sums(**{name: torch.zeros(shape[::-1]).permute(2, 1, 0)}),
                    sums(**{name: torch.zeros(shape, device="meta")})):
            with pytest.raises((ValueError, TypeError), match=name):
                m.backward(d_out, grads=bad)
    one = torch.zeros(SHAPES["w_gate"])
    with pytest.raises(ValueError, match="their own"):
        m.backward(d_out, grads=sums(w_gate=one, w_up=one))
    down = torch.zeros(SHAPES["w_down"])
    with pytest.raises(ValueError, match="their own"):
        m.backward(d_out, grads=sums(w_down=down, w_up=down.view(SHAPES["w_up"])))
    assert calls == []


@pytest.mark.parametrize("dt", [BF, F32])
def test_sums_that_fit_are_passed_on(calls, monkeypatch, dt):
    m = layer()
    forward(m, monkeypatch)
    grads = sums(w_up=torch.zeros(SHAPES["w_up"], dtype=dt), other=None)
    out = m.backward(torch.zeros((T, D), dtype=BF), grads=grads)
    added = [(a[2], k["accumulate"]) for n, a, k in calls if n == "moe_grouped_gemm_wgrad"]
    assert len(added) == 3 and all(acc for _, acc in added)
    assert {id(t) for t, _ in added} == {id(grads[n]) for n in SHAPES}
    assert all(out[n] is grads[n] for n in SHAPES)


def test_buffers_that_no_forward_has_written_are_refused(calls, monkeypatch):
    """alloc() alone, and alloc() for other tokens after a forward pass."""
    m = layer()
    with pytest.raises(RuntimeError, match="forward pass"):
        m.backward(torch.zeros((T, D), dtype=BF))
    forward(m, monkeypatch)
    m.backward(torch.zeros((T, D), dtype=BF))
    made = len(calls)
    m.alloc(T + 1)
    with pytest.raises(RuntimeError, match="forward pass"):
        m.backward(torch.zeros((T + 1, D), dtype=BF))
    assert len(calls) == made
    forward(m, monkeypatch)
    m.backward(torch.zeros((T + 1, D), dtype=BF))
    assert len(calls) == 2 * made
