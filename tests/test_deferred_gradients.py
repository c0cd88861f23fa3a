"""CPU checks of deferred norm and clip calls: the thunk holds the tensors whose
addresses it passes on, however they were listed."""
import gc
import weakref

import pytest
import torch

from grouped_gemm_router_amd import api


@pytest.fixture(autouse=True)
def host_tensors(monkeypatch):
    """Marshalling alone: host tensors (device -1), and no library call."""
    monkeypatch.setattr(api, "_gpu", lambda t, name: -1)
    monkeypatch.setattr(api, "_raw_stream", lambda s, d: 0)


def listings(tensors):
    """The ways to list tensors: (what is passed on, what the caller does then)."""
    return {"list": (tensors, lambda: None),
            "generator": ((t for t in tensors), lambda: None),
            "emptied list": (tensors, tensors.clear),
            "map": (map(lambda t: t, tensors), lambda: None),
            "tuple": (tuple(tensors), lambda: None)}


KINDS = ["list", "generator", "emptied list", "map", "tuple"]


def alive(refs):
    gc.collect()
    return [r() is not None for r in refs]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 300])
def test_the_norm_holds_its_gradients(kind, n):
    grads = [torch.zeros(3) for _ in range(n)]
    refs = [weakref.ref(g) for g in grads]
    passed, then = listings(grads)[kind]
    thunk = api.deferred(api.moe_grad_norm, passed, torch.zeros(1), ws=torch.zeros(1 << 12))
    then()
    del grads, passed, then
    assert all(alive(refs))
    del thunk
    assert not any(alive(refs))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("apart", [False, True])
def test_the_clip_holds_its_gradients_and_outputs(kind, apart):
    grads = [torch.zeros(3), torch.zeros(5, dtype=torch.bfloat16)]
    out = [torch.zeros_like(g) for g in grads] if apart else None
    refs = [weakref.ref(t) for t in grads + (out or [])]
    passed, then = listings(grads)[kind]
    into, then_out = listings(out)[kind] if apart else (None, lambda: None)
    thunk = api.deferred(api.moe_grad_clip, passed, torch.zeros(1), 1.0, out=into)
    then()
    then_out()
    del grads, out, passed, into, then, then_out
    assert all(alive(refs))
    del thunk
    assert not any(alive(refs))
