"""A shared projection with the low-rank adapters of many requests beside it.

:class:`AdaptedLinear` keeps the weights where the library's calls take them
(``include/moe_lora.h``) and allocates the outputs; every step runs in the
library's HIP kernels on the current stream, with no host synchronisation.
It serves a projection that the caller runs beside the expert layer
(attention's, say), or a router whose fp32 logits the caller hands to
``moe_route`` with ``MOE_ROUTE_FROM_LOGITS``.  ``MoELayer`` itself computes its
own logits and runs its shared experts inside the grouped GEMMs, both without
adapters.
"""
from __future__ import annotations

import torch

from . import api
from .layer import padded_weights


class AdaptedLinear:
    """W [N][K] shared and frozen; A [n][r][K], B [n][r][N] the adapters'
    factors (rank-major; an adapter of a lower rank has zero rows behind it),
    scale [n] fp32.  ``grad`` also keeps W transposed for the backward pass
    and requires N % 8 == 0 (the forward pass takes any N).
    A and B are used as they are, so an optimiser may update them in place."""

    def __init__(self, W, A, B, scale, *, grad=False):
        self.N, self.K = W.shape
        self.n, self.r, _ = A.shape
        assert A.shape == (self.n, self.r, self.K) and B.shape == (self.n, self.r, self.N)
        assert A.dtype == W.dtype and B.dtype == W.dtype
        if grad and self.N % 8:
            raise ValueError("grad=True requires N %% 8 == 0, got N = %d" % self.N)
        self.A, self.B, self.scale = A, B, scale
        # row pitch as for the expert weights
        self.W = padded_weights(W[None])[0]
        self.W_t = padded_weights(W.t().contiguous()[None])[0] if grad else None

    def forward(self, x, adapter, *, out=None, out_dtype=None):
        """(y [T][N], v [T][r]): the projection of x [T][K] with the adapter
        of each row (adapter [T] int32, outside [0, n) for none), and the
        low-rank vectors that backward() takes.  Every call has a workspace
        of its own from the allocator, so calls may run on several streams and
        be captured into graphs."""
        T = x.shape[0]
        if out is None:
            out = torch.empty((T, self.N), dtype=out_dtype or x.dtype, device=x.device)
        v = torch.empty((T, self.r), dtype=torch.float32, device=x.device)
        api.moe_lora_linear(x, self.A, self.B, self.scale, adapter, out, v, W=self.W)
        return out, v

    __call__ = forward

    def backward(self, dy, x, adapter, v):
        """(dx [T][K], dA [n][r][K], dB [n][r][N]) for the dy [T][N] of a
        forward(x, adapter) that returned v; dA and dB are fp32.  dy and dx are
        of the weights' type: the caller rounds the gradient of fp32 outputs
        of bf16 weights."""
        if self.W_t is None:
            raise RuntimeError("backward needs W transposed: build with grad=True")
        if dy.dtype != self.A.dtype:
            raise TypeError("dy must be %s, the weights' type, got %s" % (self.A.dtype, dy.dtype))
        T, f32, dev = x.shape[0], torch.float32, x.device
        u = torch.empty((T, self.r), dtype=f32, device=dev)
        dx = torch.empty((T, self.K), dtype=self.A.dtype, device=dev)
        dA = torch.empty((self.n, self.r, self.K), dtype=f32, device=dev)
        dB = torch.empty((self.n, self.r, self.N), dtype=f32, device=dev)
        api.moe_lora_linear_backward(dy, x, self.A, self.B, self.scale, adapter, v, u,
                                     W_t=self.W_t, dx=dx, dA=dA, dB=dB)
        return dx, dA, dB
