"""One block of a model around the routed FFN, and its router's gradient.

A block takes the residual stream h and the output o of the block before it:

    h', x = h + gate * N_post(o),  N_pre(h')      moe_norm_forward
    logits = x W_r^T + b_r                        moe_linear (fp32 out)
    ids, w = routing rule on the logits           moe_route_ex
    o' = sum_j w_j FFN_ids_j(x) (+ shared)        moe_forward_routed

and hands (h', o') on, so that each boundary between two blocks is one pass over the
stream.  Argument marshalling only: every arithmetic step runs in the library's
kernels.  All buffers are allocated once; a step enqueues its work on one stream
without synchronising and can be captured in a CUDA graph.

The experts have no gradient here (their weights are frozen, as when a router is
tuned): router_gradient takes the gradient of a loss into the routing weights w
back through the routing rule, the router's linear layer and the norms.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import (MOE_DTYPE_F32, MOE_GATE_CHANNEL, MOE_GATE_NONE, MOE_NORM_RMS, forward_options,
               linear_problem, moe_forward_routed, moe_linear, moe_linear_backward,
               moe_linear_backward_workspace_size, moe_linear_workspace_size, moe_norm_backward,
               moe_norm_backward_workspace_size, moe_norm_forward, moe_read_device_status, moe_route_backward,
               moe_route_ex, moe_workspace_size_ex, norm_problem, problem, route_options)


class RouterGradient(NamedTuple):
    dh: torch.Tensor          # [T, H] into the residual stream h
    d_o: torch.Tensor         # [T, H] into the block output o
    router_weight: torch.Tensor
    router_bias: torch.Tensor
    post_weight: torch.Tensor
    pre_weight: torch.Tensor
    gate: Optional[torch.Tensor]


class Block:
    """A block for T tokens, E experts of which k, hidden size H, expert size I.

    experts: (w1, w2, w1_scale, w2_scale) as moe_forward takes them in `quant`; router:
    (weight [E, H] bf16, bias [E] fp32 or None); norms: (post weight, pre weight, gate or
    None), fp32 [H] each; rule: keyword arguments of route_options; shared: (n_shared,
    w1, w2, w1_scale, w2_scale) or None."""

    def __init__(self, T: int, E: int, k: int, H: int, I: int, quant, experts, router, norms, rule: Optional[dict] = None,
                 shared=None, eps: float = 1e-6):
        self.T, self.E, self.k, self.H = T, E, k, H
        self.experts, self.router, self.norms = experts, router, norms
        self.problem = problem(T, E, k, H, I, quant)
        self.options = forward_options(*shared) if shared else None
        self._kept = (shared, rule)  # the descriptors hold their tensors' addresses
        self.rule = route_options(**(rule or {}))
        self.norm = norm_problem(T, H, MOE_NORM_RMS, MOE_NORM_RMS,
                                 gate=MOE_GATE_NONE if norms[2] is None else MOE_GATE_CHANNEL, w_dtype=MOE_DTYPE_F32,
                                 eps=eps)
        self.linear = linear_problem(T, E, H, out_dtype=MOE_DTYPE_F32)
        dev = experts[0].device

        def empty(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device=dev)

        def scratch(n):
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
            ws[:256].zero_()  # the status word, which a step clears and sets: no error before the first
            return ws

        bf16 = torch.bfloat16
        self.h_out, self.x, self.o_out = (empty(T, H, dtype=bf16) for _ in range(3))
        self.logits, self.ids, self.w = empty(T, E), empty(T, k, dtype=torch.int32), empty(T, k)
        self.ws = scratch(moe_workspace_size_ex(self.problem, self.options))
        self.ws_linear = scratch(moe_linear_workspace_size(self.linear))
        self._grad = None

    def forward(self, h: torch.Tensor, o: torch.Tensor, stream=None):
        """(h', o') of the block for the stream h and the previous block's output o, bf16 [T, H].
        Both are the block's own buffers, which the next step writes again."""
        post, pre, gate = self.norms
        weight, bias = self.router
        moe_norm_forward(self.norm, h, o, gate, post, None, pre, None, self.h_out, self.x, stream=stream)
        moe_linear(self.linear, self.x, weight, bias, None, self.logits, None, self.ws_linear, stream=stream)
        moe_route_ex(self.rule, self.logits, self.T, self.E, self.k, self.ids, self.w, stream=stream)
        w1, w2, s1, s2 = self.experts
        moe_forward_routed(self.problem, self.options, self.x, self.ids, self.w, w1, w2, s1, s2, self.o_out, self.ws,
                           stream=stream)
        return self.h_out, self.o_out

    def router_gradient(self, o: torch.Tensor, dw: torch.Tensor, dh_out: Optional[torch.Tensor] = None,
                        stream=None) -> RouterGradient:
        """Gradients of a loss with gradient dw [T, k] fp32 into the last forward's routing
        weights (and dh_out [T, H] into h', e.g. of the blocks that follow), for the o that
        forward took."""
        post, pre, gate = self.norms
        weight, _ = self.router
        if self._grad is None:
            dev, bf16 = weight.device, torch.bfloat16
            T, E, H = self.T, self.E, self.H

            def empty(*shape, dtype=torch.float32):
                return torch.empty(*shape, dtype=dtype, device=dev)

            out = RouterGradient(empty(T, H, dtype=bf16), empty(T, H, dtype=bf16), empty(E, H, dtype=bf16), empty(E),
                                 empty(H), empty(H), None if gate is None else empty(H))
            n = max(moe_linear_backward_workspace_size(self.linear), moe_norm_backward_workspace_size(self.norm))
            self._grad = (out, empty(T, E), empty(T, H, dtype=bf16), torch.empty(n, dtype=torch.uint8, device=dev))
        out, dlogits, dx, ws = self._grad
        moe_route_backward(self.rule, self.logits, self.T, self.E, self.k, self.ids, dw, dlogits, stream=stream)
        moe_linear_backward(self.linear, dlogits, self.x, weight, None, dx, out.router_weight, out.router_bias, ws,
                            stream=stream)
        moe_norm_backward(self.norm, dh_out, dx, self.h_out, o, gate, post, None, pre, out.dh, out.d_o, out.gate,
                          out.post_weight, None, out.pre_weight, None, ws, stream=stream)
        return out

    def status(self, stream=None) -> int:
        """Device status of the last forward, MOE_OK before the first (blocks until it is done)."""
        return moe_read_device_status(self.ws_linear, stream) or moe_read_device_status(self.ws, stream)
