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

DenseBlock is a block whose FFN every token passes (a model's first layers, say), with
the same boundary:

    h', x = h + gate * N_post(o),  N_pre(h')      moe_norm_forward
    a = act(x W_g^T) * (x W_u^T)                  moe_gated
    o' = a W_d^T                                  moe_linear

and its whole gradient, or, for inference, on e4m3 weights with a scale per 128 x 128 block
(moe_quantise on x, moe_gated_fp8, moe_linear_fp8).

A block's buffers are made on the stream that is current then; a step on another stream comes after it
(torch.cuda.Stream.wait_stream), as with any tensor.
"""
from __future__ import annotations

from contextlib import nullcontext
from typing import NamedTuple, Optional

import torch

from . import (MOE_ACT_SILU, MOE_BF16, MOE_DTYPE_BF16, MOE_DTYPE_E4M3, MOE_DTYPE_F16, MOE_DTYPE_F32, MOE_FP8_BLOCK128,
               MOE_GATE_CHANNEL, MOE_GATE_NONE, MOE_NORM_RMS, QUANT_BY_NAME, forward_options, gated_problem, linear_problem,
               moe_forward_routed, moe_gated, moe_gated_backward, moe_gated_backward_workspace_size, moe_gated_fp8,
               moe_gated_fp8_workspace_size, moe_gated_workspace_size, moe_linear, moe_linear_backward,
               moe_linear_backward_workspace_size, moe_linear_fp8, moe_linear_fp8_workspace_size,
               moe_linear_workspace_size, moe_norm_backward, moe_norm_backward_workspace_size, moe_norm_forward,
               moe_quantise, moe_read_device_status, moe_route_backward, moe_route_ex, moe_workspace_size_ex, norm_problem,
               problem, quantise_problem, route_options)


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


def _scratch(n: int, device) -> torch.Tensor:
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()  # the status word, which a step clears and sets: no error before the first
    return ws


def _on(stream):
    """torch's current stream becomes `stream` (a torch.cuda.Stream, a cudaStream_t, or None for the current
    one): what is allocated meanwhile may be written by it at once and is reused in its order."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return nullcontext() if stream is None else torch.cuda.stream(stream)


def quantise_dense(w_gated: torch.Tensor, w_down: torch.Tensor, stream=None):
    """The e4m3 weights of a DenseBlock from its 16- or 32-bit ones: (codes [2 N, H], scales [2, N / 128, H / 128],
    codes [H, N], scales [H / 128, N / 128]), the counts of blocks rounded up.  They belong to `stream`, which
    writes them: other streams wait for it."""
    dtype = {torch.float32: MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16}
    if w_gated.dtype not in dtype or w_down.dtype not in dtype:
        raise ValueError("w_gated and w_down are of 16 or 32 bits")
    N = w_gated.shape[0] // 2
    if w_gated.dim() != 2 or w_gated.shape[0] != 2 * N or w_down.shape != (w_gated.shape[1], N):
        raise ValueError(f"w_gated [2 N, H] and w_down [H, N] expected, not {tuple(w_gated.shape)} and {tuple(w_down.shape)}")

    def empty(matrices, rows, cols):
        dev = w_gated.device
        return (torch.empty(matrices * rows, cols, dtype=torch.uint8, device=dev),
                torch.empty(matrices, -(-rows // 128), -(-cols // 128), device=dev))

    def codes(w, q, s):
        moe_quantise(quantise_problem(*w.shape, dtype[w.dtype], 128), w, q, s, stream=stream)

    with _on(stream):
        (q, s), (q_down, s_down) = empty(2, N, w_gated.shape[1]), empty(1, *w_down.shape)
    for i in range(2):  # the halves' blocks of rows are apart
        codes(w_gated[i * N:(i + 1) * N], q[i * N:(i + 1) * N], s[i])
    codes(w_down, q_down, s_down[0])
    return q, s, q_down, s_down[0]


def _expect(tensors, **expected):
    """The tensors a block keeps (where they are given) are of the sizes and types that its kernels read."""
    for (name, (shape, dtypes)), t in zip(expected.items(), tensors):
        if t is not None and (t.shape != shape or t.dtype not in dtypes):
            raise ValueError(f"{name}: {list(shape)} of {dtypes[0]} expected, not {list(t.shape)} of {t.dtype}")


class DenseGradient(NamedTuple):
    dh: torch.Tensor          # [T, H] into the residual stream h
    d_o: torch.Tensor         # [T, H] into the block output o
    gated_weight: torch.Tensor
    down_weight: torch.Tensor
    post_weight: torch.Tensor
    pre_weight: torch.Tensor
    gate: Optional[torch.Tensor]


class DenseBlock:
    """A block for T tokens, hidden size H and N gated columns, whose FFN every token passes.

    weights: quant "bf16": (gated [2 N, H] bf16, N gate rows and then N up rows; down [H, N]
    bf16), H and N multiples of 8; "fp8_block": what quantise_dense returns, H and N
    multiples of 16.  norms as Block's.  act: a moe_act.  train (bf16): keeps what gradient needs."""

    def __init__(self, T: int, H: int, N: int, weights, norms, quant="bf16", act: int = MOE_ACT_SILU, train: bool = False,
                 eps: float = 1e-6):
        quant = QUANT_BY_NAME[quant] if isinstance(quant, str) else int(quant)
        if quant not in (MOE_BF16, MOE_FP8_BLOCK128):
            raise ValueError("a dense block's weights are bf16 or fp8_block")
        if train and quant != MOE_BF16:
            raise ValueError("FP8 weights have no gradient")
        self.T, self.H, self.N, self.fp8, self.train = T, H, N, quant == MOE_FP8_BLOCK128, train
        single, half, codes = (torch.float32,), (torch.bfloat16,), (torch.uint8, torch.float8_e4m3fn)
        if len(weights) != (4 if self.fp8 else 2):
            raise ValueError("weights: (gated, down) in bf16, what quantise_dense returns in fp8_block")
        if self.fp8:
            h, n = -(-H // 128), -(-N // 128)
            _expect(weights, gated=((2 * N, H), codes), gated_scale=((2, n, h), single), down=((H, N), codes),
                    down_scale=((h, n), single))
        else:
            _expect(weights, gated=((2 * N, H), half), down=((H, N), half))
        _expect(norms, post=((H,), single), pre=((H,), single), gate=((H,), single))
        self.weights, self.norms = weights, norms
        self.norm = norm_problem(T, H, MOE_NORM_RMS, MOE_NORM_RMS,
                                 gate=MOE_GATE_NONE if norms[2] is None else MOE_GATE_CHANNEL, w_dtype=MOE_DTYPE_F32,
                                 eps=eps)
        dev = weights[0].device

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device=dev)

        self.h_out, self.x, self.o_out = (empty(T, H) for _ in range(3))
        if self.fp8:
            self.quantise = quantise_problem(T, H)
            self.gated = gated_problem(T, N, H, MOE_DTYPE_E4M3, MOE_DTYPE_E4M3, act=act)
            self.down = linear_problem(T, H, N, dtype=MOE_DTYPE_E4M3)
            self.x_codes, self.x_scale = empty(T, H, dtype=torch.uint8), empty(T, -(-H // 128), dtype=torch.float32)
            self.a, self.a_scale = empty(T, N, dtype=torch.uint8), empty(T, -(-N // 128), dtype=torch.float32)
            sizes = moe_gated_fp8_workspace_size(self.gated), moe_linear_fp8_workspace_size(self.down)
        else:
            self.gated, self.down = gated_problem(T, N, H, act=act), linear_problem(T, H, N)
            self.a, self.z = empty(T, N), empty(T, 2 * N) if train else None
            sizes = moe_gated_workspace_size(self.gated), moe_linear_workspace_size(self.down)
        if 0 in sizes:
            raise ValueError("H and N are multiples of 8 (bf16) or 16 (fp8_block)")
        self.ws_gated, self.ws_down = (_scratch(n, dev) for n in sizes)
        self._grad = None
        if train:  # a workspace for each gradient, since the next one's call would clear its status
            f32 = torch.float32
            out = DenseGradient(empty(T, H), empty(T, H), empty(2 * N, H), empty(H, N), empty(H, dtype=f32),
                                empty(H, dtype=f32), None if norms[2] is None else empty(H, dtype=f32))
            sizes = (moe_linear_backward_workspace_size(self.down), moe_gated_backward_workspace_size(self.gated),
                     moe_norm_backward_workspace_size(self.norm))
            self._grad = (out, empty(T, N), empty(T, H), [_scratch(n, dev) for n in sizes])

    def forward(self, h: torch.Tensor, o: torch.Tensor, stream=None):
        """(h', o') as Block.forward."""
        post, pre, gate = self.norms
        moe_norm_forward(self.norm, h, o, gate, post, None, pre, None, self.h_out, self.x, stream=stream)
        if self.fp8:
            wg, sg, wd, sd = self.weights
            moe_quantise(self.quantise, self.x, self.x_codes, self.x_scale, stream=stream)
            moe_gated_fp8(self.gated, self.x_codes, self.x_scale, wg, sg, None, self.a, self.a_scale, self.ws_gated,
                          stream=stream)
            moe_linear_fp8(self.down, self.a, self.a_scale, wd, sd, None, None, self.o_out, self.ws_down, stream=stream)
        else:
            wg, wd = self.weights
            moe_gated(self.gated, self.x, wg, None, self.a, self.z, self.ws_gated, stream=stream)
            moe_linear(self.down, self.a, wd, None, None, self.o_out, None, self.ws_down, stream=stream)
        return self.h_out, self.o_out

    def gradient(self, o: torch.Tensor, do_out: torch.Tensor, dh_out: Optional[torch.Tensor] = None,
                 stream=None) -> DenseGradient:
        """Gradients of a loss with gradient do_out [T, H] bf16 into o' (and dh_out [T, H] into h') of the last
        forward, for the o that it took.  The block's own buffers, which the next gradient writes again."""
        if not self.train:
            raise ValueError("the block was made without train")
        post, pre, gate = self.norms
        wg, wd = self.weights
        out, da, dx, (ws_down, ws_gated, ws_norm) = self._grad
        moe_linear_backward(self.down, do_out, self.a, wd, None, da, out.down_weight, None, ws_down, stream=stream)
        moe_gated_backward(self.gated, da, self.x, wg, self.z, dx, out.gated_weight, None, ws_gated,
                           stream=stream)
        moe_norm_backward(self.norm, dh_out, dx, self.h_out, o, gate, post, None, pre, out.dh, out.d_o, out.gate,
                          out.post_weight, None, out.pre_weight, None, ws_norm, stream=stream)
        return out

    def status(self, stream=None) -> int:
        """Device status of the last forward and the last gradient, MOE_OK before the first (blocks until they are done)."""
        spaces = [self.ws_gated, self.ws_down] + (self._grad[3][:2] if self._grad else [])
        return next((st for st in (moe_read_device_status(ws, stream) for ws in spaces) if st), 0)
