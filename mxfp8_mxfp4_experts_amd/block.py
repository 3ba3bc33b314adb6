"""``MoEBlock``: one MoE block, from the residual stream to the experts' output.

In order, on the current stream:

1. ``moe_add_rmsnorm``   h = x + residual, y = norm(h), and y in 8 bits;
2. ``moe_gate_logits``   the router's logits from y;
3. ``moe_route_groups``  the experts of every token and their weights;
4. the experts (``MoELayer``), either on y itself, in the MXFP8 that the norm
   gave, or with ``down`` and ``up`` in a width of their own: y's 8-bit integers
   times ``down`` go into the experts, their output times ``up`` comes back.

The block's output is the experts' share only: the caller adds it to h, which
the next block's norm does on its way in (pass it as that block's ``x`` and h as
its ``residual``).  Buffers are allocated once for ``max_tokens`` and reused, so
a call allocates nothing but its two outputs, and a graph captured with up to
``max_tokens`` stays valid whatever such batches run beside it.  A larger batch
makes the buffers anew: graphs from before it are to be captured again.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _binding as B
from .layer import MoELayer


class MoEBlock:
    def __init__(self, experts: MoELayer, norm_w: torch.Tensor, gate_w: torch.Tensor, *,
                 gate_bias: Optional[torch.Tensor] = None, eps: float = 1e-6, n_group: int = 1,
                 topk_group: int = 1, score: int = B.SCORE_SIGMOID,
                 group_score: int = B.GROUP_TOP2, renormalise: bool = True,
                 down: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                 up: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, max_tokens: int = 1):
        """norm_w bf16 [H]; gate_w bf16 [E, H]; gate_bias float [E] or None.
        ``experts``, where made for fewer than ``max_tokens``, gives its weights
        only: the block then has a layer with buffers of its own.
        ``down`` / ``up``: (int8 [L, H], float [L]) into the experts' width L and
        (int8 [H, L], float [H]) back, both or none, as ``quantise`` gives them."""
        self.experts, self.norm_w, self.gate_w, self.gate_bias = experts, norm_w, gate_w, gate_bias
        self.H, self.E, self.L = norm_w.shape[0], gate_w.shape[0], experts.H
        if gate_w.shape[1] != self.H:
            raise ValueError(f"gate_w must be [E, {self.H}], got {tuple(gate_w.shape)}")
        if self.E != experts.E:
            raise ValueError(f"gate_w has {self.E} experts, the layer {experts.E}")
        if (down is None) != (up is None):
            raise ValueError("down and up go together")
        if down is None and self.L != self.H:
            raise ValueError(f"the experts' width {self.L} is not {self.H}: give down and up")
        if down is not None:
            for name, (w, w_s), shape in (("down", down, (self.L, self.H)),
                                          ("up", up, (self.H, self.L))):
                if tuple(w.shape) != shape or tuple(w_s.shape) != shape[:1]:
                    raise ValueError(f"{name} must be int8 {shape} with float {shape[:1]}")
        self.eps, self.n_group, self.topk_group = eps, n_group, topk_group
        self.score, self.group_score, self.renormalise = score, group_score, renormalise
        self.down, self.up = down, up
        self.device = norm_w.device
        self._alloc(max_tokens)

    @staticmethod
    def quantise(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        """A bf16 weight [N, K] as int8 with one scale per output channel."""
        return B.moe_quant_int8(w)

    def _alloc(self, T: int):
        dev, H, L = self.device, self.H, self.L
        self.max_tokens = T
        if self.experts.max_tokens < T:
            # Else the layer would make its buffers anew in the middle of the block's calls, and
            # graphs that use them, captured of the block or of the layer itself, would write to
            # memory given back.
            self.experts = self.experts.with_max_tokens(T)
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        self.logits = torch.empty((T, self.E), dtype=torch.float32, device=dev)
        self.topk_idx = torch.empty((T, self.experts.top_k), dtype=torch.int32, device=dev)
        self.topk_w = torch.empty((T, self.experts.top_k), dtype=torch.float32, device=dev)
        if self.down is None:
            self.xq = torch.empty((T, H), dtype=torch.uint8, device=dev)
            self.xs = torch.empty((T, H // 32), dtype=torch.uint8, device=dev)
        else:
            self.xq = torch.empty((T, H), dtype=torch.int8, device=dev)
            self.xs = torch.empty((T,), dtype=torch.float32, device=dev)
            self.z = torch.empty((T, L), dtype=torch.bfloat16, device=dev)
            self.z_out = torch.empty((T, L), dtype=torch.bfloat16, device=dev)
        # One workspace for all products: each runs after the one before on the stream.
        need = B.moe_gate_workspace_size(T, self.E, H)
        if self.down is not None:
            need = max(need, B.moe_int8_matmul_workspace_size(T, L, H),
                       B.moe_int8_workspace_size(T, H, L))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=dev)

    def __call__(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None,
                 residual_out: Optional[torch.Tensor] = None):
        """x, residual bf16 [T, H] -> (out, h): the experts' output bf16 [T, H]
        and the new residual stream (x itself without a residual)."""
        T = x.shape[0]
        if T > self.max_tokens:
            self._alloc(T)
        y, xq, xs = self.y[:T], self.xq[:T], self.xs[:T]
        h, _, _, _ = B.moe_add_rmsnorm(
            x, self.norm_w, self.eps, residual=residual,
            q8=B.Q8_MXFP8 if self.down is None else B.Q8_INT8, residual_out=residual_out, y=y,
            xq=xq, xs=xs)
        ws = self.workspace
        logits = B.moe_gate_logits(y, self.gate_w, out=self.logits[:T], workspace=ws)
        idx, w = B.moe_route_groups(
            logits, self.gate_bias, self.experts.top_k, n_group=self.n_group,
            topk_group=self.topk_group, score=self.score, group_score=self.group_score,
            renormalise=self.renormalise, routed_scaling=self.experts.routed_scaling,
            topk_idx=self.topk_idx[:T], topk_w=self.topk_w[:T])
        if self.down is None:
            out = self.experts.mxfp8(xq, xs, idx, w, out=out)
        else:
            z = B.moe_int8_matmul(xq, xs, *self.down, out=self.z[:T], workspace=ws)
            z = self.experts(z, None, None, out=self.z_out[:T], topk_idx=idx, topk_w=w)
            out = B.moe_int8_linear(z, *self.up, out=out, workspace=ws)
        return out, x if h is None else h
