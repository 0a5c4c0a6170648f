"""One GPU's MoE layer as a fixed pipeline of the library's calls:

    moe_route -> moe_layout -> moe_grouped_gate_up_gather -> moe_grouped_down -> moe_combine

where the gate/up GEMM gathers its rows from the token rows itself (the
permute fused into its operand loads, so the expert-major copy of x is never
written), or, with ``gather=False``, the permute as its own stage:

    moe_route -> moe_layout -> moe_permute -> moe_grouped_gate_up
              -> moe_grouped_down -> moe_combine

With ``gate_w`` the router projection comes first (moe_linear, fp32 logits);
with ``router`` the scored router takes moe_route's place; with ``shared`` a
shared expert runs beside the routed ones and its down projection takes their
sum as its residual:

    [moe_linear ->] moe_route | moe_route_scored -> ... -> moe_combine
              [-> moe_grouped_gate_up -> moe_linear]

All buffers are allocated once, at construction, for the worst case
(``m_cap`` local rows), so a forward pass launches kernels only: no
allocation, no host sync (the dispatch-without-waiting principle of DeepEP's
``num_worst_tokens`` in DeepEP issue #272 and the host-sync-free hot path of
xtuner PR #2056, section "Design").
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import ops


@dataclass
class Router:
    """How the layer's scored router chooses and weighs (``ops.route_scored``)."""

    score: str = "sigmoid"
    bias: torch.Tensor | None = None  # [E] fp32, steers the choice alone
    num_groups: int = 1
    top_groups: int = 1
    group_rank: str = "top2"
    renormalise: bool = True
    scale: float = 1.0


def _check(t, name: str, dtype, shape, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev} (got {t.device})")


def _check_router(r, num_experts: int, top_k: int, dev):
    """What moe_route_scored would refuse, at the layer's construction."""
    if not isinstance(r, Router):
        raise TypeError("router must be a Router")
    ops._one_of(ops._SCORES, r.score, "router.score")
    ops._one_of(ops._RANKS, r.group_rank, "router.group_rank")
    if not 1 <= r.num_groups <= 64 or num_experts % r.num_groups:
        raise ValueError(f"router.num_groups must divide {num_experts} experts, 64 at most "
                         f"(got {r.num_groups})")
    if not 1 <= r.top_groups <= r.num_groups:
        raise ValueError(f"router.top_groups must be 1 to {r.num_groups} (got {r.top_groups})")
    if not 1 <= top_k <= r.top_groups * (num_experts // r.num_groups):
        raise ValueError(f"top_k must be 1 to the experts of router.top_groups groups (got {top_k})")
    if not math.isfinite(r.scale):
        raise ValueError(f"router.scale must be finite (got {r.scale})")
    if r.bias is not None:
        _check(r.bias, "router.bias", torch.float32, (num_experts,), dev)


class MoELayer:
    def __init__(self, num_tokens: int, hidden: int, num_experts: int, top_k: int, inter: int,
                 w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor, ep_size: int = 1,
                 local_rank: int = -1, align: int = 128, gather: bool = True,
                 gate_w: torch.Tensor | None = None, router: Router | None = None,
                 shared: tuple | None = None):
        """w1, w3: [E_loc, H, I] and w2: [E_loc, I, H], bf16 on the GPU (math
        orientation); repacked once here into the GEMM's layout. gate_w: the
        router projection [E, H] bf16 (then no logits are given to the layer).
        shared: a shared expert's (w1, w3 [H, Is], w2 [Is, H]) bf16, contiguous; not
        for one rank's share of the experts, whose output the ranks add up."""
        if shared is not None and ep_size > 1 and local_rank >= 0:
            raise ValueError("a rank's share of the experts takes no shared expert: the sum over "
                             "the ranks would count it on each of them")
        dev = w1.device
        if gate_w is not None:
            _check(gate_w, "gate_w", torch.bfloat16, (num_experts, hidden), dev)
        if router is not None:
            _check_router(router, num_experts, top_k, dev)
        if shared is not None:
            if len(shared) != 3:
                raise ValueError(f"shared must be (w1, w3, w2) (got {len(shared)} entries)")
            width = shared[0].shape[-1] if isinstance(shared[0], torch.Tensor) else 0
            for t, name, shape in zip(shared, ("w1", "w3", "w2"),
                                      ((hidden, width), (hidden, width), (width, hidden))):
                _check(t, f"shared {name}", torch.bfloat16, shape, dev)
        self.T, self.H, self.E, self.k, self.I = num_tokens, hidden, num_experts, top_k, inter
        self.desc = ops.layout_desc(num_tokens, num_experts, top_k, ep_size, local_rank, align)
        self.ep_size, self.local_rank, self.align = ep_size, local_rank, align
        self.gather = gather
        self.L = ops.alloc_layout(self.desc, dev)
        self.m_cap = self.L.m_cap
        self.w1t = ops.pack_weights(w1)
        self.w3t = ops.pack_weights(w3)
        self.w2t = ops.pack_weights(w2)
        self.topk_idx = torch.empty((num_tokens, top_k), dtype=torch.int32, device=dev)
        self.topk_w = torch.empty((num_tokens, top_k), dtype=torch.float32, device=dev)
        self.x_perm = torch.empty((self.m_cap, hidden), dtype=torch.bfloat16, device=dev)
        self.h = torch.empty((self.m_cap, inter), dtype=torch.bfloat16, device=dev)
        self.y = torch.empty((self.m_cap, hidden), dtype=torch.bfloat16, device=dev)
        self.out = torch.empty((num_tokens, hidden), dtype=torch.bfloat16, device=dev)
        self.router, self.gate_w, self.shared_w2 = router, gate_w, None
        if gate_w is not None:
            self.logits = torch.empty((num_tokens, num_experts), dtype=torch.float32, device=dev)
            self.gate_ws = ops.linear_workspace(self.out, gate_w)
        if shared is not None:
            s1, s3, s2 = shared
            self.shared_w1 = ops.pack_weights(s1.unsqueeze(0))
            self.shared_w3 = ops.pack_weights(s3.unsqueeze(0))
            self.shared_w2 = s2.t()  # [H, Is], its memory in math orientation
            self.shared_h = torch.empty((num_tokens, s2.shape[0]), dtype=torch.bfloat16,
                                        device=dev)
            # one group of all the tokens
            self.shared_off = torch.tensor([0, num_tokens], dtype=torch.int32, device=dev)
            self.shared_cnt = torch.tensor([num_tokens], dtype=torch.int32, device=dev)
            self.shared_ws = ops.linear_workspace(self.shared_h, self.shared_w2)

    def stages(self, x: torch.Tensor, logits: torch.Tensor | None = None):
        """The layer as (name, thunk) pairs, in order, for timing each stage.
        logits: the router's [T, E] fp32 (left out where the layer has gate_w)."""
        L, r = self.L, self.router
        if (logits is None) != (self.gate_w is not None):
            raise ValueError("the layer takes logits, or has gate_w, and not both")
        front = []
        if self.gate_w is not None:
            logits = self.logits
            front.append(("gate", lambda: ops.linear(x, self.gate_w, out=self.logits,
                                                     workspace=self.gate_ws)))
        if r is None:
            front.append(("route", lambda: ops.route(logits, self.k, self.topk_idx,
                                                     self.topk_w)))
        else:
            front.append(("route", lambda: ops.route_scored(
                logits, self.k, r.bias, r.score, r.num_groups, r.top_groups, r.group_rank,
                r.renormalise, r.scale, self.topk_idx, self.topk_w)))
        front += [
            ("layout", lambda: ops.layout(self.topk_idx, self.E, self.ep_size, self.local_rank,
                                          self.align, out=L)),
        ]
        if self.gather:
            middle = [("gate_up", lambda: ops.grouped_gate_up_gather(
                x, L.src_row, self.k, L.offsets, L.local_counts, self.w1t, self.w3t,
                out=self.h))]
        else:
            middle = [
                ("permute", lambda: ops.permute(x, L.dst_row, L.src_row, L.offsets, self.m_cap,
                                                out=self.x_perm)),
                ("gate_up", lambda: ops.grouped_gate_up(self.x_perm, L.offsets, L.local_counts,
                                                        self.w1t, self.w3t, out=self.h)),
            ]
        back = [
            ("down", lambda: ops.grouped_down(self.h, L.offsets, L.local_counts, self.w2t,
                                              out=self.y)),
            ("combine", lambda: ops.combine(self.y, L.dst_row, self.topk_w, out=self.out)),
        ]
        if self.shared_w2 is not None:
            back += [
                ("shared_gate_up", lambda: ops.grouped_gate_up(
                    x, self.shared_off, self.shared_cnt, self.shared_w1, self.shared_w3,
                    out=self.shared_h)),
                ("shared_down", lambda: ops.linear(
                    self.shared_h, self.shared_w2, residual=self.out, out=self.out,
                    workspace=self.shared_ws)),
            ]
        return front + middle + back

    def forward(self, x: torch.Tensor, logits: torch.Tensor | None = None) -> torch.Tensor:
        for _, run in self.stages(x, logits):
            run()
        return self.out

    __call__ = forward
