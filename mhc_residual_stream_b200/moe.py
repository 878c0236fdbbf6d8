"""The MoE sublayer between two boundaries, on the CUDA library.

What the pages' executor calls MoEStep (vllm ...specialized_decode.runtime.decode,
SpecializedDecode.run): from a boundary's layer input to the unfinalized output
that the next boundary takes (mhc_boundary_moe_finalize): router logits
(mhc_linear), experts and permutation (mhc_moe_route), the experts' products
(mhc_moe_experts) and the shared expert (two mhc_linear).
"""

from __future__ import annotations

import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import mhc as M
from . import synthetic as S


@dataclass(frozen=True)
class MoeConfig:
    """Sizes and routing of a MoE sublayer. `shared` is the shared expert's
    intermediate size; `balance` draws a bias that chooses experts (not weights)."""
    experts: int
    intermediate: int
    top_k: int = 8
    shared: int = 0  # 0: as intermediate
    scoring: str = "sigmoid"
    num_groups: int = 1
    top_groups: int = 1
    group_top: int = 2
    renormalize: bool = True
    weight_scale: float = 1.0
    balance: bool = True


@dataclass
class MoeWeights:
    """router [E, H], w13 [E, 2I, H], w2 [E, H, I], shared13 [2S, H], shared2 [H, S] bf16;
    bias [E] fp32 or None."""
    router: torch.Tensor
    bias: Optional[torch.Tensor]
    w13: torch.Tensor
    w2: torch.Tensor
    shared13: torch.Tensor
    shared2: torch.Tensor

    @classmethod
    def draw(cls, cfg: MoeConfig, hidden: int, seed: int, device) -> "MoeWeights":
        """Seeded weights, N(0, 1/sqrt(fan-in)), drawn on the CPU in fp32."""
        g = S.gen(seed)
        E, I, Sh = cfg.experts, cfg.intermediate, cfg.shared or cfg.intermediate

        def w(*shape):
            return (torch.randn(*shape, generator=g) / math.sqrt(shape[-1])).to(torch.bfloat16).to(device)

        def experts(*shape):  # one at a time: 64 of 4096 x 7168 are 7.5 GB in fp32
            out = torch.empty(E, *shape, dtype=torch.bfloat16, device=device)
            for e in range(E):
                out[e] = w(*shape)
            return out
        return cls(router=w(E, hidden), bias=(torch.randn(E, generator=g) * 0.05).to(device) if cfg.balance else None,
                   w13=experts(2 * I, hidden), w2=experts(hidden, I), shared13=w(2 * Sh, hidden), shared2=w(hidden, Sh))


class MoeSublayer:
    """The buffers and workspaces of a MoE sublayer for a batch of `rows`. One serves
    every layer of a loop on one stream: a boundary has read a layer's outputs before
    the next layer's sublayer writes them."""

    def __init__(self, cfg: MoeConfig, rows: int, hidden: int, device="cuda"):
        k, E, Sh = cfg.top_k, cfg.experts, cfg.shared or cfg.intermediate

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device=device)
        self.cfg, self.rows, self.hidden = cfg, rows, hidden
        self.logits = empty(rows, E, dtype=torch.float32)
        self.expert_weights = empty(rows, k, dtype=torch.float32)
        self.expert_ids = empty(rows, k, dtype=torch.int32)
        self.e2p = empty(rows * k, dtype=torch.int32)
        self.permuted_rows = empty(rows * k, dtype=torch.int32)
        self.expert_offsets = empty(E + 1, dtype=torch.int32)
        # zero once: slots without an expert leave places behind the last pair unwritten
        self.gemm2_permuted = torch.zeros(rows * k, hidden, dtype=torch.bfloat16, device=device)
        self.shared_inner = empty(rows, Sh)
        self.shared_output = empty(rows, hidden)
        self.linear_ws = M.new_linear_workspace(rows, device)
        self.route_ws = M.new_moe_route_workspace(rows, E, k, device)
        self.experts_ws = M.new_moe_experts_workspace(rows, rows * k, cfg.intermediate, device)

    def run(self, x: torch.Tensor, w: MoeWeights, stream=None):
        """Enqueue the sublayer on layer input x [rows, hidden] bf16; its outputs are
        gemm2_permuted, expert_weights, e2p and shared_output."""
        c = self.cfg
        M.mhc_linear(x, w.router, self.logits, workspace=self.linear_ws, stream=stream)
        M.mhc_moe_route(self.logits, self.expert_weights, self.expert_ids, self.e2p, self.permuted_rows,
                        self.expert_offsets, bias=w.bias, scoring=c.scoring, num_groups=c.num_groups,
                        top_groups=c.top_groups, group_top=c.group_top, renormalize=c.renormalize,
                        weight_scale=c.weight_scale, workspace=self.route_ws, stream=stream)
        M.mhc_moe_experts(x, w.w13, w.w2, self.permuted_rows, self.expert_offsets, self.gemm2_permuted,
                          workspace=self.experts_ws, stream=stream)
        M.mhc_linear(x, w.shared13, self.shared_inner, activation="swiglu", workspace=self.linear_ws, stream=stream)
        M.mhc_linear(self.shared_inner, w.shared2, self.shared_output, workspace=self.linear_ws, stream=stream)

    def device_status(self, stream=None) -> int:
        """The first error a kernel recorded, read and cleared (synchronises)."""
        return next((s for s in [M.mhc_get_device_status(ws, stream)
                                 for ws in (self.linear_ws, self.route_ws, self.experts_ws)] if s != M.OK), M.OK)
