"""One MoE block for serving, from the residual stream to the block's output.

``MoeBlock`` holds the weights and the device buffers and makes the calls in order: the norm
before the block (with what the block before left to add), the router, the FP8 experts
(``binding.MoeLayer``) and beside them the shared expert, whose projections carry each request's
low-rank adapter.  The block's output is the next block's ``z``.
"""
from __future__ import annotations

import torch

from . import binding as B


class MoeBlock:
    """weights: dict of device tensors
         pre_norm [K], post_norm [K]   norms before this block and after the one before
         router [E, K], router_bias [E] fp32 (selection bias; None: without)
         w13, w13_s, w2, w2_s          the experts (see ``binding.MoeLayer``)
         shared_gate_up [2 Ns, K], shared_down [K, Ns]
         adapters: dict(gate_up_a [S, R, K], gate_up_b [S, 2 Ns, R], down_a [S, R, Ns],
                        down_b [S, K, R], scale fp32 [S]), or None
    T is the most tokens of a call.  The logits are the router's projection in bf16, as the
    projection rounds its output, and the experts are taken by them; moe_route takes fp32 logits
    too, from a caller who computes them."""

    def __init__(self, T, K, N, E, top_k, M_max, weights, num_groups=1, top_groups=1,
                 scoring=B.MOE_SCORE_SIGMOID, route_scale=1.0, eps=1e-6, device="cuda"):
        w = self.weights = weights
        self.T, self.K, self.E, self.top_k = T, K, E, top_k
        self.route = dict(scoring=scoring, scale=route_scale, num_groups=num_groups,
                          top_groups=top_groups, renormalize=True)
        self.eps = eps
        self.experts = B.MoeLayer(T, K, N, E, top_k, M_max, w["w13"], w["w13_s"], w["w2"],
                                  w["w2_s"], device=device)
        dev = torch.device(device)

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device=dev)

        Ns = w["shared_down"].shape[1]
        self.x, self.h, self.out = empty(T, K), empty(T, K), empty(T, K)
        self.logits, self.gate_up = empty(T, E), empty(T, 2 * Ns)
        self.ids = empty(T, top_k, dtype=torch.int32)
        self.topk_weights = empty(T, top_k, dtype=torch.float32)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        ad = w["adapters"]
        S, R = ad["gate_up_a"].shape[:2] if ad else (0, 0)
        need = max(B.lora_workspace_size(T, k, n, S, R) for k, n in ((K, 2 * Ns), (Ns, K)))
        self.workspace = empty(max(need, 256), dtype=torch.uint8)

    def _linear(self, x, weight, out, adapter=None, adapter_ids=None):
        ad = self.weights["adapters"]
        if ad is None or adapter is None or adapter_ids is None:
            B.moe_lora_linear(x, weight, None, None, None, None, out, None,
                              device_status=self.status)
        else:
            B.moe_lora_linear(x, weight, ad[adapter + "_a"], ad[adapter + "_b"], adapter_ids,
                              ad["scale"], out, self.workspace, device_status=self.status)
        return out

    def forward(self, x, z=None, adapter_ids=None, is_padding=None, residual_scale=1.0):
        """x [T, K]: the residual stream; z [T, K]: the output of the block before, not yet added.
        Returns (residual stream with z added, output of this block), both the block's own
        buffers."""
        w, T = self.weights, x.shape[0]
        res = self.x[:T] if z is not None else x
        h, out = self.h[:T], self.out[:T]
        B.moe_block_norm(x, z=z, post_weight=w["post_norm"] if z is not None else None,
                         scale=residual_scale, pre_weight=w["pre_norm"], eps=self.eps,
                         x_out=res if z is not None else None, y=h)
        logits = self._linear(h, w["router"], self.logits[:T])
        ids, tw = self.ids[:T], self.topk_weights[:T]
        B.moe_route(logits, ids, tw, bias=w["router_bias"], is_padding=is_padding, **self.route)
        gate_up = self._linear(h, w["shared_gate_up"], self.gate_up[:T], "gate_up", adapter_ids)
        gate, up = gate_up.chunk(2, dim=1)
        self._linear(torch.nn.functional.silu(gate).mul_(up), w["shared_down"], out, "down",
                     adapter_ids)
        routed = self.experts.forward(h, ids, tw, is_padding)
        return res, out.add_(routed[:T])
