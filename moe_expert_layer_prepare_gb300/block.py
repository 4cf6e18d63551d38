"""One MoE block for serving, from the residual stream to the block's output.

``MoeBlock`` holds the weights and the device buffers and makes the calls in order: the norm
before the block (with what the block before left to add), the router, the FP8 experts
(``binding.MoeLayer``) and beside them the shared expert, whose projections carry each request's
low-rank adapter.  The block's output is the next block's ``z``.  The experts may have 4-bit
weights instead (``FourBitExperts``), and the shared expert a fused gated projection or FP8
weights.
"""
from __future__ import annotations

import torch

from . import binding as B


class FourBitExperts:
    """Experts with 4-bit weights for short batches: gate and up projections with the activation,
    down projection, weighted sum of a token's experts; three launches.

    weights: dict of device tensors
         w13 uint8 [E, 2 N, K / 2], w2 uint8 [E, K, N / 2]   codes, see ``binding.moe_w4_linear``
         w13_s, w2_s                                          scales of their groups
         w13_z, w2_z                                          zero points; None or absent: without
    T: the most tokens of a call; T * top_k is at most 1024."""

    def __init__(self, T, top_k, weights, dtype=torch.bfloat16, activation=B.MOE_ACT_SILU,
                 device="cuda"):
        w = self.weights = weights
        if T * top_k > 1024:
            raise ValueError(f"{T} tokens with {top_k} experts each are more than 1024 routes")
        K, N = w["w2"].shape[1], w["w13"].shape[1] // 2
        dev = torch.device(device)
        self.top_k, self.activation = top_k, activation
        self.inter = torch.empty((T * top_k, N), dtype=dtype, device=dev)
        self.rows = torch.empty((T * top_k, K), dtype=dtype, device=dev)
        self.out = torch.empty((T, K), dtype=dtype, device=dev)
        self.route_row = torch.arange(T * top_k, dtype=torch.int32, device=dev).view(T, top_k)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def forward(self, hidden, topk_ids, topk_weights, is_padding=None):
        """hidden [T, K], topk_ids int32 or int64 [T, top_k] (< 0: no expert), topk_weights fp32;
        padding tokens are those without experts, as ``moe_route`` gives them."""
        w, T = self.weights, hidden.shape[0]
        n = T * self.top_k
        inter, rows, out = self.inter[:n], self.rows[:n], self.out[:T]
        B.moe_w4_linear(hidden, w["w13"], w["w13_s"], inter, zeros=w.get("w13_z"),
                        topk_ids=topk_ids, activation=self.activation, device_status=self.status)
        B.moe_w4_linear(inter, w["w2"], w["w2_s"], rows, zeros=w.get("w2_z"),
                        topk_ids=topk_ids.view(n, 1), device_status=self.status)
        B.moe_unpermute(rows, self.route_row[:T], topk_weights, out)
        return out


class MoeBlock:
    """weights: dict of device tensors
         pre_norm [K], post_norm [K]   norms before this block and after the one before
         router [E, K], router_bias [E] fp32 (selection bias; None: without)
         w13, w13_s, w2, w2_s          the experts (see ``binding.MoeLayer``)
         shared_gate_up [2 Ns, K], shared_down [K, Ns]
         shared_w13, shared_w13_s, shared_w2, shared_w2_s   instead of those two: an FP8 shared
                                       expert ([1, 2 Ns, K], ... as the experts'), without adapters
         adapters: dict(gate_up_a [S, R, K], gate_up_b [S, 2 Ns, R], down_a [S, R, Ns],
                        down_b [S, K, R], scale fp32 [S]), or None
    experts: takes the place of the FP8 experts, whose weights are then not needed (``FourBitExperts``,
    or an object with its ``forward`` and ``status``).  fused_shared: without adapters the shared
    expert's gate, up and activation are one call, with one rounding where three calls have four.
    With an FP8 shared expert the norm gives its input in 8 bits too; the block then has no
    post_norm (None) and no residual scale.
    status (int32 [1]): the MOE_DEV_* bits of all of the block's calls, its experts' among them; one
    word with experts.status.
    T is the most tokens of a call.  The logits are the router's projection in bf16, as the
    projection rounds its output, and the experts are taken by them; moe_route takes fp32 logits
    too, from a caller who computes them."""

    def __init__(self, T, K, N, E, top_k, M_max, weights, num_groups=1, top_groups=1,
                 scoring=B.MOE_SCORE_SIGMOID, route_scale=1.0, eps=1e-6, device="cuda",
                 experts=None, fused_shared=False):
        w = self.weights = weights
        self.T, self.K, self.E, self.top_k = T, K, E, top_k
        self.route = dict(scoring=scoring, scale=route_scale, num_groups=num_groups,
                          top_groups=top_groups, renormalize=True)
        self.eps = eps
        self.experts = experts or B.MoeLayer(T, K, N, E, top_k, M_max, w["w13"], w["w13_s"],
                                             w["w2"], w["w2_s"], device=device)
        dev = torch.device(device)

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device=dev)

        self.shared8 = w.get("shared_w13") is not None
        Ns = w["shared_w2"].shape[2] if self.shared8 else w["shared_down"].shape[1]
        self.fused_shared = fused_shared
        self.x, self.h, self.out = empty(T, K), empty(T, K), empty(T, K)
        self.logits, self.gate_up = empty(T, E), empty(T, 2 * Ns)
        self.ids = empty(T, top_k, dtype=torch.int32)
        self.topk_weights = empty(T, top_k, dtype=torch.float32)
        self.status = self.experts.status
        ad = w["adapters"]
        if self.shared8 and (ad is not None or w["post_norm"] is not None):
            raise ValueError("an FP8 shared expert goes without adapters and without post_norm")
        if fused_shared:
            self.inter = empty(T, Ns)
        if self.shared8:
            G = (K + 127) // 128
            self.q = empty(T, K, dtype=torch.uint8)
            self.q_sf = empty(T, (G + 3) // 4, dtype=torch.int32)
            self.out8 = empty(1, T, K)
            self.counts = torch.arange(T + 1, dtype=torch.int32, device=dev)
            self.ws13 = empty(B.experts_workspace_size(1, T, K, Ns, T, 13), dtype=torch.uint8)
            self.ws2 = torch.zeros(max(256, B.experts_workspace_size(1, T, K, Ns, T, 2)),
                                   dtype=torch.uint8, device=dev)
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

    def _shared(self, h, out, adapter_ids):
        w, T = self.weights, h.shape[0]
        if self.shared8:
            B.moe_batched_experts(self.out8, self.q, self.q_sf, w["shared_w13"], w["shared_w13_s"],
                                  w["shared_w2"], w["shared_w2_s"], self.counts[T:T + 1], self.ws13,
                                  self.ws2, valid_shape_m=self.T, device_status=self.status)
            return out.copy_(self.out8[0, :T])
        if self.fused_shared and (w["adapters"] is None or adapter_ids is None):
            inter = self.inter[:T]
            B.moe_gated_linear(h, w["shared_gate_up"], inter, device_status=self.status)
            return self._linear(inter, w["shared_down"], out)
        gate_up = self._linear(h, w["shared_gate_up"], self.gate_up[:T], "gate_up", adapter_ids)
        gate, up = gate_up.chunk(2, dim=1)
        return self._linear(torch.nn.functional.silu(gate).mul_(up), w["shared_down"], out, "down",
                            adapter_ids)

    def forward(self, x, z=None, adapter_ids=None, is_padding=None, residual_scale=1.0):
        """x [T, K]: the residual stream; z [T, K]: the output of the block before, not yet added.
        Returns (residual stream with z added, output of this block), both the block's own
        buffers."""
        w, T = self.weights, x.shape[0]
        res = self.x[:T] if z is not None else x
        h, out = self.h[:T], self.out[:T]
        if self.shared8:
            if residual_scale != 1.0:
                raise ValueError("an FP8 shared expert goes without a residual scale")
            B.moe_norm_quant(x, w["pre_norm"], self.q[:T], self.q_sf[:T], z=z,
                             x_out=res if z is not None else None, y=h, eps=self.eps)
        else:
            B.moe_block_norm(x, z=z, post_weight=w["post_norm"] if z is not None else None,
                             scale=residual_scale, pre_weight=w["pre_norm"], eps=self.eps,
                             x_out=res if z is not None else None, y=h)
        logits = self._linear(h, w["router"], self.logits[:T])
        ids, tw = self.ids[:T], self.topk_weights[:T]
        B.moe_route(logits, ids, tw, bias=w["router_bias"], is_padding=is_padding, **self.route)
        self._shared(h, out, adapter_ids)
        routed = self.experts.forward(h, ids, tw, is_padding)
        return res, out.add_(routed[:T])
