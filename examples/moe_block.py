"""The operators around the experts at work: a served block, and a trained one.

    python examples/moe_block.py

Serving: a batch of requests, each with its own adapter, goes through two blocks (norm, router,
FP8 experts beside a shared expert with low-rank adapters, ``moe_expert_layer_prepare_gb300.block``).
Training: a router and the scales of simple experts learn a teacher's output; every gradient but
the experts' own comes from the library (norm, unpermute, permute, router).
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from moe_expert_layer_prepare_gb300 import binding as B
from moe_expert_layer_prepare_gb300 import synthetic as syn
from moe_expert_layer_prepare_gb300.block import MoeBlock


def make_block(T, K, N, E, top_k, Ns, S, R, seed, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def rnd(*shape, std):
        return (torch.randn(shape, generator=g, device=device) * std).to(torch.bfloat16)

    w13, w13_s = syn.make_block_fp8_weights(E, 2 * N, K, seed + 1, device=device)
    w2, w2_s = syn.make_block_fp8_weights(E, K, N, seed + 2, device=device)
    ones = torch.ones(K, dtype=torch.bfloat16, device=device)
    weights = dict(
        pre_norm=ones, post_norm=ones.clone(), router=rnd(E, K, std=K ** -0.5),
        router_bias=torch.randn(E, generator=g, device=device) * 0.01,
        w13=w13, w13_s=w13_s, w2=w2, w2_s=w2_s,
        shared_gate_up=rnd(2 * Ns, K, std=K ** -0.5), shared_down=rnd(K, Ns, std=Ns ** -0.5),
        adapters=dict(gate_up_a=rnd(S, R, K, std=K ** -0.5),
                      gate_up_b=rnd(S, 2 * Ns, R, std=R ** -0.5),
                      down_a=rnd(S, R, Ns, std=Ns ** -0.5), down_b=rnd(S, K, R, std=R ** -0.5),
                      scale=torch.full((S,), 0.25, device=device)))
    return MoeBlock(T, K, N, E, top_k, T, weights, num_groups=4, top_groups=2, route_scale=2.5)


def serve():
    T, K, S = 96, 512, 6
    blocks = [make_block(T, K, 256, 16, 4, 384, S, 16, seed) for seed in (1, 11)]
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    adapter_ids = torch.randint(-1, S, (T,), device="cuda", dtype=torch.int32)
    z = None
    for b in blocks:
        x, z = b.forward(x, z, adapter_ids=adapter_ids)
    assert int(blocks[-1].status.item()) == 0 and bool(torch.isfinite(z).all())
    print(f"served {T} tokens through {len(blocks)} blocks: |x| {x.float().norm():.1f}, "
          f"|z| {z.float().norm():.1f}")


class TrainedBlock:
    """x -> x + combine(experts(sort(norm(x)))): experts are columns' scales [E, K]."""

    def __init__(self, T, K, E, k):
        f32 = dict(dtype=torch.float32, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.T, self.K, self.E, self.k = T, K, E, k
        self.norm = torch.ones(K, **f32)
        self.router = torch.randn(E, K, **f32) * K ** -0.5
        self.scales = torch.ones(E, K, **f32)
        self.ids, self.weights = torch.empty(T, k, **i32), torch.empty(T, k, **f32)
        self.offsets, self.route_row = torch.empty(E + 1, **i32), torch.empty(T, k, **i32)
        self.row_route = torch.empty(T * k, **i32)
        self.sort_ws = torch.empty(max(256, B.sort_workspace_size(T, k, E)), dtype=torch.uint8,
                                   device="cuda")
        self.norm_ws = torch.empty(B.block_norm_workspace_size(T, K), dtype=torch.uint8,
                                   device="cuda")
        self.rstd = torch.empty(T, **f32)

    def row_experts(self):
        """Expert of every row of the sorted order."""
        r = torch.arange(self.T * self.k, device="cuda", dtype=torch.int32)
        return torch.searchsorted(self.offsets[1:].contiguous(), r, right=True).clamp_max(self.E - 1)

    def forward(self, x):
        T, K = x.shape
        self.x, self.h = x, torch.empty_like(x)
        B.moe_block_norm(x, pre_weight=self.norm, y=self.h, rstd_pre=self.rstd)
        self.logits = self.h @ self.router.t()
        B.moe_route(self.logits, self.ids, self.weights)
        B.moe_sort_routes(self.ids, self.offsets, self.route_row, self.row_route, self.sort_ws)
        self.rows = torch.empty(T * self.k, K, device="cuda")
        B.moe_permute(self.h, self.route_row, self.offsets, self.rows)
        self.expert = self.row_experts()
        self.rows_out = self.rows * self.scales[self.expert]
        out = torch.empty_like(x)
        B.moe_unpermute(self.rows_out, self.route_row, self.weights, out)
        return x + out

    def backward(self, d_out):
        """Gradients of norm, router and scales, and of x."""
        d_rows_out, d_w = torch.empty_like(self.rows), torch.empty_like(self.weights)
        B.moe_unpermute_backward(d_out, self.rows_out, self.route_row, self.weights, self.offsets,
                                 d_rows_out, d_w)
        d_scales = torch.zeros_like(self.scales).index_add_(0, self.expert, d_rows_out * self.rows)
        d_h = torch.empty_like(self.x)
        B.moe_permute_backward(d_rows_out * self.scales[self.expert], self.route_row, d_h)
        d_logits = torch.empty_like(self.logits)
        B.moe_route_backward(self.logits, self.ids, d_w, d_logits)
        d_router = d_logits.t() @ self.h
        d_h += d_logits @ self.router
        d_x, d_norm = torch.empty_like(self.x), torch.empty_like(self.norm)
        B.moe_block_norm_backward(self.x, pre_weight=self.norm, rstd_pre=self.rstd, d_y=d_h,
                                  d_x=d_x, d_pre_weight=d_norm, workspace=self.norm_ws)
        return dict(norm=d_norm, router=d_router, scales=d_scales, x=d_x + d_out)


def train(steps=60, lr=80.0, router_lr=4.0):
    torch.manual_seed(0)
    T, K, E, k = 513, 256, 8, 2
    teacher, student = TrainedBlock(T, K, E, k), TrainedBlock(T, K, E, k)
    teacher.scales += 0.5 * torch.randn_like(teacher.scales)
    student.router.copy_(teacher.router)
    losses = []
    for _ in range(steps):
        x = torch.randn(T, K, device="cuda")
        err = student.forward(x) - teacher.forward(x)
        losses.append(err.square().mean().item())
        grads = student.backward(err * (2.0 / err.numel()))
        for name in ("norm", "router", "scales"):
            getattr(student, name).sub_((router_lr if name == "router" else lr) * grads[name])
    print(f"trained {steps} steps: loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    serve()
    train()
