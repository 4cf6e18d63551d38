"""The operators around the experts at work: a served block, and a trained one.

    python examples/moe_block.py

Serving: a batch of requests, each with its own adapter, goes through two blocks (norm, router,
FP8 experts beside a shared expert with low-rank adapters, ``moe_expert_layer_prepare_gb300.block``).
The same with little more than half the bytes of weights: experts with 4-bit weights and an FP8
shared expert, whose input the norm gives in 8 bits.
Training: a router and the scales of simple experts learn a teacher's output; every gradient but
the experts' own comes from the library (norm, unpermute, permute, router).  A gated feed-forward
block learns another's, with the gradients of the norm and of the gated projection.
"""
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from moe_expert_layer_prepare_gb300 import binding as B
from moe_expert_layer_prepare_gb300 import synthetic as syn
from moe_expert_layer_prepare_gb300.block import FourBitExperts, MoeBlock


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


def make_light_block(T, K, N, E, top_k, Ns, seed, group=64, zeros=True, device="cuda"):
    """A block whose experts have 4-bit weights (integers with zero points, or e2m1 values with
    group 32 and no zero points) and whose shared expert has FP8 ones."""
    g = torch.Generator(device=device).manual_seed(seed)
    dev = dict(device=device)

    def codes(rows, cols):
        return torch.randint(0, 256, (E, rows, cols // 2), dtype=torch.uint8, generator=g, **dev)

    def scales(rows, cols):
        shape = (E, rows, cols // group)
        if not zeros:  # e2m1 values are 2.7 in size on average
            e = 127 - round(math.log2(2.7 * cols ** 0.5))
            return torch.randint(e - 1, e + 2, shape, dtype=torch.uint8, generator=g, **dev)
        return ((0.5 + torch.rand(shape, generator=g, **dev)) * cols ** -0.5 / 4.6).to(torch.bfloat16)

    def zero_points(rows, cols):
        return torch.randint(6, 10, (E, rows, cols // group), dtype=torch.uint8, generator=g, **dev) \
            if zeros else None

    experts = FourBitExperts(T, top_k, dict(
        w13=codes(2 * N, K), w13_s=scales(2 * N, K), w13_z=zero_points(2 * N, K),
        w2=codes(K, N), w2_s=scales(K, N), w2_z=zero_points(K, N)), device=device)
    s13, s13_s = syn.make_block_fp8_weights(1, 2 * Ns, K, seed + 1, device=device)
    s2, s2_s = syn.make_block_fp8_weights(1, K, Ns, seed + 2, device=device)
    weights = dict(
        pre_norm=torch.ones(K, dtype=torch.bfloat16, **dev), post_norm=None,
        router=(torch.randn(E, K, generator=g, **dev) * K ** -0.5).to(torch.bfloat16),
        router_bias=None, shared_w13=s13, shared_w13_s=s13_s, shared_w2=s2, shared_w2_s=s2_s,
        adapters=None)
    return MoeBlock(T, K, N, E, top_k, T, weights, route_scale=2.5, experts=experts)


def serve_light():
    T, K = 48, 512
    blocks = [make_light_block(T, K, 256, 16, 4, 384, seed) for seed in (1, 11)]
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    z = None
    for b in blocks:
        x, z = b.forward(x, z)
    assert all(int(b.status.item()) == 0 for b in blocks) and bool(torch.isfinite(z).all())
    print(f"served {T} tokens with 4-bit experts: |x| {x.float().norm():.1f}, |z| {z.float().norm():.1f}")


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


class GatedFeedForward:
    """x -> x + (silu(h Wg^T) * (h Wu^T)) Wd^T of h = norm(x), bf16, with its gradients."""

    def __init__(self, T, K, N, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*shape, std):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.T, self.K, self.N = T, K, N
        self.norm = torch.ones(K, **bf)
        self.gate_up, self.down = rnd(2 * N, K, std=K ** -0.5), rnd(K, N, std=N ** -0.5)
        self.rstd = torch.empty(T, device="cuda")
        self.h, self.kept, self.inter = torch.empty(T, K, **bf), torch.empty(T, 2 * N, **bf), torch.empty(T, N, **bf)
        need = max(B.gated_linear_workspace_size(T, K, N), B.block_norm_workspace_size(T, K))
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")

    def forward(self, x):
        self.x = x
        B.moe_block_norm(x, pre_weight=self.norm, y=self.h, rstd_pre=self.rstd)
        B.moe_gated_linear(self.h, self.gate_up, self.inter, gate_up=self.kept)
        out = torch.empty_like(x)
        B.moe_lora_linear(self.inter, self.down, None, None, None, None, out, None)
        return out.add_(x)

    def backward(self, d_out):
        d_down = d_out.t() @ self.inter
        d_inter = d_out @ self.down
        d_h, d_gate_up = torch.empty_like(self.h), torch.empty_like(self.gate_up)
        B.moe_gated_linear_backward(d_inter, self.h, self.gate_up, self.kept, d_x=d_h,
                                    d_weight=d_gate_up, workspace=self.workspace)
        d_x, d_norm = torch.empty_like(self.x), torch.empty_like(self.norm)
        B.moe_block_norm_backward(self.x, pre_weight=self.norm, rstd_pre=self.rstd, d_y=d_h, d_x=d_x,
                                  d_pre_weight=d_norm, workspace=self.workspace)
        return dict(norm=d_norm, gate_up=d_gate_up, down=d_down, x=d_x + d_out)


def train_feed_forward(steps=40, lr=0.2):
    T, K, N = 520, 128, 200
    teacher, student = GatedFeedForward(T, K, N, 1), GatedFeedForward(T, K, N, 2)
    names = ("norm", "gate_up", "down")
    master = {n: getattr(student, n).float() for n in names}
    g = torch.Generator(device="cuda").manual_seed(3)
    losses = []
    for _ in range(steps):
        x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
        err = student.forward(x).float() - teacher.forward(x).float()
        losses.append(err.square().mean().item())
        grads = student.backward((err * (2.0 / T)).to(torch.bfloat16))
        for n in names:
            master[n] -= lr * grads[n].float()
            getattr(student, n).copy_(master[n])
    print(f"trained a feed-forward block {steps} steps: loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    serve()
    serve_light()
    train()
    train_feed_forward()
