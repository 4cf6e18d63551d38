"""The operators together: a served block against its parts in plain arithmetic, and a training
step against autograd."""
import os
import sys

import pytest
import torch

from moe_expert_layer_prepare_gb300 import binding as B
from tests._util import need_cuda

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    need_cuda()
    from moe_expert_layer_prepare_gb300 import build
    build.build()
    B.load()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_block
    return moe_block


def rel(a, b):
    a, b = a.detach().cpu().double(), b.detach().cpu().double()
    return ((a - b).norm() / b.norm()).item()


# each number is a handful of bf16 roundings (2^-9 of the norm each, independent) apart
@pytest.mark.parametrize("T", [1, 40, 96])
def test_served_block(ex, T):
    K, S = 512, 5
    b = ex.make_block(96, K, 256, 16, 4, 384, S, 16, seed=T)
    w = b.weights
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    z = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    ids = torch.randint(-1, S, (T,), device="cuda", dtype=torch.int32)
    x1, out = b.forward(x, z, adapter_ids=ids)
    assert int(b.status.item()) == 0 and int(b.experts.status.item()) == 0

    def norm(v):
        return v * torch.rsqrt(v.square().mean(1, keepdim=True) + b.eps)

    xr = x.double() + norm(z.double())
    assert rel(x1, xr) < 3e-3
    h = b.h[:T].double()
    assert rel(b.h[:T], norm(xr)) < 5e-3
    assert rel(b.logits[:T], h @ w["router"].double().t()) < 3e-3
    ids2, tw2 = torch.empty_like(b.ids[:T]), torch.empty_like(b.topk_weights[:T])
    B.moe_route(b.logits[:T], ids2, tw2, bias=w["router_bias"], **b.route)
    assert torch.equal(ids2, b.ids[:T]) and torch.equal(tw2, b.topk_weights[:T])

    def linear(v, weight, name):
        y = v @ weight.double().t()
        ad = w["adapters"]
        for a in range(S):
            at = ids == a
            low = v[at] @ ad[name + "_a"][a].double().t()
            y[at] += ad["scale"][a].double() * (low @ ad[name + "_b"][a].double().t())
        return y

    gate, up = linear(h, w["shared_gate_up"], "gate_up").chunk(2, dim=1)
    shared = linear(torch.nn.functional.silu(gate) * up, w["shared_down"], "down")
    assert rel(out, shared + b.experts.out[:T].double()) < 1e-2


def test_training_step_against_autograd(ex):
    torch.manual_seed(3)
    T, K, E, k = 70, 64, 8, 2
    t = ex.TrainedBlock(T, K, E, k)
    t.scales += 0.3 * torch.randn_like(t.scales)
    x, up = torch.randn(T, K, device="cuda"), torch.randn(T, K, device="cuda")
    out = t.forward(x)
    grads = t.backward(up)
    leaf = {n: getattr(t, n).double().requires_grad_(True) for n in ("norm", "router", "scales")}
    xd = x.double().requires_grad_(True)
    h = xd * torch.rsqrt(xd.square().mean(1, keepdim=True) + 1e-6) * leaf["norm"]
    ids = t.ids.long()
    w = torch.softmax((h @ leaf["router"].t()).gather(1, ids), dim=1)
    ref = xd + (w[:, :, None] * h[:, None, :] * leaf["scales"][ids]).sum(1)
    (ref * up.double()).sum().backward()
    # fp32 throughout: a few roundings of 2^-24 of terms about as large as the result
    assert rel(out, ref) < 1e-5
    for n, g in leaf.items():
        assert rel(grads[n], g.grad) < 2e-5, n
    assert rel(grads["x"], xd.grad) < 2e-5


def test_example_runs_and_learns(ex, capsys):
    ex.serve()
    losses = ex.train()
    assert losses[-1] < 0.2 * losses[0]
