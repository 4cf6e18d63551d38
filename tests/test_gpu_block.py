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


def test_served_block_in_a_cuda_graph(ex):
    K, S = 512, 5
    b = ex.make_block(700, K, 256, 16, 4, 384, S, 16, seed=7)
    for T in (1, 64, 600):
        g = torch.Generator(device="cuda").manual_seed(T)

        def inputs():
            return (torch.randn(T, K, generator=g, device="cuda").bfloat16(),
                    torch.randn(T, K, generator=g, device="cuda").bfloat16(),
                    torch.randint(-1, S, (T,), generator=g, device="cuda", dtype=torch.int32))

        x, z, ids = inputs()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # the first call on a stream, before the capture
            b.forward(x, z, adapter_ids=ids)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res, out = b.forward(x, z, adapter_ids=ids)
        for _ in range(2):
            for t, new in zip((x, z, ids), inputs()):
                t.copy_(new)
            graph.replay()
            got = res.clone(), out.clone()
            want = b.forward(x, z, adapter_ids=ids)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert int(b.status.item()) == 0 and int(b.experts.status.item()) == 0


def test_training_calls_in_a_cuda_graph(ex):
    T, K, E, k = 300, 256, 8, 2
    g = torch.Generator(device="cuda").manual_seed(1)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    logits, x, rows, d_out, pre = rnd(T, E), rnd(T, K), rnd(T * k, K), rnd(T, K), rnd(K)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, w = torch.empty(T, k, **i32), rnd(T, k)
    off, rr, ro = torch.empty(E + 1, **i32), torch.empty(T, k, **i32), torch.empty(T * k, **i32)
    sorted_rows, out, d_rows, d_w = rnd(T * k, K), rnd(T, K), rnd(T * k, K), rnd(T, k)
    y, rx, d_x, d_pre, d_logits = rnd(T, K), rnd(T), rnd(T, K), rnd(K), rnd(T, E)
    ws = torch.empty(B.block_norm_workspace_size(T, K), dtype=torch.uint8, device="cuda")

    def step():
        B.moe_block_norm(x, pre_weight=pre, y=y, rstd_pre=rx)
        B.moe_route(logits, ids, w)
        B.moe_sort_routes(ids, off, rr, ro)
        B.moe_permute(y, rr, off, sorted_rows)
        B.moe_unpermute(rows, rr, w, out)
        B.moe_unpermute_backward(d_out, rows, rr, w, off, d_rows, d_w)
        B.moe_route_backward(logits, ids, d_w, d_logits)
        B.moe_permute_backward(d_rows, rr, d_x)
        B.moe_block_norm_backward(x, pre_weight=pre, rstd_pre=rx, d_y=d_out, d_x=d_x,
                                  d_pre_weight=d_pre, workspace=ws)
        return [t.clone() for t in (ids, w, rr, sorted_rows, out, d_rows, d_w, d_logits, d_x, d_pre)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in (logits, x, rows, d_out):
        t.copy_(rnd(*t.shape))
    graph.replay()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)
