"""A run of the norm with an 8-bit output, the gated projection and the 4-bit products together, as a
block uses them: against its parts in plain arithmetic, in CUDA graphs, and a training step against
autograd."""
import pytest
import torch

from moe_expert_layer_prepare_gb300 import binding as B
from moe_expert_layer_prepare_gb300.block import MoeBlock
from tests.test_gpu_block import ex, rel  # noqa: F401

pytestmark = pytest.mark.gpu


def weights_of(codes, scales, zeros):
    """4-bit weights in fp64."""
    E, N, half = codes.shape
    G = 2 * half // scales.shape[2]
    q = torch.stack([codes & 15, codes >> 4], -1).view(E, N, -1, G)
    if scales.dtype == torch.uint8:
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        v = table[(q & 7).long()] * torch.where(q >= 8, -1.0, 1.0)
        s = torch.exp2(scales.double() - 127)
    else:
        v, s = q.double() - (8.0 if zeros is None else zeros.double()[..., None]), scales.double()
    return (v * s[..., None]).view(E, N, 2 * half)


def silu_mul(v):
    g, u = v.chunk(2, -1)
    return torch.nn.functional.silu(g) * u


# each number is a handful of bf16 roundings (2^-9 of the norm each, independent) apart
@pytest.mark.parametrize("T", [1, 5, 48])
@pytest.mark.parametrize("zeros", [True, False])
def test_light_block(ex, T, zeros):  # noqa: F811
    K, N, E, k, Ns = 512, 256, 16, 4, 384
    b = ex.make_light_block(48, K, N, E, k, Ns, seed=T, group=64 if zeros else 32, zeros=zeros)
    w, e = b.weights, b.experts.weights
    g = torch.Generator(device="cuda").manual_seed(T)
    x, z = (torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    x1, out = b.forward(x, z)
    assert int(b.status.item()) == 0 and int(b.experts.status.item()) == 0
    xr = x.double() + z.double()
    assert rel(x1, xr) < 3e-3
    assert rel(b.h[:T], xr * torch.rsqrt(xr.square().mean(1, keepdim=True) + b.eps)) < 3e-3
    h = b.h[:T].double()
    # the 8-bit input: half steps of 2^-4 at most, over root three on average
    scale = torch.exp2(b.q_sf[:T].contiguous().view(torch.uint8).view(T, -1)[:, :K // 128].double() - 127)
    h8 = b.q[:T].view(torch.float8_e4m3fn).double() * scale.repeat_interleave(128, 1)
    assert rel(h8, h) < 2.0 ** -4 / 3 ** 0.5
    # routed experts, from the ids that the block took
    w13, w2 = (weights_of(e[n], e[n + "_s"], e[n + "_z"]) for n in ("w13", "w2"))
    ids, tw = b.ids[:T].long(), b.topk_weights[:T].double()
    inter = silu_mul(torch.einsum("tkno,to->tkn", w13[ids], h))
    routed = (torch.einsum("tkon,tkn->tko", w2[ids], inter) * tw[..., None]).sum(1)
    assert rel(b.experts.out[:T], routed) < 1e-2
    # the shared expert from its 8-bit input; its inner rows are in 8 bits once more
    def blocks(v, s):
        return v[0].view(torch.float8_e4m3fn).double() * s[0].double().repeat_interleave(128, 0).repeat_interleave(128, 1)

    shared = silu_mul(h8 @ blocks(w["shared_w13"], w["shared_w13_s"]).t()) @ \
        blocks(w["shared_w2"], w["shared_w2_s"]).t()
    assert rel(b.out8[0, :T], shared) < 2.0 ** -4 / 3 ** 0.5
    assert rel(out, b.out8[0, :T].double() + b.experts.out[:T].double()) < 5e-3


def test_padding_tokens_get_nothing_from_the_experts(ex):  # noqa: F811
    b = ex.make_light_block(20, 512, 256, 16, 4, 384, seed=3)
    x = torch.randn(20, 512, device="cuda").to(torch.bfloat16)
    pad = torch.zeros(20, dtype=torch.uint8, device="cuda")
    pad[[0, 7, 19]] = 1
    b.forward(x, is_padding=pad)
    out = b.experts.out
    assert bool((out[pad == 1] == 0).all()) and bool((out[pad == 0] != 0).any(1).all())
    assert int(b.experts.status.item()) == 0


@pytest.mark.parametrize("T", [2, 300])
def test_fused_shared_expert_is_the_three_calls(ex, T):  # noqa: F811
    """The same block with the gated projection and with projection, activation and product one after
    another: the roundings between them apart."""
    plain = ex.make_block(300, 512, 256, 16, 4, 384, 2, 16, seed=5)
    w = dict(plain.weights, adapters=None)
    args = (300, 512, 256, 16, 4, 300, w)
    kw = dict(num_groups=4, top_groups=2, route_scale=2.5)
    a, b = MoeBlock(*args, **kw), MoeBlock(*args, fused_shared=True, **kw)
    x = torch.randn(T, 512, device="cuda").to(torch.bfloat16)
    xa, oa = a.forward(x)
    xb, ob = b.forward(x)
    assert torch.equal(xa, xb) and torch.equal(a.ids[:T], b.ids[:T])
    h = a.h[:T].double()
    shared = silu_mul(h @ w["shared_gate_up"].double().t()) @ w["shared_down"].double().t()
    ref = shared + a.experts.out[:T].double()
    assert rel(ob, ref) < 5e-3 and rel(oa, ref) < 1e-2


def test_refusals(ex):  # noqa: F811
    b = ex.make_light_block(8, 512, 256, 16, 4, 384, seed=1)
    x = torch.randn(8, 512, device="cuda").to(torch.bfloat16)
    with pytest.raises(ValueError):
        b.forward(x, residual_scale=0.5)
    with pytest.raises(ValueError):
        MoeBlock(8, 512, 256, 16, 4, 8, dict(b.weights, post_norm=b.weights["pre_norm"]), experts=b.experts)
    with pytest.raises(ValueError):
        ex.make_light_block(400, 512, 256, 16, 4, 384, seed=1)


def test_light_block_in_a_cuda_graph(ex):  # noqa: F811
    """Captured once and replayed on new inputs, other routes among them; two graphs of one block."""
    b = ex.make_light_block(48, 512, 256, 16, 4, 384, seed=9)
    graphs = []
    for T in (1, 40):
        x, z = (torch.randn(T, 512, device="cuda").bfloat16() for _ in range(2))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b.forward(x, z)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res, out = b.forward(x, z)
        graphs.append((graph, x, z, res, out))
    for _ in range(3):
        for graph, x, z, res, out in graphs:
            x.copy_(torch.randn(x.shape, device="cuda"))
            z.copy_(torch.randn(x.shape, device="cuda"))
            graph.replay()
            got = res.clone(), out.clone()
            want = b.forward(x, z)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert int(b.status.item()) == 0 and int(b.experts.status.item()) == 0


@pytest.mark.parametrize("T,K,N", [(70, 64, 40), (700, 128, 200)])
def test_feed_forward_gradients_against_autograd(ex, T, K, N):  # noqa: F811
    f = ex.GatedFeedForward(T, K, N, seed=T)
    f.norm += (0.1 * torch.randn(K, device="cuda")).to(torch.bfloat16)
    x, up = (torch.randn(T, K, device="cuda").to(torch.bfloat16) for _ in range(2))
    out = f.forward(x)
    grads = f.backward(up)
    leaf = {n: getattr(f, n).double().requires_grad_(True) for n in ("norm", "gate_up", "down")}
    xd = x.double().requires_grad_(True)
    h = xd * torch.rsqrt(xd.square().mean(1, keepdim=True) + 1e-6) * leaf["norm"]
    ref = xd + silu_mul(h @ leaf["gate_up"].t()) @ leaf["down"].t()
    (ref * up.double()).sum().backward()
    # about ten bf16 roundings in a row, each 2^-9 of the norm and independent
    assert rel(out, ref) < 1e-2
    for n, v in leaf.items():
        assert rel(grads[n], v.grad) < 1e-2, n
    assert rel(grads["x"], xd.grad) < 1e-2


def test_training_calls_in_a_cuda_graph(ex):  # noqa: F811
    f = ex.GatedFeedForward(520, 128, 200, seed=4)
    x, up = (torch.randn(520, 128, device="cuda").to(torch.bfloat16) for _ in range(2))

    def step():
        out = f.forward(x)
        return [out, *f.backward(up).values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for t in (x, up):
            t.copy_(torch.randn(t.shape, device="cuda"))
        graph.replay()
        kept = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(kept, step()))


def test_examples_run(ex):  # noqa: F811
    ex.serve_light()
    ex.train_feed_forward(steps=5)


def test_the_gradient_passes_straight_through_the_8_bit_norm(ex):  # noqa: F811
    """A layer with its forward in 8 bits: the norm's gradient from moe_norm_quant's rstd is that of
    the norm in 64 bits."""
    T, K = 33, 384
    x, z, d = (torch.randn(T, K, device="cuda").to(torch.bfloat16) for _ in range(3))
    w = (1 + 0.2 * torch.randn(K, device="cuda")).to(torch.bfloat16)
    q, sf = torch.empty(T, K, dtype=torch.uint8, device="cuda"), torch.empty(T, 3, device="cuda")
    x_out, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    B.moe_norm_quant(x, w, q, sf, z=z, x_out=x_out, rstd=rstd)
    d_x, d_z, d_w = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(B.block_norm_workspace_size(T, K), dtype=torch.uint8, device="cuda")
    B.moe_block_norm_backward(x, z=z, pre_weight=w, rstd_pre=rstd, d_y=d, d_x=d_x, d_z=d_z,
                              d_pre_weight=d_w, workspace=ws)
    xd, wd = (x.double() + z.double()).requires_grad_(True), w.double().requires_grad_(True)
    (xd * torch.rsqrt(xd.square().mean(1, keepdim=True) + 1e-6) * wd * d.double()).sum().backward()
    assert rel(d_x, xd.grad) < 3e-3 and rel(d_z, xd.grad) < 3e-3 and rel(d_w, wd.grad) < 3e-3


def test_the_blocks_status_has_its_experts_too(ex):  # noqa: F811
    """A router that knows more experts than there are, and experts with too little room: the block's
    word tells of both."""
    from moe_expert_layer_prepare_gb300.block import FourBitExperts
    x = torch.randn(20, 512, device="cuda").to(torch.bfloat16)
    b = ex.make_light_block(20, 512, 256, 16, 4, 384, seed=3)
    few = FourBitExperts(20, 4, {n: v[:3] for n, v in b.experts.weights.items()})
    short = MoeBlock(20, 512, 256, 16, 4, 20, b.weights, experts=few)
    short.forward(x)
    assert int(short.status.item()) == B.MOE_DEV_BAD_EXPERT
    b.forward(x)
    assert int(b.status.item()) == 0
    w = dict(ex.make_block(20, 512, 256, 16, 4, 384, 2, 16, seed=5).weights, adapters=None)
    full = MoeBlock(20, 512, 256, 16, 4, 1, w)
    full.forward(x)
    assert int(full.status.item()) == B.MOE_DEV_CAPACITY
