"""moe_block_norm and moe_block_norm_backward against their formulas in 64 bits."""
import pytest
import torch

from moe_expert_layer_prepare_gb300 import binding as B
from tests._block_util import DTYPES, HALF_ULP, assert_within, rounded, strided
from tests._util import need_cuda

pytestmark = pytest.mark.gpu
EPS = 1e-5
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def cuda():
    need_cuda()
    from moe_expert_layer_prepare_gb300 import build
    build.build()
    B.load()


def forward64(x, z, post, gate, scale, pre, offset):
    xo = x
    if z is not None:
        n = z
        if post is not None:
            n = z * torch.rsqrt((z * z).mean(1, keepdim=True) + EPS) * (post + offset)
        if gate is not None:
            n = n * (gate[:, None] if gate.dim() == 1 and gate.shape[0] == x.shape[0] and
                     gate.shape[0] != x.shape[1] else gate)
        xo = x + scale * n
    y = None
    if pre is not None:
        y = xo * torch.rsqrt((xo * xo).mean(1, keepdim=True) + EPS) * (pre + offset)
    return xo, y


def tensors(T, K, dtype, wdtype, gate, layout, post=True, pre=True, z=True):
    g = torch.Generator(device="cuda").manual_seed(T * 31 + K)
    dt, wt = DTYPES[dtype], DTYPES[wdtype]

    def rnd(*shape, dtype=dt, mean=0.0):
        t = (torch.randn(shape, generator=g, device="cuda") + mean).to(dtype)
        if len(shape) == 2 and layout != "plain":
            t = strided(t, 8 if layout == "padded" else 3, 0 if layout == "padded" else 1)
        return t

    gt = {"none": None, "channel": lambda: rnd(K, dtype=wt), "token": lambda: rnd(T),
          "full": lambda: rnd(T, K)}[gate]
    return dict(x=rnd(T, K), z=rnd(T, K) if z else None,
                post=rnd(K, dtype=wt, mean=1.0) if post and z else None,
                gate=gt() if gt and z else None, pre=rnd(K, dtype=wt, mean=1.0) if pre else None,
                rnd=rnd, wt=wt, dt=dt)


def check(T, K, dtype, wdtype, gate, layout="plain", offset=0.0, scale=0.6, **kw):
    s = tensors(T, K, dtype, wdtype, gate, layout, **kw)
    dt, wt, rnd = s["dt"], s["wt"], s["rnd"]
    x, z, post, gt, pre = (s[n] for n in ("x", "z", "post", "gate", "pre"))
    f32 = dict(dtype=torch.float32, device="cuda")
    xo = rnd(T, K) if z is not None else None
    y = rnd(T, K) if pre is not None else None
    rz = torch.empty(T, **f32) if post is not None else None
    rx = torch.empty(T, **f32) if pre is not None else None
    B.moe_block_norm(x, z=z, post_weight=post, gate=gt, scale=scale, pre_weight=pre,
                     weight_offset=offset, eps=EPS, x_out=xo, y=y, rstd_post=rz, rstd_pre=rx)
    leaves = [None if t is None else t.cpu().double().requires_grad_(True)
              for t in (x, z, post, gt, pre)]
    rxo, ry = forward64(*leaves[:4], scale, leaves[4], offset)
    # sums over K in fp32 by trees: a factor's relative error grows with log2(K), held to 32 units
    rel = 32 * U
    size = leaves[0].detach().abs() + (rxo - leaves[0]).detach().abs() if z is not None else \
        leaves[0].detach().abs()
    if xo is not None:
        assert_within(xo, rxo.detach(), rounded(rxo.detach(), dt, rel * size), "x_out")
    if y is not None:
        inv = torch.rsqrt((rxo * rxo).mean(1, keepdim=True) + EPS).detach()
        yerr = rel * (size * inv * (leaves[4].detach() + offset).abs() + ry.detach().abs())
        assert_within(y, ry.detach(), rounded(ry.detach(), dt, yerr), "y")
        assert_within(rx, inv[:, 0], inv[:, 0] * rel * 4, "rstd_pre")

    dxo = rnd(T, K) if z is not None else None
    dy = rnd(T, K) if pre is not None else None
    dx, dz = rnd(T, K), rnd(T, K) if z is not None else None
    dg = torch.empty_like(gt) if gt is not None and layout == "plain" else \
        (rnd(*gt.shape, dtype=gt.dtype) if gt is not None else None)
    dp = torch.empty(K, dtype=wt, device="cuda") if post is not None else None
    dq = torch.empty(K, dtype=wt, device="cuda") if pre is not None else None
    ws = torch.full((B.block_norm_workspace_size(T, K),), 0xFF, dtype=torch.uint8, device="cuda")
    B.moe_block_norm_backward(x, z=z, post_weight=post, gate=gt, scale=scale, pre_weight=pre,
                              weight_offset=offset, rstd_post=rz, rstd_pre=rx, d_x_out=dxo, d_y=dy,
                              d_x=dx, d_z=dz, d_gate=dg, d_post_weight=dp, d_pre_weight=dq,
                              workspace=ws)
    outs, ups = [], []
    if dxo is not None:
        outs.append(rxo), ups.append(dxo.cpu().double())
    if dy is not None:
        outs.append(ry), ups.append(dy.cpu().double())
    torch.autograd.backward(outs, ups)

    # The sums that each gradient is made of, by magnitude: d = dx' + rx (u - xh mean(u xh)), and
    # dz the same with v = scale gate post d.  Where they cancel (K = 1: a norm of one value is
    # constant) the rounding of the terms is what is left.
    zero = torch.zeros(T, K, dtype=torch.float64)
    val = [None if t is None else t.detach() for t in leaves]
    d_size, n = (dxo.cpu().double().abs() if dxo is not None else zero), val[1]
    xov = rxo.detach()
    if pre is not None:
        inv = torch.rsqrt((xov * xov).mean(1, keepdim=True) + EPS)
        u, xh = (dy.cpu().double() * (val[4] + offset)).abs(), (size * inv)
        d_size = d_size + inv * (u + xh * (u * xh).mean(1, keepdim=True))
    branch = zero + scale
    if gt is not None:
        per_token = gt.dim() == 1 and gt.shape[0] == T and gt.shape[0] != K
        branch = branch * (val[3][:, None] if per_token else val[3]).abs()
    dz_size = branch * d_size
    if post is not None:
        rzv = torch.rsqrt((val[1] ** 2).mean(1, keepdim=True) + EPS)
        zh, v = (val[1] * rzv).abs(), dz_size * (val[2] + offset).abs()
        dp_size = (dz_size * zh).sum(0)
        dz_size = rzv * (v + zh * (v * zh).mean(1, keepdim=True))
        n = zh * (val[2] + offset).abs()
    dg_size = scale * d_size * n.abs() if n is not None else None

    def near(got, leaf, name, magnitude):
        if got is None:
            return
        assert_within(got, leaf.grad, rounded(leaf.grad, got.dtype, 64 * U * magnitude + 1e-30), name)

    near(dx, leaves[0], "d_x", d_size)
    near(dz, leaves[1], "d_z", dz_size)
    if post is not None:
        near(dp, leaves[2], "d_post_weight", dp_size)
    if gt is not None:
        near(dg, leaves[3], "d_gate", dg_size if gt.dim() == 2 else
             dg_size.sum(1) if per_token else dg_size.sum(0))
    if pre is not None:
        near(dq, leaves[4], "d_pre_weight", (dy.cpu().double().abs() * xh).sum(0))


SHAPES = [(1, 1), (1, 7168), (3, 8), (5, 33), (17, 520), (40, 1031), (9, 4096), (600, 64),
          (2, 16384), (3, 16383), (4, 5000)]


@pytest.mark.parametrize("T,K", SHAPES)
@pytest.mark.parametrize("dtype,wdtype", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"),
                                          ("fp16", "fp16"), ("fp32", "bf16")])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_forward_and_gradient(T, K, dtype, wdtype, gate):
    if T == K and gate == "token":
        pytest.skip("a [T] gate with T == K is a channel gate")
    check(T, K, dtype, wdtype, gate)


@pytest.mark.parametrize("layout", ["padded", "odd"])
@pytest.mark.parametrize("K", [64, 4100, 7168])
@pytest.mark.parametrize("gate", ["channel", "full"])
def test_strides(layout, K, gate):
    check(21, K, "bf16", "bf16", gate, layout=layout)
    check(21, K, "fp32", "fp32", gate, layout=layout)


@pytest.mark.parametrize("kw", [dict(post=False), dict(pre=False), dict(z=False),
                                dict(post=False, pre=False)])
def test_parts(kw):
    check(19, 264, "bf16", "bf16", "none", **kw)
    check(19, 264, "fp32", "fp32", "none", offset=1.0, **kw)
    if kw.get("z", True):
        check(19, 264, "fp16", "fp32", "token", **kw)


def test_weight_offset_and_many_rows():
    check(1001, 136, "fp32", "fp32", "channel", offset=1.0)
    check(5003, 72, "bf16", "fp32", "full", offset=1.0)


@pytest.mark.parametrize("T,K,dtype,wdtype", [(701, 4096, "bf16", "bf16"), (1003, 5120, "bf16", "bf16"),
                                              (1003, 7168, "fp16", "fp16"), (701, 8192, "bf16", "fp32"),
                                              (401, 7168, "fp32", "fp32"), (333, 16384, "bf16", "bf16")])
@pytest.mark.parametrize("gate", ["token", "full"])
def test_several_long_rows_a_block(T, K, dtype, wdtype, gate):
    check(T, K, dtype, wdtype, gate)


def test_in_place_zero_rows_and_infinite_values():
    s = tensors(8, 512, "bf16", "bf16", "none", "plain")
    x, z, post, pre = s["x"], s["z"], s["post"], s["pre"]
    z[3] = 0.0
    x[4] = 0.0
    z[4] = 0.0
    a, y1, y2 = s["rnd"](8, 512), s["rnd"](8, 512), s["rnd"](8, 512)
    B.moe_block_norm(x, z=z, post_weight=post, pre_weight=pre, x_out=a, y=y1)
    assert torch.equal(a[3], x[3]) and not a[4].any() and not y1[4].any()
    b = x.clone()
    B.moe_block_norm(b, z=z, post_weight=post, pre_weight=pre, x_out=b, y=y2)
    assert torch.equal(a, b) and torch.equal(y1, y2)
    x[5, 7] = float("inf")
    x[6, 9] = float("nan")
    B.moe_block_norm(x, z=z, post_weight=post, pre_weight=pre, x_out=a, y=y1)
    rows = [0, 1, 2, 3, 4, 7]
    assert torch.equal(a[rows], b[rows]) and torch.equal(y1[rows], y2[rows])  # each row alone
    assert bool(torch.isnan(y1[6]).all()) and bool(torch.isnan(y1[5, 7]))


def test_gradient_against_differences():
    T, K, h = 3, 24, 1e-2
    s = tensors(T, K, "fp32", "fp32", "channel", "plain")
    names = ("x", "z", "post", "gate", "pre")
    v = {n: s["rnd"](*s[n].shape) for n in names}
    cx, cy = s["rnd"](T, K), s["rnd"](T, K)

    def run(at):
        t = {n: s[n] + at * v[n] for n in names}
        xo, y = s["rnd"](T, K), s["rnd"](T, K)
        rz, rx = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        B.moe_block_norm(t["x"], z=t["z"], post_weight=t["post"], gate=t["gate"], scale=0.5,
                         pre_weight=t["pre"], eps=EPS, x_out=xo, y=y, rstd_post=rz, rstd_pre=rx)
        return (xo.double() * cx).sum().item() + (y.double() * cy).sum().item(), rz, rx

    # Richardson's combination of two central differences: truncation of order h^4
    d1 = (run(h)[0] - run(-h)[0]) / (2 * h)
    d2 = (run(2 * h)[0] - run(-2 * h)[0]) / (4 * h)
    num = (4 * d1 - d2) / 3
    _, rz, rx = run(0.0)
    d = {n: torch.empty_like(s[n]) for n in names}
    ws = torch.empty(B.block_norm_workspace_size(T, K), dtype=torch.uint8, device="cuda")
    B.moe_block_norm_backward(s["x"], z=s["z"], post_weight=s["post"], gate=s["gate"], scale=0.5,
                              pre_weight=s["pre"], rstd_post=rz, rstd_pre=rx, d_x_out=cx, d_y=cy,
                              d_x=d["x"], d_z=d["z"], d_gate=d["gate"], d_post_weight=d["post"],
                              d_pre_weight=d["pre"], workspace=ws)
    ana = sum((d[n].double() * v[n].double()).sum().item() for n in names)
    size = sum((d[n].double() * v[n].double()).abs().sum().item() for n in names)
    assert abs(ana - num) <= size * 1e-3 + 2 * T * K * 4 * U / h, (ana, num, size)


def test_stream_same_bits_twice_and_refusals():
    T, K = 700, 1024
    s = tensors(T, K, "bf16", "fp32", "channel", "plain")
    rz, rx = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    xo, y = s["rnd"](T, K), s["rnd"](T, K)
    kw = dict(z=s["z"], post_weight=s["post"], gate=s["gate"], pre_weight=s["pre"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    B.moe_block_norm(s["x"], x_out=xo, y=y, rstd_post=rz, rstd_pre=rx, stream=st, **kw)
    st.synchronize()
    ws = torch.empty(B.block_norm_workspace_size(T, K), dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(2):
        dp, dq, dg = (torch.empty(K, device="cuda") for _ in range(3))
        dx, dz = s["rnd"](T, K), s["rnd"](T, K)
        B.moe_block_norm_backward(s["x"], rstd_post=rz, rstd_pre=rx, d_x_out=xo, d_y=y, d_x=dx,
                                  d_z=dz, d_gate=dg, d_post_weight=dp, d_pre_weight=dq,
                                  workspace=ws, **kw)
        got.append((dp, dq, dg, dx, dz))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    with pytest.raises(ValueError):
        B.moe_block_norm(s["x"], x_out=xo.float(), y=y, **kw)
    with pytest.raises(ValueError):
        B.moe_block_norm(s["x"].t().contiguous().t(), x_out=xo, y=y, **kw)
    with pytest.raises(B.MoeError) as e:
        B.moe_block_norm(s["x"], y=y, **kw)
    assert e.value.status == 1  # z without x_out
    with pytest.raises(B.MoeError) as e:
        B.moe_block_norm_backward(s["x"], rstd_post=rz, rstd_pre=rx, d_y=y, d_x=xo, **kw)
    assert e.value.status == 5  # no workspace


@pytest.mark.parametrize("T", [2, 48, 520])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["channel", "token"])
def test_as_many_tokens_as_columns(T, dtype, kind):
    # [T] and [K] are one shape: the caller says which
    K, dt, token = T, DTYPES[dtype], kind == "token"
    s = tensors(T, K, dtype, dtype, kind, "plain")
    code = B.MOE_GATE_TOKEN if token else B.MOE_GATE_CHANNEL
    kw = dict(z=s["z"], post_weight=s["post"], gate=s["gate"], scale=0.6, pre_weight=s["pre"])
    xo, y, dxo, dy, dx, dz = (s["rnd"](T, K) for _ in range(6))
    rz, rx = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    with pytest.raises(ValueError, match="gate_kind"):
        B.moe_block_norm(s["x"], eps=EPS, x_out=xo, y=y, rstd_post=rz, rstd_pre=rx, **kw)
    B.moe_block_norm(s["x"], eps=EPS, x_out=xo, y=y, rstd_post=rz, rstd_pre=rx, gate_kind=code, **kw)
    dg, dp, dq = (torch.empty(K, dtype=dt, device="cuda") for _ in range(3))
    ws = torch.empty(B.block_norm_workspace_size(T, K), dtype=torch.uint8, device="cuda")
    back = dict(rstd_post=rz, rstd_pre=rx, d_x_out=dxo, d_y=dy, d_x=dx, d_z=dz, d_gate=dg,
                d_post_weight=dp, d_pre_weight=dq, workspace=ws)
    with pytest.raises(ValueError, match="gate_kind"):
        B.moe_block_norm_backward(s["x"], **kw, **back)
    B.moe_block_norm_backward(s["x"], gate_kind=code, **kw, **back)

    leaf = {n: s[n].cpu().double().requires_grad_(True) for n in ("x", "z", "post", "gate", "pre")}
    g = leaf["gate"][:, None] if token else leaf["gate"][None, :]
    rxo, ry = forward64(leaf["x"], leaf["z"], leaf["post"], g, 0.6, leaf["pre"], 0.0)
    torch.autograd.backward([rxo, ry], [dxo.cpu().double(), dy.cpu().double()])
    # one rounding of each value, and fp32 sums that may cancel to a hundredth
    tol = HALF_ULP[dt] + 6400 * U
    for name, got, ref in (("x_out", xo, rxo), ("y", y, ry), ("d_x", dx, leaf["x"].grad),
                           ("d_z", dz, leaf["z"].grad), ("d_gate", dg, leaf["gate"].grad),
                           ("d_post", dp, leaf["post"].grad), ("d_pre", dq, leaf["pre"].grad)):
        off = ((got.cpu().double() - ref).norm() / ref.norm()).item()
        assert off <= tol, (name, off)


def test_gate_kinds_that_shape_and_type_settle_and_refusals():
    T = K = 32
    s = tensors(T, K, "bf16", "fp32", "token", "plain")
    kw = dict(z=s["z"], post_weight=s["post"], pre_weight=s["pre"])

    def run(gate, **more):
        xo, y = s["rnd"](T, K), s["rnd"](T, K)
        B.moe_block_norm(s["x"], gate=gate, x_out=xo, y=y, **kw, **more)
        return torch.cat([xo, y])

    token, channel = s["gate"], s["rnd"](K, dtype=torch.float32)
    assert torch.equal(run(token), run(token[:, None]))  # bf16, where channel gates are fp32
    assert torch.equal(run(token), run(token, gate_kind=B.MOE_GATE_TOKEN))
    assert torch.equal(run(channel), run(channel, gate_kind=B.MOE_GATE_CHANNEL))
    full = token[:, None].expand(T, K).contiguous()
    assert torch.equal(run(full), run(full, gate_kind=B.MOE_GATE_FULL))
    for gate, kind in ((token, B.MOE_GATE_CHANNEL), (channel, B.MOE_GATE_TOKEN),
                       (token, B.MOE_GATE_FULL), (full, B.MOE_GATE_TOKEN), (token, 7),
                       (full, B.MOE_GATE_NONE), (None, B.MOE_GATE_TOKEN)):
        with pytest.raises(ValueError):
            run(gate, gate_kind=kind)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_no_tokens(gate):
    K = 72
    s = tensors(0, K, "bf16", "fp32", gate, "plain")
    kw = dict(z=s["z"], post_weight=s["post"], gate=s["gate"], pre_weight=s["pre"])
    e, r = s["rnd"](0, K), torch.empty(0, device="cuda")
    B.moe_block_norm(s["x"], x_out=e, y=e.clone(), rstd_post=r, rstd_pre=r.clone(), **kw)
    B.moe_block_norm(s["x"], pre_weight=s["pre"], y=e)
    dp, dq = torch.full((K,), 7.0, device="cuda"), torch.full((K,), 7.0, device="cuda")
    dg = None if s["gate"] is None else torch.full_like(s["gate"], 7.0)
    n = B.block_norm_workspace_size(0, K)
    B.moe_block_norm_backward(s["x"], rstd_post=r, rstd_pre=r, d_x_out=e, d_y=e, d_x=e, d_z=e,
                              d_gate=dg, d_post_weight=dp, d_pre_weight=dq,
                              workspace=torch.empty(n, dtype=torch.uint8, device="cuda"), **kw)
    assert not dp.any() and not dq.any() and (dg is None or not dg.any())
    dq.fill_(7.0)
    B.moe_block_norm_backward(s["x"], pre_weight=s["pre"], rstd_pre=r, d_y=e, d_x=e,
                              d_pre_weight=dq)
    assert not dq.any()


def test_no_columns():
    x, w = torch.empty(5, 0, device="cuda"), torch.empty(0, device="cuda")
    B.moe_block_norm(x, z=x, post_weight=w, pre_weight=w, x_out=x, y=x)
    B.moe_block_norm_backward(x, z=x, post_weight=w, pre_weight=w, d_x=x, d_z=x, d_y=x,
                              d_post_weight=w, d_pre_weight=w)


# rows of two packs a thread, in each case of how many blocks one or two stages leave an SM
@pytest.mark.parametrize("K,wdtype", [(6144, "fp32"), (7168, "bf16"), (7672, "bf16"),
                                      (7680, "bf16"), (8192, "bf16"), (8192, "fp32")])
@pytest.mark.parametrize("gate", ["none", "channel", "full"])
def test_stages_of_long_rows(K, wdtype, gate):
    check(503, K, "bf16", wdtype, gate)
