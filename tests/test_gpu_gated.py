"""moe_gated_linear and its gradients against the formulas in 64 bits."""
import ctypes
import math
import time

import pytest
import torch

from moe_expert_layer_prepare_gb300 import binding as B
from tests._block_util import DTYPES, HALF_ULP, assert_within, rounded, strided
from tests._util import need_cuda

pytestmark = pytest.mark.gpu
ACTS = {"silu": B.MOE_ACT_SILU, "gelu_tanh": B.MOE_ACT_GELU_TANH}

# fp32 sums of K products: their error is below 2^-16 of the sum of magnitudes.  The activation in
# fp32, relative: its argument's few roundings, at most 17 times amplified by the exponential where
# the result is not yet below 2^-24 of its argument, and the exponential's and quotient's own.
SUM, ACT = 2.0 ** -16, 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def cuda():
    need_cuda()
    from moe_expert_layer_prepare_gb300 import build
    build.build()
    B.load()


def act(name, g):
    """Value and slope in the precision of g."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def problem(T, K, N, dtype, seed=0, layout="plain", gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + 11 * K + N)
    dt = DTYPES[dtype]

    def rnd(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)

    x, w, d = rnd(T, K), rnd(2 * N, K, std=gain * K ** -0.5), rnd(T, N)
    if layout != "plain":
        x, d = strided(x, 8), strided(d, 5, 1)
    return x, w, d


def new(shape, dt, layout="plain", pad=3, offset=1):
    t = torch.full(shape, float("nan"), dtype=dt, device="cuda")
    return t if layout == "plain" else strided(t, pad, offset)


def check_forward(x, w, name, layout="plain", keep=True):
    T, N, dt = x.shape[0], w.shape[0] // 2, x.dtype
    out = new((T, N), dt, layout)
    gate_up = new((T, 2 * N), dt, layout) if keep else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.moe_gated_linear(x, w, out, activation=ACTS[name], gate_up=gate_up, device_status=status)
    xd, wd = x.double(), w.double()
    gu, mag = xd @ wd.t(), xd.abs() @ wd.abs().t() * SUM
    (g, u), (eg, eu) = gu.split(N, 1), mag.split(N, 1)
    a, _ = act(name, g)
    # the slope is at most 1.13 in size; the error's own product is of the second order
    extra = 1.2 * eg * (u.abs() + eu) + a.abs() * eu + (a * u).abs() * ACT
    assert_within(out, a * u, rounded(a * u, dt, extra), "out")
    if keep:
        assert_within(gate_up, gu, rounded(gu, dt, mag), "gate_up")
    assert int(status.item()) == 0
    return out, gate_up


def backward(d, x, w, gate_up, name, layout="plain", want=("x", "w"), pad=3, offset=1):
    T, K = x.shape
    N, dt = w.shape[0] // 2, x.dtype
    ws = torch.full((B.gated_linear_workspace_size(T, K, N),), 0xFF, dtype=torch.uint8, device="cuda")
    d_x = new((T, K), dt, layout, pad, offset) if "x" in want else None
    d_w = new((2 * N, K), dt) if "w" in want else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.moe_gated_linear_backward(d, x, w, gate_up, d_x=d_x, d_weight=d_w, activation=ACTS[name],
                                workspace=ws, device_status=status)
    assert int(status.item()) == 0
    return d_x, d_w


def check_backward(d, x, w, gate_up, name, **kw):
    d_x, d_w = backward(d, x, w, gate_up, name, **kw)
    N, dt = w.shape[0] // 2, x.dtype
    g, u = gate_up.double().split(N, 1)
    dd, xd, wd = d.double(), x.double(), w.double()
    a, slope = act(name, g)
    d_gu = torch.cat([dd * u * slope, dd * a], 1)
    # each gradient of gate and up: computed in fp32 (the slope's terms are up to 1 + |g| in
    # size), then rounded once
    size = torch.cat([(dd * u).abs() * (1 + slope.abs()), (dd * a).abs()], 1)
    off = rounded(d_gu, dt, size * 2 * ACT)
    for got, ref, extra in ((d_x, d_gu @ wd, off @ wd.abs() + d_gu.abs() @ wd.abs() * SUM),
                            (d_w, d_gu.t() @ xd, off.t() @ xd.abs() + d_gu.abs().t() @ xd.abs() * SUM)):
        if got is None:
            continue
        assert_within(got, ref, rounded(ref, dt, extra), "gradient")
        # the roundings are independent: together they are off by about half a step over root
        # three, twice; a product left out of the sums is more
        assert (got.double() - ref).norm() <= 2 * HALF_ULP[dt] * ref.norm() + 1e-30
    return d_x, d_w


SIZES = [(1, 8, 1), (1, 7168, 130), (2, 72, 100), (5, 520, 64), (16, 1000, 257), (17, 512, 33),
         (33, 2048, 384), (64, 256, 129), (65, 320, 300), (128, 4096, 256), (130, 136, 65),
         (300, 1032, 260), (512, 192, 264), (513, 72, 513), (700, 512, 512), (1031, 2056, 203)]


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_forward(T, K, N, dtype, name):
    x, w, _ = problem(T, K, N, dtype)
    check_forward(x, w, name)


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_backward(T, K, N, dtype, name):
    x, w, d = problem(T, K, N, dtype)
    gate_up = (x.float() @ w.float().t()).to(x.dtype)
    check_backward(d, x, w, gate_up, name)


@pytest.mark.parametrize("T", [3, 70, 600])
@pytest.mark.parametrize("N", [96, 201])
def test_strides_and_parts(T, N):
    x, w, d = problem(T, 328, N, "bf16", layout="strided")
    out, gate_up = check_forward(x, w, "silu", layout="strided")
    alone, _ = check_forward(x, w, "silu", keep=False)
    assert torch.equal(out, alone)
    both = check_backward(d, x, w, gate_up, "silu", layout="strided")
    wide = check_backward(d, x, w, gate_up, "silu", layout="strided", pad=8, offset=8)
    for want, at in ((("x",), 0), (("w",), 1)):
        one = check_backward(d, x, w, gate_up, "silu", want=want)
        assert one[1 - at] is None and torch.equal(one[at], both[at])
    assert torch.equal(wide[0], both[0])


@pytest.mark.parametrize("T,K,N", [(40, 264, 70), (600, 520, 300), (1500, 72, 65), (300, 4096, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_integers_give_exact_gradients(T, K, N, dtype):
    """Whole numbers that the gradients of gate and up hold exactly (silu's slope at 32 is 1 in
    fp32): every sum is exact, so the results are the sums rounded once."""
    g = torch.Generator(device="cuda").manual_seed(T + K)
    dt = DTYPES[dtype]

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=g, device="cuda").to(dt)

    x, w, d = whole(T, K), whole(2 * N, K), whole(T, N)
    gate_up = torch.cat([torch.full((T, N), 32.0, dtype=dt, device="cuda"), whole(T, N)], 1)
    d_gu = torch.cat([d.double() * gate_up[:, N:].double(), d.double() * 32], 1)
    d_x, d_w = backward(d, x, w, gate_up, "silu")
    assert torch.equal(d_x, (d_gu @ w.double()).to(dt))
    assert torch.equal(d_w, (d_gu.t() @ x.double()).to(dt))


def test_gradients_against_differences():
    T, K, N = 6, 64, 40
    x, w, d = problem(T, K, N, "fp16")
    for name in ACTS:
        _, gate_up = check_forward(x, w, name)
        d_x, d_w = check_backward(d, x, w, gate_up, name)

        def loss(xx, ww):
            g, u = (xx @ ww.t()).split(N, 1)
            return (act(name, g)[0] * u * d.double()).sum().item()

        h = 1e-6
        for t, k, r in ((0, 0, 0), (5, 63, 79), (2, 17, 41)):
            e, f = torch.zeros_like(x, dtype=torch.float64), torch.zeros_like(w, dtype=torch.float64)
            e[t, k], f[r, k] = h, h
            xd, wd = x.double(), w.double()
            sx = (loss(xd + e, wd) - loss(xd - e, wd)) / (2 * h)
            sw = (loss(xd, wd + f) - loss(xd, wd - f)) / (2 * h)
            # sums of 80 and of 6 terms, each within a few fp16 roundings (2^-11) of its size
            assert abs(d_x[t, k].item() - sx) <= 80 * 2.0 ** -10 * 3 * K ** -0.5 + 2.0 ** -10 * abs(sx)
            assert abs(d_w[r, k].item() - sw) <= 6 * 2.0 ** -10 * 12 + 2.0 ** -10 * abs(sw)


@pytest.mark.parametrize("T", [2, 600])
@pytest.mark.parametrize("name", list(ACTS))
def test_large_arguments(T, name):
    """Gates far beyond where the activation is flat: 0 or the gate itself, never NaN."""
    x, w, d = problem(T, 64, 24, "bf16", gain=300.0)
    _, gate_up = check_forward(x, w, name)
    check_backward(d, x, w, gate_up, name)
    gate_up[:, :24] = torch.tensor([1e30, -1e30, 3e4, -3e4, 90.0, -90.0, 0.0, -0.0] * 3, device="cuda")
    gate_up[:, 24:] = 1.0
    d_x, d_w = backward(d, x, w, gate_up, name)
    assert bool(d_x.isfinite().all()) and bool(d_w.isfinite().all())


@pytest.mark.parametrize("T", [4, 700])
def test_a_broken_token_stays_in_its_row(T):
    x, w, d = problem(T, 256, 96, "bf16")
    clean, gate_up = check_forward(x, w, "silu")
    clean_x, _ = backward(d, x, w, gate_up, "silu")
    x[1, 3] = float("nan")
    out, gu = new((T, 96), x.dtype), new((T, 192), x.dtype)
    B.moe_gated_linear(x, w, out, gate_up=gu)
    d_x, _ = backward(d, x, w, gu, "silu")
    other = torch.arange(T, device="cuda") != 1
    assert bool(out[1].isnan().all()) and torch.equal(out[other], clean[other])
    assert bool(d_x[1].isnan().all()) and torch.equal(d_x[other], clean_x[other])


def test_rows_behind_the_last_and_empty_batches():
    x, w, d = problem(20, 64, 40, "bf16")
    out, gu = torch.full((20, 40), 7.0, device="cuda").to(x.dtype), torch.full((20, 80), 7.0, device="cuda").to(x.dtype)
    B.moe_gated_linear(x[:13], w, out[:13], gate_up=gu[:13])
    B.moe_gated_linear(x[:0], w, out[:0], gate_up=gu[:0])
    assert bool((out[13:] == 7).all()) and bool((gu[13:] == 7).all())
    d_w, d_x = torch.full_like(w, 7.0), torch.full_like(x, 7.0)
    ws = torch.empty(B.gated_linear_workspace_size(20, 64, 40), dtype=torch.uint8, device="cuda")
    B.moe_gated_linear_backward(d[:13], x[:13], w, gu[:13], d_x=d_x[:13], workspace=ws)
    assert bool((d_x[13:] == 7).all())
    B.moe_gated_linear_backward(d[:0], x[:0], w, gu[:0], d_x=d_x[:0], d_weight=d_w)
    assert bool((d_w == 0).all()) and bool((d_x[13:] == 7).all())


def test_stream_same_bits_twice_and_a_shared_workspace():
    """Batches of different sizes behind one another on another stream and one workspace."""
    s = torch.cuda.Stream()
    cases = [problem(T, 520, 200, "bf16", seed=T) for T in (700, 3, 130, 1031)]
    ws = torch.empty(max(B.gated_linear_workspace_size(x.shape[0], 520, 200) for x, _, _ in cases),
                     dtype=torch.uint8, device="cuda")
    want = []
    for x, w, d in cases:
        out, gu = check_forward(x, w, "silu")
        want.append((out, *backward(d, x, w, gu, "silu")))
    torch.cuda.synchronize()
    got = []
    with torch.cuda.stream(s):
        for x, w, d in cases * 2:
            out, gu = new((x.shape[0], 200), x.dtype), new((x.shape[0], 400), x.dtype)
            d_x, d_w = new(x.shape, x.dtype), new(w.shape, x.dtype)
            B.moe_gated_linear(x, w, out, gate_up=gu)
            B.moe_gated_linear_backward(d, x, w, gu, d_x=d_x, d_weight=d_w, workspace=ws)
            got.append((out, d_x, d_w))
    s.synchronize()
    for a, b in zip(want * 2, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_workspace_serves_shorter_batches():
    sizes = [B.gated_linear_workspace_size(T, 512, 203) for T in range(1, 1200)]
    assert sizes == sorted(sizes)


def test_refusals():
    x, w, d = problem(4, 64, 24, "bf16")
    out, gu, dx, dw = new((4, 24), x.dtype), new((4, 48), x.dtype), new((4, 64), x.dtype), new((48, 64), x.dtype)
    ws = torch.empty(B.gated_linear_workspace_size(4, 64, 24), dtype=torch.uint8, device="cuda")
    for kw in (dict(weight=w[:47]), dict(weight=w.float()), dict(out=out[:, :23]), dict(out=out.t()),
               dict(gate_up=gu[:, :47]), dict(x=x.cpu()), dict(weight=strided(w, 8))):
        with pytest.raises(ValueError):
            B.moe_gated_linear(**{**dict(x=x, weight=w, out=out), **kw})
    good = dict(d_out=d, x=x, weight=w, gate_up=gu, d_x=dx, d_weight=dw, workspace=ws)
    for kw in (dict(d_out=d[:3]), dict(gate_up=gu[:, :24]), dict(d_x=dx[:3]), dict(d_weight=dw[:24]),
               dict(d_weight=dw.float())):
        with pytest.raises(ValueError):
            B.moe_gated_linear_backward(**{**good, **kw})
    for kw in (dict(workspace=None), dict(workspace=ws[:-1]), dict(activation=B.MOE_ACT_NONE),
               dict(x=strided(x, 3))):
        with pytest.raises(B.MoeError):
            B.moe_gated_linear_backward(**{**good, **kw})
    with pytest.raises(B.MoeError):
        B.moe_gated_linear(x.float(), w.float(), out.float())


@pytest.mark.parametrize("T", [16, 700])
def test_wait_timeout_sets_status_and_context_survives(T):
    """As in test_gpu_timeout: the first CTAs of the test build withhold a stage; the call sets the
    status and returns, and the regular library goes on in the same process."""
    from moe_expert_layer_prepare_gb300 import build
    test_lib = B.configure(ctypes.CDLL(build.build_test_variant("timeout")))
    x, w, d = problem(T, 1024, 128, "bf16")
    out, gu = check_forward(x, w, "silu")
    ws = torch.empty(B.gated_linear_workspace_size(T, 1024, 128), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    regular = B._lib
    status = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
    t0 = time.perf_counter()
    try:
        B._lib = test_lib
        B.moe_gated_linear(x, w, new(out.shape, x.dtype), device_status=status[0])
        B.moe_gated_linear_backward(d, x, w, gu, d_x=new(x.shape, x.dtype), workspace=ws,
                                    device_status=status[1])
        torch.cuda.synchronize()
    finally:
        B._lib = regular
    assert time.perf_counter() - t0 < 5.0
    assert all(int(s.item()) & B.MOE_DEV_TIMEOUT for s in status)
    again, gu = check_forward(x, w, "silu")
    assert torch.equal(again, out)
    check_backward(d, x, w, gu, "silu")


@pytest.mark.parametrize("T,N", [(1024, 2048), (700, 3000), (1300, 2100), (600, 2600), (2000, 1100), (513, 4000),
                                 (1500, 1700), (600, 3700), (513, 3300), (129, 70), (256, 2048), (512, 1990)])
def test_tiles_of_every_width(T, N):
    """Batches for which the forward's tiles are 64 to 128 outputs wide, whole or shared by two pairs
    of CTAs, with a last tile that is not full."""
    x, w, _ = problem(T, 520, N, "bf16")
    check_forward(x, w, "silu")
    check_forward(x, w, "gelu_tanh", layout="strided")


@pytest.mark.parametrize("T,K,N", [(1, 512, 5000), (3, 1024, 3001), (9, 4096, 700), (700, 1000, 300)])
def test_gradients_of_few_tokens_and_a_workspace_on_16_bytes(T, K, N):
    """Wide blocks of few tokens; tiles cut along k keep their sums in a workspace that starts on 16
    bytes and on no more; results on 16 bytes too."""
    x, w, d = problem(T, K, N, "bf16")
    gate_up = (x.float() @ w.float().t()).to(x.dtype)
    want = check_backward(d, x, w, gate_up, "silu")
    need = B.gated_linear_workspace_size(T, K, N)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    ws = ws[(16 - ws.data_ptr()) % 32:][:need]
    assert ws.data_ptr() % 32 == 16
    d_x = torch.empty(T * K + 8, dtype=x.dtype, device="cuda")[8:].view(T, K)
    d_w = torch.empty(2 * N * K + 8, dtype=x.dtype, device="cuda")[8:].view(2 * N, K)
    B.moe_gated_linear_backward(d, x, w, gate_up, d_x=d_x, d_weight=d_w, workspace=ws)
    assert torch.equal(d_x, want[0]) and torch.equal(d_w, want[1])


@pytest.mark.parametrize("T", [64, 65, 100, 128, 129])
def test_wide_blocks_around_the_kernels_limits(T):
    """Around as many features as give every second pair of CTAs a tile, and every one."""
    for N in (4800, 4900, 9600, 9800):
        x, w, _ = problem(T, 136, N, "fp16")
        check_forward(x, w, "gelu_tanh")


@pytest.mark.parametrize("T,K,N", [(129, 3528, 384), (256, 3592, 601), (300, 4104, 203),
                                   (256, 3592, 4608), (256, 3592, 4736), (385, 3520, 264)])
@pytest.mark.parametrize("layout", ["plain", "strided"])
def test_two_pairs_a_tile_and_the_tiles_alone(T, K, N, layout):
    """K and tiles around what two pairs share, an odd number of slabs, odd rows."""
    x, w, _ = problem(T, K, N, "bf16", layout=layout)
    out, _ = check_forward(x, w, "silu", layout=layout)
    alone, _ = check_forward(x, w, "silu", layout=layout, keep=False)
    assert torch.equal(out, alone)


@pytest.mark.parametrize("T", [1, 32, 64, 128])
@pytest.mark.parametrize("N", [1024, 1160, 1216, 2304, 2432, 2500, 4736, 4864])
def test_shares_of_k_around_the_clusters_that_run_at_once(T, N):
    x, w, _ = problem(T, 2056, N, "bf16")
    check_forward(x, w, "silu")


@pytest.mark.parametrize("keep", [False, True])
def test_a_tile_of_two_pairs_that_gave_up_is_not_stored(keep):
    """As test_wait_timeout_sets_status_and_context_survives, where two pairs share a tile: the first
    pair withholds a stage, so no CTA of its cluster stores; the other tile is whole."""
    from moe_expert_layer_prepare_gb300 import build
    test_lib = B.configure(ctypes.CDLL(build.build_test_variant("timeout")))
    T, K, N = 256, 4096, 256
    x, w, _ = problem(T, K, N, "bf16")
    out, gate_up = check_forward(x, w, "silu")
    got, gu = torch.full_like(out, 7.0), torch.full_like(gate_up, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    regular = B._lib
    t0 = time.perf_counter()
    try:
        B._lib = test_lib
        B.moe_gated_linear(x, w, got, gate_up=gu if keep else None, device_status=status)
        torch.cuda.synchronize()
    finally:
        B._lib = regular
    assert time.perf_counter() - t0 < 5.0
    assert int(status.item()) == B.MOE_DEV_TIMEOUT
    assert bool((got[:, :128] == 7).all()) and torch.equal(got[:, 128:], out[:, 128:])
    if keep:
        for at in (0, N):
            assert bool((gu[:, at:at + 128] == 7).all())
            assert torch.equal(gu[:, at + 128:at + N], gate_up[:, at + 128:at + N])
    again, _ = check_forward(x, w, "silu")
    assert torch.equal(again, out)
