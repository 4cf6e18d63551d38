"""moe_w4_linear against its formula in 64 bits."""
import math

import pytest
import torch

from moe_expert_layer_prepare_gb300 import binding as B
from tests._block_util import DTYPES, assert_within, rounded, strided
from tests._util import need_cuda

pytestmark = pytest.mark.gpu
ACTS = {"none": B.MOE_ACT_NONE, "silu": B.MOE_ACT_SILU, "gelu_tanh": B.MOE_ACT_GELU_TANH}
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
# fp32 sums of exact products, at most 32 additions of a group behind one another and 512 groups in
# eight parts: below 2^-16 of the sum of magnitudes.  The activation as in test_gpu_gated.
SUM, ACT = 2.0 ** -16, 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def cuda():
    need_cuda()
    from moe_expert_layer_prepare_gb300 import build
    build.build()
    B.load()


def matrices(lead, K, fmt, G, dtype, zeros, g, whole=False):
    """(bytes, scales, zeros) on the GPU and the weights in fp64."""
    w = torch.randint(0, 256, (*lead, K // 2), dtype=torch.uint8, generator=g, device="cuda")
    codes = torch.stack([w & 15, w >> 4], -1).view(*lead, K // G, G)
    z = None
    if fmt == "e2m1":
        s = torch.randint(124, 131, (*lead, K // G), dtype=torch.uint8, generator=g, device="cuda")
        scale, value = torch.exp2(s.double() - 127), E2M1.cuda()[codes.long()]
    else:
        s = 0.01 + torch.rand((*lead, K // G), generator=g, device="cuda")
        if whole:
            s = torch.exp2(torch.floor(s * 4) - 2)
        s = s.to(dtype)
        if zeros:
            z = torch.randint(0, 256, (*lead, K // G), dtype=torch.uint8, generator=g, device="cuda")
        scale = s.double()
        value = codes.double() - ((z & 15).double()[..., None] if zeros else 8.0)
    return w, s, z, (value * scale[..., None]).view(*lead, K)


def act(name, v):
    if name == "none":
        return v
    g, u = v.chunk(2, -1)
    if name == "silu":
        return g * torch.sigmoid(g) * u
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) * u


def bound(name, v, extra, dt):
    """Bound of out from the products v and the error of their fp32 sums."""
    ref = act(name, v)
    if name != "none":
        g, u = v.chunk(2, -1)
        eg, eu = extra.chunk(2, -1)
        extra = 1.2 * eg * (u.abs() + eu) + g.abs() * eu + ref.abs() * ACT
    return ref, rounded(ref, dt, extra)


def problem(T, K, N, dtype, fmt="int4", G=32, zeros=False, E=0, k=0, seed=0, pad=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 3 * T + K + 7 * N)
    dt = DTYPES[dtype]
    lead = (E, N) if E else (N,)
    w, s, z, values = matrices(lead, K, fmt, G, dt, zeros, g)
    x = (torch.randn(T, K, generator=g, device="cuda") * K ** -0.5 / 3).to(dt)
    ids = None
    if E:
        ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
        ids[torch.rand(T, k, generator=g, device="cuda") < pad] = -1
    return dict(x=x, weight=w, scales=s, zeros=z, topk_ids=ids), values


def expect(p, values):
    x, ids = p["x"].double(), p["topk_ids"]
    if ids is None:
        return x @ values.t(), x.abs() @ values.abs().t() * SUM
    flat = ids.reshape(-1).tolist()
    v = torch.zeros(len(flat), values.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(v)
    for r, e in enumerate(flat):
        if 0 <= e < values.shape[0]:
            row = x[r // ids.shape[1]]
            v[r], mag[r] = values[e] @ row, values[e].abs() @ row.abs() * SUM
    return v, mag


def run(p, name="none", layout="plain", status=None, stream=None):
    n, dt = p["weight"].shape[-2], p["x"].dtype
    rows = p["x"].shape[0] if p["topk_ids"] is None else p["topk_ids"].numel()
    out = torch.full((rows, n if name == "none" else n // 2), float("nan"), dtype=dt, device="cuda")
    if layout != "plain":
        out = strided(out, 3, 1)
    B.moe_w4_linear(out=out, activation=ACTS[name], device_status=status, stream=stream, **p)
    return out


def check(p, values, name="none", **kw):
    out = run(p, name, **kw)
    ref, tol = bound(name, *expect(p, values), out.dtype)
    assert_within(out, ref, tol, "out")
    return out


FORMATS = [("int4", 32, False), ("int4", 64, True), ("int4", 128, False), ("int4", 128, True),
           ("int4", 32, True), ("e2m1", 32, False)]


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,K,N", [(1, 128, 1), (1, 7168, 130), (2, 256, 16), (3, 384, 100),
                                   (8, 2048, 514), (9, 640, 66), (16, 4096, 258), (17, 512, 34),
                                   (33, 2176, 18), (70, 1152, 30)])
def test_one_matrix(T, K, N, dtype, fmt, G, zeros):
    p, values = problem(T, K, N, dtype, fmt, G, zeros)
    check(p, values)
    if N % 2 == 0:
        check(p, values, "silu")


@pytest.mark.parametrize("K", [32, 96, 224, 288, 1056])
@pytest.mark.parametrize("fmt", ["int4", "e2m1"])
def test_short_and_ragged_rows(K, fmt):
    p, values = problem(5, K, 44, "bf16", fmt)
    for name in ACTS:
        check(p, values, name)


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("T,K,N,E,k", [(1, 512, 64, 16, 8), (1, 2048, 66, 256, 8), (5, 256, 130, 7, 3),
                                       (16, 640, 48, 300, 8), (128, 384, 18, 8, 1),
                                       (60, 256, 34, 3, 2), (1024, 128, 16, 1024, 1)])
def test_experts(T, K, N, E, k, name, fmt, G, zeros):
    p, values = problem(T, K, N, "bf16", fmt, G, zeros, E, k, pad=0.1)
    check(p, values, name)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_all_routes_to_one_expert_or_none(dtype):
    p, values = problem(40, 512, 50, dtype, "int4", 64, True, 5, 2)
    p["topk_ids"].fill_(3)
    check(p, values, "silu")
    p["topk_ids"].fill_(-1)
    assert bool((run(p) == 0).all())
    p["topk_ids"][7, 1] = 4
    check(p, values)


def test_every_code_scale_and_zero_point():
    """Each code alone under a one of x, with the scales' whole range of exponents: exact values."""
    codes = torch.arange(16, device="cuda", dtype=torch.uint8)
    for dtype in ("bf16", "fp16"):
        dt = DTYPES[dtype]
        x = torch.eye(32, device="cuda").to(dt)
        w = (codes[:, None] * 17).expand(16, 16).contiguous()
        for z in range(16):
            s = torch.full((16, 1), 0.25, device="cuda").to(dt)
            zs = torch.full((16, 1), z + 16 * (z % 3), dtype=torch.uint8, device="cuda")
            out = torch.empty(32, 16, dtype=dt, device="cuda")
            B.moe_w4_linear(x, w, s, out, zeros=zs)
            assert torch.equal(out, ((codes.float() - z) * 0.25).to(dt).expand(32, 16))
        exps = range(0, 255) if dtype == "bf16" else range(106, 141)
        for e in exps:
            s = torch.full((16, 1), e, dtype=torch.uint8, device="cuda")
            B.moe_w4_linear(x, w, s, out)
            want = (E2M1.cuda()[codes.long()] * 2.0 ** (e - 127)).float().to(dt)
            assert torch.equal(out, want.expand(32, 16)), e
        s.fill_(255)
        B.moe_w4_linear(x, w, s, out)
        assert bool(out.isnan().all())


@pytest.mark.parametrize("T", [1, 8, 20])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_whole_numbers_are_exact(T, G):
    g = torch.Generator(device="cuda").manual_seed(T + G)
    w, s, z, values = matrices((70,), 896, "int4", G, torch.bfloat16, True, g, whole=True)
    x = torch.randint(-4, 5, (T, 896), generator=g, device="cuda").to(torch.bfloat16)
    p = dict(x=x, weight=w, scales=s, zeros=z, topk_ids=None)
    assert torch.equal(run(p), (x.double() @ values.t()).to(torch.bfloat16))


def test_strides_types_of_ids_and_streams():
    p, values = problem(6, 512, 66, "bf16", "int4", 64, True, 9, 3, pad=0.2)
    a = check(p, values, "silu", layout="strided")
    q = dict(p, x=strided(p["x"], 8, 8), topk_ids=p["topk_ids"].long())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = run(q, "silu", stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    for _ in range(3):
        assert torch.equal(run(p, "silu"), b)


def test_scales_off_their_alignment():
    """Scales and zero points that start anywhere."""
    p, values = problem(3, 512, 40, "fp16", "int4", 32, True)
    s = torch.empty(p["scales"].numel() + 1, dtype=torch.float16, device="cuda")[1:].view_as(p["scales"])
    z = torch.empty(p["zeros"].numel() + 1, dtype=torch.uint8, device="cuda")[1:].view_as(p["zeros"])
    q = dict(p, scales=s.copy_(p["scales"]), zeros=z.copy_(p["zeros"]))
    assert torch.equal(check(q, values), run(p))


def test_ids_out_of_range():
    p, values = problem(4, 256, 32, "bf16", "e2m1", 32, False, 6, 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p["topk_ids"][1, 0] = -7
    check(p, values, status=status)
    assert int(status.item()) == 0
    p["topk_ids"][2, 1] = 6
    out = check(p, values, status=status)
    assert int(status.item()) == B.MOE_DEV_BAD_EXPERT and bool((out[5] == 0).all())


@pytest.mark.parametrize("experts", [False, True])
def test_a_broken_row_stays_alone(experts):
    p, values = problem(12, 512, 48, "bf16", "int4", 32, False, 4 if experts else 0, 1)
    clean = check(p, values)
    p["x"][5, 100] = float("inf")
    p["x"][7, 3] = float("nan")
    out = run(p)
    other = torch.tensor([t not in (5, 7) for t in range(12)], device="cuda")
    assert torch.equal(out[other], clean[other]) and not bool(out[5].isfinite().any())
    assert bool(out[7].isnan().all())


def test_a_broken_matrix_stays_with_its_rows():
    p, values = problem(10, 256, 40, "bf16", "int4", 64, False, 6, 2)
    clean = run(p)
    hit = (p["topk_ids"] == 2).reshape(-1)
    p["scales"][2] = float("nan")
    out = run(p)
    assert bool(hit.any()) and torch.equal(out[~hit], clean[~hit]) and bool(out[hit].isnan().all())


def test_rows_behind_the_last_and_empty_batches():
    p, _ = problem(9, 256, 40, "bf16")
    out = torch.full((9, 40), 7.0, device="cuda").to(torch.bfloat16)
    for n in (0, 5):
        B.moe_w4_linear(p["x"][:n], p["weight"], p["scales"], out[:n])
    assert bool((out[5:] == 7).all()) and bool((out[:5] != 7).any())
    ids = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    B.moe_w4_linear(p["x"][:0], p["weight"][None], p["scales"][None], out[:0], topk_ids=ids)


def test_offsets_beyond_32_bits():
    """The last of so many matrices that their bytes pass 2^31 (and their scales' bytes 2^30)."""
    E, N, K = 200, 4096, 5632
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(E, N, K // 32, dtype=torch.bfloat16, device="cuda")
    assert w.numel() > 2 ** 31
    w[-1], s[-1], _, values = matrices((N,), K, "int4", 32, torch.bfloat16, False, g)
    x = (torch.randn(2, K, generator=g, device="cuda") / 75).to(torch.bfloat16)
    ids = torch.tensor([[E - 1], [0]], dtype=torch.int32, device="cuda")
    out = run(dict(x=x, weight=w, scales=s, zeros=None, topk_ids=ids))
    ref, mag = values @ x[0].double(), values.abs() @ x[0].double().abs() * SUM
    assert_within(out[0], ref, rounded(ref, out.dtype, mag), "last matrix")
    assert bool((out[1] == 0).all())


def test_refusals():
    p, _ = problem(4, 256, 32, "bf16", "int4", 32, True)
    x, w, s, z = p["x"], p["weight"], p["scales"], p["zeros"]
    out = torch.empty(4, 32, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    good = dict(x=x, weight=w, scales=s, out=out, zeros=z)
    for kw in (dict(topk_ids=ids), dict(weight=w[None]), dict(weight=w[:, :-1]), dict(out=out[:, :31]),
               dict(scales=s.float()), dict(scales=s[:31]), dict(zeros=z[:, :7]), dict(x=x.cpu()),
               dict(scales=s[:, :7]), dict(out=out.half()), dict(activation=B.MOE_ACT_SILU),
               dict(weight=w[None], scales=s[None], zeros=z[None], topk_ids=ids.float())):
        with pytest.raises(ValueError):
            B.moe_w4_linear(**{**good, **kw})
    for kw in (dict(scales=s[:, ::4].contiguous().view(torch.uint8)[:, :2].contiguous(), zeros=None),
               dict(scales=torch.zeros(32, 8, dtype=torch.uint8, device="cuda")),
               dict(scales=torch.zeros(32, 1, dtype=torch.bfloat16, device="cuda"), zeros=None),
               dict(activation=5)):
        with pytest.raises((B.MoeError, ValueError)):
            B.moe_w4_linear(**{**good, **kw})
    long = torch.zeros(1025, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.MoeError):
        B.moe_w4_linear(long, w, s, torch.empty(1025, 32, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("T,K,N", [(5, 16384, 34), (7, 8192, 66), (16, 4096, 98), (12, 7168, 40), (20, 2304, 70),
                                   (9, 6400, 33), (2, 32768, 17)])
def test_rows_that_fill_shared_memory(T, K, N, fmt, G, zeros):
    """Batches whose rows leave room for fewer warps, or for some of the rows only."""
    p, values = problem(T, K, N, "bf16", fmt, G, zeros)
    check(p, values, "silu" if N % 2 == 0 else "none")


@pytest.mark.parametrize("fmt,G,zeros", [("int4", 128, True), ("e2m1", 32, False)])
@pytest.mark.parametrize("T,K,k,E", [(40, 7168, 2, 3), (12, 8192, 8, 9), (6, 16384, 2, 5)])
def test_experts_with_more_rows_than_there_is_room_for(T, K, k, E, fmt, G, zeros):
    p, values = problem(T, K, 48, "bf16", fmt, G, zeros, E, k, pad=0.05)
    check(p, values, "gelu_tanh")


@pytest.mark.parametrize("fmt", ["int4", "e2m1"])
@pytest.mark.parametrize("size", [2.0 ** -130, 2.0 ** -118, 2.0 ** -90, 2.0 ** -40, 2.0 ** 40, 2.0 ** 100, 2.0 ** 117])
def test_rows_of_any_size(fmt, size):
    """bf16 rows near the ends of their exponents: as exact as others."""
    g = torch.Generator(device="cuda").manual_seed(7)
    w, s, _, values = matrices((40,), 512, fmt, 32, torch.bfloat16, False, g, whole=True)
    x = torch.randint(-4, 5, (3, 512), generator=g, device="cuda").double()
    x[1] *= size
    p = dict(x=x.to(torch.bfloat16), weight=w, scales=s, zeros=None, topk_ids=None)
    assert torch.equal(p["x"].double(), x)
    assert torch.equal(run(p), (x @ values.t()).to(torch.float32).to(torch.bfloat16))


def test_a_huge_value_with_zero_weight_changes_nothing():
    g = torch.Generator(device="cuda").manual_seed(8)
    w, s, _, values = matrices((24,), 256, "int4", 64, torch.bfloat16, False, g)
    w[:, 50] = 0x88  # columns 100 and 101: code 8 is zero
    s = (s.float() * 64).to(torch.bfloat16)
    values = (torch.stack([w & 15, w >> 4], -1).view(24, 4, 64).double() - 8) * s.double()[..., None]
    x = torch.randn(2, 256, generator=g, device="cuda").to(torch.bfloat16)
    clean = run(dict(x=x, weight=w, scales=s, zeros=None, topk_ids=None))
    x[0, 100] = 3e38
    out = run(dict(x=x, weight=w, scales=s, zeros=None, topk_ids=None))
    # the others are below 2^-31 of the row's largest value: some 2^-40 of it is all that is left
    assert bool(out[0].isfinite().all()) and torch.equal(out[1], clean[1])


@pytest.mark.parametrize("fmt,G,zeros", [("int4", 32, False), ("int4", 128, True), ("e2m1", 32, False)])
@pytest.mark.parametrize("T,K,E,k", [(33, 29312, 4, 1), (8, 28672, 5, 8), (64, 32768, 3, 1), (64, 28672, 6, 8),
                                     (128, 25600, 3, 8), (1024, 32768, 2, 1)])
def test_long_rows_of_many_routes(T, K, E, k, fmt, G, zeros):
    """Rows beside which the longer blocks have no room, and some beside which they have.  Whole
    numbers, so that every sum is exact in fp32: far below 2^24 of their unit, 1/16 or 1/4."""
    g = torch.Generator(device="cuda").manual_seed(T + K + G)
    w, s, z, values = matrices((E, 18), K, fmt, G, torch.bfloat16, zeros, g, whole=True)
    x = torch.randint(-4, 5, (T, K), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    p = dict(x=x, weight=w, scales=s, zeros=z, topk_ids=ids)
    each = torch.einsum("tk,enk->ten", x.double(), values)
    ref = each.gather(1, ids.clamp_min(0).long()[:, :, None].expand(T, k, 18))
    ref = ref.masked_fill(ids[:, :, None] < 0, 0.0).view(T * k, 18)
    assert ref.abs().max() < 2 ** 17
    assert torch.equal(run(p), ref.to(torch.bfloat16))
    # gate and up are exact, so the activation and one rounding are all
    want, tol = bound("silu", ref * 2.0 ** -10, torch.zeros_like(ref), torch.bfloat16)
    assert_within(run(dict(p, x=x * 2.0 ** -10), "silu"), want, tol, "gated")


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_small_values_beside_a_large_one_keep_their_bits(dtype, fmt, G, zeros):
    """One value with all its significant bits, down to 2^-31 (fp16 2^-28) of the row's largest, whose
    weight is zero, in each of 32 columns behind it: the product alone is left, rounded once."""
    g = torch.Generator(device="cuda").manual_seed(G)
    w, s, z, _ = matrices((48,), 512, fmt, G, DTYPES[dtype], zeros, g)
    zero = (z[:, :1] & 15) if zeros else 8 if fmt == "int4" else 0
    w[:, :1] = (w[:, :1] & 0xF0) | zero  # column 0
    q = torch.stack([w & 15, w >> 4], -1).view(48, 512)[:, :33]
    if fmt == "e2m1":
        values = E2M1.cuda()[q.long()] * torch.exp2(s[:, 0:2].double() - 127).repeat_interleave(32, 1)[:, :33]
    else:
        z0 = (z & 15).double().repeat_interleave(G, 1)[:, :33] if zeros else 8.0
        values = (q.double() - z0) * s.double().repeat_interleave(G, 1)[:, :33]
    assert bool((values[:, 0] == 0).all())
    large, bits, below = (1.0, 8, 31) if dtype == "bf16" else (2.0 ** 15, 11, 28)
    smallest = torch.exp2(torch.arange(below - 10, below + 1, device="cuda", dtype=torch.float64).neg()) * large
    x = torch.zeros(11, 32, 512, dtype=torch.float64, device="cuda")
    x[:, :, 0] = large
    col = torch.arange(32, device="cuda")
    x[:, col, col + 1] = smallest[:, None] * (2 - 2.0 ** (1 - bits))
    x = x.view(11 * 32, 512)
    p = dict(x=x.to(DTYPES[dtype]), weight=w, scales=s, zeros=z, topk_ids=None)
    assert torch.equal(p["x"].double(), x)
    out = run(p)
    want = x[:, :33] @ values.t()  # one product and zeros
    assert torch.equal(out, want.float().to(out.dtype))


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_large_value_of_zero_weight(dtype, fmt, G, zeros):
    """Rows of which a value with zero weight is far the largest: the others are as exact as ever
    to 2^-31 (fp16 2^-28) of it, and below off by at most 2^-39 of it each."""
    p, values = problem(3, 512, 40, dtype, fmt, G, zeros)
    codes = torch.stack([p["weight"] & 15, p["weight"] >> 4], -1).view(40, 512)
    codes[:, 100] = (p["zeros"][:, 100 // G] & 15) if zeros else 8 if fmt == "int4" else 0
    p["weight"] = codes[:, 0::2] | codes[:, 1::2] << 4
    values[:, 100] = 0
    large = [2.0 ** 8, 2.0 ** 14, 2.0 ** 15] if dtype == "fp16" else [2.0 ** 12, 2.0 ** 60, 3e38]
    p["x"][:, 100] = torch.tensor(large, device="cuda").to(p["x"].dtype)
    ref, tol = expect(p, values)
    most = p["x"][:, 100:101].double()
    assert_within(run(p), ref, rounded(ref, p["x"].dtype, tol + 2.0 ** -39 * most * values.abs().sum(1)), "out")


@pytest.mark.parametrize("fmt", ["int4", "e2m1"])
def test_scales_and_rows_of_any_size_together(fmt):
    """bf16 rows and scales whose product is finite, however large either is; a group of zeros under
    the largest scale is zero.  One product a column: exact."""
    codes = torch.arange(16, device="cuda", dtype=torch.uint8)
    w = (codes[:, None] * 17).expand(16, 32).contiguous()  # two groups
    w[:, 16:] = 0x88 if fmt == "int4" else 0
    value = codes.double() - 8 if fmt == "int4" else E2M1.cuda()
    out = torch.empty(1, 16, dtype=torch.bfloat16, device="cuda")
    for ex in (-126, -100, -60, -20, 0, 20, 60, 100, 120):
        x = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
        x[0, 5], x[0, 40] = 2.0 ** ex, 2.0 ** ex
        for es in (-120, -100, -40, 0, 40, 100, 122, 124):
            if not -120 <= ex + es <= 124:
                continue
            if fmt == "int4":
                s = torch.full((16, 2), 2.0 ** es, device="cuda").to(torch.bfloat16)
                s[:, 1] = 2.0 ** 127
            else:
                s = torch.full((16, 2), es + 127, dtype=torch.uint8, device="cuda")
                s[:, 1] = 254
            B.moe_w4_linear(x, w, s, out)
            assert torch.equal(out[0], (value * 2.0 ** (ex + es)).float().to(torch.bfloat16)), (ex, es)
