"""moe_sort_routes, moe_permute, moe_unpermute and their gradients in 64 bits."""
import numpy as np
import pytest
import torch

from moe_expert_layer_prepare_gb300 import binding as B
from tests._block_util import DTYPES, assert_within, rounded, strided
from tests._util import need_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    need_cuda()
    from moe_expert_layer_prepare_gb300 import build
    build.build()
    B.load()


def sort_routes(ids, E, status=None):
    T, k = ids.shape
    off = torch.full((E + 1,), 77, dtype=torch.int32, device="cuda")
    rr = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    ro = torch.full((T * k,), 77, dtype=torch.int32, device="cuda")
    ws = torch.full((max(1, B.sort_workspace_size(T, k, E)),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    B.moe_sort_routes(ids, off, rr, ro, ws, device_status=status)
    return off, rr, ro


def plan(ids, E):
    """The definition in numpy: offsets, route_row, row_route."""
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(ok, flat, E), kind="stable")
    n = int(ok.sum())
    rr = np.full(flat.size, -1, np.int32)
    rr[order[:n]] = np.arange(n)
    ro = np.full(flat.size, -1, np.int32)
    ro[:n] = order[:n]
    off = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))]).astype(np.int32)
    return off, rr.reshape(ids.shape), ro


# 4096 routes are the most of one block, 131,072 the most of 128 blocks of 1024
@pytest.mark.parametrize("T,k,E", [(0, 2, 8), (1, 1, 1), (1, 8, 256), (7, 2, 8), (33, 6, 1024),
                                   (512, 8, 3), (4096, 1, 16), (4097, 1, 256), (2051, 6, 32),
                                   (8192, 8, 256), (16385, 8, 1000), (70001, 4, 7)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(T, k, E, dtype):
    rng = np.random.default_rng(T + E)
    ids = rng.integers(-1, E, size=(T, k))
    ids[: T // 3] = rng.integers(0, max(1, E // 8), size=(T // 3, k))  # a crowded third
    off, rr, ro = sort_routes(torch.from_numpy(ids).to("cuda", dtype), E)
    for got, want in zip((off, rr, ro), plan(ids, E)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_sort_more_routes_of_an_expert_than_16_bits_count():
    T = 9_000_001
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    ids[5::1000] = 1
    off, rr, ro = sort_routes(ids, 2)
    order = torch.sort(ids[:, 0], stable=True).indices.int()
    n = int((ids == 0).sum())
    assert off.tolist() == [0, n, T]
    assert torch.equal(ro, order)
    assert torch.equal(rr[:, 0][order.long()], torch.arange(T, dtype=torch.int32, device="cuda"))


def test_sort_ids_out_of_range():
    ids = np.array([[0, 9], [3, -5], [2 ** 31 - 1, 1]])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    off, rr, ro = sort_routes(torch.from_numpy(ids).to("cuda", torch.int32), 4, st)
    for got, want in zip((off, rr, ro), plan(ids, 4)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert int(st.item()) == B.MOE_DEV_BAD_EXPERT
    big = torch.full((5000, 1), 2 ** 40, dtype=torch.int64, device="cuda")
    st.zero_()
    off, rr, _ = sort_routes(big, 4, st)
    assert int(st.item()) == B.MOE_DEV_BAD_EXPERT and not off.any() and bool((rr == -1).all())


def make(T, k, E, K, dtype, seed, layout):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    ids = rng.integers(-1, E, size=(T, k))
    if T > 2:
        ids[1] = -1  # a token that no expert takes
    off, rr, ro = sort_routes(torch.from_numpy(ids).to("cuda", torch.int32), E)

    def rnd(n):
        t = torch.randn(n, K, generator=g, device="cuda").to(dtype)
        return t if layout == "plain" else strided(t, 8 if layout == "padded" else 3,
                                                   0 if layout == "padded" else 1)

    w = torch.randn(T, k, generator=g, device="cuda")
    return ids, off, rr, ro, rnd, w


SHAPES = [(1, 1, 1, 1), (1, 8, 16, 7168), (5, 2, 4, 8), (33, 8, 8, 520), (40, 9, 16, 1031),
          (300, 2, 8, 4096), (19, 32, 64, 264), (64, 3, 4, 129)]


@pytest.mark.parametrize("T,k,E,K", SHAPES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("layout", ["plain", "padded", "odd"])
def test_rows_there_and_back(T, k, E, K, dtype, layout):
    dt = DTYPES[dtype]
    ids, off, rr, ro, rnd, w = make(T, k, E, K, dt, T + K, layout)
    n = int(off[-1].item())
    R = T * k + 2  # two rows more than there are routes
    x, eo, up, dr = rnd(T), rnd(R), rnd(T), rnd(R)
    eo[n:] = float("nan")  # rows that no route names are not read
    dr[n:] = float("nan")
    rows, d_eo = rnd(R), rnd(R)
    out, dx = rnd(T), rnd(T)
    dw = torch.full((T, k), 77.0, device="cuda")
    B.moe_permute(x, rr, off, rows)
    B.moe_unpermute(eo, rr, w, out)
    B.moe_unpermute_backward(up, eo, rr, w, off, d_eo, dw)
    B.moe_permute_backward(dr, rr, dx)

    token = (ro[:n] // k).long().cpu()
    assert torch.equal(rows[:n].cpu(), x.cpu()[token]) and not rows[n:].any()
    at = rr.cpu().long()
    placed = (at >= 0)[:, :, None]
    wf = w.cpu().double()
    eps = 2.0 ** -24 * (k + 1)

    def gather(t):
        v = t.cpu().double()[at.clamp_min(0)]
        return torch.where(placed, v, torch.zeros_like(v))

    terms = gather(eo) * wf[:, :, None]
    assert_within(out, terms.sum(1), rounded(terms.sum(1), dt, terms.abs().sum(1) * eps), "out")
    terms = gather(dr)
    assert_within(dx, terms.sum(1), rounded(terms.sum(1), dt, terms.abs().sum(1) * eps), "d_x")
    u = up.cpu().double()
    terms = gather(eo) * u[:, None, :]
    assert_within(dw, terms.sum(2), terms.abs().sum(2) * 2.0 ** -24 * (K / 32 + 16) + 1e-30, "d_w")
    want = u[token] * wf.reshape(-1)[ro[:n].long().cpu()][:, None]
    assert_within(d_eo[:n], want, rounded(want, dt, want.abs() * 2.0 ** -24), "d_rows")
    assert not d_eo[n:].any()


def test_rows_beyond_the_buffer_are_left_out():
    ids, off, rr, ro, rnd, w = make(50, 4, 8, 64, torch.float32, 3, "plain")
    n = int(off[-1].item())
    short = n - 20
    guard = torch.full((n, 64), 5.0, device="cuda")
    x = rnd(50)
    B.moe_permute(x, rr, off, guard[:short])
    assert torch.equal(guard[:short].cpu(), x.cpu()[(ro[:short] // 4).long().cpu()])
    assert bool((guard[short:] == 5.0).all())
    out, out2 = rnd(50), rnd(50)
    B.moe_unpermute(guard[:short], rr, w, out)
    cut = torch.where(rr < short, rr, -1)
    B.moe_unpermute(guard, cut, w, out2)
    assert torch.equal(out, out2)
    dw = torch.full((50, 4), 77.0, device="cuda")
    dg = torch.full((n, 64), 5.0, device="cuda")
    B.moe_unpermute_backward(x, guard[:short], rr, w, off, dg[:short], dw)
    assert bool((dw[cut < 0] == 0).all()) and bool((dg[short:] == 5.0).all())


def test_shared_weights_with_the_bf16_reduce():
    # the contiguous form of moe_topk_reduce is the same sum
    ids, off, rr, ro, rnd, w = make(90, 8, 16, 2048, torch.bfloat16, 9, "plain")
    eo = rnd(90 * 8)
    a, b = rnd(90), rnd(90)
    B.moe_unpermute(eo, rr, w, a)
    B.moe_topk_reduce(eo, None, rr, w, b)
    assert torch.equal(a, b)


def test_gradients_against_differences():
    # the forward is linear in the rows and in the weights, so differences are exact up to rounding
    ids, off, rr, ro, rnd, w = make(12, 3, 4, 40, torch.float32, 11, "plain")
    eo, up, v = rnd(36), rnd(12), rnd(36)
    vw = torch.randn(12, 3, generator=torch.Generator().manual_seed(1)).cuda()
    dw, d_eo, out = torch.empty(12, 3, device="cuda"), rnd(36), rnd(12)
    B.moe_unpermute_backward(up, eo, rr, w, off, d_eo, dw)

    def loss(rows, weights):
        B.moe_unpermute(rows, rr, weights, out)
        return (out.double() * up.double()).sum(1).cpu()

    zero = torch.zeros(1)
    num = loss(v, w)
    ana = torch.zeros(12, dtype=torch.float64)
    n = int(off[-1].item())
    ana.index_add_(0, (ro[:n] // 3).long().cpu(), (d_eo.double() * v.double()).sum(1).cpu()[:n])
    assert_within(ana, num, zero + 3 * 40 * 16 * 2.0 ** -22, "rows")
    num = loss(eo, w + vw) - loss(eo, w - vw)
    ana = 2 * (dw.double() * vw.double()).sum(1).cpu()
    assert_within(ana, num, zero + 3 * 40 * 32 * 2.0 ** -22, "weights")


def test_stream_and_refusals():
    ids, off, rr, ro, rnd, w = make(20, 2, 4, 64, torch.bfloat16, 2, "plain")
    x, rows, again = rnd(20), rnd(40), rnd(40)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.moe_permute(x, rr, off, rows, stream=s)
    s.synchronize()
    B.moe_permute(x, rr, off, again)
    assert torch.equal(rows, again)
    with pytest.raises(ValueError):
        B.moe_permute(x.float(), rr, off, rows)
    with pytest.raises(ValueError):
        B.moe_permute(x, rr.long(), off, rows)
    with pytest.raises(ValueError):
        B.moe_unpermute(rows, rr, w.half(), x)
    with pytest.raises(ValueError):
        B.moe_unpermute(rows.double(), rr, w, x.double())
    with pytest.raises(B.MoeError) as e:
        B.moe_sort_routes(torch.zeros(5000, 1, dtype=torch.int32, device="cuda"),
                          torch.empty(5, dtype=torch.int32, device="cuda"),
                          torch.empty(5000, 1, dtype=torch.int32, device="cuda"),
                          torch.empty(5000, dtype=torch.int32, device="cuda"))
    assert e.value.status == 5  # above one block's routes a workspace is needed


def test_tokens_without_routes():
    # top_k 0: nothing of x is read (the address may be NULL), every row is cleared
    T, K, R = 70, 520, 9
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    rr = torch.empty(T, 0, dtype=torch.int32, device="cuda")
    x = torch.full((T, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    for null in (False, True):
        rows = torch.full((R, K), 7.0, dtype=torch.bfloat16, device="cuda")
        if null:
            st = B.load().moe_permute(B.PermuteArgs.pack(
                T, K, 0, 4, R, B.MOE_DTYPE_BF16, 0, K, 0, off.data_ptr(), rows.data_ptr(), K),
                torch.cuda.current_stream().cuda_stream)
            assert st == B.MOE_OK
        else:
            B.moe_permute(x, rr, off, rows)
        assert not rows.any()
    out = torch.full((T, K), 7.0, dtype=torch.bfloat16, device="cuda")
    B.moe_unpermute(rows, rr, None, out)
    assert not out.any()


def test_no_tokens():
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    rr = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    w, e = torch.empty(0, 2, device="cuda"), torch.empty(0, 64, device="cuda")
    for R in (0, 3):
        rows, d_rows = torch.full((R, 64), 7.0, device="cuda"), torch.full((R, 64), 7.0, device="cuda")
        B.moe_permute(e, rr, off, rows)
        B.moe_unpermute(rows, rr, w, e)
        B.moe_unpermute_backward(e, rows, rr, w, off, d_rows, w)
        B.moe_permute_backward(rows, rr, e)
        assert not rows.any() and not d_rows.any()


# 2048 routes are the most that one block sorts, 131,072 the most of blocks of 1024 routes each
@pytest.mark.parametrize("R", [2047, 2048, 2049, 3072, 131071, 131073])
@pytest.mark.parametrize("E", [1, 256, 1024])
def test_sort_at_the_steps_of_the_split(R, E):
    rng = np.random.default_rng(R + E)
    ids = rng.integers(-1, E, size=(R, 1))
    off, rr, ro = sort_routes(torch.from_numpy(ids).to("cuda", torch.int32), E)
    for got, want in zip((off, rr, ro), plan(ids, E)):
        assert np.array_equal(got.cpu().numpy(), want)
