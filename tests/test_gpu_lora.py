"""moe_lora_linear against its formula in 64 bits."""
import ctypes
import time

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


def problem(T, K, N, S, R, dtype, seed=0, order="mixed", layout="plain"):
    g = torch.Generator(device="cuda").manual_seed(seed + T + K + N)
    dt = DTYPES[dtype]

    def rnd(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)

    ids = torch.randint(-1, S, (T,), generator=g, device="cuda", dtype=torch.int32)
    if order == "sorted":
        ids = ids.sort().values
    elif order == "none":
        ids.fill_(-1)
    x = rnd(T, K)
    out = torch.full((T, N), float("nan"), dtype=dt, device="cuda")
    if layout != "plain":
        x = strided(x, 8)
        out = strided(out, 3, 1)
    a = rnd(S, R, K, std=K ** -0.5)
    b = rnd(S, N, R, std=max(R, 1) ** -0.5)
    return dict(x=x, weight=rnd(N, K, std=K ** -0.5), lora_a=a, lora_b=b, adapter_ids=ids,
                lora_scale=torch.rand(S, generator=g, device="cuda") * 2, out=out)


def run(p, status=None, stream=None):
    T, K = p["x"].shape
    S, R = p["lora_a"].shape[:2] if p["lora_a"] is not None else (0, 0)
    ws = torch.full((max(16, B.lora_workspace_size(T, K, p["weight"].shape[0], S, R)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    B.moe_lora_linear(workspace=ws, device_status=status, stream=stream, **p)
    return p["out"]


def expect(p):
    """(value, bound of the fp32 sums' error) in fp64, adapter by adapter."""
    x, w = p["x"].cpu().double(), p["weight"].cpu().double()
    ref, mag = x @ w.t(), x.abs() @ w.abs().t()
    if p["lora_a"] is not None:
        ids = p["adapter_ids"].cpu()
        for s in range(p["lora_a"].shape[0]):
            at = (ids == s).nonzero()[:, 0]
            if not len(at):
                continue
            a, b = p["lora_a"][s].cpu().double(), p["lora_b"][s].cpu().double()
            c = p["lora_scale"][s].item()
            ref[at] += c * ((x[at] @ a.t()) @ b.t())
            mag[at] += c * ((x[at].abs() @ a.abs().t()) @ b.abs().t())
    # fp32 accumulation, and s h as a 16-bit value and its 16-bit remainder (2^-17 for bf16)
    return ref, mag * 2.0 ** -16


def check(p, **kw):
    out = run(p, **kw)
    ref, extra = expect(p)
    assert_within(out, ref, rounded(ref, out.dtype, extra), "out")


# token counts around every tile, features and K that fill no tile, ranks with one and two parts
@pytest.mark.parametrize("T,K,N,S,R", [
    (1, 8, 1, 1, 8), (1, 7168, 512, 8, 16), (2, 72, 100, 3, 24), (15, 64, 128, 3, 8),
    (16, 1000, 257, 20, 16), (17, 512, 130, 5, 32), (33, 2048, 384, 40, 32),
    (64, 256, 129, 70, 40), (65, 320, 300, 4, 64), (128, 4096, 256, 9, 72),
    (129, 136, 64, 3, 128), (257, 264, 140, 6, 16), (300, 1032, 260, 30, 48),
    (512, 192, 264, 11, 64), (513, 72, 513, 5, 8), (700, 512, 512, 2, 128), (1500, 192, 72, 100, 8),
    (2100, 136, 300, 24, 48)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["mixed", "sorted"])
def test_against_the_formula(T, K, N, S, R, dtype, order):
    check(problem(T, K, N, S, R, dtype, order=order))


@pytest.mark.parametrize("T", [3, 40, 200])
def test_strides_and_no_adapter(T):
    check(problem(T, 520, 200, 4, 16, "bf16", layout="strided"))
    check(problem(T, 520, 200, 4, 16, "bf16", order="none"))
    p = problem(T, 520, 200, 4, 16, "fp16")
    p.update(lora_a=None, lora_b=None, adapter_ids=None, lora_scale=None)
    check(p)


def test_every_token_its_own_adapter():
    p = problem(64, 512, 256, 64, 16, "bf16")
    p["adapter_ids"] = torch.randperm(64, device="cuda").to(torch.int32)
    check(p)
    p = problem(300, 128, 128, 300, 8, "bf16")
    p["adapter_ids"] = torch.arange(300, device="cuda", dtype=torch.int32)
    check(p)


@pytest.mark.parametrize("T", [9, 100, 900])
def test_a_broken_adapter_stays_with_its_tokens(T):
    p = problem(T, 256, 200, 5, 40, "bf16")
    q = dict(p, adapter_ids=torch.where(p["adapter_ids"] == 3, -1, p["adapter_ids"]))
    p["lora_a"][3, 1] = float("inf")
    p["lora_b"][3] = float("nan")
    out = run(p)
    others = (p["adapter_ids"] != 3).cpu()
    ref, extra = expect(q)
    assert_within(out[others], ref[others], rounded(ref, out.dtype, extra)[others], "others")
    assert bool(torch.isnan(out.cpu()[~others]).all())


@pytest.mark.parametrize("T", [30, 120, 800])
def test_ids_out_of_range_and_nan_in_unused_adapters(T):
    p = problem(T, 256, 200, 5, 16, "bf16")
    p["adapter_ids"][3] = 5
    p["adapter_ids"][4] = 2 ** 31 - 1
    p["adapter_ids"][p["adapter_ids"] == 2] = -7
    p["lora_a"][2] = float("nan")
    p["lora_b"][2] = float("nan")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(p, status=st)
    q = dict(p, adapter_ids=torch.where(p["adapter_ids"] >= 5, -1, p["adapter_ids"]))
    ref, extra = expect(q)
    assert_within(out, ref, rounded(ref, out.dtype, extra), "out")
    assert int(st.item()) == B.MOE_DEV_BAD_ADAPTER


def test_stream_and_same_bits_twice():
    p = problem(50, 1024, 512, 12, 32, "bf16")
    first = run(p).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p["out"].zero_()
    torch.cuda.synchronize()
    run(p, stream=s)
    s.synchronize()
    assert torch.equal(first, p["out"])


def test_back_to_back_calls_share_a_workspace():
    ps = [problem(T, 512, 384, 6, 16, "bf16", seed=T) for T in (40, 33, 64, 7)]
    ws = torch.empty(max(B.lora_workspace_size(p["x"].shape[0], 512, 384, 6, 16) for p in ps),
                     dtype=torch.uint8, device="cuda")
    for _ in range(5):
        for p in ps:
            B.moe_lora_linear(workspace=ws, **p)
    torch.cuda.synchronize()
    for p in ps:
        ref, extra = expect(p)
        assert_within(p["out"], ref, rounded(ref, p["out"].dtype, extra), "out")


def test_refusals():
    p = problem(4, 64, 32, 2, 8, "bf16")
    with pytest.raises(ValueError):
        run(dict(p, out=p["out"].float()))
    with pytest.raises(ValueError):
        run(dict(p, weight=p["weight"].t().contiguous().t()))
    with pytest.raises(B.MoeError) as e:
        B.moe_lora_linear(workspace=None, **p)
    assert e.value.status == 5
    q = {k: (v.float() if v.is_floating_point() else v) for k, v in p.items()}
    with pytest.raises(B.MoeError) as e:
        run(q)
    assert e.value.status == 3
    with pytest.raises(B.MoeError) as e:
        run(problem(4, 60, 32, 2, 8, "bf16"))
    assert e.value.status == 4


def test_wait_timeout_sets_status_and_context_survives():
    """The test build's CTA 0 issues no slab after its first, so the MMA warp's wait on it runs
    out after 5 ms; the CTA drains what it issued and returns, alone and inside a cluster."""
    from moe_expert_layer_prepare_gb300 import build
    test_lib = B.configure(ctypes.CDLL(build.build_test_variant("timeout")))
    regular = B.load()
    # eight CTAs share a tile's K; one each; a pair of CTAs a tile
    for T, N in ((8, 256), (300, 20000), (600, 512)):
        p = problem(T, 2048, N, 3, 16, "bf16")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        B._lib = test_lib
        try:
            t0 = time.perf_counter()
            run(p, status=st)
            torch.cuda.synchronize()
            assert time.perf_counter() - t0 < 5.0
        finally:
            B._lib = regular
        assert int(st.item()) & B.MOE_DEV_TIMEOUT
        check(p)


@pytest.mark.parametrize("T", [130, 200, 400, 512])
def test_a_broken_adapter_and_bad_ids_in_batches_of_two_to_four_tiles(T):
    # tokens as they come through the tcgen05 shrink, then tiles of 64 or 128 tokens
    for R in (16, 72):
        p = problem(T, 264, 200, 6, R, "bf16")
        p["adapter_ids"][3], p["adapter_ids"][T - 1] = 6, 2 ** 31 - 1
        p["adapter_ids"][p["adapter_ids"] == 2] = -7
        p["lora_a"][2] = float("nan")
        p["lora_b"][2] = float("nan")
        good = torch.where((p["adapter_ids"] == 3) | (p["adapter_ids"] >= 6), -1, p["adapter_ids"])
        q = dict(p, adapter_ids=good)
        p["lora_a"][3, 1] = float("inf")
        p["lora_b"][3] = float("nan")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = run(p, status=st)
        others = (p["adapter_ids"] != 3).cpu()
        ref, extra = expect(q)
        assert_within(out[others], ref[others], rounded(ref, out.dtype, extra)[others], "others")
        assert bool(torch.isnan(out.cpu()[~others]).all())
        assert int(st.item()) == B.MOE_DEV_BAD_ADAPTER


def test_batches_of_every_path_share_a_workspace_back_to_back():
    # order, copied rows, pieces of tiles and sums of one call right behind those of another
    sizes = (700, 300, 2100, 40, 1500, 513, 512, 1, 900)
    ps = [problem(T, 520, 776, 9, 40, "bf16", seed=T) for T in sizes]
    need = max(B.lora_workspace_size(T, 520, 776, 9, 40) for T in sizes)
    assert need == B.lora_workspace_size(max(sizes), 520, 776, 9, 40)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(4):
        for p in ps:
            p["out"].fill_(float("nan"))
        for p in ps:
            B.moe_lora_linear(workspace=ws, **p)
    torch.cuda.synchronize()
    for p in ps:
        ref, extra = expect(p)
        assert_within(p["out"], ref, rounded(ref, p["out"].dtype, extra), "out")


@pytest.mark.parametrize("T,dtype,order", [(600, "bf16", "mixed"), (1024, "fp16", "mixed"),
                                           (2000, "bf16", "mixed"), (2000, "bf16", "sorted")])
def test_mixed_batches_of_real_width(T, dtype, order):
    p = problem(T, 2048, 7168, 16, 64, dtype, order=order)
    check(p)
    first = p["out"].clone()
    for _ in range(10):  # the same bits each time
        p["out"].fill_(0.0)
        assert torch.equal(run(p), first)


def test_norm_router_and_projection_behind_one_another():
    # the chain of a block without a synchronisation, against the same calls one at a time
    T, K, N, E = 1500, 2048, 1024, 64
    p = problem(T, K, N, 8, 16, "bf16")
    g = torch.Generator(device="cuda").manual_seed(1)
    x, z = (torch.randn(T, K, generator=g, device="cuda").bfloat16() for _ in range(2))
    ones = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    router = (torch.randn(E, K, generator=g, device="cuda") * K ** -0.5).bfloat16()
    ws = torch.empty(B.lora_workspace_size(T, K, N, 8, 16), dtype=torch.uint8, device="cuda")

    def chain(pause):
        bufs = dict(xo=torch.zeros_like(x), h=torch.zeros_like(x),
                    logits=torch.zeros(T, E, dtype=torch.bfloat16, device="cuda"),
                    ids=torch.zeros(T, 4, dtype=torch.int32, device="cuda"),
                    w=torch.zeros(T, 4, device="cuda"), out=torch.zeros_like(p["out"]))
        torch.cuda.synchronize()
        steps = [
            lambda: B.moe_block_norm(x, z=z, post_weight=ones, pre_weight=ones, x_out=bufs["xo"],
                                     y=bufs["h"]),
            lambda: B.moe_lora_linear(bufs["h"], router, None, None, None, None, bufs["logits"],
                                      None),
            lambda: B.moe_route(bufs["logits"], bufs["ids"], bufs["w"]),
            lambda: B.moe_lora_linear(bufs["h"], p["weight"], p["lora_a"], p["lora_b"],
                                      p["adapter_ids"], p["lora_scale"], bufs["out"], ws)]
        for _ in range(3):
            for step in steps:
                step()
                if pause:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return bufs

    a, b = chain(True), chain(False)
    for name in a:
        assert torch.equal(a[name], b[name]), name


@pytest.mark.parametrize("T", [1, 3, 16, 40, 100, 200, 512, 700, 1500])
@pytest.mark.parametrize("R", [8, 24, 72, 128])
@pytest.mark.parametrize("how", ["large", "small", "all"])
def test_fp16_products_beyond_its_range(T, R, how):
    # s h about 2^17 with rows of B about 2^-10, about 2^-20 with B about 2^10, and both beside
    # ordinary ones and zeros: the sums are ordinary numbers, their middle factor is not
    p = problem(T, 512, 264, 5, R, "fp16")
    up = torch.ones(5, device="cuda")
    if how != "small":
        up[[0, 3]] = 2.0 ** 17
    if how != "large":
        up[[1, 4]] = 2.0 ** -20
    if how == "large":
        up.fill_(2.0 ** 17)
    p["lora_scale"] = p["lora_scale"] * up
    # B back by 2^-10 or 2^10 (its own range); what is left is up to 2^7 or 2^-10
    back = torch.where(up > 1, 2.0 ** -10, torch.where(up < 1, 2.0 ** 10, 1.0))
    p["lora_b"] = (p["lora_b"].float() * back[:, None, None]).half()
    if how == "small":
        p["weight"] *= 2.0 ** -9  # so that the adapters' part is the larger one
    if T > 2:
        p["x"][T // 2] = 0.0
    out = run(p)
    ref, extra = expect(p)
    assert_within(out, ref, rounded(ref, out.dtype, extra), "out")


@pytest.mark.parametrize("T", [5, 200, 1100])
def test_fp16_rows_with_pieces_of_every_size(T):
    # ranks 0..7 overflow, 8..15 vanish, 16..23 are ordinary, 24..31 zero, within each row
    p = problem(T, 512, 300, 3, 32, "fp16")
    size = torch.tensor([2.0 ** 13, 2.0 ** -16, 1.0, 0.0], device="cuda").repeat_interleave(8)
    p["lora_a"] = (p["lora_a"].float() * size[:, None]).half()
    p["lora_b"] = (p["lora_b"].float() / size.clamp_min(2.0 ** -16) / 16).half()
    p["lora_scale"] = p["lora_scale"] * 16
    out = run(p)
    ref, extra = expect(p)
    assert_within(out, ref, rounded(ref, out.dtype, extra), "out")


@pytest.mark.parametrize("T", [2, 70, 300, 1000])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_an_infinite_sum_stays_one(T, dtype):
    # h infinite: out is that infinity with the sign of B's value, not NaN
    p = problem(T, 256, 200, 3, 24, dtype)
    p["adapter_ids"][0] = 1
    p["x"][:, 7] = 0.5
    p["lora_a"][1, 2, 7] = float("inf")
    p["lora_b"][1, :, 2] = torch.where(p["lora_b"][1, :, 2] > 0, 1.0, -1.0).to(p["x"].dtype)
    out = run(p)
    mine = (p["adapter_ids"] == 1).cpu()
    want = torch.where(p["lora_b"][1, :, 2] > 0, float("inf"), -float("inf")).cpu()
    assert bool((out.cpu()[mine].float() == want).all())
    q = dict(p, adapter_ids=torch.where(p["adapter_ids"] == 1, -1, p["adapter_ids"]))
    ref, extra = expect(q)
    assert_within(out[~mine.cuda()], ref[~mine], rounded(ref, out.dtype, extra)[~mine], "others")


@pytest.mark.parametrize("T,K,N,R", [(600, 64, 2000, 8), (2100, 128, 1100, 64), (1500, 2048, 512, 128)])
def test_fp16_wide_and_ordinary_batches_in_turn(T, K, N, R):
    # one workspace, calls right behind one another: what one batch found wide is not the next one's
    ps = []
    for seed, up in ((1, 1.0), (2, 2.0 ** 17), (3, 1.0), (4, 2.0 ** -18)):
        p = problem(T, K, N, 7, R, "fp16", seed=seed)
        p["lora_scale"][::2] *= up
        p["lora_b"][::2] = (p["lora_b"][::2].float() / up ** 0.5).half()
        ps.append(p)
    ws = torch.empty(B.lora_workspace_size(T, K, N, 7, R), dtype=torch.uint8, device="cuda")
    first = []
    for p in ps:
        ws.fill_(0xFF)
        B.moe_lora_linear(workspace=ws, **p)
        ref, extra = expect(p)
        assert_within(p["out"], ref, rounded(ref, p["out"].dtype, extra), "out")
        first.append(p["out"].clone())
    differs = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(60):
        for p in ps:
            B.moe_lora_linear(workspace=ws, **p)
        for p, f in zip(ps, first):
            differs += (p["out"] != f).sum()
            p["out"].zero_()
    assert differs.item() == 0
