"""moe_route and moe_route_backward against their formulas in 64 bits."""
import numpy as np
import pytest
import torch

from moe_expert_layer_prepare_gb300 import binding as B
from tests._block_util import DTYPES, HALF_ULP, assert_within, rounded
from tests._util import need_cuda

pytestmark = pytest.mark.gpu
SCORING = {"softmax": B.MOE_SCORE_SOFTMAX, "sigmoid": B.MOE_SCORE_SIGMOID}


@pytest.fixture(scope="module", autouse=True)
def cuda():
    need_cuda()
    from moe_expert_layer_prepare_gb300 import build
    build.build()
    B.load()


def select(l, bias, scoring, k, groups, top_groups):
    """ids of the definition, row by row (l: fp32 numpy [T, E])."""
    T, E = l.shape
    key = l.astype(np.float32)
    if bias is not None:
        if scoring == "sigmoid":
            with np.errstate(over="ignore"):
                key = (np.float32(1) / (np.float32(1) + np.exp(-key))).astype(np.float32)
        key = (key + bias).astype(np.float32)
    ids = np.full((T, k), -1, np.int64)
    size = E // groups
    for t in range(T):
        ok = [e for e in range(E) if key[t, e] > -np.inf]
        if groups > 1:
            value = {}
            for g in range(groups):
                mine = sorted((key[t, e] for e in ok if e // size == g), reverse=True)
                if mine:
                    second = mine[1] if len(mine) > 1 else np.float32(0)
                    value[g] = mine[0] if bias is None else np.float32(mine[0] + second)
            best = sorted(value, key=lambda g: (-value[g], g))[:top_groups]
            ok = [e for e in ok if e // size in best]
        taken = sorted(ok, key=lambda e: (-key[t, e], e))[:k]
        ids[t, :len(taken)] = taken
    return ids


def weights64(l, ids, scoring, renorm, scale):
    """Weights in fp64 of logits l (fp64 tensor, may require grad) with the selection given."""
    taken = ids >= 0
    at = l.gather(1, ids.clamp_min(0))
    if scoring == "sigmoid":
        s = torch.where(taken, torch.sigmoid(at), torch.zeros_like(at))
        w = s / (s.sum(dim=1, keepdim=True) + 1e-20) if renorm else s
    else:
        # exponentials relative to the largest logit in the sum; rows that take nothing give 0
        if renorm:
            pool, mine = at, taken
        else:
            pool, mine = l, l > -float("inf")
        some = taken.any(dim=1, keepdim=True)
        mine = mine & some
        ninf = torch.full_like(pool, -float("inf"))
        m = torch.where(mine, pool, ninf).amax(dim=1, keepdim=True).detach()
        m = torch.where(some, m, torch.zeros_like(m))

        def ex(v, use):
            return torch.where(use, torch.exp(torch.where(use, v - m, torch.zeros_like(v))),
                               torch.zeros_like(v))
        total = ex(pool, mine).sum(dim=1, keepdim=True)
        w = ex(at, taken) / torch.where(some, total, torch.ones_like(total))
    return w * scale


def route(l, k, scoring="softmax", renorm=True, scale=1.0, bias=None, pad=None, groups=1,
          top_groups=1, ids_dtype=torch.int32):
    T = l.shape[0]
    ids = torch.full((T, k), 77, dtype=ids_dtype, device="cuda")
    w = torch.full((T, k), 77.0, device="cuda")
    B.moe_route(l, ids, w, bias=bias, is_padding=pad, scoring=SCORING[scoring],
                renormalize=renorm, scale=scale, num_groups=groups, top_groups=top_groups)
    return ids, w


CASES = [(1, 1, 1), (3, 5, 5), (7, 8, 2), (9, 32, 32), (65, 33, 4), (40, 100, 8), (130, 256, 8),
         (17, 300, 7), (5, 1000, 32)]


@pytest.mark.parametrize("T,E,k", CASES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("scoring,renorm", [("softmax", True), ("softmax", False),
                                            ("sigmoid", True), ("sigmoid", False)])
def test_forward_and_gradient(T, E, k, dtype, scoring, renorm):
    g = torch.Generator().manual_seed(T * 1000 + E)
    l = (torch.randn(T, E, generator=g) * 2).to(DTYPES[dtype])  # 16-bit logits tie often
    pad = (torch.rand(T, generator=g) < 0.2).to(torch.uint8)
    ids, w = route(l.cuda(), k, scoring, renorm, 1.7, pad=pad.cuda())
    want = select(l.float().numpy(), None, scoring, k, 1, 1)
    want[pad.numpy() != 0] = -1
    assert np.array_equal(ids.cpu().numpy(), want)
    l64 = l.double().requires_grad_(True)
    wid = torch.from_numpy(want)
    ref = weights64(l64, wid, scoring, renorm, 1.7)
    # exp and the quotient: a few units in the last place of fp32, the sum's E of them
    assert_within(w, ref.detach(), ref.detach().abs() * (E + 16) * 2.0 ** -24 + 1e-30, "weights")

    dw = torch.randn(T, k, generator=g)
    dl = torch.full((T, E), 77.0, dtype=l.dtype, device="cuda")
    B.moe_route_backward(l.cuda(), ids, dw.cuda(), dl, scoring=SCORING[scoring],
                         renormalize=renorm, scale=1.7)
    (ref * dw.double()).sum().backward()
    mag = 1.7 * dw.abs().double().sum(dim=1, keepdim=True).expand(T, E)
    assert_within(dl, l64.grad, rounded(l64.grad, l.dtype, mag * (E + 32) * 2.0 ** -24),
                  "d_logits")
    assert bool((dl[pad.cuda() != 0] == 0).all())


@pytest.mark.parametrize("E,groups,top_groups,k", [(256, 8, 4, 8), (96, 4, 1, 5), (60, 3, 2, 6),
                                                   (64, 32, 16, 8), (40, 5, 5, 8), (1024, 8, 3, 32)])
@pytest.mark.parametrize("scoring,with_bias", [("sigmoid", True), ("softmax", True),
                                               ("softmax", False), ("sigmoid", False)])
def test_groups_and_bias(E, groups, top_groups, k, scoring, with_bias):
    T = 50
    g = torch.Generator().manual_seed(E + groups)
    l = torch.randn(T, E, generator=g)
    # a coarse grid: keys tie often, and no two differ by less than exp's rounding
    l = torch.round(l * 4) / 4
    bias = torch.round(torch.randn(E, generator=g) * 4) / 64 if with_bias else None
    ids, w = route(l.cuda(), k, scoring, True, 2.5, groups=groups, top_groups=top_groups,
                   bias=None if bias is None else bias.cuda(), ids_dtype=torch.int64)
    got = ids.cpu().numpy()
    if scoring == "sigmoid" and with_bias:
        # the key's exp is the GPU's: take the keys from the same elementary operations there
        key = (1.0 / (1.0 + torch.exp(-l.cuda())) + bias.cuda()).cpu().numpy()
        want = select(key, None, "softmax", k, 1, 1) if groups == 1 else \
            select(key, np.zeros(E, np.float32), "softmax", k, groups, top_groups)
    else:
        want = select(l.numpy(), None if bias is None else bias.numpy(), scoring, k, groups,
                      top_groups)
    assert np.array_equal(got, want)
    ref = weights64(l.double(), torch.from_numpy(want), scoring, True, 2.5)
    assert_within(w, ref, ref.abs() * (E + 16) * 2.0 ** -24 + 1e-30, "weights")


@pytest.mark.parametrize("scoring,renorm", [("softmax", True), ("softmax", False),
                                            ("sigmoid", True), ("sigmoid", False)])
def test_masked_and_extreme_logits(scoring, renorm):
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(torch.float32).min
    rows = [[-inf] * 8, [nan] * 8, [-inf, 1.0, -inf, nan, 0.5, -inf, nan, -inf],
            [low] * 8, [low, 0.0, low, 1.0, low, low, low, low], [0.0, -0.0, 0.0, -0.0] * 2,
            [inf, 0.0, inf, 1.0, 2.0, -inf, nan, 3.0], [3e38, 3e38, 1.0, 0.0, 0.0, 0.0, 0.0, 0.0],
            [-200.0, -300.0, -250.0, low, low, low, low, low]]
    l = torch.tensor(rows)
    ids, w = route(l.cuda(), 4, scoring, renorm)
    want = select(l.numpy(), None, scoring, 4, 1, 1)
    assert np.array_equal(ids.cpu().numpy(), want)
    w = w.cpu()
    assert bool(torch.isfinite(w).all())
    assert bool((w[torch.from_numpy(want) < 0] == 0).all())
    finite = [r for r in range(len(rows)) if r != 6]
    ref = weights64(l[finite].double(), torch.from_numpy(want[finite]), scoring, renorm, 1.0)
    assert_within(w[finite], ref, ref.abs() * 1e-5 + 1e-30, "weights")
    if scoring == "softmax":  # infinite logits share the weight
        assert w[6].tolist() == [0.5, 0.5, 0.0, 0.0]
    dw = torch.ones(len(rows), 4)
    dl = torch.full((len(rows), 8), 77.0, device="cuda")
    B.moe_route_backward(l.cuda(), ids, dw.cuda(), dl, scoring=SCORING[scoring],
                         renormalize=renorm)
    assert bool(torch.isfinite(dl).all())
    assert bool((dl[0] == 0).all()) and bool((dl[1] == 0).all())


def test_strided_logits_other_stream_and_no_tokens():
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn(20, 70, generator=g, device="cuda")
    part = wide[:, 3:67]
    s = torch.cuda.Stream()
    ids = torch.empty(20, 6, dtype=torch.int32, device="cuda")
    w = torch.empty(20, 6, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    B.moe_route(part, ids, w, stream=s)
    s.synchronize()
    ids2, w2 = route(part.contiguous(), 6)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    route(torch.empty(0, 8, device="cuda"), 2)


def test_gradient_against_differences():
    # logits 0.2 apart or more keep the selection under steps of 1e-2
    g = torch.Generator().manual_seed(5)
    T, E, k, h = 6, 12, 4, 1e-2
    l = torch.stack([torch.randperm(E, generator=g).float() * 0.25 for _ in range(T)])
    c = torch.randn(T, k, generator=g)
    v = torch.randn(T, E, generator=g).clamp(-2, 2)
    for scoring in SCORING:
        for renorm in (True, False):
            def loss(x):
                return (route(x.cuda(), k, scoring, renorm)[1].cpu().double() * c).sum(dim=1)
            num = (loss(l + h * v) - loss(l - h * v)) / (2 * h)
            ids, _ = route(l.cuda(), k, scoring, renorm)
            dl = torch.empty(T, E, device="cuda")
            B.moe_route_backward(l.cuda(), ids, c.cuda(), dl, scoring=SCORING[scoring],
                                 renormalize=renorm)
            ana = (dl.cpu().double() * v).sum(dim=1)
            # truncation h^2 |v|^3 |c| / 6 and the forward's rounding over h
            size = c.abs().sum(dim=1).double()
            bound = size * (h * h * 8 + 32 * HALF_ULP[torch.float32] / h)
            assert_within(ana, num, bound, f"{scoring} {renorm}")


def test_refusals():
    l = torch.randn(4, 8, device="cuda")
    ids = torch.empty(4, 2, dtype=torch.int32, device="cuda")
    w = torch.empty(4, 2, device="cuda")
    with pytest.raises(ValueError):
        B.moe_route(l, ids, w.half())
    with pytest.raises(ValueError):
        B.moe_route(l, ids.float(), w)
    with pytest.raises(ValueError):
        B.moe_route(l.t(), torch.empty(8, 2, dtype=torch.int32, device="cuda"),
                    torch.empty(8, 2, device="cuda"))
    with pytest.raises(B.MoeError) as e:
        B.moe_route(l, ids, w, num_groups=3)
    assert e.value.status == 2


@pytest.mark.parametrize("E,groups", [(64, 2), (128, 2), (12, 3), (60, 3)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_groups_whose_best_two_keys_add_up_to_minus_infinity(E, groups, scoring):
    # masked by the type's lowest value, through the logits or the bias: such a group is the
    # last to be taken, but it has experts, and comes before a group that has none
    low, size = torch.finfo(torch.float32).min, E // groups
    l, bias = torch.zeros(4, E), torch.zeros(E)
    if scoring == "softmax":
        l.fill_(low)
    else:
        bias.fill_(low)
        bias[1] = 0.25
    l[:, 1] = 1.0
    l[1] = torch.arange(E) % 7
    l[2, :size] = -float("inf") if scoring == "softmax" else float("nan")
    l[3] = float("nan")
    l[3, -2:] = low if scoring == "softmax" else 0.0
    ids, w = route(l.cuda(), 6, scoring, True, bias=bias.cuda(), groups=groups, top_groups=2)
    key = l if scoring == "softmax" else 1.0 / (1.0 + torch.exp(-l))
    with np.errstate(over="ignore", invalid="ignore"):
        want = select(key.numpy(), bias.numpy(), "softmax", 6, groups, 2)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert bool(torch.isfinite(w).all())


def chosen64(l, bias, k, groups, top_groups, apart):
    """Experts by softmax(l) + bias in 64 bits, and the rows where no two keys (or groups' values)
    that decide are closer than `apart` times the row's largest score or key."""
    l, bias = l.double().numpy(), bias.double().numpy()
    T, E = l.shape
    ids, clear = np.full((T, k), -1, np.int64), np.ones(T, bool)
    for t in range(T):
        ok = [e for e in range(E) if l[t, e] > -np.inf]
        if not ok:
            continue
        ex = {e: np.exp(l[t, e] - max(l[t, i] for i in ok)) for e in ok}
        z = sum(ex.values())
        key = {e: ex[e] / z + bias[e] for e in ok if bias[e] > -np.inf}
        least = apart * max([1 / z] + [abs(v) for v in key.values()])
        if groups > 1:
            value = {}
            for e, v in key.items():
                value.setdefault(e * groups // E, []).append(v)
            value = {g: sum(sorted(v)[-2:]) for g, v in value.items()}
            rank = sorted(value, key=lambda g: (-value[g], g))
            if len(rank) > top_groups:
                clear[t] &= value[rank[top_groups - 1]] - value[rank[top_groups]] > least
            key = {e: v for e, v in key.items() if e * groups // E in rank[:top_groups]}
        rank = sorted(key, key=lambda e: (-key[e], e))
        ids[t, :min(k, len(rank))] = rank[:k]
        clear[t] &= all(key[a] - key[b] > least for a, b in zip(rank[:k], rank[1:k + 1]))
    return ids, clear


@pytest.mark.parametrize("E,groups,top_groups,k", [(1, 1, 1, 1), (8, 1, 1, 2), (40, 5, 2, 8),
                                                   (256, 1, 1, 8), (256, 8, 4, 8), (60, 3, 2, 6),
                                                   (1000, 1, 1, 32)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
def test_softmax_with_a_bias_on_the_score(E, groups, top_groups, k, dtype, renorm):
    T = 60
    g = torch.Generator().manual_seed(E + groups)
    l = (torch.randn(T, E, generator=g) * 2).to(DTYPES[dtype])
    bias = torch.randn(E, generator=g) * 0.03
    if E > 8:
        l[:, 3] = -float("inf")
        l[1::7, 5] = float("nan")
        l[2, :] = -float("inf")
        l[3, 8:] = -float("inf")
        bias[3] = 5.0  # a masked expert stays masked
        bias[7] = -float("inf")
    ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 77.0, device="cuda")
    scoring = B.MOE_SCORE_SOFTMAX | B.MOE_SCORE_BIAS_ON_SCORE
    B.moe_route(l.cuda(), ids, w, bias=bias.cuda(), scoring=scoring, renormalize=renorm, scale=1.5,
                num_groups=groups, top_groups=top_groups)
    # a score's fp32 error: E / 32 + 5 sums after one another, exp, quotient, sum with the bias
    # (twice for a group), in units of 2^-24; two keys are compared
    want, clear = chosen64(l.float(), bias, k, groups, top_groups, 4 * (E / 32 + 16) * 2.0 ** -24)
    assert clear.sum() > T // 2
    assert np.array_equal(ids.cpu().numpy()[clear], want[clear])
    l64 = l.double()
    l64 = torch.where(torch.isnan(l64), torch.full_like(l64, -float("inf")), l64)
    at = ids.cpu().long()
    ref = weights64(l64, at, "softmax", renorm, 1.5)
    assert_within(w, ref, ref.abs() * (E + 16) * 2.0 ** -24 + 1e-30, "weights")
    # the gradient is the softmax's
    dw = torch.randn(T, k, generator=g).cuda()
    a, b = (torch.empty(T, E, dtype=l.dtype, device="cuda") for _ in range(2))
    B.moe_route_backward(l.cuda(), ids, dw, a, scoring=scoring, renormalize=renorm)
    B.moe_route_backward(l.cuda(), ids, dw, b, scoring=B.MOE_SCORE_SOFTMAX, renormalize=renorm)
    assert torch.equal(a, b)


def test_bias_on_the_score_where_it_says_nothing():
    g = torch.Generator().manual_seed(2)
    l, bias = torch.randn(30, 64, generator=g).cuda(), torch.randn(64, generator=g).cuda()
    for form, b in ((B.MOE_SCORE_SOFTMAX, None), (B.MOE_SCORE_SIGMOID, None),
                    (B.MOE_SCORE_SIGMOID, bias)):
        got = []
        for scoring in (form, form | B.MOE_SCORE_BIAS_ON_SCORE):
            ids = torch.empty(30, 4, dtype=torch.int32, device="cuda")
            w = torch.empty(30, 4, device="cuda")
            B.moe_route(l, ids, w, bias=b, scoring=scoring)
            got.append((ids, w))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    for scoring in (2, 3, 6, 7, 8, -1):
        with pytest.raises(B.MoeError):
            B.moe_route(l, ids, w, scoring=scoring)
