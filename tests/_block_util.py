"""Shared by the tests of the operators around the experts: types, strided tensors, bounds."""
import torch

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
# half a unit in the last place, relative: the error of one rounding
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# one rounding of a value below the type's normal range
TINY = {torch.float32: 1e-40, torch.bfloat16: 1e-40, torch.float16: 2.0 ** -25}


def strided(t, pad, offset=0):
    """The same values in a wider allocation: row stride K + pad, `offset` elements in front, NaN
    around them."""
    T, K = t.shape
    buf = torch.full((T * (K + pad) + offset + 8,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[offset:offset + T * (K + pad)].view(T, K + pad)[:, :K]
    v.copy_(t)
    return v


def assert_within(got, ref, bound, what):
    """|got - ref| <= bound, all in fp64 on the CPU; NaN nowhere."""
    got = got.detach().cpu().double()
    ref, bound = ref.cpu().double(), bound.cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    d = (got - ref).abs()
    ok = d <= bound
    assert bool(ok.all()), (f"{what}: {(~ok).sum().item()} of {ok.numel()} off, worst "
                            f"{(d / bound.clamp_min(1e-300)).max().item():.2f} x the bound")


def rounded(ref, dtype, extra):
    """Bound of a value rounded once to dtype whose fp32 sum is off by at most `extra`."""
    return ref.abs() * HALF_ULP[dtype] * 1.01 + extra * (1 + 2 * HALF_ULP[dtype]) + TINY[dtype]
