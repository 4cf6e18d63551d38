"""moe_norm_quant against the norm in 64 bits: residual sum, norm, 8-bit codes and scales."""
import pytest
import torch

from tests._block_util import DTYPES, assert_within, rounded, strided

pytestmark = pytest.mark.gpu

# Relative error of the kernel's fp32 y before any rounding to fewer bits: the square sum's (at most
# 64 additions deep: 32 of a thread, 5 and 5 levels of the block), halved by the root, and six
# single roundings.  64 units of 2^-24 hold both.
REL = 64 * 2.0 ** -24


def reference(x, z, w, offset, eps):
    x = x.double()
    if z is not None:
        x = x + z.double()
    rstd = 1 / torch.sqrt((x * x).mean(dim=1) + eps)
    return x, x * rstd[:, None] * (w.double() + offset), rstd


def exponent(amax):
    """The exponent byte of moe_prepare_inputs: 2^(e - 127) is the power of two at or above
    max(amax, 1e-4) / 448."""
    e = torch.ceil(torch.log2(amax.clamp_min(1e-4) / 448)) + 127
    return e.clamp(1, 254)


def check_codes(q, sf, y, mode):
    """Codes and scales against y (fp64): a scale is that of amax within REL, a code the nearest
    one within REL of its value."""
    T, K = y.shape
    G = (K + 127) // 128
    yp = torch.nn.functional.pad(y, (0, -K % 128)).view(T, G, 128)
    amax = yp.abs().amax(dim=2)
    if mode == "fp32":
        scale = sf.double()
        assert_within(scale, amax.clamp_min(1e-4) / 448, amax.clamp_min(1e-4) / 448 * (REL + 2.0 ** -23),
                      "scale")
    else:
        b = sf.contiguous().view(torch.uint8).view(T, -1)
        assert bool((b[:, G:] == 0).all()), "the last word is filled up with zeros"
        got = b[:, :G].double()
        assert bool((got >= exponent(amax * (1 - REL))).all())
        assert bool((got <= exponent(amax * (1 + REL))).all())
        scale = torch.exp2(got - 127)
    v = yp / scale[:, :, None]
    step = torch.exp2(torch.floor(torch.log2((v.abs() * (1 + REL)).clamp_min(2.0 ** -6))) - 3)
    codes = torch.nn.functional.pad(q.contiguous().view(torch.float8_e4m3fn).double(), (0, -K % 128))
    # amax / scale is at most 448 (1 + REL + 2^-23): the largest code
    assert_within(codes.view(T, G, 128), v.clamp(-448, 448), step / 2 + v.abs() * 2 * REL, "codes")


def run(x, w, z=None, mode="ue8m0", y=True, pad=0, offset=0.0, eps=1e-6, in_place=False):
    from moe_expert_layer_prepare_gb300 import binding as B
    T, K = x.shape
    G = (K + 127) // 128
    q = strided(torch.zeros(T, K, device="cuda"), pad).to(torch.uint8) if not pad else \
        torch.zeros(T, K + pad, dtype=torch.uint8, device="cuda")[:, :K]
    cols = G if mode == "fp32" else (G + 3) // 4
    sf = torch.full((T, cols + (1 if pad else 0)), 7, device="cuda",
                    dtype=torch.float32 if mode == "fp32" else torch.int32)[:, :cols]
    x_out = None if z is None else (x if in_place else strided(torch.zeros_like(x), pad))
    yy = strided(torch.zeros_like(x), pad) if y else None
    rstd = torch.empty(T, device="cuda")
    ref = reference(x, z, w, offset, eps)
    B.moe_norm_quant(x, w, q, sf, z=z, x_out=x_out, y=yy, rstd=rstd, weight_offset=offset, eps=eps)
    torch.cuda.synchronize()
    check_codes(q, sf, ref[1], mode)
    if z is not None:
        assert_within(x_out, ref[0], rounded(ref[0], x.dtype, ref[0].abs() * 2.0 ** -24), "x_out")
    if y:
        assert_within(yy, ref[1], rounded(ref[1], x.dtype, ref[1].abs() * REL), "y")
    assert_within(rstd, ref[2], ref[2] * REL, "rstd")
    return q, sf, x_out, yy


def inputs(T, K, dtype, wdtype, z, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 1009 + T * 131 + K)
    x = torch.randn(T, K, device="cuda", generator=g) * 2
    x[:, ::97] *= 20
    zz = torch.randn(T, K, device="cuda", generator=g).to(DTYPES[dtype]) if z else None
    w = (1 + 0.2 * torch.randn(K, device="cuda", generator=g)).to(DTYPES[wdtype])
    return x.to(DTYPES[dtype]), w, zz


@pytest.mark.parametrize("mode", ["ue8m0", "fp32"])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"),
                                          ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("T,K", [(1, 128), (1, 1), (3, 7), (5, 129), (64, 4096), (33, 7168),
                                 (2, 16384), (7, 8200), (9, 4095), (700, 2048), (16, 520)])
def test_sizes(T, K, dtype, wdtype, mode):
    x, w, z = inputs(T, K, dtype, wdtype, True)
    run(x, w, z, mode=mode)


@pytest.mark.parametrize("mode", ["ue8m0", "fp32"])
@pytest.mark.parametrize("K", [4096, 4095, 640])
def test_forms(K, mode):
    """Without a residual, without y, in place, with strides, an offset and another eps."""
    x, w, z = inputs(17, K, "bf16", "bf16", True)
    run(x, w, None, mode=mode)
    run(x, w, None, mode=mode, y=False)
    run(x, w, z, mode=mode, y=False)
    run(x.clone(), w, z, mode=mode, in_place=True)
    for pad in (8, 3):
        run(strided(x, pad), w, strided(z, pad), mode=mode, pad=pad)
    run(strided(x, 8, offset=1), w, z, mode=mode)
    run(x, w - 1, z, mode=mode, offset=1.0, eps=1e-2)


def test_small_and_large_values():
    """Rows of zeros (the smallest scale, zero codes), tiny rows and rows whose squares are large."""
    x = torch.zeros(4, 256, device="cuda")
    x[1] = 1e-12
    x[2] = torch.linspace(-1, 1, 256, device="cuda") * 1e15
    x[3, 5] = 3.0
    w = torch.ones(256, device="cuda")
    for mode in ("ue8m0", "fp32"):
        q, sf, _, _ = run(x, w, mode=mode)
        assert bool((q[0] == 0).all())


def test_an_infinity_or_nan_stays_in_its_row():
    x, w, z = inputs(6, 512, "bf16", "bf16", True)
    clean = run(x.clone(), w, z)
    x[2, 3], x[4, 7] = float("nan"), float("inf")
    from moe_expert_layer_prepare_gb300 import binding as B
    q = torch.empty(6, 512, dtype=torch.uint8, device="cuda")
    sf = torch.empty(6, 1, dtype=torch.int32, device="cuda")
    x_out, y = torch.empty_like(x), torch.empty_like(x)
    B.moe_norm_quant(x, w, q, sf, z=z, x_out=x_out, y=y)
    for t in (0, 1, 3, 5):
        assert torch.equal(q[t], clean[0][t]) and torch.equal(sf[t], clean[1][t])
        assert torch.equal(y[t], clean[3][t])
    assert bool(y[2].isnan().all()) and bool(y[4, 7].isnan()) and bool((y[4, :7] == 0).all())


def test_rows_behind_the_last_are_left():
    from moe_expert_layer_prepare_gb300 import binding as B
    x, w, z = inputs(8, 384, "fp16", "fp16", True)
    q = torch.full((8, 384), 77, dtype=torch.uint8, device="cuda")
    sf = torch.full((8, 1), 77, dtype=torch.int32, device="cuda")
    x_out, y = torch.full_like(x, 77), torch.full_like(x, 77)
    B.moe_norm_quant(x[:5], w, q[:5], sf[:5], z=z[:5], x_out=x_out[:5], y=y[:5])
    B.moe_norm_quant(x[:0], w, q[:0], sf[:0], z=z[:0], x_out=x_out[:0], y=y[:0])
    for t in (q, sf, x_out, y):
        assert bool((t[5:] == 77).all())


def test_same_results_each_time_and_as_the_rows_norm():
    """Two calls agree in every bit, and y is moe_block_norm's to its own bound."""
    from moe_expert_layer_prepare_gb300 import binding as B
    x, w, z = inputs(300, 7168, "bf16", "bf16", True)
    a, b = run(x, w, z), run(x, w, z)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[3], b[3])
    xo, y = torch.empty_like(x), torch.empty_like(x)
    B.moe_block_norm(x, z=z, pre_weight=w, x_out=xo, y=y)
    assert torch.equal(xo, a[2])
    assert_within(a[3], y.double(), y.double().abs() * 2.0 ** -7, "y")


def test_the_gradient_of_the_norm_takes_rstd():
    """moe_block_norm_backward from this call's rstd, against differences in 64 bits."""
    from moe_expert_layer_prepare_gb300 import binding as B
    x, w, z = inputs(5, 256, "fp32", "fp32", True)
    q = torch.empty(5, 256, dtype=torch.uint8, device="cuda")
    sf = torch.empty(5, 2, device="cuda")
    x_out, rstd = torch.empty_like(x), torch.empty(5, device="cuda")
    B.moe_norm_quant(x, w, q, sf, z=z, x_out=x_out, rstd=rstd)
    d_y = torch.randn_like(x)
    d_x, d_z, d_w = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(B.block_norm_workspace_size(5, 256), dtype=torch.uint8, device="cuda")
    B.moe_block_norm_backward(x, z=z, pre_weight=w, rstd_pre=rstd, d_y=d_y, d_x=d_x, d_z=d_z,
                              d_pre_weight=d_w, workspace=ws)
    h = 1e-5
    for t, k in ((0, 0), (3, 97), (4, 255)):
        e = torch.zeros_like(x, dtype=torch.float64)
        e[t, k] = h
        up = (reference(x.double() + e, z, w, 0.0, 1e-6)[1] * d_y.double()).sum()
        down = (reference(x.double() - e, z, w, 0.0, 1e-6)[1] * d_y.double()).sum()
        slope = ((up - down) / (2 * h)).item()
        # gradient's terms are of size |d_y| rstd w: 1e-4 of them holds fp32's sums of 256
        tol = 1e-4 * (rstd[t].item() * (d_y[t] * w).abs().max().item()) * 16
        assert abs(d_x[t, k].item() - slope) <= tol and abs(d_z[t, k].item() - slope) <= tol


def test_refusals():
    from moe_expert_layer_prepare_gb300 import binding as B
    x, w, z = inputs(4, 256, "bf16", "bf16", True)
    q = torch.empty(4, 256, dtype=torch.uint8, device="cuda")
    sf = torch.empty(4, 1, dtype=torch.int32, device="cuda")
    for kw in (dict(q=q[:, :255]), dict(q_sf=sf.repeat(1, 2)), dict(q_sf=torch.empty(4, 1, device="cuda")),
               dict(weight=w[:255]), dict(z=z.float(), x_out=x), dict(x=x.t()), dict(q=q.cpu()),
               dict(rstd=torch.empty(3, device="cuda")), dict(y=x[:3]), dict(x=x.double())):
        with pytest.raises(ValueError):
            B.moe_norm_quant(**{**dict(x=x, weight=w, q=q, q_sf=sf), **kw})
    with pytest.raises(B.MoeError):
        B.moe_norm_quant(x, w, q, sf, z=z)  # no x_out
