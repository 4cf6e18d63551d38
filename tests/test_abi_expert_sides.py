"""Host-side refusals of the norm with an 8-bit output, the gated projection and the products with
4-bit weights (no GPU: every call below returns before its first CUDA call)."""
import ctypes

from moe_expert_layer_prepare_gb300 import binding as B
from tests.test_abi_block import (ALIGNMENT, FAKE, INVALID, OK, SHAPE, UNSUPPORTED, WORKSPACE,  # noqa: F401
                                  fill, lib)


def packed_layout(cls):
    values = [float(i) if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(cls._fields_)]
    raw = cls.pack(*values)
    assert bytes(cls(*values))[:len(raw)] == raw and len(raw) > ctypes.sizeof(cls) - 8


def test_norm_quant(lib):  # noqa: F811
    packed_layout(B.NormQuantArgs)

    def call(**kw):
        base = dict(num_tokens=8, hidden_size=256, dtype=B.MOE_DTYPE_BF16,
                    weight_dtype=B.MOE_DTYPE_FP32, x_stride0=256, z_stride0=256, x_out_stride0=256,
                    y_stride0=256, q_stride0=256, q_sf_stride0=2, sf_mode=B.MOE_SF_FP32, eps=1e-6)
        base.update(kw)
        return lib.moe_norm_quant(ctypes.byref(fill(B.NormQuantArgs, **base)), None)

    assert lib.moe_norm_quant(None, None) == INVALID
    assert call(num_tokens=-1) == INVALID
    assert call(num_tokens=0, x=None, q=None) == OK
    assert call(hidden_size=0) == OK
    assert call(dtype=3) == INVALID
    assert call(weight_dtype=-1) == INVALID
    assert call(sf_mode=B.MOE_SF_NONE) == INVALID
    assert call(sf_mode=3) == INVALID
    assert call(hidden_size=16385) == UNSUPPORTED
    assert call(z=None) == INVALID
    assert call(x_out=None) == INVALID
    for name in ("x", "weight", "q", "q_sf"):
        assert call(**{name: None}) == INVALID
        assert b"NULL" in lib.moe_last_error()
    for name in ("x_stride0", "z_stride0", "x_out_stride0", "y_stride0", "q_stride0"):
        assert call(**{name: 255}) == SHAPE
    assert call(q_sf_stride0=1) == SHAPE
    assert call(q_sf_stride0=0, sf_mode=B.MOE_SF_UE8M0_PACKED) == SHAPE
