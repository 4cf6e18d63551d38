"""Host-side refusals of the norm with an 8-bit output, the gated projection and the products with
4-bit weights (no GPU: every call below returns before its first CUDA call)."""
import ctypes
import os
import subprocess
import sys

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


def test_gated_linear(lib):  # noqa: F811
    packed_layout(B.GatedLinearArgs)
    packed_layout(B.GatedLinearBackwardArgs)
    sizes = dict(num_tokens=8, in_features=64, out_features=24, dtype=B.MOE_DTYPE_BF16,
                 activation=B.MOE_ACT_SILU, x_stride0=64, gate_up_stride0=48)

    def forward(**kw):
        return lib.moe_gated_linear(
            ctypes.byref(fill(B.GatedLinearArgs, **{**sizes, **dict(out_stride0=24), **kw})), None)

    def backward(**kw):
        base = {**sizes, **dict(d_out_stride0=24, d_x_stride0=64, workspace_bytes=1 << 40)}
        return lib.moe_gated_linear_backward(
            ctypes.byref(fill(B.GatedLinearBackwardArgs, **{**base, **kw})), None)

    assert lib.moe_gated_linear(None, None) == INVALID
    assert lib.moe_gated_linear_backward(None, None) == INVALID
    for call in (forward, backward):
        for name in ("num_tokens", "in_features", "out_features"):
            assert call(**{name: -1}) == INVALID
        assert call(dtype=5) == INVALID
        assert call(activation=3) == INVALID
        assert call(activation=B.MOE_ACT_NONE) == UNSUPPORTED
        assert call(dtype=B.MOE_DTYPE_FP32) == UNSUPPORTED
        assert call(num_tokens=1 << 22) == UNSUPPORTED
        assert call(out_features=1 << 28) == UNSUPPORTED
        assert call(x=None) == INVALID
        assert call(weight=None) == INVALID
        assert call(x_stride0=56) == SHAPE
        assert call(gate_up_stride0=47) == SHAPE
        assert call(in_features=60) == ALIGNMENT
        assert call(x_stride0=68) == ALIGNMENT
        assert call(x=FAKE + 8) == ALIGNMENT
        assert call(weight=FAKE + 2) == ALIGNMENT
    assert forward(num_tokens=0, x=None, out=None) == OK
    assert forward(in_features=0) == SHAPE
    assert forward(out=None) == INVALID
    assert forward(out_stride0=23) == SHAPE
    assert backward(in_features=0) == OK
    assert backward(num_tokens=0, d_weight=None, x=None) == OK
    assert backward(d_x=None, d_weight=None) == OK
    assert backward(d_out=None) == INVALID
    assert backward(gate_up=None) == INVALID
    assert backward(d_out_stride0=23) == SHAPE
    assert backward(d_x_stride0=63) == SHAPE
    assert backward(workspace=None) == WORKSPACE
    assert backward(workspace_bytes=1 << 10) == WORKSPACE
    assert backward(workspace=FAKE + 4) == ALIGNMENT
    assert lib.moe_gated_linear_workspace_size(0, 64, 24) == 0


def test_w4_linear(lib):  # noqa: F811
    packed_layout(B.W4LinearArgs)

    def call(**kw):
        base = dict(num_tokens=8, in_features=256, matrix_rows=32, num_experts=4, top_k=2,
                    group_size=64, dtype=B.MOE_DTYPE_BF16, format=B.MOE_W4_INT4,
                    activation=B.MOE_ACT_NONE, x_stride0=256, topk_ids_dtype=B.MOE_IDS_INT32,
                    out_stride0=32)
        return lib.moe_w4_linear(ctypes.byref(fill(B.W4LinearArgs, **{**base, **kw})), None)

    assert lib.moe_w4_linear(None, None) == INVALID
    for name in ("num_tokens", "in_features", "matrix_rows", "num_experts", "top_k"):
        assert call(**{name: -1}) == INVALID
    assert call(dtype=7) == INVALID
    assert call(format=2) == INVALID
    assert call(activation=3) == INVALID
    assert call(activation=-1) == INVALID
    assert call(topk_ids_dtype=2) == INVALID
    assert call(dtype=B.MOE_DTYPE_FP32) == UNSUPPORTED
    assert call(group_size=16) == UNSUPPORTED
    assert call(group_size=0) == UNSUPPORTED
    assert call(group_size=64, format=B.MOE_W4_E2M1, zeros=None) == UNSUPPORTED
    assert call(group_size=32, format=B.MOE_W4_E2M1) == UNSUPPORTED  # zeros
    assert call(matrix_rows=33, activation=B.MOE_ACT_SILU) == SHAPE
    assert call(num_tokens=0) == OK
    assert call(top_k=0) == OK
    assert call(matrix_rows=0) == OK
    assert call(in_features=0) == SHAPE
    assert call(in_features=224) == SHAPE
    assert call(num_experts=0) == SHAPE
    assert call(num_tokens=513) == UNSUPPORTED
    assert call(num_experts=1025) == UNSUPPORTED
    assert call(num_tokens=1025, topk_ids=None) == UNSUPPORTED
    for name in ("x", "weight", "scales", "out"):
        assert call(**{name: None}) == INVALID
    assert call(x_stride0=248) == SHAPE
    assert call(out_stride0=31) == SHAPE
    assert call(x_stride0=257) == ALIGNMENT
    assert call(x=FAKE + 2) == ALIGNMENT
    assert call(weight=FAKE + 8) == ALIGNMENT


def test_w4_linear_counts_routes_without_wrapping(lib):  # noqa: F811
    """tokens * top_k that would wrap to none, and to a few."""
    for T, k in ((1 << 40, 1 << 40), ((1 << 62) + 1, 4)):
        args = fill(B.W4LinearArgs, num_tokens=T, in_features=256, matrix_rows=32, num_experts=4,
                    top_k=k, group_size=64, dtype=B.MOE_DTYPE_BF16, format=B.MOE_W4_INT4,
                    activation=B.MOE_ACT_NONE, x_stride0=256, topk_ids_dtype=B.MOE_IDS_INT32,
                    out_stride0=31)
        assert lib.moe_w4_linear(ctypes.byref(args), None) == UNSUPPORTED


# Every length of the rows above 24,000 with every count of routes, with no GPU in sight: a call that
# the checks let pass ends at its first CUDA call, before its pointers are read.
SWEEP = """
import ctypes
from moe_expert_layer_prepare_gb300 import binding as B
from tests.test_abi_block import fill
lib, calls = B.load(), 0
for fmt, G in ((B.MOE_W4_INT4, 32), (B.MOE_W4_INT4, 64), (B.MOE_W4_INT4, 128), (B.MOE_W4_E2M1, 32)):
    for routes, k in ((1, 1), (32, 1), (33, 1), (64, 8), (216, 8), (512, 8), (1024, 1), (1024, 8)):
        for K in range(24064, 32769, 128):
            zeros = 0x10000 if calls % 2 and fmt == B.MOE_W4_INT4 else None
            a = fill(B.W4LinearArgs, num_tokens=routes // k, in_features=K, matrix_rows=7168,
                     num_experts=(3, 256)[calls // 2 % 2], top_k=k, group_size=G, dtype=1 + calls // 4 % 2,
                     format=fmt, activation=(B.MOE_ACT_NONE, B.MOE_ACT_SILU)[calls // 8 % 2],
                     zeros=zeros, x_stride0=K, topk_ids_dtype=B.MOE_IDS_INT32, out_stride0=7168)
            st = lib.moe_w4_linear(ctypes.byref(a), None)
            assert st == 6, (st, fmt, G, routes, K, lib.moe_last_error())
            calls += 1
print(calls)
"""


def test_w4_linear_has_a_form_for_long_rows_of_many_routes(lib):  # noqa: F811
    """In a process of its own, which an integer division by zero would end."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SWEEP], cwd=root, capture_output=True, text=True,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=root))
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    assert int(r.stdout) == 4 * 8 * 69
