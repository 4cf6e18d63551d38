"""Host-side refusals of the operators around the experts (no GPU: every call below returns
before its first CUDA call)."""
import ctypes

import pytest

from moe_expert_layer_prepare_gb300 import binding as B

FAKE = 0x10000  # never dereferenced
OK, INVALID, SHAPE, UNSUPPORTED, ALIGNMENT, WORKSPACE = range(6)


@pytest.fixture(scope="module")
def lib():
    from moe_expert_layer_prepare_gb300 import build
    build.build()
    return B.load()


def fill(cls, **kw):
    a = cls()
    for n, t in cls._fields_:
        if t is ctypes.c_void_p:
            setattr(a, n, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def route(lib, cls=B.RouteArgs, fn="moe_route", **kw):
    base = dict(num_tokens=8, num_experts=16, top_k=2, logits_dtype=B.MOE_DTYPE_BF16,
                logits_stride0=16, topk_ids_dtype=B.MOE_IDS_INT32)
    base.update(dict(num_groups=1, top_groups=1) if cls is B.RouteArgs else
                dict(d_logits_stride0=16))
    base.update(kw)
    return getattr(lib, fn)(ctypes.byref(fill(cls, **base)), None)


def test_route(lib):
    assert lib.moe_route(None, None) == INVALID
    assert route(lib, num_tokens=-1) == INVALID
    assert route(lib, num_tokens=0) == OK
    assert route(lib, top_k=0) == SHAPE
    assert route(lib, top_k=17) == SHAPE
    assert route(lib, num_experts=1025, logits_stride0=1025) == UNSUPPORTED
    assert route(lib, num_experts=64, logits_stride0=64, top_k=33) == UNSUPPORTED
    assert route(lib, logits_dtype=3) == INVALID
    assert route(lib, scoring=2) == INVALID
    assert route(lib, topk_ids_dtype=2) == INVALID
    assert route(lib, num_groups=3) == SHAPE
    assert route(lib, num_groups=0) == SHAPE
    assert route(lib, num_groups=4, top_groups=5) == SHAPE
    assert route(lib, num_groups=16, top_groups=1) == SHAPE  # two experts of one-expert groups
    assert route(lib, num_experts=64, logits_stride0=64, num_groups=64, top_groups=8) == UNSUPPORTED
    assert route(lib, logits_stride0=15) == SHAPE
    assert route(lib, logits=None) == INVALID
    assert route(lib, topk_weights=None) == INVALID
    assert b"NULL" in lib.moe_last_error()
    back = dict(cls=B.RouteBackwardArgs, fn="moe_route_backward")
    assert route(lib, num_tokens=0, **back) == OK
    assert lib.moe_last_error() == b""
    assert route(lib, d_logits=None, **back) == INVALID
    assert route(lib, d_logits_stride0=8, **back) == SHAPE
    assert route(lib, top_k=33, num_experts=64, **back) == UNSUPPORTED


def test_packed_structs_have_the_c_layout():
    for cls in (B.RouteArgs, B.RouteBackwardArgs, B.SortArgs, B.PermuteArgs, B.UnpermuteArgs,
                B.UnpermuteBackwardArgs, B.BlockNormArgs, B.BlockNormBackwardArgs, B.LoraArgs):
        values = [float(i) if t is ctypes.c_float else i + 1
                  for i, (_, t) in enumerate(cls._fields_)]
        raw = cls.pack(*values)
        a = cls(*values)
        assert bytes(a)[:len(raw)] == raw and len(raw) > ctypes.sizeof(cls) - 8


def test_sort(lib):
    def sort(**kw):
        base = dict(num_tokens=8, top_k=2, num_experts=4, workspace_bytes=1 << 20)
        base.update(kw)
        return lib.moe_sort_routes(ctypes.byref(fill(B.SortArgs, **base)), None)
    assert lib.moe_sort_routes(None, None) == INVALID
    assert sort(num_tokens=-1) == INVALID
    assert sort(topk_ids_dtype=7) == INVALID
    assert sort(num_experts=0) == SHAPE
    assert sort(num_experts=1025) == UNSUPPORTED
    assert sort(num_tokens=1 << 26) == UNSUPPORTED
    for name in ("expert_offsets", "topk_ids", "route_row", "row_route"):
        assert sort(**{name: None}) == INVALID
    assert sort(num_tokens=100000, workspace=None) == WORKSPACE
    assert sort(num_tokens=100000, workspace_bytes=16) == WORKSPACE
    assert sort(num_tokens=100000, workspace=FAKE + 4) == ALIGNMENT
    assert lib.moe_sort_workspace_size(64, 2, 8) == 0
    assert lib.moe_sort_workspace_size(-1, 2, 8) == 0
    assert lib.moe_sort_workspace_size(8192, 8, 256) > 0


def test_rows(lib):
    def call(fn, cls, **kw):
        base = dict(num_tokens=4, hidden_size=64, top_k=2, num_rows=8, dtype=B.MOE_DTYPE_BF16)
        if cls is not B.UnpermuteArgs:
            base["num_experts"] = 4
        base.update({n: 64 for n, _ in cls._fields_ if n.endswith("stride0")})
        base.update(kw)
        return getattr(lib, fn)(ctypes.byref(fill(cls, **base)), None)

    def permute(**kw):
        return call("moe_permute", B.PermuteArgs, **kw)

    def unpermute(**kw):
        return call("moe_unpermute", B.UnpermuteArgs, **kw)

    def back(**kw):
        return call("moe_unpermute_backward", B.UnpermuteBackwardArgs, **kw)

    for f in (permute, unpermute, back):
        assert f(num_tokens=-1) == INVALID and f(dtype=9) == INVALID
        assert f(top_k=33) == UNSUPPORTED and f(num_rows=1 << 31) == UNSUPPORTED
        assert f(rows=None) == INVALID and f(route_row=None) == INVALID
        assert f(rows_stride0=63) == SHAPE
    assert permute(hidden_size=0) == OK and permute(num_rows=0) == OK
    assert permute(x=None) == INVALID and permute(expert_offsets=None) == INVALID
    assert permute(x_stride0=63) == SHAPE and permute(num_experts=-1) == INVALID
    assert unpermute(num_tokens=0) == OK
    assert unpermute(out=None) == INVALID and unpermute(out_stride0=3) == SHAPE
    assert back(num_tokens=0, num_rows=0) == OK
    for name in ("d_out", "topk_weights", "expert_offsets", "d_rows", "d_weights"):
        assert back(**{name: None}) == INVALID
    assert back(d_rows_stride0=1) == SHAPE and back(d_out_stride0=1) == SHAPE


def norm(lib, cls=B.BlockNormArgs, fn="moe_block_norm", **kw):
    base = dict(num_tokens=4, hidden_size=64, dtype=1, weight_dtype=1, gate_kind=1, gate_stride0=64)
    base.update({n: 64 for n, _ in cls._fields_ if n.endswith("stride0")})
    if cls is B.BlockNormBackwardArgs:
        base["workspace_bytes"] = 1 << 20
    base.update(kw)
    return getattr(lib, fn)(ctypes.byref(fill(cls, **base)), None)


def test_block_norm(lib):
    assert lib.moe_block_norm(None, None) == INVALID
    assert norm(lib, num_tokens=0) == OK
    assert norm(lib, hidden_size=-1) == INVALID
    assert norm(lib, hidden_size=16385) == UNSUPPORTED
    assert norm(lib, dtype=4) == INVALID and norm(lib, weight_dtype=-1) == INVALID
    assert norm(lib, gate_kind=4) == INVALID
    assert norm(lib, gate_kind=0) == INVALID and norm(lib, gate=None) == INVALID
    assert norm(lib, x=None) == INVALID
    assert norm(lib, z=None) == INVALID and norm(lib, x_out=None) == INVALID
    assert norm(lib, y=None) == INVALID and norm(lib, pre_weight=None) == INVALID
    assert norm(lib, y_stride0=8) == SHAPE and norm(lib, z_stride0=8) == SHAPE
    back = dict(cls=B.BlockNormBackwardArgs, fn="moe_block_norm_backward")
    assert norm(lib, hidden_size=0, **back) == OK
    assert norm(lib, x=None, **back) == INVALID and norm(lib, d_x=None, **back) == INVALID
    assert norm(lib, rstd_pre=None, **back) == INVALID
    assert norm(lib, rstd_post=None, **back) == INVALID
    assert norm(lib, z=None, **back) == INVALID
    assert norm(lib, pre_weight=None, **back) == INVALID
    assert norm(lib, gate=None, gate_kind=0, **back) == INVALID  # d_gate without a gate
    assert norm(lib, d_z_stride0=1, **back) == SHAPE
    assert norm(lib, workspace=None, **back) == WORKSPACE
    assert norm(lib, workspace_bytes=64, **back) == WORKSPACE
    assert norm(lib, workspace=FAKE + 4, **back) == ALIGNMENT
    assert lib.moe_block_norm_workspace_size(0, 64) == 0
    assert lib.moe_block_norm_workspace_size(4, 64) > 0


def test_workspaces_serve_shorter_calls(lib):
    ts = [1, 2, 7, 31, 63, 64, 65, 100, 127, 128, 129, 300, 511, 512, 513, 700, 1024, 1500, 2048,
          2049, 3500, 5000, 8192, 16385, 16500, 40000, 131073, 300000]
    for k, n, s, r in ((64, 64, 1, 8), (7168, 4096, 16, 64), (2048, 7168, 1000, 128)):
        sizes = [lib.moe_lora_workspace_size(t, k, n, s, r) for t in ts]
        assert sizes == sorted(sizes)
    for f in (lambda t: lib.moe_sort_workspace_size(t, 1, 256),
              lambda t: lib.moe_sort_workspace_size(t, 8, 1000),
              lambda t: lib.moe_block_norm_workspace_size(t, 4096)):
        sizes = [f(t) for t in ts]
        assert sizes == sorted(sizes)


def test_lora(lib):
    def lora(**kw):
        base = dict(num_tokens=4, in_features=64, out_features=32, num_adapters=2, rank=8,
                    dtype=B.MOE_DTYPE_BF16, x_stride0=64, out_stride0=32, workspace_bytes=1 << 20)
        base.update(kw)
        return lib.moe_lora_linear(ctypes.byref(fill(B.LoraArgs, **base)), None)
    assert lib.moe_lora_linear(None, None) == INVALID
    assert lora(num_tokens=0) == OK and lora(out_features=0) == OK
    assert lora(rank=-8) == INVALID
    assert lora(dtype=B.MOE_DTYPE_FP32) == UNSUPPORTED and lora(dtype=5) == INVALID
    assert lora(in_features=0) == SHAPE and lora(rank=0) == SHAPE
    assert lora(rank=136) == UNSUPPORTED and lora(num_adapters=1024) == UNSUPPORTED
    for name in ("x", "weight", "out", "lora_a", "lora_b", "adapter_ids", "lora_scale"):
        assert lora(**{name: None}) == INVALID
    assert lora(x_stride0=63) == SHAPE and lora(out_stride0=31) == SHAPE
    assert lora(in_features=60) == ALIGNMENT and lora(rank=12) == ALIGNMENT
    assert lora(x=FAKE + 8) == ALIGNMENT and lora(lora_b=FAKE + 2) == ALIGNMENT
    assert lora(x_stride0=68) == ALIGNMENT
    assert lora(workspace=None) == WORKSPACE and lora(workspace_bytes=8) == WORKSPACE
    assert lora(workspace=FAKE + 4) == ALIGNMENT
    assert lora(out_features=1 << 30, out_stride0=1 << 30) == UNSUPPORTED
    assert lib.moe_lora_workspace_size(4, 64, 32, 0, 8) == 0
    assert lib.moe_lora_workspace_size(4, 64, 32, 2, 8) > 0


def test_workspaces_grow_with_the_tokens(lib):
    # every step, at the counts where a plan changes: one block or many of the sort, its blocks'
    # share, the projection's path and the shrink's tokens a block
    steps = sorted({t + d for t in (16, 32, 64, 128, 256, 512, 1024, 2048, 4096, 32768, 65536,
                                    131072, 132096, 196608, 262144, 1048576, 4063232)
                    for d in (-1025, -129, -2, -1, 0, 1, 2, 97, 129, 1025) if t + d > 0})
    for k, n, s, r in ((4096, 4096, 256, 16), (64, 64, 1023, 8), (7168, 4096, 16, 64),
                       (2048, 7168, 48, 32), (512, 512, 1, 128)):
        sizes = [lib.moe_lora_workspace_size(t, k, n, s, r) for t in steps]
        assert sizes == sorted(sizes), (k, n, s, r)
    for e in (1, 8, 1024):
        sizes = [lib.moe_sort_workspace_size(t, 1, e) for t in steps]
        assert sizes == sorted(sizes), e
