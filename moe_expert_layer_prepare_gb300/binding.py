"""Thin ctypes binding of ``libmoe_prep.so`` (argument marshalling only).

The functions keep the C names: ``moe_prepare_inputs``, ``moe_batched_experts``,
``moe_topk_reduce``; around them ``moe_route``, ``moe_sort_routes``, ``moe_permute``,
``moe_unpermute``, ``moe_block_norm``, ``moe_lora_linear``, ``moe_norm_quant``,
``moe_gated_linear``, ``moe_w4_linear`` and their gradients.  Tensors are PyTorch CUDA tensors; only
their data pointers, shapes and strides cross the boundary.  Every step of the path runs
in the library's kernels; if the library is missing this module raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_prep.so")

MOE_OK = 0
MOE_SF_NONE, MOE_SF_UE8M0_PACKED, MOE_SF_FP32 = 0, 1, 2
MOE_IDS_INT32, MOE_IDS_INT64 = 0, 1
MOE_WEIGHTS_FP32, MOE_WEIGHTS_BF16 = 0, 1
MOE_ACT_SILU, MOE_ACT_GELU_TANH, MOE_ACT_NONE = 0, 1, 2
MOE_W4_INT4, MOE_W4_E2M1 = 0, 1
MOE_SHARED_BF16, MOE_SHARED_FP8 = 0, 1
MOE_STAGE_W13, MOE_STAGE_W2, MOE_STAGE_ALL = 1, 2, 3
MOE_DTYPE_FP32, MOE_DTYPE_BF16, MOE_DTYPE_FP16 = 0, 1, 2
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID, MOE_SCORE_BIAS_ON_SCORE = 0, 1, 4
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN, MOE_GATE_FULL = 0, 1, 2, 3
MOE_DEV_CAPACITY, MOE_DEV_BAD_EXPERT, MOE_DEV_TIMEOUT, MOE_DEV_BAD_ADAPTER = 1, 2, 4, 8
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARGUMENT", 2: "MOE_ERR_SHAPE",
                3: "MOE_ERR_UNSUPPORTED", 4: "MOE_ERR_ALIGNMENT", 5: "MOE_ERR_WORKSPACE",
                6: "MOE_ERR_CUDA"}

_i64, _i32, _vp, _sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t


class PrepareArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("hidden_size", _i64), ("top_k", _i64),
        ("hidden", _vp), ("hidden_stride0", _i64),
        ("topk_ids", _vp), ("topk_ids_dtype", _i32),
        ("topk_ids_stride0", _i64), ("topk_ids_stride1", _i64),
        ("topk_weights", _vp), ("topk_weights_dtype", _i32),
        ("topk_weights_stride0", _i64), ("topk_weights_stride1", _i64),
        ("is_padding", _vp), ("is_padding_stride0", _i64),
        ("x", _vp), ("x_stride0", _i64),
        ("x_sf", _vp), ("sf_mode", _i32), ("x_sf_stride0", _i64), ("x_sf_stride1", _i64),
        ("shared_x_sf", _vp), ("shared_x_sf_stride0", _i64), ("shared_x_sf_stride1", _i64),
        ("shared_x_sf_rows", _i64), ("shared_block_m", _i64),
        ("topk_idx_out", _vp), ("topk_idx_out_stride0", _i64), ("topk_idx_out_stride1", _i64),
        ("topk_weights_out", _vp), ("topk_weights_out_stride0", _i64),
        ("topk_weights_out_stride1", _i64),
        ("logical_to_physical", _vp), ("num_logical", _i64), ("map_stride", _i64),
        ("logical_replica_count", _vp), ("expert_load", _vp), ("num_physical", _i64),
        ("should_record", _vp), ("num_unpadded_tokens", _vp),
        ("num_experts", _i64), ("max_tokens_per_expert", _i64),
        ("x_b", _vp), ("sf_b", _vp), ("expert_num_tokens", _vp), ("route_slot", _vp),
        ("expert_offsets", _vp),
        ("workspace", _vp), ("workspace_bytes", _sz),
        ("device_status", _vp),
    ]


class Nvfp4Args(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("hidden_size", _i64), ("top_k", _i64),
        ("hidden", _vp), ("hidden_stride0", _i64),
        ("topk_ids", _vp), ("topk_ids_dtype", _i32),
        ("topk_ids_stride0", _i64), ("topk_ids_stride1", _i64),
        ("topk_weights", _vp), ("topk_weights_dtype", _i32),
        ("topk_weights_stride0", _i64), ("topk_weights_stride1", _i64),
        ("is_padding", _vp), ("is_padding_stride0", _i64),
        ("x", _vp), ("x_stride0", _i64),
        ("x_sf", _vp), ("x_sf_stride0", _i64),
        ("x_scales", _vp),
        ("shared_x", _vp), ("shared_x_stride0", _i64), ("shared_x_dtype", _i32),
        ("shared_x_sf", _vp), ("shared_x_sf_stride0", _i64), ("shared_x_sf_stride1", _i64),
        ("shared_x_sf_rows", _i64), ("shared_block_m", _i64),
        ("topk_idx_out", _vp), ("topk_idx_out_stride0", _i64), ("topk_idx_out_stride1", _i64),
        ("topk_weights_out", _vp), ("topk_weights_out_stride0", _i64),
        ("topk_weights_out_stride1", _i64),
        ("logical_to_physical", _vp), ("num_logical", _i64), ("map_stride", _i64),
        ("logical_replica_count", _vp), ("expert_load", _vp), ("num_physical", _i64),
        ("should_record", _vp), ("num_unpadded_tokens", _vp),
        ("w2_global_scale", _vp), ("l2_alpha", _vp), ("num_local_experts", _i64),
        ("l2_activation_scale", ctypes.c_float),
        ("device_status", _vp),
    ]


class ExpertsArgs(ctypes.Structure):
    _fields_ = [
        ("num_experts", _i64), ("max_tokens_per_expert", _i64), ("hidden_size", _i64),
        ("intermediate_size", _i64), ("activation", _i32), ("stages", _i32),
        ("output", _vp), ("hidden", _vp), ("a_scale", _vp), ("a_scale_mode", _i32),
        ("w13", _vp), ("w13_scale", _vp), ("w2", _vp), ("w2_scale", _vp),
        ("expert_num_tokens", _vp), ("expert_offsets", _vp),
        ("inter_q", _vp), ("inter_sf", _vp),
        ("workspace13", _vp), ("workspace13_bytes", _sz),
        ("workspace2", _vp), ("workspace2_bytes", _sz),
        ("valid_shape_m", _i64), ("gate_up_dump", _vp), ("device_status", _vp),
    ]


_f32 = ctypes.c_float


# Argument structs of the operators around the experts.  A call fills one with
# ``pack`` (the struct's bytes from its values in order, None not allowed: a NULL
# pointer is 0), a quarter of the time that filling the ctypes object takes, which
# counts where a call's kernel runs for two microseconds.
_FORMAT = {_i64: "q", _i32: "i", _vp: "P", _sz: "N", _f32: "f"}


def _packer(cls):
    cls.pack = staticmethod(struct.Struct("@" + "".join(_FORMAT[t] for _, t in cls._fields_)).pack)
    return cls


@_packer
class RouteArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("num_experts", _i64), ("top_k", _i64),
        ("logits", _vp), ("logits_dtype", _i32), ("logits_stride0", _i64),
        ("bias", _vp), ("is_padding", _vp), ("scoring", _i32), ("renormalize", _i32),
        ("scale", _f32), ("num_groups", _i64), ("top_groups", _i64),
        ("topk_ids", _vp), ("topk_ids_dtype", _i32), ("topk_weights", _vp),
    ]


@_packer
class RouteBackwardArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("num_experts", _i64), ("top_k", _i64),
        ("logits", _vp), ("logits_dtype", _i32), ("logits_stride0", _i64),
        ("scoring", _i32), ("renormalize", _i32), ("scale", _f32),
        ("topk_ids", _vp), ("topk_ids_dtype", _i32), ("d_weights", _vp),
        ("d_logits", _vp), ("d_logits_stride0", _i64),
    ]


@_packer
class SortArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("top_k", _i64), ("num_experts", _i64), ("topk_ids", _vp),
        ("topk_ids_dtype", _i32), ("expert_offsets", _vp), ("route_row", _vp),
        ("row_route", _vp), ("workspace", _vp), ("workspace_bytes", _sz), ("device_status", _vp),
    ]


@_packer
class PermuteArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("hidden_size", _i64), ("top_k", _i64), ("num_experts", _i64),
        ("num_rows", _i64), ("dtype", _i32), ("x", _vp), ("x_stride0", _i64), ("route_row", _vp),
        ("expert_offsets", _vp), ("rows", _vp), ("rows_stride0", _i64),
    ]


@_packer
class UnpermuteArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("hidden_size", _i64), ("top_k", _i64), ("num_rows", _i64),
        ("dtype", _i32), ("rows", _vp), ("rows_stride0", _i64), ("route_row", _vp),
        ("topk_weights", _vp), ("out", _vp), ("out_stride0", _i64),
    ]


@_packer
class UnpermuteBackwardArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("hidden_size", _i64), ("top_k", _i64), ("num_experts", _i64),
        ("num_rows", _i64), ("dtype", _i32), ("d_out", _vp), ("d_out_stride0", _i64),
        ("rows", _vp), ("rows_stride0", _i64), ("route_row", _vp), ("topk_weights", _vp),
        ("expert_offsets", _vp), ("d_rows", _vp), ("d_rows_stride0", _i64), ("d_weights", _vp),
    ]


@_packer
class BlockNormArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("hidden_size", _i64), ("dtype", _i32), ("weight_dtype", _i32),
        ("x", _vp), ("x_stride0", _i64), ("z", _vp), ("z_stride0", _i64),
        ("post_weight", _vp), ("gate", _vp), ("gate_kind", _i32), ("gate_stride0", _i64),
        ("scale", _f32), ("pre_weight", _vp), ("weight_offset", _f32), ("eps", _f32),
        ("x_out", _vp), ("x_out_stride0", _i64), ("y", _vp), ("y_stride0", _i64),
        ("rstd_post", _vp), ("rstd_pre", _vp),
    ]


@_packer
class BlockNormBackwardArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("hidden_size", _i64), ("dtype", _i32), ("weight_dtype", _i32),
        ("x", _vp), ("x_stride0", _i64), ("z", _vp), ("z_stride0", _i64),
        ("post_weight", _vp), ("gate", _vp), ("gate_kind", _i32), ("gate_stride0", _i64),
        ("scale", _f32), ("pre_weight", _vp), ("weight_offset", _f32),
        ("rstd_post", _vp), ("rstd_pre", _vp),
        ("d_x_out", _vp), ("d_x_out_stride0", _i64), ("d_y", _vp), ("d_y_stride0", _i64),
        ("d_x", _vp), ("d_x_stride0", _i64), ("d_z", _vp), ("d_z_stride0", _i64),
        ("d_gate", _vp), ("d_gate_stride0", _i64), ("d_post_weight", _vp), ("d_pre_weight", _vp),
        ("workspace", _vp), ("workspace_bytes", _sz),
    ]


@_packer
class LoraArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("in_features", _i64), ("out_features", _i64),
        ("num_adapters", _i64), ("rank", _i64), ("dtype", _i32),
        ("x", _vp), ("x_stride0", _i64), ("weight", _vp), ("lora_a", _vp), ("lora_b", _vp),
        ("adapter_ids", _vp), ("lora_scale", _vp), ("out", _vp), ("out_stride0", _i64),
        ("workspace", _vp), ("workspace_bytes", _sz), ("device_status", _vp),
    ]


@_packer
class NormQuantArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("hidden_size", _i64), ("dtype", _i32), ("weight_dtype", _i32),
        ("x", _vp), ("x_stride0", _i64), ("z", _vp), ("z_stride0", _i64), ("weight", _vp),
        ("weight_offset", _f32), ("eps", _f32), ("x_out", _vp), ("x_out_stride0", _i64),
        ("y", _vp), ("y_stride0", _i64), ("q", _vp), ("q_stride0", _i64), ("q_sf", _vp),
        ("sf_mode", _i32), ("q_sf_stride0", _i64), ("rstd", _vp),
    ]


@_packer
class GatedLinearArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("in_features", _i64), ("out_features", _i64), ("dtype", _i32),
        ("activation", _i32), ("x", _vp), ("x_stride0", _i64), ("weight", _vp), ("out", _vp),
        ("out_stride0", _i64), ("gate_up", _vp), ("gate_up_stride0", _i64),
        ("device_status", _vp),
    ]


@_packer
class GatedLinearBackwardArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("in_features", _i64), ("out_features", _i64), ("dtype", _i32),
        ("activation", _i32), ("d_out", _vp), ("d_out_stride0", _i64), ("x", _vp),
        ("x_stride0", _i64), ("weight", _vp), ("gate_up", _vp), ("gate_up_stride0", _i64),
        ("d_x", _vp), ("d_x_stride0", _i64), ("d_weight", _vp), ("workspace", _vp),
        ("workspace_bytes", _sz), ("device_status", _vp),
    ]


@_packer
class W4LinearArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", _i64), ("in_features", _i64), ("matrix_rows", _i64),
        ("num_experts", _i64), ("top_k", _i64), ("group_size", _i64), ("dtype", _i32),
        ("format", _i32), ("activation", _i32), ("x", _vp), ("x_stride0", _i64), ("weight", _vp),
        ("scales", _vp), ("zeros", _vp), ("topk_ids", _vp), ("topk_ids_dtype", _i32),
        ("out", _vp), ("out_stride0", _i64), ("device_status", _vp),
    ]


_lib = None


def load():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    _lib = configure(ctypes.CDLL(LIB_PATH))
    return _lib


def configure(lib):
    """Declare the C signatures on a loaded copy of the library."""
    lib.moe_abi_version.restype = ctypes.c_int
    lib.moe_last_error.restype = ctypes.c_char_p
    lib.moe_prepare_inputs.restype = ctypes.c_int
    lib.moe_prepare_inputs.argtypes = [ctypes.POINTER(PrepareArgs), _vp]
    lib.moe_prepare_workspace_size.restype = _sz
    lib.moe_prepare_workspace_size.argtypes = [_i64, _i64, _i64]
    lib.moe_prepare_inputs_noalloc.restype = ctypes.c_int
    lib.moe_prepare_inputs_noalloc.argtypes = [ctypes.POINTER(PrepareArgs), _vp]
    lib.moe_batched_experts.restype = ctypes.c_int
    lib.moe_batched_experts.argtypes = [ctypes.POINTER(ExpertsArgs), _vp]
    lib.moe_batched_experts_workspace_size.restype = _sz
    lib.moe_batched_experts_workspace_size.argtypes = [_i64, _i64, _i64, _i64, _i64,
                                                       ctypes.c_int]
    lib.moe_topk_reduce.restype = ctypes.c_int
    lib.moe_topk_reduce.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _vp,
                                    _vp]
    for name in ("moe_route", "moe_route_backward", "moe_sort_routes", "moe_permute",
                 "moe_unpermute", "moe_unpermute_backward", "moe_block_norm",
                 "moe_block_norm_backward", "moe_lora_linear", "moe_norm_quant",
                 "moe_gated_linear", "moe_gated_linear_backward", "moe_w4_linear"):
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = [_vp, _vp]  # the packed struct's bytes, the stream
    for name, n in (("moe_sort_workspace_size", 3), ("moe_block_norm_workspace_size", 2),
                    ("moe_lora_workspace_size", 5), ("moe_gated_linear_workspace_size", 3)):
        getattr(lib, name).restype = _sz
        getattr(lib, name).argtypes = [_i64] * n
    return lib


class MoeError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def _check(fn, st):
    if st != MOE_OK:
        raise MoeError(fn, st, load().moe_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def prepare_workspace_size(num_tokens, top_k, num_experts) -> int:
    return int(load().moe_prepare_workspace_size(num_tokens, top_k, num_experts))


def experts_workspace_size(E, M_max, K, N, valid_shape_m, which) -> int:
    return int(load().moe_batched_experts_workspace_size(E, M_max, K, N, valid_shape_m, which))


def moe_prepare_inputs(hidden, topk_ids, topk_weights, x, x_sf, topk_idx_out, topk_weights_out,
                       is_padding=None, sf_mode=MOE_SF_UE8M0_PACKED, eplb=None, dispatch=None,
                       device_status=None, stream=None, shared_x_sf=None, shared_block_m=None):
    """Input staging (and optional dispatch).  See include/moe_prep.h.

    shared_x_sf: uint8 [rows, K/128] shared-expert scale pages, given together
    with shared_block_m (UE8M0 scales only).

    eplb: dict(logical_to_physical, logical_replica_count, expert_load=None,
               should_record=None, num_unpadded_tokens=None) -- device tensors.
    dispatch: dict(num_experts, max_tokens_per_expert, x_b, sf_b, expert_num_tokens,
                   route_slot, workspace[, expert_offsets]) -- with expert_offsets
              ([E+1] int32) the rows are laid out contiguously per expert.
    """
    T, K = hidden.shape
    a = PrepareArgs()
    a.num_tokens, a.hidden_size = T, K
    a.top_k = topk_ids.shape[1] if topk_ids.dim() == 2 else 0
    a.hidden, a.hidden_stride0 = _ptr(hidden), hidden.stride(0)
    a.topk_ids = _ptr(topk_ids)
    a.topk_ids_dtype = MOE_IDS_INT64 if topk_ids.dtype == torch.int64 else MOE_IDS_INT32
    a.topk_ids_stride0, a.topk_ids_stride1 = topk_ids.stride(0), topk_ids.stride(1)
    a.topk_weights = _ptr(topk_weights)
    a.topk_weights_dtype = MOE_WEIGHTS_BF16 if topk_weights.dtype == torch.bfloat16 else \
        MOE_WEIGHTS_FP32
    a.topk_weights_stride0, a.topk_weights_stride1 = topk_weights.stride(0), topk_weights.stride(1)
    if is_padding is not None:
        a.is_padding, a.is_padding_stride0 = _ptr(is_padding), is_padding.stride(0)
    a.x, a.x_stride0 = _ptr(x), x.stride(0)
    a.sf_mode = sf_mode
    if x_sf is not None:
        a.x_sf, a.x_sf_stride0 = _ptr(x_sf), x_sf.stride(0)
        a.x_sf_stride1 = x_sf.stride(1) if x_sf.dim() > 1 else 1
    a.topk_idx_out = _ptr(topk_idx_out)
    a.topk_idx_out_stride0, a.topk_idx_out_stride1 = topk_idx_out.stride(0), topk_idx_out.stride(1)
    a.topk_weights_out = _ptr(topk_weights_out)
    a.topk_weights_out_stride0 = topk_weights_out.stride(0)
    a.topk_weights_out_stride1 = topk_weights_out.stride(1)
    if shared_x_sf is not None:
        a.shared_x_sf = _ptr(shared_x_sf)
        a.shared_x_sf_stride0, a.shared_x_sf_stride1 = shared_x_sf.stride(0), shared_x_sf.stride(1)
        a.shared_x_sf_rows = shared_x_sf.shape[0]
    if shared_block_m is not None:
        a.shared_block_m = int(shared_block_m)
    if eplb:
        l2p = eplb["logical_to_physical"]
        a.logical_to_physical, a.num_logical, a.map_stride = _ptr(l2p), l2p.shape[0], l2p.stride(0)
        a.logical_replica_count = _ptr(eplb["logical_replica_count"])
        load_t = eplb.get("expert_load")
        if load_t is not None:
            a.expert_load, a.num_physical = _ptr(load_t), load_t.numel()
        a.should_record = _ptr(eplb.get("should_record"))
        a.num_unpadded_tokens = _ptr(eplb.get("num_unpadded_tokens"))
    if dispatch:
        a.num_experts = dispatch["num_experts"]
        a.max_tokens_per_expert = dispatch["max_tokens_per_expert"]
        a.x_b, a.sf_b = _ptr(dispatch["x_b"]), _ptr(dispatch["sf_b"])
        a.expert_num_tokens = _ptr(dispatch["expert_num_tokens"])
        a.route_slot = _ptr(dispatch["route_slot"])
        a.expert_offsets = _ptr(dispatch.get("expert_offsets"))
        ws = dispatch["workspace"]
        a.workspace, a.workspace_bytes = _ptr(ws), ws.numel() * ws.element_size()
    a.device_status = _ptr(device_status)
    _check("moe_prepare_inputs", load().moe_prepare_inputs(ctypes.byref(a), _stream(stream)))


def moe_prepare_inputs_noalloc(hidden, topk_ids, topk_weights, x, x_sf, topk_idx_out,
                               topk_weights_out, is_padding=None, sf_mode=MOE_SF_UE8M0_PACKED,
                               eplb=None, dispatch=None, device_status=None, stream=None):
    """Staging + dispatch for callers that cannot allocate device memory.

    Same arguments as ``moe_prepare_inputs`` except that ``dispatch`` needs no
    ``workspace``: the scratch of the dispatch is a fixed array inside the
    library (MOE_PREPARE_NOALLOC_SCRATCH_BYTES, 4 MiB, per GPU).  Calls on one
    device share that array, so calls that may overlap on the GPU must be
    serialised; the first call on a device looks the array up, so make it
    before any stream capture.
    """
    T, K = hidden.shape
    a = PrepareArgs()
    a.num_tokens, a.hidden_size = T, K
    a.top_k = topk_ids.shape[1] if topk_ids.dim() == 2 else 0
    a.hidden, a.hidden_stride0 = _ptr(hidden), hidden.stride(0)
    a.topk_ids = _ptr(topk_ids)
    a.topk_ids_dtype = MOE_IDS_INT64 if topk_ids.dtype == torch.int64 else MOE_IDS_INT32
    a.topk_ids_stride0, a.topk_ids_stride1 = topk_ids.stride(0), topk_ids.stride(1)
    a.topk_weights = _ptr(topk_weights)
    a.topk_weights_dtype = MOE_WEIGHTS_BF16 if topk_weights.dtype == torch.bfloat16 else \
        MOE_WEIGHTS_FP32
    a.topk_weights_stride0, a.topk_weights_stride1 = topk_weights.stride(0), topk_weights.stride(1)
    if is_padding is not None:
        a.is_padding, a.is_padding_stride0 = _ptr(is_padding), is_padding.stride(0)
    a.x, a.x_stride0 = _ptr(x), x.stride(0)
    a.sf_mode = sf_mode
    if x_sf is not None:
        a.x_sf, a.x_sf_stride0 = _ptr(x_sf), x_sf.stride(0)
        a.x_sf_stride1 = x_sf.stride(1) if x_sf.dim() > 1 else 1
    a.topk_idx_out = _ptr(topk_idx_out)
    a.topk_idx_out_stride0, a.topk_idx_out_stride1 = topk_idx_out.stride(0), topk_idx_out.stride(1)
    a.topk_weights_out = _ptr(topk_weights_out)
    a.topk_weights_out_stride0 = topk_weights_out.stride(0)
    a.topk_weights_out_stride1 = topk_weights_out.stride(1)
    if eplb:
        l2p = eplb["logical_to_physical"]
        a.logical_to_physical, a.num_logical, a.map_stride = _ptr(l2p), l2p.shape[0], l2p.stride(0)
        a.logical_replica_count = _ptr(eplb["logical_replica_count"])
        load_t = eplb.get("expert_load")
        if load_t is not None:
            a.expert_load, a.num_physical = _ptr(load_t), load_t.numel()
        a.should_record = _ptr(eplb.get("should_record"))
        a.num_unpadded_tokens = _ptr(eplb.get("num_unpadded_tokens"))
    if dispatch:
        a.num_experts = dispatch["num_experts"]
        a.max_tokens_per_expert = dispatch["max_tokens_per_expert"]
        a.x_b, a.sf_b = _ptr(dispatch["x_b"]), _ptr(dispatch["sf_b"])
        a.expert_num_tokens = _ptr(dispatch["expert_num_tokens"])
        a.route_slot = _ptr(dispatch["route_slot"])
    a.device_status = _ptr(device_status)
    _check("moe_prepare_inputs_noalloc",
           load().moe_prepare_inputs_noalloc(ctypes.byref(a), _stream(stream)))


def moe_prepare_nvfp4_inputs(hidden, topk_ids, topk_weights, x, x_sf, x_scales, topk_idx_out,
                             topk_weights_out, is_padding=None, shared_x=None, eplb=None,
                             w2_global_scale=None, l2_alpha=None, l2_activation_scale=1.0,
                             device_status=None, stream=None, shared_x_sf=None,
                             shared_block_m=None):
    """NVFP4 token staging (E2M1 + E4M3 per 16 + fp32 per-token scale) and the
    top-k repack.  x: uint8 [T, K/2]; x_sf: int32 [T, K/64]; x_scales: fp32 [T].
    shared_x: bf16 [T, K] (a copy of the hidden rows) or uint8 [T, K] (the
    MXFP8 shared input, fp8 codes, given with shared_x_sf uint8 [rows, K/128]
    and shared_block_m).  See include/moe_prep.h."""
    T, K = hidden.shape
    a = Nvfp4Args()
    a.num_tokens, a.hidden_size = T, K
    a.top_k = topk_ids.shape[1] if topk_ids.dim() == 2 else 0
    a.hidden, a.hidden_stride0 = _ptr(hidden), hidden.stride(0)
    a.topk_ids = _ptr(topk_ids)
    a.topk_ids_dtype = MOE_IDS_INT64 if topk_ids.dtype == torch.int64 else MOE_IDS_INT32
    a.topk_ids_stride0, a.topk_ids_stride1 = topk_ids.stride(0), topk_ids.stride(1)
    a.topk_weights = _ptr(topk_weights)
    a.topk_weights_dtype = MOE_WEIGHTS_BF16 if topk_weights.dtype == torch.bfloat16 else \
        MOE_WEIGHTS_FP32
    a.topk_weights_stride0, a.topk_weights_stride1 = topk_weights.stride(0), topk_weights.stride(1)
    if is_padding is not None:
        a.is_padding, a.is_padding_stride0 = _ptr(is_padding), is_padding.stride(0)
    a.x, a.x_stride0 = _ptr(x), x.stride(0)
    a.x_sf, a.x_sf_stride0 = _ptr(x_sf), x_sf.stride(0)
    a.x_scales = _ptr(x_scales)
    if shared_x is not None:
        a.shared_x, a.shared_x_stride0 = _ptr(shared_x), shared_x.stride(0)
        a.shared_x_dtype = MOE_SHARED_BF16 if shared_x.dtype == torch.bfloat16 else MOE_SHARED_FP8
    if shared_x_sf is not None:
        a.shared_x_sf = _ptr(shared_x_sf)
        a.shared_x_sf_stride0, a.shared_x_sf_stride1 = shared_x_sf.stride(0), shared_x_sf.stride(1)
        a.shared_x_sf_rows = shared_x_sf.shape[0]
    if shared_block_m is not None:
        a.shared_block_m = int(shared_block_m)
    a.topk_idx_out = _ptr(topk_idx_out)
    a.topk_idx_out_stride0, a.topk_idx_out_stride1 = topk_idx_out.stride(0), topk_idx_out.stride(1)
    a.topk_weights_out = _ptr(topk_weights_out)
    a.topk_weights_out_stride0 = topk_weights_out.stride(0)
    a.topk_weights_out_stride1 = topk_weights_out.stride(1)
    if eplb:
        l2p = eplb["logical_to_physical"]
        a.logical_to_physical, a.num_logical, a.map_stride = _ptr(l2p), l2p.shape[0], l2p.stride(0)
        a.logical_replica_count = _ptr(eplb["logical_replica_count"])
        load_t = eplb.get("expert_load")
        if load_t is not None:
            a.expert_load, a.num_physical = _ptr(load_t), load_t.numel()
        a.should_record = _ptr(eplb.get("should_record"))
        a.num_unpadded_tokens = _ptr(eplb.get("num_unpadded_tokens"))
    if l2_alpha is not None:
        a.w2_global_scale, a.l2_alpha = _ptr(w2_global_scale), _ptr(l2_alpha)
        a.num_local_experts = l2_alpha.numel()
    a.l2_activation_scale = float(l2_activation_scale)
    a.device_status = _ptr(device_status)
    _check("moe_prepare_nvfp4_inputs",
           load().moe_prepare_nvfp4_inputs(ctypes.byref(a), _stream(stream)))


def moe_batched_experts(output, hidden, a_scale, w13, w13_scale, w2, w2_scale,
                        expert_num_tokens, workspace13=None, workspace2=None, valid_shape_m=0,
                        inter_q=None, inter_sf=None, gate_up_dump=None, stages=MOE_STAGE_ALL,
                        device_status=None, stream=None, expert_offsets=None):
    """w13 GEMM + SiLU-and-mul requant + w2 GEMM.  See include/moe_prep.h.

    expert_offsets ([E+1] int32, nullable) selects the contiguous layout.
    """
    E = w13.shape[0]
    K = w13.shape[2]
    N = w2.shape[2]
    if output is not None:
        M_max = output.shape[1] if output.dim() == 3 else output.shape[0] // E
    else:
        M_max = hidden.shape[0] // E
    a = ExpertsArgs()
    a.num_experts, a.max_tokens_per_expert, a.hidden_size, a.intermediate_size = E, M_max, K, N
    a.activation, a.stages = MOE_ACT_SILU, stages
    a.output, a.hidden, a.a_scale = _ptr(output), _ptr(hidden), _ptr(a_scale)
    # fp32 activation scales [E*M_max, K/128] select the fp32 dequantisation
    a.a_scale_mode = (MOE_SF_FP32 if a_scale is not None and a_scale.dtype == torch.float32
                      else MOE_SF_UE8M0_PACKED)
    a.w13, a.w13_scale, a.w2, a.w2_scale = _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale)
    a.expert_num_tokens = _ptr(expert_num_tokens)
    a.expert_offsets = _ptr(expert_offsets)
    a.inter_q, a.inter_sf = _ptr(inter_q), _ptr(inter_sf)
    if workspace13 is not None:
        a.workspace13 = _ptr(workspace13)
        a.workspace13_bytes = workspace13.numel() * workspace13.element_size()
    if workspace2 is not None:
        a.workspace2 = _ptr(workspace2)
        a.workspace2_bytes = workspace2.numel() * workspace2.element_size()
    a.valid_shape_m = valid_shape_m
    a.gate_up_dump = _ptr(gate_up_dump)
    a.device_status = _ptr(device_status)
    _check("moe_batched_experts", load().moe_batched_experts(ctypes.byref(a), _stream(stream)))


def moe_topk_reduce(expert_out, topk_idx, route_slot, topk_weights, out, stream=None,
                    num_valid_tokens=None):
    """Top-k weighted sum back to token order.  See include/moe_prep.h.

    topk_idx None: route_slot holds rows of expert_out (contiguous layout).
    num_valid_tokens: optional int32 device scalar; tokens at or past it are
    not written.
    """
    if expert_out.dim() == 3:
        E, M_max, K = expert_out.shape
    else:
        (E, K), M_max = (1, expert_out.shape[1]), expert_out.shape[0]
    T, k = route_slot.shape
    _check("moe_topk_reduce", load().moe_topk_reduce(
        _ptr(expert_out), E, M_max, K, _ptr(topk_idx), _ptr(route_slot), _ptr(topk_weights), T, k,
        _ptr(num_valid_tokens), _ptr(out), _stream(stream)))


# ---------------------------------------------------------------------------
# The operators around the experts.  The library sees pointers, sizes and
# strides; what only the tensors know (types, shapes, inner strides) is checked
# here and raises ValueError.
# ---------------------------------------------------------------------------
_BF16, _FP16, _FP32, _INT32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
_DTYPE = {_FP32: MOE_DTYPE_FP32, _BF16: MOE_DTYPE_BF16, _FP16: MOE_DTYPE_FP16}
_IDS = {_INT32: MOE_IDS_INT32, torch.int64: MOE_IDS_INT64}
_current_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _raw_stream(stream):
    if stream is None:
        return _current_stream(_current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(name, args, stream):
    st = getattr(_lib or load(), name)(args, _raw_stream(stream))
    if st != MOE_OK:
        _check(name, st)


def _at(t):
    return 0 if t is None else t.data_ptr()


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _rows(name, t, shape, dtype):
    """Row stride of a tensor of this shape with inner stride 1 (0 for None)."""
    if t is None:
        return 0
    s0, s1 = t.stride() if t.dim() == 2 else (0, 0)
    if t.dtype is not dtype or t.shape != shape or (s1 != 1 and shape[1] > 1):
        raise ValueError(f"{name}: want {dtype} {list(shape)} with inner stride 1, got {t.dtype} "
                         f"{list(t.shape)} with strides {t.stride()}")
    return s0


def _flat(name, t, shape, dtype):
    """Address of a contiguous tensor of this shape and type (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: want contiguous {dtype} {list(shape)}, got {t.dtype} "
                         f"{list(t.shape)} with strides {t.stride()}")
    return t.data_ptr()


def _here(*tensors):
    """Every tensor on the current device, whose stream a call goes to."""
    dev = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor {list(t.shape)} is on {t.device}, and the current device is "
                             f"cuda:{dev}")


def _code(name, dtype, table=_DTYPE):
    d = table.get(dtype)
    if d is None:
        raise ValueError(f"{name}: unsupported type {dtype}")
    return d


def moe_route(logits, topk_ids, topk_weights, bias=None, is_padding=None,
              scoring=MOE_SCORE_SOFTMAX, renormalize=True, scale=1.0, num_groups=1, top_groups=1,
              stream=None):
    """Router: top-k ids (int32 or int64 [T, k]) and weights (fp32 [T, k]) of logits [T, E].

    bias: fp32 [E], added for the selection alone: to the score of MOE_SCORE_SIGMOID and of
    MOE_SCORE_SOFTMAX | MOE_SCORE_BIAS_ON_SCORE, to the logit of MOE_SCORE_SOFTMAX by itself.
    is_padding: uint8 [T]; num_groups, top_groups: only the experts of the best groups are taken.
    See include/moe_prep.h."""
    T, E = logits.shape
    k = topk_ids.shape[1]
    dt, idt, tk = logits.dtype, topk_ids.dtype, (T, k)
    _call("moe_route", RouteArgs.pack(
        T, E, k, logits.data_ptr(), _code("logits", dt), _rows("logits", logits, (T, E), dt),
        _flat("bias", bias, (E,), _FP32), _flat("is_padding", is_padding, (T,), torch.uint8),
        scoring, 1 if renormalize else 0, scale, num_groups, top_groups,
        _flat("topk_ids", topk_ids, tk, idt), _code("topk_ids", idt, _IDS),
        _flat("topk_weights", topk_weights, tk, _FP32)), stream)


def moe_route_backward(logits, topk_ids, d_weights, d_logits, scoring=MOE_SCORE_SOFTMAX,
                       renormalize=True, scale=1.0, stream=None):
    """Gradient of the logits (every value written) from that of ``moe_route``'s weights; scoring,
    renormalize and scale as in the forward call.  See include/moe_prep.h."""
    T, E = shape = logits.shape
    k = topk_ids.shape[1]
    dt, idt, tk = logits.dtype, topk_ids.dtype, (T, k)
    _call("moe_route_backward", RouteBackwardArgs.pack(
        T, E, k, logits.data_ptr(), _code("logits", dt), _rows("logits", logits, shape, dt),
        scoring, 1 if renormalize else 0, scale, _flat("topk_ids", topk_ids, tk, idt),
        _code("topk_ids", idt, _IDS), _flat("d_weights", d_weights, tk, _FP32),
        d_logits.data_ptr(), _rows("d_logits", d_logits, shape, dt)), stream)


def sort_workspace_size(num_tokens, top_k, num_experts) -> int:
    return int(load().moe_sort_workspace_size(num_tokens, top_k, num_experts))


def moe_sort_routes(topk_ids, expert_offsets, route_row, row_route, workspace=None,
                    device_status=None, stream=None):
    """Rows of the routes in expert order.  topk_ids: int32 or int64 [T, k]; expert_offsets: int32
    [E + 1]; route_row: int32 [T, k]; row_route: int32 [T * k]; workspace: uint8,
    sort_workspace_size() bytes.  See include/moe_prep.h."""
    T, k = tk = topk_ids.shape
    n, idt = expert_offsets.shape[0], topk_ids.dtype
    _call("moe_sort_routes", SortArgs.pack(
        T, k, n - 1, _flat("topk_ids", topk_ids, tk, idt), _code("topk_ids", idt, _IDS),
        _flat("expert_offsets", expert_offsets, (n,), _INT32),
        _flat("route_row", route_row, tk, _INT32), _flat("row_route", row_route, (T * k,), _INT32),
        _at(workspace), _bytes(workspace), _at(device_status)), stream)


def moe_permute(x, route_row, expert_offsets, rows, stream=None):
    """rows[route_row[t, j]] = x[t]; rows past the last routed one become zeros.  x: [T, K] and
    rows: [num_rows, K] of one type (fp32, bf16, fp16).  See include/moe_prep.h."""
    T, k = tk = route_row.shape
    R, K = shape = rows.shape
    n, dt = expert_offsets.shape[0], rows.dtype
    _call("moe_permute", PermuteArgs.pack(
        T, K, k, n - 1, R, _code("rows", dt), x.data_ptr(), _rows("x", x, (T, K), dt),
        _flat("route_row", route_row, tk, _INT32),
        _flat("expert_offsets", expert_offsets, (n,), _INT32), rows.data_ptr(),
        _rows("rows", rows, shape, dt)), stream)


def moe_unpermute(rows, route_row, topk_weights, out, stream=None):
    """out[t] = sum_j topk_weights[t, j] * rows[route_row[t, j]], summed in fp32; topk_weights None:
    every weight is 1.  See include/moe_prep.h."""
    T, k = tk = route_row.shape
    R, K = shape = rows.shape
    dt = rows.dtype
    _call("moe_unpermute", UnpermuteArgs.pack(
        T, K, k, R, _code("rows", dt), rows.data_ptr(), _rows("rows", rows, shape, dt),
        _flat("route_row", route_row, tk, _INT32),
        _flat("topk_weights", topk_weights, tk, _FP32), out.data_ptr(),
        _rows("out", out, (T, K), dt)), stream)


def moe_permute_backward(d_rows, route_row, d_x, stream=None):
    """d_x[t] = sum_j d_rows[route_row[t, j]]: the gradient of ``moe_permute``."""
    moe_unpermute(d_rows, route_row, None, d_x, stream=stream)


def moe_unpermute_backward(d_out, rows, route_row, topk_weights, expert_offsets, d_rows, d_weights,
                           stream=None):
    """Gradients of ``moe_unpermute``: d_rows [num_rows, K] (zeros past the last routed row) and
    d_weights fp32 [T, k].  See include/moe_prep.h."""
    T, k = tk = route_row.shape
    R, K = shape = rows.shape
    n, dt = expert_offsets.shape[0], rows.dtype
    _call("moe_unpermute_backward", UnpermuteBackwardArgs.pack(
        T, K, k, n - 1, R, _code("rows", dt), d_out.data_ptr(), _rows("d_out", d_out, (T, K), dt),
        rows.data_ptr(), _rows("rows", rows, shape, dt),
        _flat("route_row", route_row, tk, _INT32), _flat("topk_weights", topk_weights, tk, _FP32),
        _flat("expert_offsets", expert_offsets, (n,), _INT32), d_rows.data_ptr(),
        _rows("d_rows", d_rows, shape, dt), _flat("d_weights", d_weights, tk, _FP32)), stream)


def _gate(gate, name, shape, dtype, wdtype, kind=None):
    """(kind, stride) of a gate, or of its gradient: the given kind, else by its shape and type,
    [K] of wdtype, [T] or [T, 1] of dtype, or [T, K] of dtype.  A 1-D gate that T == K lets be
    either of two kinds is refused without one (T == K == 1: both are the same)."""
    if gate is None:
        if kind not in (None, MOE_GATE_NONE):
            raise ValueError(f"{name}: gate_kind {kind} without a gate")
        return MOE_GATE_NONE, 0
    T, K = shape
    gs = gate.shape
    if kind is None:
        channel = gs == (K,) and gate.dtype is wdtype
        token = gate.dtype is dtype and (gs == (T,) or (gs == (T, 1) and K != 1))
        if channel and token and K != 1:
            raise ValueError(f"{name}: {list(gs)} with {T} tokens of {K} values is a channel gate "
                             "or a token gate: give gate_kind (or a token gate as [T, 1])")
        kind = MOE_GATE_CHANNEL if channel else MOE_GATE_TOKEN if token else MOE_GATE_FULL
    if kind == MOE_GATE_CHANNEL:
        _flat(name, gate, (K,), wdtype)
        return kind, 0
    if kind == MOE_GATE_TOKEN:
        if gate.dtype is not dtype or gs not in ((T,), (T, 1)):
            raise ValueError(f"{name}: want {dtype} [{T}] or [{T}, 1], got {gate.dtype} {list(gs)}")
        return kind, gate.stride(0)
    if kind != MOE_GATE_FULL:
        raise ValueError(f"{name}: gate_kind {kind} with a gate")
    return kind, _rows(name, gate, shape, dtype)


def _weight_type(x, pre_weight, post_weight, gate):
    for t in (pre_weight, post_weight, gate):
        if t is not None:
            return t.dtype
    return x.dtype


def moe_block_norm(x, z=None, post_weight=None, gate=None, scale=1.0, pre_weight=None,
                   weight_offset=0.0, eps=1e-6, x_out=None, y=None, rstd_post=None, rstd_pre=None,
                   stream=None, gate_kind=None):
    """x_out = x + scale * gate * rmsnorm(z, post_weight) and y = rmsnorm(x_out, pre_weight).

    x, z, x_out, y: [T, K] of one type; post_weight, pre_weight and a channel gate: [K] of one
    type (fp32, bf16 or fp16); a token gate: [T] or [T, 1] of x's type; a full gate: [T, K].
    gate_kind: MOE_GATE_CHANNEL, MOE_GATE_TOKEN or MOE_GATE_FULL; without it the gate's shape and
    type tell, and a 1-D gate that could be a channel's or a token's, as T == K, raises ValueError.
    Without z only y = rmsnorm(x) is written, without pre_weight only x_out.  rstd_post, rstd_pre:
    fp32 [T], kept for the gradient.  See include/moe_prep.h."""
    T, K = shape = x.shape
    dt, wdt = x.dtype, _weight_type(x, pre_weight, post_weight, gate)
    kind, gs = _gate(gate, "gate", shape, dt, wdt, gate_kind)
    _call("moe_block_norm", BlockNormArgs.pack(
        T, K, _code("x", dt), _code("weights", wdt), x.data_ptr(), _rows("x", x, shape, dt),
        _at(z), _rows("z", z, shape, dt), _flat("post_weight", post_weight, (K,), wdt), _at(gate),
        kind, gs, scale, _flat("pre_weight", pre_weight, (K,), wdt), weight_offset, eps,
        _at(x_out), _rows("x_out", x_out, shape, dt), _at(y), _rows("y", y, shape, dt),
        _flat("rstd_post", rstd_post, (T,), _FP32), _flat("rstd_pre", rstd_pre, (T,), _FP32)),
        stream)


def block_norm_workspace_size(num_tokens, hidden_size) -> int:
    return int(load().moe_block_norm_workspace_size(num_tokens, hidden_size))


def moe_block_norm_backward(x, z=None, post_weight=None, gate=None, scale=1.0, pre_weight=None,
                            weight_offset=0.0, rstd_post=None, rstd_pre=None, d_x_out=None,
                            d_y=None, d_x=None, d_z=None, d_gate=None, d_post_weight=None,
                            d_pre_weight=None, workspace=None, stream=None, gate_kind=None):
    """Gradients of ``moe_block_norm`` from d_x_out and d_y (either may be None) and the forward's
    inputs, rstd_post and rstd_pre; gate_kind as there.  d_x is always written, the others where
    given.  workspace: uint8, block_norm_workspace_size() bytes.  See include/moe_prep.h."""
    T, K = shape = x.shape
    dt, wdt = x.dtype, _weight_type(x, pre_weight, post_weight, gate)
    kind, gs = _gate(gate, "gate", shape, dt, wdt, gate_kind)
    dgs = 0
    if d_gate is not None:
        if gate is None or d_gate.shape != gate.shape:
            raise ValueError("d_gate must have the gate's shape and type")
        dgs = _gate(d_gate, "d_gate", shape, dt, wdt, kind)[1]
    _call("moe_block_norm_backward", BlockNormBackwardArgs.pack(
        T, K, _code("x", dt), _code("weights", wdt), x.data_ptr(), _rows("x", x, shape, dt),
        _at(z), _rows("z", z, shape, dt), _flat("post_weight", post_weight, (K,), wdt), _at(gate),
        kind, gs, scale, _flat("pre_weight", pre_weight, (K,), wdt), weight_offset,
        _flat("rstd_post", rstd_post, (T,), _FP32), _flat("rstd_pre", rstd_pre, (T,), _FP32),
        _at(d_x_out), _rows("d_x_out", d_x_out, shape, dt), _at(d_y),
        _rows("d_y", d_y, shape, dt), _at(d_x), _rows("d_x", d_x, shape, dt), _at(d_z),
        _rows("d_z", d_z, shape, dt), _at(d_gate), dgs,
        _flat("d_post_weight", d_post_weight, (K,), wdt),
        _flat("d_pre_weight", d_pre_weight, (K,), wdt), _at(workspace), _bytes(workspace)),
        stream)


def lora_workspace_size(num_tokens, in_features, out_features, num_adapters, rank) -> int:
    return int(load().moe_lora_workspace_size(num_tokens, in_features, out_features, num_adapters,
                                              rank))


def moe_lora_linear(x, weight, lora_a, lora_b, adapter_ids, lora_scale, out, workspace,
                    device_status=None, stream=None):
    """out[t] = x[t] weight^T + lora_scale[a] * (x[t] lora_a[a]^T) lora_b[a]^T, a = adapter_ids[t]
    (< 0: no adapter).  x [T, K], weight [N, K], lora_a [S, R, K], lora_b [S, N, R], out [T, N] of
    one type (bf16 or fp16); adapter_ids int32 [T]; lora_scale fp32 [S].  lora_a None: the
    projection alone.  workspace: uint8, lora_workspace_size() bytes.  See include/moe_prep.h."""
    T, K = shape = x.shape
    N, dt = weight.shape[0], x.dtype
    S, R = lora_a.shape[:2] if lora_a is not None else (0, 0)
    _call("moe_lora_linear", LoraArgs.pack(
        T, K, N, S, R, _code("x", dt), x.data_ptr(), _rows("x", x, shape, dt),
        _flat("weight", weight, (N, K), dt), _flat("lora_a", lora_a, (S, R, K), dt),
        _flat("lora_b", lora_b, (S, N, R), dt), _flat("adapter_ids", adapter_ids, (T,), _INT32),
        _flat("lora_scale", lora_scale, (S,), _FP32), out.data_ptr(),
        _rows("out", out, (T, N), dt), _at(workspace), _bytes(workspace), _at(device_status)),
        stream)


def moe_norm_quant(x, weight, q, q_sf, z=None, x_out=None, y=None, rstd=None, weight_offset=0.0,
                   eps=1e-6, stream=None):
    """x_out = x + z and rmsnorm(x_out, weight) in 8 bits, its 1x128 groups scaled as by
    ``moe_prepare_inputs``.

    x, z, x_out, y: [T, K] of one type (fp32, bf16 or fp16); weight: [K] (any of them); q: uint8
    [T, K]; q_sf: packed UE8M0 exponents, int32 [T, ceil(G / 4)], or scales, fp32 [T, G], of the
    G = ceil(K / 128) groups; y: the norm's output in x's type as well; rstd: fp32 [T], what
    ``moe_block_norm_backward`` takes as rstd_pre.  See include/moe_prep.h."""
    T, K = shape = x.shape
    dt, wdt, sdt = x.dtype, weight.dtype, q_sf.dtype
    G = (K + 127) // 128
    mode = MOE_SF_FP32 if sdt is _FP32 else MOE_SF_UE8M0_PACKED
    _here(x, weight, q, q_sf, z, x_out, y, rstd)
    _call("moe_norm_quant", NormQuantArgs.pack(
        T, K, _code("x", dt), _code("weight", wdt), x.data_ptr(), _rows("x", x, shape, dt),
        _at(z), _rows("z", z, shape, dt), _flat("weight", weight, (K,), wdt), weight_offset, eps,
        _at(x_out), _rows("x_out", x_out, shape, dt), _at(y), _rows("y", y, shape, dt),
        q.data_ptr(), _rows("q", q, shape, torch.uint8), q_sf.data_ptr(), mode,
        _rows("q_sf", q_sf, (T, G), _FP32) if mode == MOE_SF_FP32 else
        _rows("q_sf", q_sf, (T, (G + 3) // 4), _INT32),
        _flat("rstd", rstd, (T,), _FP32)), stream)


def moe_gated_linear(x, weight, out, activation=MOE_ACT_SILU, gate_up=None, device_status=None,
                     stream=None):
    """out = act(x Wg^T) * (x Wu^T), Wg and Wu the first and the second half of weight's rows.

    x [T, K], weight [2 N, K], out [T, N] of one type (bf16 or fp16); activation: MOE_ACT_SILU or
    MOE_ACT_GELU_TANH; gate_up [T, 2 N]: both projections, kept for the gradient.  See
    include/moe_prep.h."""
    T, K = shape = x.shape
    rows, dt = weight.shape[0], x.dtype
    if rows % 2:
        raise ValueError(f"weight: {rows} rows are not as many gate rows as up rows")
    N = rows // 2
    _here(x, weight, out, gate_up, device_status)
    _call("moe_gated_linear", GatedLinearArgs.pack(
        T, K, N, _code("x", dt), activation, x.data_ptr(), _rows("x", x, shape, dt),
        _flat("weight", weight, (rows, K), dt), out.data_ptr(), _rows("out", out, (T, N), dt),
        _at(gate_up), _rows("gate_up", gate_up, (T, rows), dt), _at(device_status)), stream)


def gated_linear_workspace_size(num_tokens, in_features, out_features) -> int:
    """Bytes of ``moe_gated_linear_backward``'s workspace."""
    return int(load().moe_gated_linear_workspace_size(num_tokens, in_features, out_features))


def moe_gated_linear_backward(d_out, x, weight, gate_up, d_x=None, d_weight=None,
                              activation=MOE_ACT_SILU, workspace=None, device_status=None,
                              stream=None):
    """Gradients of ``moe_gated_linear``: d_x [T, K] and d_weight [2 N, K], each where given, from
    d_out [T, N], the forward's x and weight and the gate_up that it wrote.  workspace: uint8,
    gated_linear_workspace_size() bytes.  See include/moe_prep.h."""
    T, K = shape = x.shape
    rows, dt = weight.shape[0], x.dtype
    if rows % 2:
        raise ValueError(f"weight: {rows} rows are not as many gate rows as up rows")
    N = rows // 2
    _here(d_out, x, weight, gate_up, d_x, d_weight, workspace, device_status)
    _call("moe_gated_linear_backward", GatedLinearBackwardArgs.pack(
        T, K, N, _code("x", dt), activation, d_out.data_ptr(), _rows("d_out", d_out, (T, N), dt),
        x.data_ptr(), _rows("x", x, shape, dt), _flat("weight", weight, (rows, K), dt),
        gate_up.data_ptr(), _rows("gate_up", gate_up, (T, rows), dt), _at(d_x),
        _rows("d_x", d_x, shape, dt), _flat("d_weight", d_weight, (rows, K), dt), _at(workspace),
        _bytes(workspace), _at(device_status)), stream)


def moe_w4_linear(x, weight, scales, out, zeros=None, topk_ids=None, activation=MOE_ACT_NONE,
                  device_status=None, stream=None):
    """Products of few rows with 4-bit weights and group scales.

    x: [T, K] bf16 or fp16; weight: uint8 [N, K / 2], two codes a byte, the lower half first, or
    with topk_ids [E, N, K / 2]; scales: [(E,) N, K / G], of x's type for integer codes
    (scale * (q - 8), or with zeros, uint8 of the same shape, scale * (q - zero)), uint8 exponents
    for e2m1 codes (2^(s - 127), G = 32); G is 32, 64 or 128.
    topk_ids: int32 or int64 [T, k]; out: [T, N], with topk_ids [T * k, N], a row a route (zeros
    where the id is none of an expert).  With an activation the first half of a matrix's rows is a
    gate, the second up, and out has N / 2 columns, act(gate) * up.  Up to 1024 rows of out, read
    again by the weights' passes for every 16 of a matrix or fewer, by K.  See include/moe_prep.h."""
    T, K = shape = x.shape
    dt, ws, sdt = x.dtype, weight.shape, scales.dtype
    E, k, idt = 0, 0, _INT32
    if topk_ids is not None:
        if len(ws) != 3:
            raise ValueError(f"weight: want [E, N, K / 2] with topk_ids, got {list(ws)}")
        E, k, idt = ws[0], topk_ids.shape[1], topk_ids.dtype
    elif len(ws) != 2:
        raise ValueError(f"weight: want [N, K / 2] without topk_ids, got {list(ws)}")
    N, groups = ws[-2], scales.shape[-1]
    if K % 2 or groups == 0 or K % groups:
        raise ValueError(f"scales: {groups} groups of {K} values")
    if sdt is not torch.uint8 and sdt is not dt:
        raise ValueError(f"scales: want {dt} or torch.uint8 exponents, got {sdt}")
    lead, rows = tuple(ws[:-1]), T * k if E else T
    _here(x, weight, scales, out, zeros, topk_ids, device_status)
    n_out = N if activation == MOE_ACT_NONE else N // 2
    _call("moe_w4_linear", W4LinearArgs.pack(
        T, K, N, E, k, K // groups, _code("x", dt),
        MOE_W4_E2M1 if sdt is torch.uint8 else MOE_W4_INT4, activation, x.data_ptr(),
        _rows("x", x, shape, dt), _flat("weight", weight, (*lead, K // 2), torch.uint8),
        _flat("scales", scales, (*lead, groups), sdt),
        _flat("zeros", zeros, (*lead, groups), torch.uint8),
        _flat("topk_ids", topk_ids, (T, k), idt), _code("topk_ids", idt, _IDS), out.data_ptr(),
        _rows("out", out, (rows, n_out), dt), _at(device_status)), stream)


class MoeLayer:
    """Device buffers of one batched MoE expert layer and the three calls.

    ``forward`` runs staging + dispatch, the batched experts and the top-k
    reduce on the current stream and returns the bf16 [T, K] output.
    """

    def __init__(self, T, K, N, E, top_k, M_max, w13, w13_s, w2, w2_s, device="cuda",
                 valid_shape_m=None, eplb=None, contiguous=False, fp32_scales=False):
        # contiguous: rows are packed per expert (expert_offsets); the buffers
        # hold E * ceil(T*k/E) rows, whatever the per-expert load
        if contiguous:
            M_max = max(1, -(-(T * top_k) // E))
        self.contiguous = contiguous
        # fp32_scales: 1x128 activation scales kept as fp32 (amax / 448) instead
        # of packed UE8M0 exponents
        self.sf_mode = MOE_SF_FP32 if fp32_scales else MOE_SF_UE8M0_PACKED
        self.T, self.K, self.N, self.E, self.top_k, self.M_max = T, K, N, E, top_k, M_max
        self.w13, self.w13_s, self.w2, self.w2_s = w13, w13_s, w2, w2_s
        self.eplb = eplb
        G = K // 128
        W = (G + 3) // 4
        dev = torch.device(device)
        u8 = dict(dtype=torch.uint8, device=dev)
        self.x = torch.empty((T, K), **u8)
        self.x_sf = (torch.empty((T, G), dtype=torch.float32, device=dev) if fp32_scales else
                     torch.empty((T, W), dtype=torch.int32, device=dev))
        self.ids_out = torch.empty((T, top_k), dtype=torch.int64, device=dev)
        self.w_out = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        self.x_b = torch.empty((E * M_max, K), **u8)
        self.sf_b = (torch.empty((E * M_max, G), dtype=torch.float32, device=dev) if fp32_scales
                     else torch.empty((E * M_max, W), dtype=torch.int32, device=dev))
        self.expert_num_tokens = torch.zeros(E, dtype=torch.int32, device=dev)
        self.route_slot = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        self.expert_offsets = (torch.zeros(E + 1, dtype=torch.int32, device=dev) if contiguous
                               else None)
        self.ws_prep = torch.empty(max(prepare_workspace_size(T, top_k, E), 256), **u8)
        self.valid_shape_m = valid_shape_m if valid_shape_m is not None else T * top_k
        self.ws13 = torch.empty(experts_workspace_size(E, M_max, K, N, self.valid_shape_m, 13), **u8)
        self.ws2 = torch.zeros(max(experts_workspace_size(E, M_max, K, N, self.valid_shape_m, 2),
                                   256), **u8)
        self.out_b = torch.empty((E, M_max, K), dtype=torch.bfloat16, device=dev)
        self.out = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def dispatch_args(self):
        return dict(num_experts=self.E, max_tokens_per_expert=self.M_max, x_b=self.x_b,
                    sf_b=self.sf_b, expert_num_tokens=self.expert_num_tokens,
                    route_slot=self.route_slot, workspace=self.ws_prep,
                    expert_offsets=self.expert_offsets)

    def prepare(self, hidden, topk_ids, topk_weights, is_padding=None, stream=None):
        moe_prepare_inputs(hidden, topk_ids, topk_weights, self.x, self.x_sf, self.ids_out,
                           self.w_out, is_padding=is_padding, sf_mode=self.sf_mode,
                           eplb=self.eplb, dispatch=self.dispatch_args(),
                           device_status=self.status, stream=stream)

    def experts(self, gate_up_dump=None, stream=None):
        moe_batched_experts(self.out_b, self.x_b, self.sf_b, self.w13, self.w13_s, self.w2,
                            self.w2_s, self.expert_num_tokens, self.ws13, self.ws2,
                            valid_shape_m=self.valid_shape_m, gate_up_dump=gate_up_dump,
                            device_status=self.status, stream=stream,
                            expert_offsets=self.expert_offsets)

    def reduce(self, stream=None):
        moe_topk_reduce(self.out_b, None if self.contiguous else self.ids_out, self.route_slot,
                        self.w_out, self.out, stream=stream)

    def forward(self, hidden, topk_ids, topk_weights, is_padding=None, stream=None):
        self.prepare(hidden, topk_ids, topk_weights, is_padding, stream)
        self.experts(stream=stream)
        self.reduce(stream=stream)
        return self.out

    def inter(self):
        """(inter_q, inter_sf) views of workspace13 as written by the w13 stage."""
        EM, N = self.E * self.M_max, self.N
        off = ((EM * N + 255) // 256) * 256
        Wy = (N // 128 + 3) // 4
        q = self.ws13[:EM * N].view(EM, N)
        sf = self.ws13[off:off + EM * Wy * 4].view(torch.int32).view(EM, Wy)
        return q, sf

    def forward_host(self, hidden_h, topk_ids_h, topk_weights_h, is_padding_h, out_h,
                     stream=None, chunks=None):
        """End-to-end call from pinned host buffers: copy the step's inputs to
        the device, run the three stages, copy the bf16 output back into
        ``out_h`` (pinned).  Nothing synchronises with the host.

        The reduce runs in token chunks (``chunks``; by default 4 from 1024
        tokens on, else 1), and each chunk's output rows go back to the host
        on a second stream while the next chunk is reduced (prefill: the
        output copy then costs 0.13 ms less).  The call's stream waits for the
        last copy, so work queued on it afterwards, or a synchronisation of
        it, sees ``out_h`` complete."""
        s = stream if stream is not None else torch.cuda.current_stream()
        if not hasattr(self, "_in_dev"):
            dev = self.x.device
            self._in_dev = (torch.empty(hidden_h.shape, dtype=hidden_h.dtype, device=dev),
                            torch.empty(topk_ids_h.shape, dtype=topk_ids_h.dtype, device=dev),
                            torch.empty(topk_weights_h.shape, dtype=topk_weights_h.dtype,
                                        device=dev),
                            None if is_padding_h is None else
                            torch.empty(is_padding_h.shape, dtype=is_padding_h.dtype, device=dev))
            self._copy_stream = torch.cuda.Stream(device=dev)
        h, i, w, p = self._in_dev
        with torch.cuda.stream(s):
            h.copy_(hidden_h, non_blocking=True)
            i.copy_(topk_ids_h, non_blocking=True)
            w.copy_(topk_weights_h, non_blocking=True)
            if p is not None:
                p.copy_(is_padding_h, non_blocking=True)
        self.prepare(h, i, w, p, stream=s)
        self.experts(stream=s)
        T = self.out.shape[0]
        n = chunks if chunks is not None else (4 if T >= 1024 else 1)
        n = max(1, min(n, T))
        if n == 1:
            self.reduce(stream=s)
            with torch.cuda.stream(s):
                out_h.copy_(self.out, non_blocking=True)
            return out_h
        cs = self._copy_stream
        idx = None if self.contiguous else self.ids_out
        bounds = [T * c // n for c in range(n + 1)]
        for c in range(n):
            t0, t1 = bounds[c], bounds[c + 1]
            moe_topk_reduce(self.out_b, None if idx is None else idx[t0:t1],
                            self.route_slot[t0:t1], self.w_out[t0:t1], self.out[t0:t1],
                            stream=s)
            cs.wait_stream(s)
            with torch.cuda.stream(cs):
                out_h[t0:t1].copy_(self.out[t0:t1], non_blocking=True)
        s.wait_stream(cs)
        return out_h
