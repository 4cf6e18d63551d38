// Typed loads, stores and reductions of the operators around the experts.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// VEC consecutive elements of T held as raw bits: 16 bytes, or one element
// where rows do not start on 16-byte boundaries.
template <typename T, int VEC>
struct Pack {
  static_assert(VEC == 1 || VEC * sizeof(T) == 16, "one element or 16 bytes");
  T v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* p) {
  Pack<T, VEC> r;
  if constexpr (VEC == 1) {
    r.v[0] = *p;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    memcpy(r.v, &u, 16);
  }
  return r;
}

// As load_pack, for data that this kernel reads once.
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack_stream(const T* p) {
  Pack<T, VEC> r;
  if constexpr (VEC == 1) {
    r.v[0] = *p;
  } else {
    const uint4 u = ld_stream_v4(p);
    memcpy(r.v, &u, 16);
  }
  return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, VEC>& r) {
  if constexpr (VEC == 1) {
    *p = r.v[0];
  } else {
    uint4 u;
    memcpy(&u, r.v, 16);
    st_v4(p, u);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> zero_pack() {
  Pack<T, VEC> r;
#pragma unroll
  for (int i = 0; i < VEC; ++i) r.v[i] = from_f32<T>(0.0f);
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

}  // namespace moe

namespace moe_host {

inline void clear_error() { set_error(MOE_OK, "%s", ""); }
inline size_t dtype_size(int32_t dtype) { return dtype == MOE_DTYPE_FP32 ? 4 : 2; }
inline bool dtype_ok(int32_t dtype) {
  return dtype == MOE_DTYPE_FP32 || dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_FP16;
}

// Whether rows of a tensor start on 16-byte boundaries (rows == 1 ignores the stride).
inline bool rows_aligned16(const void* p, int64_t stride0, size_t elem, int64_t rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 &&
         (rows <= 1 || (stride0 * (int64_t)elem) % 16 == 0);
}

// Calls f with a value of the element type of `dtype`.
template <typename F>
moe_status_t with_dtype(int32_t dtype, F&& f) {
  switch (dtype) {
    case MOE_DTYPE_FP32: return f(float{});
    case MOE_DTYPE_BF16: return f(__nv_bfloat16{});
    default: return f(__half{});
  }
}

inline moe_status_t launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return MOE_OK;
}

}  // namespace moe_host
