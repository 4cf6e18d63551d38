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

// Two 16-bit values of a word (the lower first) as floats, and back.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float2 f);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float2 f) {
  const __nv_bfloat162 h = __float22bfloat162_rn(f);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float2 f) {
  const __half2 h = __float22half2_rn(f);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// VEC consecutive elements of T as they lie in memory: 16 bytes as four words,
// or one element where rows do not start on 16-byte boundaries.
template <typename T, int VEC>
struct Pack {
  static_assert(VEC * sizeof(T) == 16, "16 bytes");
  uint4 w;
  __device__ __forceinline__ uint32_t word(int i) const {
    return i == 0 ? w.x : (i == 1 ? w.y : (i == 2 ? w.z : w.w));
  }
  __device__ __forceinline__ void set_word(int i, uint32_t v) {
    (i == 0 ? w.x : (i == 1 ? w.y : (i == 2 ? w.z : w.w))) = v;
  }
  // elements 2 q and 2 q + 1
  __device__ __forceinline__ float2 get2(int q) const {
    if constexpr (sizeof(T) == 4)
      return make_float2(__uint_as_float(word(2 * q)), __uint_as_float(word(2 * q + 1)));
    else
      return unpack2<T>(word(q));
  }
  __device__ __forceinline__ void set2(int q, float2 f) {
    if constexpr (sizeof(T) == 4) {
      set_word(2 * q, __float_as_uint(f.x));
      set_word(2 * q + 1, __float_as_uint(f.y));
    } else {
      set_word(q, pack2<T>(f));
    }
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
#pragma unroll
    for (int q = 0; q < VEC / 2; ++q) {
      const float2 v = get2(q);
      f[2 * q] = v.x, f[2 * q + 1] = v.y;
    }
  }
  __device__ __forceinline__ void set(const float (&f)[VEC]) {
#pragma unroll
    for (int q = 0; q < VEC / 2; ++q) set2(q, make_float2(f[2 * q], f[2 * q + 1]));
  }
};
template <typename T>
struct Pack<T, 1> {
  T v;
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f32(v); }
  __device__ __forceinline__ void set(const float (&f)[1]) { v = from_f32<T>(f[0]); }
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* p) {
  Pack<T, VEC> r;
  if constexpr (VEC == 1)
    r.v = *p;
  else
    r.w = *reinterpret_cast<const uint4*>(p);
  return r;
}

// As load_pack, for data that this kernel reads once.
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack_stream(const T* p) {
  Pack<T, VEC> r;
  if constexpr (VEC == 1)
    r.v = *p;
  else
    r.w = ld_stream_v4(p);
  return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, VEC>& r) {
  if constexpr (VEC == 1)
    *p = r.v;
  else
    st_v4(p, r.w);
}

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> zero_pack() {
  Pack<T, VEC> r;
  if constexpr (VEC == 1)
    r.v = from_f32<T>(0.0f);
  else
    r.w = make_uint4(0, 0, 0, 0);
  return r;
}

// Arithmetic in pairs (fma.rn.f32x2 and its like).
__device__ __forceinline__ float2 both(float f) { return make_float2(f, f); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

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
