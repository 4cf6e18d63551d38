// What the forward and the gradient of moe_block_norm share.
#pragma once

#include <mutex>

#include "block_common.cuh"

namespace moe {

struct NormParams {
  int64_t T, K;
  const void *x, *z, *gate, *post_w, *pre_w;
  int64_t x_stride, z_stride, gate_stride;
  int w_dtype, gate_kind;
  float scale, offset, eps;
  void *x_out, *y;
  int64_t x_out_stride, y_stride;
  float *rstd_post, *rstd_pre;
  // gradient
  const float *rz, *rx;
  const void *d_x_out, *d_y;
  int64_t d_x_out_stride, d_y_stride;
  void *d_x, *d_z, *d_gate, *d_post_w, *d_pre_w;
  int64_t d_x_stride, d_z_stride, d_gate_stride;
  float4* row_sums;  // [T]
  float* partials;   // [row blocks][3][K]: dwq, dwp, dg
  int rows_per_block, row_blocks;
};

// VEC weights of a [K] tensor of any of the three types, plus offset.
template <int VEC>
__device__ __forceinline__ void load_weights(const void* w, int dtype, int64_t c, float offset,
                                             float (&o)[VEC]) {
  if (dtype == MOE_DTYPE_FP32) {
    const float* p = static_cast<const float*>(w) + c;
    if constexpr (VEC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
        o[i] = v.x, o[i + 1] = v.y, o[i + 2] = v.z, o[i + 3] = v.w;
      }
    } else {
      o[0] = __ldg(p);
    }
  } else {
    uint32_t u[(VEC + 1) / 2];
    const uint16_t* p = static_cast<const uint16_t*>(w) + c;
    if constexpr (VEC == 8) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
    } else if constexpr (VEC == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      u[0] = v.x, u[1] = v.y;
    } else {
      u[0] = __ldg(p);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const uint16_t h = (uint16_t)(u[i / 2] >> (16 * (i & 1)));
      o[i] = dtype == MOE_DTYPE_BF16 ? bf16_bits_to_f32(h) : __half2float(__ushort_as_half(h));
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] += offset;
}

template <int VEC>
__device__ __forceinline__ void load_weights_or_one(const void* w, int dtype, int64_t c,
                                                    float offset, float (&o)[VEC]) {
  if (w != nullptr) {
    load_weights<VEC>(w, dtype, c, offset, o);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = 1.0f;
  }
}

// A token's own gate, 1 for the other kinds.
template <typename T>
__device__ __forceinline__ float token_factor(const NormParams& p, int64_t t) {
  return p.gate_kind == MOE_GATE_TOKEN
             ? to_f32(static_cast<const T*>(p.gate)[t * p.gate_stride])
             : 1.0f;
}

// Gate of VEC columns (1 without a channel or full gate).
template <typename T, int VEC>
__device__ __forceinline__ void load_gate(const NormParams& p, int64_t t, int64_t c,
                                          float (&g)[VEC]) {
  if (p.gate_kind == MOE_GATE_CHANNEL) {
    load_weights<VEC>(p.gate, p.w_dtype, c, 0.0f, g);
  } else if (p.gate_kind == MOE_GATE_FULL) {
    load_pack<T, VEC>(static_cast<const T*>(p.gate) + t * p.gate_stride + c).get(g);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = 1.0f;
  }
}

// Sum over the block, given to every thread; `part` holds 32 floats and is
// free again after the caller's next barrier.
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < (int)(blockDim.x >> 5) ? part[lane] : 0.0f);
}

// 16-byte asynchronous copies to shared memory.  In the kernels that use them
// every thread copies exactly the packs that it reads itself, so waiting for its
// own copies is enough and rows ahead cost neither registers nor barriers.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// VEC weights of a pack as they lie in shared memory, in their own type; fp32 ones
// four a plane, so that neighbouring threads read neighbouring 16 bytes.
template <int VEC>
__device__ __forceinline__ void read_weights(const uint8_t* s, int dtype, int c, int packs,
                                             float2 (&w)[VEC / 2]) {
  if (dtype == MOE_DTYPE_FP32) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(s + ((size_t)i * packs + c) * 16);
      w[2 * i] = make_float2(v.x, v.y), w[2 * i + 1] = make_float2(v.z, v.w);
    }
    return;
  }
  uint32_t u[VEC / 2];
  if constexpr (VEC == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(s + (size_t)c * 16);
    u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(s + (size_t)c * 8);
    u[0] = v.x, u[1] = v.y;
  }
  if (dtype == MOE_DTYPE_BF16) {
#pragma unroll
    for (int q = 0; q < VEC / 2; ++q) w[q] = unpack2<__nv_bfloat16>(u[q]);
  } else {
#pragma unroll
    for (int q = 0; q < VEC / 2; ++q) w[q] = unpack2<__half>(u[q]);
  }
}

// Copies a thread's packs of a [K] tensor to shared memory.
template <int VEC, int NV>
__device__ __forceinline__ void fetch_weights(uint8_t* dst, const void* src, int dtype, int packs) {
  const int bytes = VEC * (dtype == MOE_DTYPE_FP32 ? 4 : 2);  // of a pack: 8, 16 or 32
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c >= packs) break;
    const size_t o = (size_t)c * bytes;
    const uint8_t* g = static_cast<const uint8_t*>(src) + o;
    if (bytes == 8) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(
                       (uint32_t)__cvta_generic_to_shared(dst + o)),
                   "l"(g)
                   : "memory");
    } else {
      copy16(dst + (size_t)c * 16, g);
      if (bytes == 32) copy16(dst + (size_t)(packs + c) * 16, g + 16);
    }
  }
}

}  // namespace moe

namespace moe_host {

constexpr int64_t kMaxHidden = 16384;
constexpr size_t kMaxBlockSmem = 232448 - 2048;  // dynamic, beside the static part

// Resident blocks an SM of a kernel with dynamic shared memory; its limit is
// raised to what one block may have.  Kept per device, block and size.
template <auto Kernel>
int resident_with(int threads, size_t smem) {
  static std::mutex mu;
  struct Entry {
    int dev, threads, blocks;
    size_t smem;
  };
  static Entry table[64];
  static int used = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < used; ++i)
    if (table[i].dev == dev && table[i].threads == threads && table[i].smem == smem)
      return table[i].blocks;
  int n = 0;
  if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kMaxBlockSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, Kernel, threads, smem) != cudaSuccess)
    return 0;
  if (used < 64) table[used++] = Entry{dev, threads, n, smem};
  return n;
}

inline moe_status_t check_norm(int64_t T, int64_t K, int32_t dtype, int32_t wdtype, int32_t gate) {
  if (T < 0 || K < 0) return set_error(MOE_ERR_INVALID_ARGUMENT, "negative size");
  if (!dtype_ok(dtype) || !dtype_ok(wdtype))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "bad dtype %d or weight_dtype %d", dtype, wdtype);
  if (gate < MOE_GATE_NONE || gate > MOE_GATE_FULL)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "bad gate_kind %d", gate);
  if (K > kMaxHidden)
    return set_error(MOE_ERR_UNSUPPORTED, "hidden_size %lld above %lld", (long long)K,
                     (long long)kMaxHidden);
  if (T >= ((int64_t)1 << 31)) return set_error(MOE_ERR_UNSUPPORTED, "too many tokens");
  return MOE_OK;
}

// Whether rows and weights may be read 16 bytes at a time.
struct Wide {
  int64_t T;
  size_t elem;
  bool ok = true;
  void rows(const void* q, int64_t stride) { ok = ok && rows_aligned16(q, stride, elem, T); }
  void weights(const void* q) { ok = ok && (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }
};

}  // namespace moe_host
