// The norm before a block with its output in 8 bits:
//   x' = x + z,  y = x' rstd (w + offset),  q = e4m3(y / s),
// s of each 128 neighbouring columns by moe_prepare_inputs' recipe.
//
// A block of threads per row.  A thread has packs of 16 bytes, so 16 lanes (32 in fp32)
// have one group: its largest value is a matter of shuffles, and x' stays in registers
// between the row's sum and the rounding.  Bound by HBM, and not far from it by the some
// thirty instructions a value.  Measured, with z and y: 8192 x 7168 bf16 82 us, 6.4 TB/s;
// 2051 x 4096 fp16 with fp32 weights and scales, without y, 15 us; one row of 7168 2.7 us.
#include "block_norm.cuh"

namespace moe {

struct NormQuantParams {
  int64_t T, K;
  const void *x, *z, *w;
  int64_t x_stride, z_stride;
  int w_dtype;
  float offset, eps;
  void *x_out, *y;
  int64_t x_out_stride, y_stride;
  uint8_t* q;
  int64_t q_stride;
  void* sf;  // int32 words of four exponents, or fp32
  int64_t sf_stride;
  float* rstd;
};

// Scale of a group from its largest value: what the values are multiplied by, and the
// group's entry.
struct GroupScale {
  float inverse;
  uint32_t bits;  // the exponent's byte, or the fp32 scale
};
template <bool FP32>
__device__ __forceinline__ GroupScale group_scale(float amax) {
  if constexpr (FP32) {
    const float s = __fdiv_rn(fmaxf(amax, 1.0e-4f), 448.0f);
    return GroupScale{__frcp_rn(s), __float_as_uint(s)};
  } else {
    const uint32_t e = ue8m0_exponent(amax);
    return GroupScale{ue8m0_inverse(e), e};
  }
}

// The largest of three sizes; NaN is passed over.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Entry of group g of token t; the bytes that fill up the last word are zero.
template <bool FP32>
__device__ __forceinline__ void store_scale(const NormQuantParams& p, int64_t t, int g,
                                            uint32_t bits) {
  if constexpr (FP32) {
    (static_cast<uint32_t*>(p.sf) + t * p.sf_stride)[g] = bits;
  } else {
    uint8_t* row = reinterpret_cast<uint8_t*>(static_cast<uint32_t*>(p.sf) + t * p.sf_stride);
    row[g] = (uint8_t)bits;
    if (g == (int)((p.K + kGroup - 1) / kGroup) - 1)
      for (int e = g + 1; e % 4 != 0; ++e) row[e] = 0;
  }
}

// Rows of 16-byte packs, NV a thread: a block takes every gridDim.x-th row and has the next
// one's x and z on their way to shared memory while it works; the weights come there once.
// Each thread reads only packs that it copied.  With one STAGE the next row is copied over
// this one as soon as x' is in registers, with two from the row's start.
template <typename T, int NV, int STAGES, bool FP32>
__global__ void __launch_bounds__(512, NV == 1 ? 2 : (NV == 2 ? 3 : 1))
    norm_quant_rows_kernel(NormQuantParams p) {
  constexpr int VEC = 16 / sizeof(T), H = VEC / 2, LANES = kGroup / VEC;
  using P = Pack<T, VEC>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float part[2][32];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int packs = (int)(p.K / VEC), w_dtype = p.w_dtype;
  const float inv_k = 1.0f / (float)p.K;
  P* stage0 = reinterpret_cast<P*>(smem);
  const int stage_packs = (1 + (p.z != nullptr)) * packs;
  uint8_t* s_w = smem + (size_t)STAGES * stage_packs * 16;
  pdl_wait();
  pdl_launch_dependents();
  auto fetch = [&](int64_t t, int s) {
    if (t < p.T) {
      P* dst = stage0 + s * stage_packs;
      const T* x = static_cast<const T*>(p.x) + t * p.x_stride;
      const T* z = static_cast<const T*>(p.z) + t * p.z_stride;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + i * threads;
        if (c >= packs) break;
        copy16(dst + c, x + c * VEC);
        if (p.z != nullptr) copy16(dst + packs + c, z + c * VEC);
      }
    }
  };
  fetch(blockIdx.x, 0);
  fetch_weights<VEC, NV>(s_w, p.w, w_dtype, packs);
  copies_commit();
  const float2 offset = both(p.offset);
  int it = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, it ^= 1) {
    if (STAGES == 2) {
      fetch(t + gridDim.x, it ^ 1);
      copies_commit();
    }
    copies_wait<STAGES - 1>();
    const P* st = STAGES == 2 ? stage0 + it * stage_packs : stage0;
    float2 v[NV][H];
    float2 ss = both(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * threads;
      if (c >= packs) {
#pragma unroll
        for (int h = 0; h < H; ++h) v[i][h] = both(0.0f);
        continue;
      }
      const P x = st[c];
#pragma unroll
      for (int h = 0; h < H; ++h) v[i][h] = x.get2(h);
      if (p.z != nullptr) {
        const P z = st[packs + c];
        P o;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          v[i][h] = add2(v[i][h], z.get2(h));
          o.set2(h, v[i][h]);
        }
        store_pack<T, VEC>(static_cast<T*>(p.x_out) + t * p.x_out_stride + c * VEC, o);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) ss = fma2(v[i][h], v[i][h], ss);
    }
    if (STAGES == 1) {
      fetch(t + gridDim.x, 0);
      copies_commit();
    }
    const float r = rsqrtf(fmaf(block_sum(ss.x + ss.y, part[it]), inv_k, p.eps));
    if (tid == 0 && p.rstd != nullptr) p.rstd[t] = r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * threads;
      const bool live = c < packs;
      if (i * threads + (tid & ~31) >= packs) break;  // the same in a whole warp
      float amax = 0.0f;
      if (live) {
        float2 w[H];
        read_weights<VEC>(s_w, w_dtype, c, packs, w);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          v[i][h] = mul2(mul2(v[i][h], both(r)), add2(w[h], offset));
          amax = max3_abs(amax, v[i][h].x, v[i][h].y);
        }
      }
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
      const GroupScale s = group_scale<FP32>(amax);
      if (!live) continue;
      if (tid % LANES == 0) store_scale<FP32>(p, t, c / LANES, s.bits);
      if (p.y != nullptr) {
        P o;
#pragma unroll
        for (int h = 0; h < H; ++h) o.set2(h, v[i][h]);
        store_pack<T, VEC>(static_cast<T*>(p.y) + t * p.y_stride + c * VEC, o);
      }
      uint32_t q[VEC / 4];
#pragma unroll
      for (int h = 0; h < H; h += 2) {
        const float2 a = mul2(v[i][h], both(s.inverse)), b = mul2(v[i][h + 1], both(s.inverse));
        q[h / 2] = pack4_e4m3(a.x, a.y, b.x, b.y);
      }
      uint8_t* dst = p.q + t * p.q_stride + c * VEC;
      if constexpr (VEC == 8)
        *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
      else
        *reinterpret_cast<uint32_t*>(dst) = q[0];
    }
  }
  copies_wait<0>();
}

// Any other rows: a warp has a group, four columns a lane, in a second pass over the
// row, which computes x' again.  A lane stores only columns that it has itself read, so
// that x_out may be x or z.
template <typename T, bool FP32>
__global__ void __launch_bounds__(512) norm_quant_kernel(NormQuantParams p) {
  __shared__ float part[2][32];
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
  const int K = (int)p.K;
  pdl_wait();
  pdl_launch_dependents();
  int it = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, it ^= 1) {
    const T* xr = static_cast<const T*>(p.x) + t * p.x_stride;
    const T* zr = static_cast<const T*>(p.z) + t * p.z_stride;
    auto x_next = [&](int c) {
      return p.z != nullptr ? to_f32(xr[c]) + to_f32(zr[c]) : to_f32(xr[c]);
    };
    float ss = 0.0f;
    for (int c = tid; c < K; c += threads) {
      const float x = x_next(c);
      ss = fmaf(x, x, ss);
    }
    const float r = rsqrtf(block_sum(ss, part[it]) / (float)K + p.eps);
    if (tid == 0 && p.rstd != nullptr) p.rstd[t] = r;
    for (int g = tid >> 5; g * kGroup < K; g += threads >> 5) {
      float x[4], y[4], amax = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = g * kGroup + e * 32 + lane;
        x[e] = y[e] = 0.0f;
        if (c < K) {
          float w[1];
          load_weights<1>(p.w, p.w_dtype, c, p.offset, w);
          x[e] = x_next(c);
          y[e] = x[e] * r * w[0];
        }
        amax = fmaxf(amax, fabsf(y[e]));
      }
      const GroupScale s = group_scale<FP32>(warp_max(amax));
      if (lane == 0) store_scale<FP32>(p, t, g, s.bits);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = g * kGroup + e * 32 + lane;
        if (c >= K) break;
        if (p.z != nullptr) (static_cast<T*>(p.x_out) + t * p.x_out_stride)[c] = from_f32<T>(x[e]);
        if (p.y != nullptr) (static_cast<T*>(p.y) + t * p.y_stride)[c] = from_f32<T>(y[e]);
        (p.q + t * p.q_stride)[c] = (uint8_t)e4m3x2(y[e] * s.inverse, 0.0f);
      }
    }
  }
}

}  // namespace moe

namespace moe_host {

using moe::NormQuantParams;

static size_t quant_rows_smem(const NormQuantParams& p, size_t elem, int stages) {
  return (size_t)p.K * (stages * (1 + (p.z != nullptr)) * elem + dtype_size(p.w_dtype));
}

template <typename E, int NV, int STAGES, bool FP32>
static moe_status_t launch_quant_rows(const NormQuantParams& p, int threads, cudaStream_t s) {
  constexpr auto kernel = moe::norm_quant_rows_kernel<E, NV, STAGES, FP32>;
  const size_t smem = quant_rows_smem(p, sizeof(E), STAGES);
  const int64_t cap = (int64_t)num_sms() * resident_with<kernel>(threads, smem);
  if (cap == 0) return set_error(MOE_ERR_CUDA, "norm quant: no resident block");
  return launched(launch_pdl(kernel, dim3((unsigned)(p.T < cap ? p.T : cap)), dim3(threads), smem, s, p),
                  "norm quant");
}

template <typename E, bool FP32>
static moe_status_t run_norm_quant(const NormQuantParams& p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(E);
  Wide w{p.T, sizeof(E)};
  w.ok = p.K % V == 0;
  w.rows(p.x, p.x_stride);
  w.rows(p.z, p.z_stride);
  w.rows(p.x_out, p.x_out_stride);
  w.rows(p.y, p.y_stride);
  w.weights(p.w);
  w.ok = w.ok && reinterpret_cast<uintptr_t>(p.q) % V == 0 && (p.T <= 1 || p.q_stride % V == 0);
  if (!w.ok) {
    constexpr auto kernel = moe::norm_quant_kernel<E, FP32>;
    const int64_t groups = (p.K + moe::kGroup - 1) / moe::kGroup;
    const int threads = (int)(groups < 16 ? groups : 16) * 32;
    const int64_t cap =
        (int64_t)num_sms() * resident_blocks(reinterpret_cast<const void*>(kernel), threads);
    return launched(launch_pdl(kernel, dim3((unsigned)(p.T < cap ? p.T : cap)), dim3(threads), 0, s, p),
                    "norm quant");
  }
  const int64_t packs = p.K / V;
  auto threads = [&](int nv) { return (int)(((packs + nv - 1) / nv + 31) / 32 * 32); };
  // One pack a thread up to 512, in two stages (8192 x 4096 52 us; two packs 56, four 54).
  // Above, four packs a thread and one stage, so that more blocks of fewer threads share an
  // SM and fewer warps wait at a row's barrier (8192 x 7168 82 us, two packs 94; 4000 x 7168
  // fp32 76 us, two stages 82); with a row for each SM or less two packs, the shorter way
  // through one row (40 x 7168 2.8 us, four packs 3.2).
  if (packs <= 512) return launch_quant_rows<E, 1, 2, FP32>(p, threads(1), s);
  if (packs <= 1024 && p.T <= num_sms()) return launch_quant_rows<E, 2, 1, FP32>(p, threads(2), s);
  if (packs <= 2048) return launch_quant_rows<E, 4, 1, FP32>(p, threads(4), s);
  if constexpr (sizeof(E) == 4) return launch_quant_rows<E, 8, 1, FP32>(p, threads(8), s);
  return set_error(MOE_ERR_UNSUPPORTED, "hidden_size too large");  // not reached: K <= 16384
}

}  // namespace moe_host

using namespace moe_host;

extern "C" {

moe_status_t moe_norm_quant(const moe_norm_quant_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t T = a->num_tokens, K = a->hidden_size;
  moe_status_t st = check_norm(T, K, a->dtype, a->weight_dtype, MOE_GATE_NONE);
  if (st != MOE_OK) return st;
  if (a->sf_mode != MOE_SF_UE8M0_PACKED && a->sf_mode != MOE_SF_FP32)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "bad sf_mode %d", a->sf_mode);
  if (T == 0 || K == 0) return MOE_OK;
  if ((a->z != nullptr) != (a->x_out != nullptr))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "x_out must be given iff z is");
  if (!a->x || !a->weight || !a->q || !a->q_sf)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  const int64_t groups = (K + moe::kGroup - 1) / moe::kGroup;
  const bool fp32 = a->sf_mode == MOE_SF_FP32;
  if (T > 1 && (a->x_stride0 < K || (a->z && (a->z_stride0 < K || a->x_out_stride0 < K)) ||
                (a->y && a->y_stride0 < K) || a->q_stride0 < K ||
                a->q_sf_stride0 < (fp32 ? groups : (groups + 3) / 4)))
    return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
  NormQuantParams p{};
  p.T = T;
  p.K = K;
  p.x = a->x;
  p.x_stride = a->x_stride0;
  p.z = a->z;
  p.z_stride = a->z_stride0;
  p.w = a->weight;
  p.w_dtype = a->weight_dtype;
  p.offset = a->weight_offset;
  p.eps = a->eps;
  p.x_out = a->x_out;
  p.x_out_stride = a->x_out_stride0;
  p.y = a->y;
  p.y_stride = a->y_stride0;
  p.q = static_cast<uint8_t*>(a->q);
  p.q_stride = a->q_stride0;
  p.sf = a->q_sf;
  p.sf_stride = a->q_sf_stride0;
  p.rstd = a->rstd;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return with_dtype(a->dtype, [&](auto v) {
    using E = decltype(v);
    return fp32 ? run_norm_quant<E, true>(p, s) : run_norm_quant<E, false>(p, s);
  });
}

}  // extern "C"
