// The seam between two blocks: RMS norm of the block's output, gate, residual
// scale and sum, and the RMS norm before the next block; and its gradient.
//
//   n = z rz wp,  x' = x + s g n,  y = x' rx wq      (rz, rx: inverse RMS)
//
// Forward: one block of threads per row, the row in registers, so x and z are
// read once and x' and y written once; two sums over the row, one after the
// other, since x' needs rz.  Bound by HBM.
//
// Backward, with xh = x' rx, zh = z rz, u = dy wq, mean over the row:
//   d = dx' + rx (u - xh mean(u xh))                  (= dx)
//   dz = rz (v - zh mean(v zh)),  v = s g wp d
//   dwq = sum_t dy xh,  dwp = sum_t s g d zh,  dg = s d n (summed as the gate is)
// mean(v zh) is linear in d, so with a = g n the row needs only the sums of
// u xh, a (dx' + rx u) and a xh, all from one reading.
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
  // backward
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

__device__ __forceinline__ void store_weight(void* w, int dtype, int64_t c, float v) {
  if (dtype == MOE_DTYPE_FP32)
    static_cast<float*>(w)[c] = v;
  else if (dtype == MOE_DTYPE_BF16)
    static_cast<__nv_bfloat16*>(w)[c] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(w)[c] = __float2half_rn(v);
}

// Sum over the block, given to every thread; `part` holds 32 floats and is
// free again after the next barrier of the caller.
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < (int)(blockDim.x >> 5) ? part[lane] : 0.0f);
}

// The branch's factor of a token (residual scale, and a token's own gate).
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
    const Pack<T, VEC> v =
        load_pack<T, VEC>(static_cast<const T*>(p.gate) + t * p.gate_stride + c);
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = to_f32(v.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = 1.0f;
  }
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

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(512) block_norm_kernel(NormParams p) {
  __shared__ float part[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t stride = (int64_t)blockDim.x * VEC;
  const int64_t c0 = (int64_t)threadIdx.x * VEC;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    Pack<T, VEC> xv[NV], zv[NV];
    const T* xr = static_cast<const T*>(p.x) + t * p.x_stride;
    const T* zr = static_cast<const T*>(p.z) + t * p.z_stride;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = c0 + i * stride;
      if (c < p.K) {
        if (p.z != nullptr) zv[i] = load_pack_stream<T, VEC>(zr + c);
        xv[i] = load_pack<T, VEC>(xr + c);
      }
    }
    float rz = 1.0f;
    if (p.post_w != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (c0 + i * stride < p.K)
#pragma unroll
          for (int q = 0; q < VEC; ++q) ss = fmaf(to_f32(zv[i].v[q]), to_f32(zv[i].v[q]), ss);
      rz = rsqrtf(block_sum(ss, part[0]) / (float)p.K + p.eps);
      if (threadIdx.x == 0 && p.rstd_post != nullptr) p.rstd_post[t] = rz;
    }
    const float branch = p.z != nullptr ? p.scale * token_factor<T>(p, t) : 0.0f;
    float xo[NV][VEC];
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = c0 + i * stride;
      if (c >= p.K) continue;
#pragma unroll
      for (int q = 0; q < VEC; ++q) xo[i][q] = to_f32(xv[i].v[q]);
      if (p.z != nullptr) {
        float w[VEC], g[VEC];
        load_weights_or_one<VEC>(p.post_w, p.w_dtype, c, p.offset, w);
        load_gate<T, VEC>(p, t, c, g);
        Pack<T, VEC> o;
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
          xo[i][q] = fmaf(branch, g[q] * (to_f32(zv[i].v[q]) * rz * w[q]), xo[i][q]);
          o.v[q] = from_f32<T>(xo[i][q]);
        }
        store_pack<T, VEC>(static_cast<T*>(p.x_out) + t * p.x_out_stride + c, o);
      }
#pragma unroll
      for (int q = 0; q < VEC; ++q) ss = fmaf(xo[i][q], xo[i][q], ss);
    }
    if (p.pre_w != nullptr) {
      const float rx = rsqrtf(block_sum(ss, part[1]) / (float)p.K + p.eps);
      if (threadIdx.x == 0 && p.rstd_pre != nullptr) p.rstd_pre[t] = rx;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t c = c0 + i * stride;
        if (c >= p.K) continue;
        float w[VEC];
        load_weights<VEC>(p.pre_w, p.w_dtype, c, p.offset, w);
        Pack<T, VEC> o;
#pragma unroll
        for (int q = 0; q < VEC; ++q) o.v[q] = from_f32<T>(xo[i][q] * rx * w[q]);
        store_pack<T, VEC>(static_cast<T*>(p.y) + t * p.y_stride + c, o);
      }
    }
    __syncthreads();  // both parts are free for the next row
  }
}

// What the gradient needs of VEC columns of a row.
template <int VEC>
struct BackCols {
  float xh[VEC];  // x' rx
  float zh[VEC];  // z rz
  float n[VEC];   // z rz wp
  float g[VEC];   // channel or full gate
  float wp[VEC];
  float u[VEC];   // dy wq
  float dy[VEC];
  float e[VEC];   // dx' + rx u
};

template <typename T, int VEC>
__device__ __forceinline__ void back_columns(const NormParams& p, int64_t t, int64_t c, float rz,
                                             float rx, float branch, BackCols<VEC>& b) {
  const Pack<T, VEC> xv =
      load_pack<T, VEC>(static_cast<const T*>(p.x) + t * p.x_stride + c);
  Pack<T, VEC> zv = zero_pack<T, VEC>(), dxv = zv, dyv = zv;
  if (p.z != nullptr) zv = load_pack<T, VEC>(static_cast<const T*>(p.z) + t * p.z_stride + c);
  if (p.d_x_out != nullptr)
    dxv = load_pack<T, VEC>(static_cast<const T*>(p.d_x_out) + t * p.d_x_out_stride + c);
  if (p.d_y != nullptr)
    dyv = load_pack<T, VEC>(static_cast<const T*>(p.d_y) + t * p.d_y_stride + c);
  float wq[VEC];
  load_gate<T, VEC>(p, t, c, b.g);
  load_weights_or_one<VEC>(p.post_w, p.w_dtype, c, p.offset, b.wp);
  load_weights_or_one<VEC>(p.pre_w, p.w_dtype, c, p.offset, wq);
#pragma unroll
  for (int q = 0; q < VEC; ++q) {
    b.zh[q] = to_f32(zv.v[q]) * rz;
    b.n[q] = b.zh[q] * b.wp[q];
    b.xh[q] = fmaf(branch, b.g[q] * b.n[q], to_f32(xv.v[q])) * rx;
    b.dy[q] = to_f32(dyv.v[q]);
    b.u[q] = b.dy[q] * wq[q];
    b.e[q] = fmaf(rx, b.u[q], to_f32(dxv.v[q]));
  }
}

// First launch: the row's three sums.  row_sums[t] = (mean(u xh), sum a e,
// sum a xh, 0) with a = g n over channel or full gates.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) block_norm_sums_kernel(NormParams p) {
  __shared__ float part[3][32];
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const float rz = p.post_w != nullptr ? p.rz[t] : 1.0f;
    const float rx = p.pre_w != nullptr ? p.rx[t] : 0.0f;
    const float branch = p.z != nullptr ? p.scale * token_factor<T>(p, t) : 0.0f;
    float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < p.K; c += (int64_t)blockDim.x * VEC) {
      BackCols<VEC> b;
      back_columns<T, VEC>(p, t, c, rz, rx, branch, b);
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        const float a = b.g[q] * b.n[q];
        s0 = fmaf(b.u[q], b.xh[q], s0);
        s1 = fmaf(a, b.e[q], s1);
        s2 = fmaf(a, b.xh[q], s2);
      }
    }
    s0 = block_sum(s0, part[0]);
    s1 = block_sum(s1, part[1]);
    s2 = block_sum(s2, part[2]);
    if (threadIdx.x == 0) p.row_sums[t] = make_float4(s0 / (float)p.K, s1, s2, 0.0f);
    __syncthreads();
  }
}

// Second launch: gradients of the rows, and each row block's column sums.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) block_norm_apply_kernel(NormParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t c = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * VEC;
  if (c >= p.K) return;
  const int64_t t0 = (int64_t)blockIdx.y * p.rows_per_block;
  const int64_t t1 = min(p.T, t0 + p.rows_per_block);
  float dwq[VEC], dwp[VEC], dg[VEC];
#pragma unroll
  for (int q = 0; q < VEC; ++q) dwq[q] = dwp[q] = dg[q] = 0.0f;
  for (int64_t t = t0; t < t1; ++t) {
    const float rz = p.post_w != nullptr ? p.rz[t] : 1.0f;
    const float rx = p.pre_w != nullptr ? p.rx[t] : 0.0f;
    const float tg = token_factor<T>(p, t);
    const float branch = p.z != nullptr ? p.scale * tg : 0.0f;
    const float4 s = p.row_sums[t];
    const float dot = s.y - rx * s.x * s.z;  // sum over the row of g n d
    const float c2 = p.post_w != nullptr ? branch * dot / (float)p.K : 0.0f;  // mean(v zh)
    if (p.gate_kind == MOE_GATE_TOKEN && p.d_gate != nullptr && c == 0)
      static_cast<T*>(p.d_gate)[t * p.d_gate_stride] = from_f32<T>(p.scale * dot);
    BackCols<VEC> b;
    back_columns<T, VEC>(p, t, c, rz, rx, branch, b);
    Pack<T, VEC> ox, oz, og;
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      const float d = fmaf(-rx * s.x, b.xh[q], b.e[q]);
      const float bg = branch * b.g[q];
      ox.v[q] = from_f32<T>(d);
      oz.v[q] = from_f32<T>(rz * (bg * b.wp[q] * d - b.zh[q] * c2));
      const float gd = p.scale * (d * b.n[q]);
      og.v[q] = from_f32<T>(gd);
      dwq[q] = fmaf(b.dy[q], b.xh[q], dwq[q]);
      dwp[q] = fmaf(bg * d, b.zh[q], dwp[q]);
      dg[q] += gd;
    }
    store_pack<T, VEC>(static_cast<T*>(p.d_x) + t * p.d_x_stride + c, ox);
    if (p.d_z != nullptr)
      store_pack<T, VEC>(static_cast<T*>(p.d_z) + t * p.d_z_stride + c, oz);
    if (p.gate_kind == MOE_GATE_FULL && p.d_gate != nullptr)
      store_pack<T, VEC>(static_cast<T*>(p.d_gate) + t * p.d_gate_stride + c, og);
  }
  float* out = p.partials + (int64_t)blockIdx.y * 3 * p.K + c;
  const bool want[3] = {p.d_pre_w != nullptr, p.d_post_w != nullptr,
                        p.d_gate != nullptr && p.gate_kind == MOE_GATE_CHANNEL};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (!want[k]) continue;
#pragma unroll
    for (int q = 0; q < VEC; ++q) out[k * p.K + q] = k == 0 ? dwq[q] : (k == 1 ? dwp[q] : dg[q]);
  }
}

// Third launch: column sums over the row blocks, in their order: 32 columns by
// 8 interleaved shares of the row blocks, joined in shared memory.
__global__ void __launch_bounds__(256) block_norm_columns_kernel(NormParams p) {
  __shared__ float part[8][33];
  pdl_wait();
  pdl_launch_dependents();
  const int col = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + col;
  const int k = blockIdx.y;
  void* out = k == 0 ? p.d_pre_w : (k == 1 ? p.d_post_w : p.d_gate);
  if (out == nullptr || (k == 2 && p.gate_kind != MOE_GATE_CHANNEL)) return;
  float sum = 0.0f;
  if (c < p.K)
    for (int b = share; b < p.row_blocks; b += 8) sum += p.partials[((int64_t)b * 3 + k) * p.K + c];
  part[share][col] = sum;
  __syncthreads();
  if (share == 0 && c < p.K) {
    for (int i = 1; i < 8; ++i) sum += part[i][col];
    store_weight(out, p.w_dtype, c, sum);
  }
}

}  // namespace moe

namespace moe_host {

using moe::NormParams;

constexpr int64_t kMaxHidden = 16384;

// Row blocks of the second launch: at least eight rows each, at most 512.
static int64_t norm_row_blocks(int64_t T) {
  int64_t n = (T + 7) / 8;
  return n > 512 ? 512 : (n < 1 ? 1 : n);
}

static size_t norm_workspace(int64_t T, int64_t K) {
  return (size_t)(T * 16 + norm_row_blocks(T) * 3 * K * 4);
}

static moe_status_t check_norm(int64_t T, int64_t K, int32_t dtype, int32_t wdtype, int32_t gate) {
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

// Rows or weights that the wide path reads 16 bytes at a time.
struct Wide {
  int64_t T;
  size_t elem;
  bool ok = true;
  void rows(const void* q, int64_t stride) { ok = ok && rows_aligned16(q, stride, elem, T); }
  void weights(const void* q) { ok = ok && (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }
};

template <typename T, int VEC, int NV>
static moe_status_t launch_forward(const NormParams& p, int threads, cudaStream_t s) {
  auto kernel = moe::block_norm_kernel<T, VEC, NV>;
  const int64_t cap =
      (int64_t)num_sms() * resident_blocks(reinterpret_cast<const void*>(kernel), threads);
  return launched(launch_pdl(kernel, dim3((unsigned)(p.T < cap ? p.T : cap)), dim3(threads), 0, s, p),
                  "block norm");
}

}  // namespace moe_host

using namespace moe_host;

extern "C" {

size_t moe_block_norm_workspace_size(int64_t num_tokens, int64_t hidden_size) {
  if (num_tokens <= 0 || hidden_size <= 0) return 0;
  return norm_workspace(num_tokens, hidden_size);
}

moe_status_t moe_block_norm(const moe_block_norm_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t T = a->num_tokens, K = a->hidden_size;
  moe_status_t st = check_norm(T, K, a->dtype, a->weight_dtype, a->gate_kind);
  if (st != MOE_OK) return st;
  if ((a->z != nullptr) != (a->x_out != nullptr))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "x_out must be given iff z is");
  if ((a->pre_weight != nullptr) != (a->y != nullptr))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "y must be given iff pre_weight is");
  if ((a->gate != nullptr) != (a->gate_kind != MOE_GATE_NONE))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "gate must be given iff gate_kind is not NONE");
  if (a->z == nullptr && (a->gate != nullptr || a->post_weight != nullptr))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a gate or post_weight needs z");
  if (T == 0 || K == 0) return MOE_OK;
  if (a->x == nullptr || (a->z == nullptr && a->y == nullptr))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if (T > 1 && (a->x_stride0 < K || (a->z && (a->z_stride0 < K || a->x_out_stride0 < K)) ||
                (a->y && a->y_stride0 < K) ||
                (a->gate_kind == MOE_GATE_FULL && a->gate_stride0 < K)))
    return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
  NormParams p{};
  p.T = T;
  p.K = K;
  p.x = a->x;
  p.x_stride = a->x_stride0;
  p.z = a->z;
  p.z_stride = a->z_stride0;
  p.gate = a->gate;
  p.gate_stride = a->gate_stride0;
  p.gate_kind = a->gate_kind;
  p.post_w = a->post_weight;
  p.pre_w = a->pre_weight;
  p.w_dtype = a->weight_dtype;
  p.scale = a->scale;
  p.offset = a->weight_offset;
  p.eps = a->eps;
  p.x_out = a->x_out;
  p.x_out_stride = a->x_out_stride0;
  p.y = a->y;
  p.y_stride = a->y_stride0;
  p.rstd_post = a->rstd_post;
  p.rstd_pre = a->rstd_pre;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return with_dtype(a->dtype, [&](auto v) {
    using E = decltype(v);
    constexpr int V = 16 / sizeof(E);
    Wide w{T, sizeof(E)};
    w.ok = K % V == 0;
    w.rows(p.x, p.x_stride);
    w.rows(p.z, p.z_stride);
    w.rows(p.x_out, p.x_out_stride);
    w.rows(p.y, p.y_stride);
    if (p.gate_kind == MOE_GATE_FULL) w.rows(p.gate, p.gate_stride);
    if (p.gate_kind == MOE_GATE_CHANNEL) w.weights(p.gate);
    w.weights(p.post_w);
    w.weights(p.pre_w);
    const int64_t packs = w.ok ? K / V : K;
    auto threads = [&](int nv) { return (int)(((packs + nv - 1) / nv + 31) / 32 * 32); };
    if (w.ok) {
      if (packs <= 512) return launch_forward<E, V, 1>(p, threads(1), s);
      if (packs <= 1024) return launch_forward<E, V, 2>(p, threads(2), s);
      if (packs <= 2048) return launch_forward<E, V, 4>(p, threads(4), s);
      return launch_forward<E, V, 8>(p, threads(8), s);
    }
    if (packs <= 2048) return launch_forward<E, 1, 4>(p, threads(4), s);
    if (packs <= 8192) return launch_forward<E, 1, 16>(p, threads(16), s);
    return launch_forward<E, 1, 32>(p, threads(32), s);
  });
}

moe_status_t moe_block_norm_backward(const moe_block_norm_backward_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t T = a->num_tokens, K = a->hidden_size;
  moe_status_t st = check_norm(T, K, a->dtype, a->weight_dtype, a->gate_kind);
  if (st != MOE_OK) return st;
  if ((a->gate != nullptr) != (a->gate_kind != MOE_GATE_NONE))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "gate must be given iff gate_kind is not NONE");
  if (a->z == nullptr && (a->gate != nullptr || a->post_weight != nullptr || a->d_z != nullptr))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a gate, post_weight or d_z needs z");
  if ((a->d_gate != nullptr && a->gate == nullptr) ||
      (a->d_post_weight != nullptr && a->post_weight == nullptr) ||
      (a->d_pre_weight != nullptr && a->pre_weight == nullptr))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a gradient of an input that is not given");
  if (a->d_y != nullptr && a->pre_weight == nullptr)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "d_y needs pre_weight");
  if (K == 0 || (T == 0 && !a->d_post_weight && !a->d_pre_weight &&
                 !(a->d_gate && a->gate_kind == MOE_GATE_CHANNEL)))
    return MOE_OK;
  if (T > 0 && (!a->x || !a->d_x || (a->post_weight && !a->rstd_post) ||
                (a->pre_weight && !a->rstd_pre)))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if (T > 1 && (a->x_stride0 < K || a->d_x_stride0 < K || (a->z && a->z_stride0 < K) ||
                (a->d_z && a->d_z_stride0 < K) || (a->d_y && a->d_y_stride0 < K) ||
                (a->d_x_out && a->d_x_out_stride0 < K) ||
                (a->gate_kind == MOE_GATE_FULL &&
                 (a->gate_stride0 < K || (a->d_gate && a->d_gate_stride0 < K)))))
    return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
  const size_t need = norm_workspace(T, K);
  if (a->workspace == nullptr || a->workspace_bytes < need)
    return set_error(MOE_ERR_WORKSPACE, "the gradient needs %zu bytes of workspace, got %zu", need,
                     a->workspace_bytes);
  if ((reinterpret_cast<uintptr_t>(a->workspace) & 15u) != 0)
    return set_error(MOE_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  NormParams p{};
  p.T = T;
  p.K = K;
  p.x = a->x;
  p.x_stride = a->x_stride0;
  p.z = a->z;
  p.z_stride = a->z_stride0;
  p.gate = a->gate;
  p.gate_stride = a->gate_stride0;
  p.gate_kind = a->gate_kind;
  p.post_w = a->post_weight;
  p.pre_w = a->pre_weight;
  p.w_dtype = a->weight_dtype;
  p.scale = a->scale;
  p.offset = a->weight_offset;
  p.rz = a->rstd_post;
  p.rx = a->rstd_pre;
  p.d_x_out = a->d_x_out;
  p.d_x_out_stride = a->d_x_out_stride0;
  p.d_y = a->d_y;
  p.d_y_stride = a->d_y_stride0;
  p.d_x = a->d_x;
  p.d_x_stride = a->d_x_stride0;
  p.d_z = a->d_z;
  p.d_z_stride = a->d_z_stride0;
  p.d_gate = a->d_gate;
  p.d_gate_stride = a->d_gate_stride0;
  p.d_post_w = a->d_post_weight;
  p.d_pre_w = a->d_pre_weight;
  p.row_sums = static_cast<float4*>(a->workspace);
  p.partials = reinterpret_cast<float*>(p.row_sums + T);
  const int64_t blocks = norm_row_blocks(T);
  p.rows_per_block = (int)((T + blocks - 1) / blocks);
  p.row_blocks = p.rows_per_block > 0 ? (int)((T + p.rows_per_block - 1) / p.rows_per_block) : 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T > 0) {
    st = with_dtype(a->dtype, [&](auto v) {
      using E = decltype(v);
      constexpr int V = 16 / sizeof(E);
      Wide w{T, sizeof(E)};
      w.ok = K % V == 0;
      w.rows(p.x, p.x_stride);
      w.rows(p.z, p.z_stride);
      w.rows(p.d_x_out, p.d_x_out_stride);
      w.rows(p.d_y, p.d_y_stride);
      w.rows(p.d_x, p.d_x_stride);
      w.rows(p.d_z, p.d_z_stride);
      if (p.gate_kind == MOE_GATE_FULL) {
        w.rows(p.gate, p.gate_stride);
        w.rows(p.d_gate, p.d_gate_stride);
      }
      if (p.gate_kind == MOE_GATE_CHANNEL) w.weights(p.gate);
      w.weights(p.post_w);
      w.weights(p.pre_w);
      auto go = [&](auto sums, auto apply, int vec) {
        const int64_t cap =
            (int64_t)num_sms() * resident_blocks(reinterpret_cast<const void*>(sums), 256);
        moe_status_t r = launched(
            launch_pdl(sums, dim3((unsigned)(T < cap ? T : cap)), dim3(256), 0, s, p),
            "block norm sums");
        if (r != MOE_OK) return r;
        const int64_t cols = (K + vec - 1) / vec;
        return launched(launch_pdl(apply, dim3((unsigned)((cols + 255) / 256), (unsigned)p.row_blocks),
                                   dim3(256), 0, s, p), "block norm gradient");
      };
      return w.ok ? go(moe::block_norm_sums_kernel<E, V>, moe::block_norm_apply_kernel<E, V>, V)
                  : go(moe::block_norm_sums_kernel<E, 1>, moe::block_norm_apply_kernel<E, 1>, 1);
    });
    if (st != MOE_OK) return st;
  }
  if (!p.d_pre_w && !p.d_post_w && !(p.d_gate && p.gate_kind == MOE_GATE_CHANNEL)) return MOE_OK;
  return launched(launch_pdl(moe::block_norm_columns_kernel, dim3((unsigned)((K + 31) / 32), 3),
                             dim3(256), 0, s, p), "block norm columns");
}

}  // extern "C"
