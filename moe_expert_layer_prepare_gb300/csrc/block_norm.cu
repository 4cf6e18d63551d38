// The seam between two blocks: RMS norm of the block's output, gate, residual
// scale and sum, and the RMS norm before the next block.
//
//   n = z rz wp,  x' = x + s g n,  y = x' rx wq      (rz, rx: inverse RMS)
//
// A block of threads per row, so x and z are read once and x' and y written
// once; two sums over the row, one after the other, since x' needs rz (one pass
// with the square of x + s g n multiplied out would cancel).  Bound by HBM, as
// long as enough rows are at work to cover the two sums' barriers: the next row is
// copied to shared memory meanwhile, and up to three blocks share an SM.
// Measured: 8192 x 7168 bf16, token gate: 73 us, 6.4 TB/s; 8192 x 4096 with a full
// gate 52 us, 6.4 TB/s; one row of 7168: 3.6 us.
#include "block_norm.cuh"

namespace moe {

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

// Rows of 16-byte packs: a block takes every gridDim.x-th row and has the next
// one's x, z and full gate on their way to shared memory while it works; the
// [K] tensors come there once.  With one STAGE the next row is copied over this
// one as soon as x' is in registers (each thread reads only packs that it copied),
// with two from the row's start.
template <typename T, int NV, int STAGES>
__global__ void __launch_bounds__(512, NV <= 2 ? (STAGES == 1 ? 3 : 2) : 1)
    block_norm_rows_kernel(NormParams p) {
  constexpr int VEC = 16 / sizeof(T), H = VEC / 2;
  using P = Pack<T, VEC>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float part[2][2][32];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int packs = (int)(p.K / VEC);
  const int arrays = 1 + (p.z != nullptr) + (p.gate_kind == MOE_GATE_FULL);
  P* stage0 = reinterpret_cast<P*>(smem);
  const int stage_packs = arrays * packs;
  const int w_dtype = p.w_dtype;
  const size_t w_bytes = (size_t)p.K * (w_dtype == MOE_DTYPE_FP32 ? 4 : 2);
  uint8_t* s_post = smem + (size_t)STAGES * stage_packs * 16;
  uint8_t* s_pre = s_post + (p.post_w != nullptr ? w_bytes : 0);
  uint8_t* s_gate = s_pre + (p.pre_w != nullptr ? w_bytes : 0);
  pdl_wait();
  pdl_launch_dependents();
  auto fetch = [&](int64_t t, int s) {
    if (t < p.T) {
      P* dst = stage0 + s * stage_packs;
      const T* x = static_cast<const T*>(p.x) + t * p.x_stride;
      const T* z = static_cast<const T*>(p.z) + t * p.z_stride;
      const T* g = static_cast<const T*>(p.gate) + t * p.gate_stride;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + i * threads;
        if (c >= packs) break;
        if (p.z != nullptr) copy16(dst + packs + c, z + c * VEC);
        copy16(dst + c, x + c * VEC);
        if (p.gate_kind == MOE_GATE_FULL) copy16(dst + 2 * packs + c, g + c * VEC);
      }
    }
  };
  fetch(blockIdx.x, 0);
  if (p.post_w != nullptr) fetch_weights<VEC, NV>(s_post, p.post_w, w_dtype, packs);
  if (p.pre_w != nullptr) fetch_weights<VEC, NV>(s_pre, p.pre_w, w_dtype, packs);
  if (p.gate_kind == MOE_GATE_CHANNEL) fetch_weights<VEC, NV>(s_gate, p.gate, w_dtype, packs);
  copies_commit();
  const float2 offset = both(p.offset);
  const float inv_k = 1.0f / (float)p.K;
  auto factor = [&](int64_t t) { return t < p.T ? p.scale * token_factor<T>(p, t) : 0.0f; };
  float ahead = factor(blockIdx.x);
  int it = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, it ^= 1) {
    if (STAGES == 2) {
      fetch(t + gridDim.x, it ^ 1);
      copies_commit();
    }
    const float2 branch = both(ahead);
    ahead = factor(t + gridDim.x);
    copies_wait<STAGES - 1>();
    const P* st = STAGES == 2 ? stage0 + it * stage_packs : stage0;
    float rz = 1.0f;
    if (p.post_w != nullptr) {
      float2 ss = both(0.0f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + i * threads;
        if (c >= packs) break;
        const P z = st[packs + c];
#pragma unroll
        for (int q = 0; q < H; ++q) ss = fma2(z.get2(q), z.get2(q), ss);
      }
      rz = rsqrtf(fmaf(block_sum(ss.x + ss.y, part[it][0]), inv_k, p.eps));
      if (tid == 0 && p.rstd_post != nullptr) p.rstd_post[t] = rz;
    }
    float2 xo[NV][H];
    float2 ss = both(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * threads;
      if (c >= packs) break;
      float2(&v)[H] = xo[i];
      const P x = st[c];
      if (p.z != nullptr) {
        const P z = st[packs + c];
#pragma unroll
        for (int q = 0; q < H; ++q) v[q] = z.get2(q);
        if (p.post_w != nullptr) {
          float2 w[H];
          read_weights<VEC>(s_post, w_dtype, c, packs, w);
#pragma unroll
          for (int q = 0; q < H; ++q) v[q] = mul2(mul2(v[q], both(rz)), add2(w[q], offset));
        }
        if (p.gate_kind == MOE_GATE_CHANNEL) {
          float2 g[H];
          read_weights<VEC>(s_gate, w_dtype, c, packs, g);
#pragma unroll
          for (int q = 0; q < H; ++q) v[q] = mul2(v[q], g[q]);
        } else if (p.gate_kind == MOE_GATE_FULL) {
          const P g = st[2 * packs + c];
#pragma unroll
          for (int q = 0; q < H; ++q) v[q] = mul2(v[q], g.get2(q));
        }
        P o;
#pragma unroll
        for (int q = 0; q < H; ++q) {
          v[q] = fma2(branch, v[q], x.get2(q));
          o.set2(q, v[q]);
        }
        store_pack<T, VEC>(static_cast<T*>(p.x_out) + t * p.x_out_stride + c * VEC, o);
      } else {
#pragma unroll
        for (int q = 0; q < H; ++q) v[q] = x.get2(q);
      }
#pragma unroll
      for (int q = 0; q < H; ++q) ss = fma2(v[q], v[q], ss);
    }
    if (STAGES == 1) {
      fetch(t + gridDim.x, 0);
      copies_commit();
    }
    if (p.pre_w == nullptr) continue;
    const float rx = rsqrtf(fmaf(block_sum(ss.x + ss.y, part[it][1]), inv_k, p.eps));
    if (tid == 0 && p.rstd_pre != nullptr) p.rstd_pre[t] = rx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * threads;
      if (c >= packs) break;
      float2 w[H];
      read_weights<VEC>(s_pre, w_dtype, c, packs, w);
      P o;
#pragma unroll
      for (int q = 0; q < H; ++q) o.set2(q, mul2(mul2(xo[i][q], both(rx)), add2(w[q], offset)));
      store_pack<T, VEC>(static_cast<T*>(p.y) + t * p.y_stride + c * VEC, o);
    }
  }
  copies_wait<0>();
}

// Any other rows (and 16-byte packs too long for shared memory): up to three passes over
// a row, which stays in L1; x' is computed again in each, U packs of a thread in flight.
// Stores come in the last one, each behind the thread's own reads of the same columns,
// so that x_out may be x.  4099 x 4095 bf16 with a channel gate, two elements at a time:
// 107 us (one: 118, four: 160, the row kept in registers: 225).
template <typename T, int VEC, int U>
__global__ void __launch_bounds__(512) block_norm_kernel(NormParams p) {
  __shared__ float part[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int K = (int)p.K, stride = blockDim.x * VEC, c0 = threadIdx.x * VEC;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + t * p.x_stride;
    const T* zr = static_cast<const T*>(p.z) + t * p.z_stride;
    float rz = 1.0f;
    if (p.post_w != nullptr) {
      float ss = 0.0f;
      for (int c = c0; c < K; c += U * stride) {
        float z[U][VEC];
#pragma unroll
        for (int i = 0; i < U; ++i)  // past the row its last pack, not summed
          load_pack<T, VEC>(zr + min(c + i * stride, K - VEC)).get(z[i]);
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int q = 0; q < VEC; ++q)
            ss = c + i * stride < K ? fmaf(z[i][q], z[i][q], ss) : ss;
      }
      rz = rsqrtf(block_sum(ss, part[0]) / (float)K + p.eps);
      if (threadIdx.x == 0 && p.rstd_post != nullptr) p.rstd_post[t] = rz;
    }
    const float branch = p.z != nullptr ? p.scale * token_factor<T>(p, t) : 0.0f;
    auto x_next = [&](int c, float (&x)[VEC]) {
      load_pack<T, VEC>(xr + c).get(x);
      if (p.z != nullptr) {
        float w[VEC], g[VEC], z[VEC];
        load_pack<T, VEC>(zr + c).get(z);
        load_weights_or_one<VEC>(p.post_w, p.w_dtype, c, p.offset, w);
        load_gate<T, VEC>(p, t, c, g);
#pragma unroll
        for (int q = 0; q < VEC; ++q) x[q] = fmaf(branch, z[q] * rz * w[q] * g[q], x[q]);
      }
    };
    float rx = 0.0f;
    if (p.pre_w != nullptr) {
      float ss = 0.0f;
      for (int c = c0; c < K; c += U * stride) {
        float x[U][VEC];
#pragma unroll
        for (int i = 0; i < U; ++i) x_next(min(c + i * stride, K - VEC), x[i]);
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int q = 0; q < VEC; ++q)
            ss = c + i * stride < K ? fmaf(x[i][q], x[i][q], ss) : ss;
      }
      rx = rsqrtf(block_sum(ss, part[1]) / (float)K + p.eps);
      if (threadIdx.x == 0 && p.rstd_pre != nullptr) p.rstd_pre[t] = rx;
    }
    for (int c = c0; c < K; c += U * stride) {
      float x[U][VEC], w[U][VEC];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int at = min(c + i * stride, K - VEC);
        x_next(at, x[i]);
        load_weights_or_one<VEC>(p.pre_w, p.w_dtype, at, p.offset, w[i]);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int at = c + i * stride;
        if (at >= K) break;
        Pack<T, VEC> o;
        o.set(x[i]);
        if (p.z != nullptr)
          store_pack<T, VEC>(static_cast<T*>(p.x_out) + t * p.x_out_stride + at, o);
        if (p.pre_w == nullptr) continue;
#pragma unroll
        for (int q = 0; q < VEC; ++q) w[i][q] *= x[i][q] * rx;
        o.set(w[i]);
        store_pack<T, VEC>(static_cast<T*>(p.y) + t * p.y_stride + at, o);
      }
    }
    __syncthreads();  // both parts are free for the next row
  }
}

}  // namespace moe

namespace moe_host {

using moe::NormParams;

// Shared memory of a row block: the stages and the [K] tensors.
static size_t rows_smem(const NormParams& p, size_t elem, int stages) {
  const int arrays = 1 + (p.z != nullptr) + (p.gate_kind == MOE_GATE_FULL);
  const int weights = (p.post_w != nullptr) + (p.pre_w != nullptr) +
                      (p.gate_kind == MOE_GATE_CHANNEL);
  return (size_t)p.K * (stages * arrays * elem + weights * dtype_size(p.w_dtype));
}

template <typename T, int NV, int STAGES>
static int rows_resident(const NormParams& p, int threads) {
  return resident_with<moe::block_norm_rows_kernel<T, NV, STAGES>>(threads,
                                                                   rows_smem(p, sizeof(T), STAGES));
}

template <typename T, int NV, int STAGES = 2>
static moe_status_t launch_rows(const NormParams& p, int threads, cudaStream_t s) {
  const size_t smem = rows_smem(p, sizeof(T), STAGES);
  const int64_t cap = (int64_t)num_sms() * rows_resident<T, NV, STAGES>(p, threads);
  if (cap == 0) return set_error(MOE_ERR_CUDA, "block norm: no resident block");
  return launched(launch_pdl(moe::block_norm_rows_kernel<T, NV, STAGES>,
                             dim3((unsigned)(p.T < cap ? p.T : cap)), dim3(threads), smem, s, p),
                  "block norm");
}

template <typename T, int VEC, int U>
static moe_status_t launch_passes(const NormParams& p, cudaStream_t s) {
  auto kernel = moe::block_norm_kernel<T, VEC, U>;
  const int64_t packs = (p.K + VEC - 1) / VEC;
  const int threads = packs < 512 ? (int)((packs + 31) / 32 * 32) : 512;
  const int64_t cap =
      (int64_t)num_sms() * resident_blocks(reinterpret_cast<const void*>(kernel), threads);
  return launched(launch_pdl(kernel, dim3((unsigned)(p.T < cap ? p.T : cap)), dim3(threads), 0, s, p),
                  "block norm");
}

}  // namespace moe_host

using namespace moe_host;

extern "C" {

moe_status_t moe_block_norm(const moe_block_norm_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t T = a->num_tokens, K = a->hidden_size;
  moe_status_t st = check_norm(T, K, a->dtype, a->weight_dtype, a->gate_kind);
  if (st != MOE_OK) return st;
  if (T == 0 || K == 0) return MOE_OK;  // before the pointers: empty tensors have no address
  if ((a->z != nullptr) != (a->x_out != nullptr))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "x_out must be given iff z is");
  if ((a->pre_weight != nullptr) != (a->y != nullptr))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "y must be given iff pre_weight is");
  if ((a->gate != nullptr) != (a->gate_kind != MOE_GATE_NONE))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "gate must be given iff gate_kind is not NONE");
  if (a->z == nullptr && (a->gate != nullptr || a->post_weight != nullptr))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a gate or post_weight needs z");
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
    // One pack a thread up to 512, in two stages (8192 x 4096 full gate: 52 us; two
    // packs a thread: 56; one stage and a third block: 55).  Above, two packs and, where
    // three blocks fit, one stage: 8192 x 7168 73 us against 90 with two stages and two
    // blocks, 8192 x 8192 88 against 91.  Where one stage fits twice and two stages do not,
    // one with 16-bit weights (full gate, 8192 x 7680: 97 us, two: 102; x 7672: 105 and
    // 116), two with fp32 ones (channel gate, 8192 x 6144: 88 us, one: 99; full gate, 1000 x
    // 8192: 20 and 23).  Where both fit twice, two (channel gate, 8192 x 7680: 78 us, one:
    // 93).  Longer rows: two stages (1000 x 16384: 24 us, one stage: 46), the sums' barriers
    // being rarer there.
    if (w.ok && rows_smem(p, sizeof(E), 2) <= kMaxBlockSmem) {
      if (packs <= 512) return launch_rows<E, 1>(p, threads(1), s);
      if (packs <= 1024) {
        const int one = rows_resident<E, 2, 1>(p, threads(2));
        if (one >= 3 ||
            (one > rows_resident<E, 2, 2>(p, threads(2)) && p.w_dtype != MOE_DTYPE_FP32))
          return launch_rows<E, 2, 1>(p, threads(2), s);
        return launch_rows<E, 2>(p, threads(2), s);
      }
      if (packs <= 2048) return launch_rows<E, 4>(p, threads(4), s);
      return launch_rows<E, 8>(p, threads(8), s);
    }
    return w.ok ? launch_passes<E, V, 1>(p, s) : launch_passes<E, 1, 2>(p, s);
  });
}

}  // extern "C"
