// Gradient of the seam between two blocks (block_norm.cu).  With xh = x' rx,
// zh = z rz, u = dy wq and mean over the row:
//   d = dx' + rx (u - xh mean(u xh))                  (= dx)
//   dz = rz (v - zh mean(v zh)),  v = s g wp d
//   dwq = sum_t dy xh,  dwp = sum_t s g d zh,  dg = s d n (summed as the gate is)
// mean(v zh) is linear in d, so with a = g n the row needs only the sums of
// u xh, a (dx' + rx u) and a xh, all from one reading.
#include "block_norm.cuh"

namespace moe {

// Rows of 16-byte packs, at most 1024, that fit shared memory twice: everything from one
// reading.  A block takes every gridDim.x-th row, the next one's tensors on their
// way to shared memory (a third stage changes little: 4099 x 4096 with a full gate 102
// us with the forward, 103 with it); the row's three sums cost one barrier, then the packs
// (kept in registers, or with two a thread read again) give the gradients.  The [K]
// tensors lie there in fp32, offset added, a pack's first four values in one plane and
// the rest in the next, so that neighbouring threads read neighbouring 16 bytes.  Each
// thread keeps the column sums of its packs in registers over all rows of the block.
//
// Issue slots and the barrier bound it, at 16 warps an SM (the column sums leave room for
// no more): 4099 x 4096 with a full gate 66 us (268 MB, 4.1 TB/s), 8192 x 7168 with a
// token gate 165 us (705 MB, 4.3 TB/s).
template <typename T, int NV, int GATE>  // GATE: channel, full, or none for the others
__global__ void __launch_bounds__(512) block_norm_backward_kernel(NormParams p) {
  constexpr int VEC = 16 / sizeof(T), H = VEC / 2;
  constexpr bool channel = GATE == MOE_GATE_CHANNEL, full = GATE == MOE_GATE_FULL;
  using P = Pack<T, VEC>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float part[2][3][32];
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
  const int packs = (int)(p.K / VEC);
  const bool has_z = p.z != nullptr, has_dx = p.d_x_out != nullptr, has_dy = p.d_y != nullptr;
  const bool post = p.post_w != nullptr, pre = p.pre_w != nullptr;
  // places of the tensors in a stage
  const int at_z = packs, at_dx = at_z + (has_z ? packs : 0), at_dy = at_dx + (has_dx ? packs : 0);
  const int at_g = at_dy + (has_dy ? packs : 0), stage_packs = at_g + (full ? packs : 0);
  P* stage0 = reinterpret_cast<P*>(smem);
  float2* s_post = reinterpret_cast<float2*>(smem + (size_t)2 * stage_packs * 16);
  float2* s_pre = s_post + (post ? p.K / 2 : 0);
  float2* s_gate = s_pre + (pre ? p.K / 2 : 0);
  pdl_wait();
  pdl_launch_dependents();
  auto fetch = [&](int64_t t, int s) {
    if (t < p.T) {
      P* dst = stage0 + s * stage_packs;
      const T* x = static_cast<const T*>(p.x) + t * p.x_stride;
      const T* z = static_cast<const T*>(p.z) + t * p.z_stride;
      const T* dx = static_cast<const T*>(p.d_x_out) + t * p.d_x_out_stride;
      const T* dy = static_cast<const T*>(p.d_y) + t * p.d_y_stride;
      const T* g = static_cast<const T*>(p.gate) + t * p.gate_stride;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + i * threads;
        if (c >= packs) break;
        copy16(dst + c, x + c * VEC);
        if (has_z) copy16(dst + at_z + c, z + c * VEC);
        if (has_dx) copy16(dst + at_dx + c, dx + c * VEC);
        if (has_dy) copy16(dst + at_dy + c, dy + c * VEC);
        if (full) copy16(dst + at_g + c, g + c * VEC);
      }
    }
  };
  fetch(blockIdx.x, 0);
  copies_commit();
#pragma unroll
  for (int i = 0; i < NV; ++i) {  // each thread its own packs
    const int c = tid + i * threads;
    if (c >= packs) break;
    auto keep = [&](float2* to, const void* w, float offset) {
      float v[VEC];
      load_weights<VEC>(w, p.w_dtype, (int64_t)c * VEC, offset, v);
#pragma unroll
      for (int q = 0; q < H; q += 2)
        *reinterpret_cast<float4*>(to + (q / 2 * packs + c) * 2) =
            make_float4(v[2 * q], v[2 * q + 1], v[2 * q + 2], v[2 * q + 3]);
    };
    if (post) keep(s_post, p.post_w, p.offset);
    if (pre) keep(s_pre, p.pre_w, p.offset);
    if (channel) keep(s_gate, p.gate, 0.0f);
  }
  float2 dwq[NV][H], dwp[NV][H], dgc[channel ? NV : 1][H];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < H; ++q) {
      dwq[i][q] = dwp[i][q] = both(0.0f);
      if (channel) dgc[i][q] = both(0.0f);
    }
  auto read = [&](const float2* s, int c, float2 (&w)[H]) {
#pragma unroll
    for (int q = 0; q < H; q += 2) {
      const float4 v = *reinterpret_cast<const float4*>(s + (q / 2 * packs + c) * 2);
      w[q] = make_float2(v.x, v.y), w[q + 1] = make_float2(v.z, v.w);
    }
  };

  // the row's own numbers are read a row ahead as well
  struct Scalars {
    float rz, rx, branch;
  };
  auto scalars = [&](int64_t t) {
    Scalars v{1.0f, 0.0f, 0.0f};
    if (t >= p.T) return v;
    if (post) v.rz = p.rz[t];
    if (pre) v.rx = p.rx[t];
    if (has_z) v.branch = p.scale * token_factor<T>(p, t);
    return v;
  };
  Scalars ahead = scalars(blockIdx.x);
  const float inv_k = 1.0f / (float)p.K;
  int it = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, it ^= 1) {
    fetch(t + gridDim.x, it ^ 1);
    copies_commit();
    const float rx = ahead.rx, branch = ahead.branch;
    const float2 rz2 = both(ahead.rz), rx2 = both(rx), branch2 = both(branch);
    const float rz = ahead.rz;
    ahead = scalars(t + gridDim.x);
    copies_wait<1>();
    const P* st = stage0 + it * stage_packs;

    // Of a pack: zh, the gate times wp (gw), a = gate n, xh, dy and e.
    auto columns = [&](int c, float2 (&zh)[H], float2 (&gw)[H], float2 (&a)[H], float2 (&xh)[H],
                       float2 (&dy)[H], float2 (&e)[H]) {
      const P x = st[c];
      if (has_z) {
        const P z = st[at_z + c];
#pragma unroll
        for (int q = 0; q < H; ++q) zh[q] = mul2(z.get2(q), rz2);
      } else {
#pragma unroll
        for (int q = 0; q < H; ++q) zh[q] = both(0.0f);
      }
      if (post) {
        read(s_post, c, gw);
      } else {
#pragma unroll
        for (int q = 0; q < H; ++q) gw[q] = both(1.0f);
      }
      if (channel) {
        float2 g[H];
        read(s_gate, c, g);
#pragma unroll
        for (int q = 0; q < H; ++q) gw[q] = mul2(gw[q], g[q]);
      } else if (full) {
        const P g = st[at_g + c];
#pragma unroll
        for (int q = 0; q < H; ++q) gw[q] = mul2(gw[q], g.get2(q));
      }
#pragma unroll
      for (int q = 0; q < H; ++q) {
        a[q] = mul2(zh[q], gw[q]);
        xh[q] = mul2(fma2(branch2, a[q], x.get2(q)), rx2);
        e[q] = both(0.0f);
        dy[q] = both(0.0f);
      }
      if (has_dx) {
        const P dx = st[at_dx + c];
#pragma unroll
        for (int q = 0; q < H; ++q) e[q] = dx.get2(q);
      }
      if (has_dy) {
        const P v = st[at_dy + c];
        float2 wq[H];
        read(s_pre, c, wq);
#pragma unroll
        for (int q = 0; q < H; ++q) {
          dy[q] = v.get2(q);
          wq[q] = mul2(wq[q], dy[q]);  // u
          e[q] = fma2(rx2, wq[q], e[q]);
        }
        float2 dot = both(0.0f);
#pragma unroll
        for (int q = 0; q < H; ++q) dot = fma2(wq[q], xh[q], dot);
        return dot;
      }
      return both(0.0f);
    };
    float2 t0 = both(0.0f), t1 = t0, t2 = t0;
    float2 zh[H], gw[H], xh[H], dy[H], e[H];  // with one pack a thread kept to the end
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * threads;
      if (c >= packs) break;
      float2 a[H];
      t0 = add2(t0, columns(c, zh, gw, a, xh, dy, e));
#pragma unroll
      for (int q = 0; q < H; ++q) {
        t1 = fma2(a[q], e[q], t1);
        t2 = fma2(a[q], xh[q], t2);
      }
    }
    float(&pt)[3][32] = part[it];
    float s0 = warp_sum(t0.x + t0.y), s1 = warp_sum(t1.x + t1.y), s2 = warp_sum(t2.x + t2.y);
    if (lane == 0) pt[0][tid >> 5] = s0, pt[1][tid >> 5] = s1, pt[2][tid >> 5] = s2;
    __syncthreads();
    const bool has = lane < (threads >> 5);
    s0 = warp_sum(has ? pt[0][lane] : 0.0f) * inv_k;
    s1 = warp_sum(has ? pt[1][lane] : 0.0f);
    s2 = warp_sum(has ? pt[2][lane] : 0.0f);
    const float dot = s1 - rx * s0 * s2;  // sum over the row of g n d
    const float c2 = post ? branch * dot * inv_k : 0.0f;
    if (p.gate_kind == MOE_GATE_TOKEN && p.d_gate != nullptr && tid == 0)
      static_cast<T*>(p.d_gate)[t * p.d_gate_stride] = from_f32<T>(p.scale * dot);
    const float2 k0 = both(-rx * s0), kz = both(-rz * c2), kv = both(rz * branch);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * threads;
      if (c >= packs) break;
      if (NV > 1) {
        float2 a[H];
        columns(c, zh, gw, a, xh, dy, e);
      }
      P ox, oz;
#pragma unroll
      for (int q = 0; q < H; ++q) {
        const float2 d = fma2(k0, xh[q], e[q]);
        ox.set2(q, d);
        oz.set2(q, fma2(kv, mul2(gw[q], d), mul2(kz, zh[q])));
        dwq[i][q] = fma2(dy[q], xh[q], dwq[i][q]);
        e[q] = d;
      }
      store_pack<T, VEC>(static_cast<T*>(p.d_x) + t * p.d_x_stride + c * VEC, ox);
      if (p.d_z != nullptr)
        store_pack<T, VEC>(static_cast<T*>(p.d_z) + t * p.d_z_stride + c * VEC, oz);
      if (channel || full) {  // the gate's gradient, and s g d for the post weight's
        float2 wp[H];
        if (post) {
          read(s_post, c, wp);
        } else {
#pragma unroll
          for (int q = 0; q < H; ++q) wp[q] = both(1.0f);
        }
        P og;
#pragma unroll
        for (int q = 0; q < H; ++q) {
          const float2 gd = mul2(both(p.scale), mul2(mul2(zh[q], wp[q]), e[q]));
          if (channel) dgc[i][q] = add2(dgc[i][q], gd);
          if (full) og.set2(q, gd);
        }
        if (full && p.d_gate != nullptr)
          store_pack<T, VEC>(static_cast<T*>(p.d_gate) + t * p.d_gate_stride + c * VEC, og);
        if (channel) {
          read(s_gate, c, wp);
        } else {
          const P g = st[at_g + c];
#pragma unroll
          for (int q = 0; q < H; ++q) wp[q] = g.get2(q);
        }
#pragma unroll
        for (int q = 0; q < H; ++q) e[q] = mul2(e[q], wp[q]);
      }
#pragma unroll
      for (int q = 0; q < H; ++q) dwp[i][q] = fma2(mul2(branch2, e[q]), zh[q], dwp[i][q]);
    }
  }
  copies_wait<0>();
  float* out = p.partials + (int64_t)blockIdx.x * 3 * p.K;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + i * threads;
    if (c >= packs) break;
    auto put = [&](float* to, const float2 (&v)[H]) {
#pragma unroll
      for (int q = 0; q < H; q += 2)
        *reinterpret_cast<float4*>(to + c * VEC + 2 * q) =
            make_float4(v[q].x, v[q].y, v[q + 1].x, v[q + 1].y);
    };
    if (p.d_pre_w != nullptr) put(out, dwq[i]);
    if (p.d_post_w != nullptr) put(out + p.K, dwp[i]);
    if (channel && p.d_gate != nullptr) put(out + 2 * p.K, dgc[i]);
  }
}

__device__ __forceinline__ void store_weight(void* w, int dtype, int64_t c, float v) {
  if (dtype == MOE_DTYPE_FP32)
    static_cast<float*>(w)[c] = v;
  else if (dtype == MOE_DTYPE_BF16)
    static_cast<__nv_bfloat16*>(w)[c] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(w)[c] = __float2half_rn(v);
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
  float x[VEC], z[VEC] = {}, dx[VEC] = {}, wq[VEC];
  load_pack<T, VEC>(static_cast<const T*>(p.x) + t * p.x_stride + c).get(x);
  if (p.z != nullptr) load_pack<T, VEC>(static_cast<const T*>(p.z) + t * p.z_stride + c).get(z);
  if (p.d_x_out != nullptr)
    load_pack<T, VEC>(static_cast<const T*>(p.d_x_out) + t * p.d_x_out_stride + c).get(dx);
#pragma unroll
  for (int q = 0; q < VEC; ++q) b.dy[q] = 0.0f;
  if (p.d_y != nullptr)
    load_pack<T, VEC>(static_cast<const T*>(p.d_y) + t * p.d_y_stride + c).get(b.dy);
  load_gate<T, VEC>(p, t, c, b.g);
  load_weights_or_one<VEC>(p.post_w, p.w_dtype, c, p.offset, b.wp);
  load_weights_or_one<VEC>(p.pre_w, p.w_dtype, c, p.offset, wq);
#pragma unroll
  for (int q = 0; q < VEC; ++q) {
    b.zh[q] = z[q] * rz;
    b.n[q] = b.zh[q] * b.wp[q];
    b.xh[q] = fmaf(branch, b.g[q] * b.n[q], x[q]) * rx;
    b.u[q] = b.dy[q] * wq[q];
    b.e[q] = fmaf(rx, b.u[q], dx[q]);
  }
}

// Any other rows, in two launches that each read everything (2048 x 7168 fp32: 112 us,
// where one reading would need twice the shared memory that there is; 4099 x 4095 bf16,
// element by element: 196 us).  The first: the row's sums,
// row_sums[t] = (mean(u xh), sum a e, sum a xh, 0) with a = g n over channel or full gates.
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

// The second: gradients of the rows, and each row block's column sums.
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
    float fx[VEC], fz[VEC], fg[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      const float d = fmaf(-rx * s.x, b.xh[q], b.e[q]);
      const float bg = branch * b.g[q];
      const float gd = p.scale * (d * b.n[q]);
      fx[q] = d;
      fz[q] = rz * (bg * b.wp[q] * d - b.zh[q] * c2);
      fg[q] = gd;
      dwq[q] = fmaf(b.dy[q], b.xh[q], dwq[q]);
      dwp[q] = fmaf(bg * d, b.zh[q], dwp[q]);
      dg[q] += gd;
    }
    Pack<T, VEC> ox, oz, og;
    ox.set(fx);
    oz.set(fz);
    og.set(fg);
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

// Last launch: column sums over the blocks of rows, in a fixed order: 32
// columns by 32 interleaved shares of the blocks, four reads of a share in
// flight, joined in shared memory.
constexpr int COL_SHARES = 32;

__global__ void __launch_bounds__(32 * COL_SHARES) block_norm_columns_kernel(NormParams p) {
  __shared__ float part[COL_SHARES][33];
  pdl_wait();
  pdl_launch_dependents();
  const int col = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + col;
  const int k = blockIdx.y;
  void* out = k == 0 ? p.d_pre_w : (k == 1 ? p.d_post_w : p.d_gate);
  if (out == nullptr || (k == 2 && p.gate_kind != MOE_GATE_CHANNEL)) return;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < p.K) {
    const float* src = p.partials + k * p.K + c;
    const int64_t step = 3 * p.K;
    for (int b = share; b < p.row_blocks; b += 4 * COL_SHARES) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (b + i * COL_SHARES < p.row_blocks) sum[i] += __ldcg(src + (b + i * COL_SHARES) * step);
    }
  }
  part[share][col] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  __syncthreads();
  // warp w joins column w: lane i has share i
  const float total = warp_sum(part[col][share]);
  const int64_t oc = (int64_t)blockIdx.x * 32 + share;
  if (col == 0 && oc < p.K) store_weight(out, p.w_dtype, oc, total);
}

}  // namespace moe

namespace moe_host {

using moe::NormParams;

// Blocks that write column sums: one a token, at most 512.
constexpr int64_t kMaxRowBlocks = 512;
static int64_t norm_row_blocks(int64_t T) {
  return T < 1 ? 1 : (T < kMaxRowBlocks ? T : kMaxRowBlocks);
}

// Without tokens the columns' sums, all zero, come from no block of rows.
static size_t norm_workspace(int64_t T, int64_t K) {
  if (T <= 0 || K <= 0) return 0;
  return (size_t)(T * 16 + norm_row_blocks(T) * 3 * K * 4);
}

// The one-reading gradient; false when the rows do not fit.
template <typename T, int NV, int GATE>
static bool launch_gated(NormParams& p, int threads, cudaStream_t s, moe_status_t* st) {
  constexpr auto kernel = moe::block_norm_backward_kernel<T, NV, GATE>;
  const int arrays = 1 + (p.z != nullptr) + (p.d_x_out != nullptr) + (p.d_y != nullptr) +
                     (GATE == MOE_GATE_FULL);
  const int kept = (p.post_w != nullptr) + (p.pre_w != nullptr) + (GATE == MOE_GATE_CHANNEL);
  const size_t row = (size_t)arrays * p.K * sizeof(T), weights = (size_t)kept * p.K * 4;
  const size_t smem = 2 * row + weights;
  if (smem > kMaxBlockSmem) return false;
  int64_t blocks = resident_with<kernel>(threads, smem);
  if (blocks == 0) return false;
  blocks *= num_sms();
  if (blocks > kMaxRowBlocks) blocks = kMaxRowBlocks;
  if (blocks > p.T) blocks = p.T;
  p.row_blocks = (int)blocks;
  *st = launched(launch_pdl(kernel, dim3((unsigned)blocks), dim3(threads), smem, s, p),
                 "block norm gradient");
  return true;
}

template <typename T, int NV>
static bool launch_backward(NormParams& p, int threads, cudaStream_t s, moe_status_t* st) {
  if (p.gate_kind == MOE_GATE_CHANNEL)
    return launch_gated<T, NV, MOE_GATE_CHANNEL>(p, threads, s, st);
  if (p.gate_kind == MOE_GATE_FULL) return launch_gated<T, NV, MOE_GATE_FULL>(p, threads, s, st);
  return launch_gated<T, NV, MOE_GATE_NONE>(p, threads, s, st);
}

}  // namespace moe_host

using namespace moe_host;

extern "C" {

size_t moe_block_norm_workspace_size(int64_t num_tokens, int64_t hidden_size) {
  return norm_workspace(num_tokens, hidden_size);
}

moe_status_t moe_block_norm_backward(const moe_block_norm_backward_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t T = a->num_tokens, K = a->hidden_size;
  moe_status_t st = check_norm(T, K, a->dtype, a->weight_dtype, a->gate_kind);
  if (st != MOE_OK) return st;
  if (K == 0) return MOE_OK;
  // (without tokens their tensors have no address)
  if (T > 0 && (a->gate != nullptr) != (a->gate_kind != MOE_GATE_NONE))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "gate must be given iff gate_kind is not NONE");
  if (T > 0 && a->z == nullptr &&
      (a->gate != nullptr || a->post_weight != nullptr || a->d_z != nullptr))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a gate, post_weight or d_z needs z");
  if ((a->d_gate != nullptr && a->gate == nullptr) ||
      (a->d_post_weight != nullptr && a->post_weight == nullptr) ||
      (a->d_pre_weight != nullptr && a->pre_weight == nullptr))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a gradient of an input that is not given");
  if (a->d_y != nullptr && a->pre_weight == nullptr)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "d_y needs pre_weight");
  if (T == 0 && !a->d_post_weight && !a->d_pre_weight &&
      !(a->d_gate && a->gate_kind == MOE_GATE_CHANNEL))
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
  if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need))
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
      if (w.ok) {
        const int64_t packs = K / V;
        moe_status_t r = MOE_OK;
        const int threads = (int)((packs + 31) / 32 * 32);
        const int half = (threads / 2 + 31) / 32 * 32;
        // one pack a thread kept to the end: 4099 x 4096 with a full gate 102 us with the
        // forward, two a thread read again 107
        if (packs <= 512 && launch_backward<E, 1>(p, threads, s, &r)) return r;
        if (packs > 512 && packs <= 1024 && launch_backward<E, 2>(p, half, s, &r)) return r;
      }
      auto go = [&](auto sums, auto apply, int vec) {
        const int64_t cap =
            (int64_t)num_sms() * resident_blocks(reinterpret_cast<const void*>(sums), 256);
        moe_status_t r = launched(
            launch_pdl(sums, dim3((unsigned)(T < cap ? T : cap)), dim3(256), 0, s, p),
            "block norm sums");
        if (r != MOE_OK) return r;
        // blocks of rows for one full round of the SMs, as each writes column sums (2048 x
        // 7168 fp32: 112 us of gradient, with 512 blocks of rows 126)
        const int64_t across = (K + 256 * vec - 1) / (256 * vec);
        int64_t blocks = (int64_t)num_sms() *
                         resident_blocks(reinterpret_cast<const void*>(apply), 256) / across;
        if (blocks < 1) blocks = 1;
        if (blocks > norm_row_blocks(T)) blocks = norm_row_blocks(T);
        p.rows_per_block = (int)((T + blocks - 1) / blocks);
        p.row_blocks = (int)((T + p.rows_per_block - 1) / p.rows_per_block);
        return launched(launch_pdl(apply, dim3((unsigned)across, (unsigned)p.row_blocks), dim3(256),
                                   0, s, p), "block norm gradient");
      };
      return w.ok ? go(moe::block_norm_sums_kernel<E, V>, moe::block_norm_apply_kernel<E, V>, V)
                  : go(moe::block_norm_sums_kernel<E, 1>, moe::block_norm_apply_kernel<E, 1>, 1);
    });
    if (st != MOE_OK) return st;
  }
  if (!p.d_pre_w && !p.d_post_w && !(p.d_gate && p.gate_kind == MOE_GATE_CHANNEL)) return MOE_OK;
  return launched(launch_pdl(moe::block_norm_columns_kernel, dim3((unsigned)((K + 31) / 32), 3),
                             dim3(32 * moe::COL_SHARES), 0, s, p), "block norm columns");
}

}  // extern "C"
