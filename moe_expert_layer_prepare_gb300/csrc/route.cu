// Router: top-k ids and weights of logits, and the gradient of the logits.
//
// One warp per token; lane i holds logits i, i + 32, i + 64, ... in registers,
// so a row is read once and coalesced.  Selection compares order-preserving
// 32-bit integers of the keys.  Without a bias the key is the logit itself (softmax
// and sigmoid are monotone), so the choice does not depend on how exp rounds.  With a
// sigmoid and a bias the key is 1/(1+expf(-l)) + bias with IEEE division and no
// contraction, the value that elementary fp32 tensor operations give.  With a softmax the
// bias is on the logit, or, where the caller says so, on the score like the sigmoid's.
//
// Issue slots bound it, not memory.  Up to 256 experts each lane sorts its keys,
// cut to make room for the expert's index in the low bits, and k rounds take the
// largest head (one redux.sync) and pop it.  The cut keys decide unless two of the
// taken ones, or the last taken and the next, are equal in what is left; then, and
// above 256 experts, k rounds over the whole keys take the warp's maximum and the
// lowest index among equal ones.
//
// Measured: 64 tokens of 8 experts 1.9 us; 8192 of 256 in groups with a bias 14.3 us
// (8.9 MB, 1.3 us of HBM; 1,420 instructions a token, 62% of the issue slots);
// 16,384 of 256 with the gradient 22 us (42 MB).  Whole keys instead of cut ones: 17.8
// and 30 us.
#include "block_common.cuh"

namespace moe {

constexpr int ROUTE_WARPS = 8;

struct RouteParams {
  int64_t T;
  int E, k;
  const void* logits;
  int64_t stride0;
  const float* bias;
  const uint8_t* is_padding;
  int sigmoid, renorm;
  int score_key;  // softmax with a bias: it is added to the score
  float scale;
  int groups, top_groups;
  void* ids;
  int ids64;
  float* weights;
  const float* d_weights;  // backward
  void* d_logits;
  int64_t d_stride0;
};

// Order-preserving key of a float; 0 for NaN and -inf (not selectable).
// Adding +0 makes -0 and +0 one key.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return f > -INFINITY ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// exp(l - m), 1 where l is the maximum itself (also an infinite one), 0 for NaN.
__device__ __forceinline__ float exp_rel(float l, float m) {
  return l == m ? 1.0f : (l < m ? expf(l - m) : 0.0f);
}

// l becomes exp(l - m) for the warp's largest logit m; NaN and -inf give 0.
template <int VPL>
__device__ __forceinline__ void exp_row(float (&l)[VPL], float m) {
  if (fabsf(m) < INFINITY) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = expf((l[i] > -INFINITY ? l[i] : -INFINITY) - m);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = l[i] > -INFINITY ? exp_rel(l[i], m) : 0.0f;
  }
}

__device__ __forceinline__ int64_t load_id(const void* ids, int ids64, int64_t i) {
  return ids64 ? static_cast<const int64_t*>(ids)[i] : (int64_t)static_cast<const int32_t*>(ids)[i];
}

// Largest key of the warp, as the logit that it stands for.
__device__ __forceinline__ float warp_max_key(uint32_t k) {
  return key_value(__reduce_max_sync(0xFFFFFFFFu, k));
}

// A group's value from its two highest keys (0: none).  Two keys near the lowest float
// (masked experts) add up to -inf; such a group comes after all others and before those
// that have no expert to take, so its value is 1.
__device__ __forceinline__ uint32_t group_key(const RouteParams& p, uint32_t k1, uint32_t k2) {
  if (p.bias == nullptr || k1 == 0) return k1;
  return max(order_key(__fadd_rn(key_value(k1), k2 ? key_value(k2) : 0.0f)), 1u);
}

// Whether group g, whose value lane g << shift has in gk, is among the best
// top_groups: fewer than these come before it.  Bit g << shift of the answer.
__device__ __forceinline__ uint32_t best_groups(const RouteParams& p, uint32_t gk, int g,
                                                int shift) {
  int before = 0;
  for (int o = 0; o < p.groups; ++o) {
    const uint32_t v = __shfl_sync(0xFFFFFFFFu, gk, o << shift);
    before += (v > gk || (v == gk && o < g)) ? 1 : 0;
  }
  return __ballot_sync(0xFFFFFFFFu, g < p.groups && gk != 0 && before < p.top_groups);
}

// Clears the keys of experts outside the best top_groups groups.  Where groups
// are whole multiples of 32 experts, a register of the warp belongs to one group.
// Otherwise the keys go through shared memory; lpg lanes share a group, each
// starting at an offset of its own so that the groups' lanes fall into different
// banks.
template <int VPL>
__device__ __forceinline__ void limit_groups(const RouteParams& p, uint32_t (&key)[VPL],
                                             uint32_t* sk, int lane) {
  const int size = p.E / p.groups;
  if (size % 32 == 0) {
    const int regs = size / 32;
    uint32_t gk = 0, k1 = 0, k2 = 0;
    int g = 0, in = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (i * 32 >= p.E) break;
      k2 = max(k2, min(k1, key[i]));
      k1 = max(k1, key[i]);
      if (++in < regs) continue;
      const uint32_t m1 = __reduce_max_sync(0xFFFFFFFFu, k1);
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, k1 == m1);
      const uint32_t m2 =
          __reduce_max_sync(0xFFFFFFFFu, lane == __ffs(who) - 1 ? k2 : k1);
      if (lane == g) gk = group_key(p, m1, m2);
      k1 = k2 = 0;
      in = 0;
      ++g;
    }
    const uint32_t kept = best_groups(p, gk, lane, 0);
    g = in = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (!((kept >> g) & 1u)) key[i] = 0;
      if (++in == regs) in = 0, ++g;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    if (e < p.E) sk[e] = key[i];
  }
  __syncwarp();
  int lpg = 1, shift = 0;  // lanes per group, a power of two
  while (lpg * 2 * p.groups <= 32) lpg *= 2, ++shift;
  const int g = lane >> shift, sub = lane & (lpg - 1);
  uint32_t k1 = 0, k2 = 0;
  if (g < p.groups) {
    const int n = (size - sub + lpg - 1) >> shift;  // this lane's elements sub, sub + lpg, ...
    int j = n > 0 ? g % n : 0;
    for (int i = 0; i < n; ++i) {
      const uint32_t v = sk[g * size + sub + (j << shift)];
      k2 = max(k2, min(k1, v));
      k1 = max(k1, v);
      if (++j == n) j = 0;
    }
  }
  for (int o = 1; o < lpg; o <<= 1) {
    const uint32_t a = __shfl_xor_sync(0xFFFFFFFFu, k1, o), b = __shfl_xor_sync(0xFFFFFFFFu, k2, o);
    k2 = max(max(k2, b), min(k1, a));
    k1 = max(k1, a);
  }
  const uint32_t kept = best_groups(p, g < p.groups ? group_key(p, k1, k2) : 0, g, shift);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    if (e < p.E && !((kept >> ((e / size) << shift)) & 1u)) key[i] = 0;
  }
}

__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {  // a >= b
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
// Descending, by a sorting network.
template <int VPL>
__device__ __forceinline__ void sort_keys(uint32_t (&c)[VPL]) {
  if constexpr (VPL == 2) order2(c[0], c[1]);
  if constexpr (VPL == 4 || VPL == 8) {
#pragma unroll
    for (int h = 0; h < VPL; h += 4) {
      order2(c[h], c[h + 1]), order2(c[h + 2], c[h + 3]);
      order2(c[h], c[h + 2]), order2(c[h + 1], c[h + 3]);
      order2(c[h + 1], c[h + 2]);
    }
  }
  if constexpr (VPL == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) order2(c[i], c[i + 4]);
    order2(c[2], c[4]), order2(c[3], c[5]);
    order2(c[1], c[2]), order2(c[3], c[4]), order2(c[5], c[6]);
  }
}

// The k experts of highest key, lane j the j-th (-1: none left).  Uses keys up.
template <int VPL>
__device__ __forceinline__ int take_exact(uint32_t (&key)[VPL], int k, int lane) {
  uint32_t bk = 0;
  int bi = 0, my_id = -1;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (key[i] > bk) bk = key[i], bi = i;
  for (int j = 0; j < k; ++j) {
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, bk);
    if (m == 0) break;
    const uint32_t win =
        __reduce_min_sync(0xFFFFFFFFu, bk == m ? (uint32_t)(bi * 32 + lane) : 0x7FFFFFFFu);
    if (lane == j) my_id = (int)win;
    if ((int)(win & 31u) == lane) {
      const int wi = (int)(win >> 5);
      bk = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (i == wi) key[i] = 0;
        if (key[i] > bk) bk = key[i], bi = i;
      }
    }
  }
  return my_id;
}

// The same by cut keys; `whole`: the cut bits of every key are zero.  False when the
// cut keys do not decide (the same for the whole warp).
template <int VPL>
__device__ __forceinline__ bool take_cut(const uint32_t (&key)[VPL], int k, int lane, bool whole,
                                         int* id) {
  constexpr uint32_t mask = VPL * 32 - 1;
  uint32_t c[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    c[i] = key[i] ? (key[i] & ~mask) | (mask - (uint32_t)(i * 32 + lane)) : 0u;
  sort_keys<VPL>(c);
  uint32_t mine = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, c[0]);
    if (lane == j) mine = m;
    if (c[0] == m) {
#pragma unroll
      for (int i = 0; i + 1 < VPL; ++i) c[i] = c[i + 1];
      c[VPL - 1] = 0;
    }
  }
  // lane j against the one taken after it, the last against the largest left
  const uint32_t left = __reduce_max_sync(0xFFFFFFFFu, c[0]);
  const uint32_t after = __shfl_down_sync(0xFFFFFFFFu, mine, 1);
  const uint32_t next = lane == k - 1 ? left : after;
  const bool tie =
      __any_sync(0xFFFFFFFFu, lane < k && next != 0 && ((mine ^ next) & ~mask) == 0);
  *id = mine != 0 ? (int)(mask - (mine & mask)) : -1;
  return whole || !tie;
}

// SCORE_KEY: softmax with the bias on the score, exp(l - m) / z + bias; an expert whose logit
// is NaN or -inf is not selectable then, whatever its bias.
template <typename T, int VPL, bool SCORE_KEY>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) route_kernel(RouteParams p) {
  extern __shared__ uint32_t smem_keys[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp;
  pdl_wait();
  pdl_launch_dependents();
  if (t >= p.T) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.stride0;
  float l[VPL];
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    l[i] = e < p.E ? to_f32(row[e]) : -INFINITY;
  }
  float m_all = -INFINITY, z_all = 0.0f;
  // l becomes exp(l - m), m and z the row's
  auto row_softmax = [&](uint32_t top) {
    m_all = warp_max_key(top);
    exp_row<VPL>(l, m_all);
#pragma unroll
    for (int i = 0; i < VPL; ++i) z_all += l[i];
    z_all = warp_sum(z_all);
  };
  if constexpr (SCORE_KEY) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      key[i] = order_key(l[i]);
      top = max(top, key[i]);
    }
    row_softmax(top);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 32 + lane;
      if (key[i] != 0) key[i] = order_key(__fadd_rn(__fdiv_rn(l[i], z_all), __ldg(p.bias + e)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 32 + lane;
      float v = l[i];
      if (p.bias != nullptr && e < p.E)
        v = __fadd_rn(p.sigmoid ? sigmoid(v) : v, __ldg(p.bias + e));
      key[i] = e < p.E ? order_key(v) : 0u;
    }
    if (!p.sigmoid && !p.renorm) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) top = max(top, p.bias == nullptr ? key[i] : order_key(l[i]));
      row_softmax(top);
    }
  }
  if (p.groups > 1) limit_groups<VPL>(p, key, smem_keys + warp * p.E, lane);
  const bool padding = p.is_padding != nullptr && p.is_padding[t] != 0;
  int my_id = -1;
  if (!padding) {
    bool decided = false;
    if constexpr (VPL <= 8)
      decided = take_cut<VPL>(key, p.k, lane, sizeof(T) == 2 && p.bias == nullptr, &my_id);
    if (!decided) my_id = take_exact<VPL>(key, p.k, lane);
  }
  // lane j holds the j-th expert
  const float lv = my_id >= 0 ? to_f32(row[my_id]) : -INFINITY;
  float w = 0.0f, total = 1.0f;
  if (p.sigmoid) {
    if (my_id >= 0) w = sigmoid(lv);
    if (p.renorm) total = warp_sum(w) + 1e-20f;
  } else if (p.renorm) {
    const float m = warp_max(lv);
    if (my_id >= 0) w = exp_rel(lv, m);
    total = fmaxf(warp_sum(w), 1e-20f);
  } else {
    if (my_id >= 0) w = exp_rel(lv, m_all);
    total = z_all;
  }
  if (lane < p.k) {
    const int64_t o = t * p.k + lane;
    if (p.ids64)
      static_cast<int64_t*>(p.ids)[o] = my_id;
    else
      static_cast<int32_t*>(p.ids)[o] = my_id;
    p.weights[o] = my_id >= 0 ? w / total * p.scale : 0.0f;
  }
}

// Gradient of the logits.  With dw scaled and p the weight before the scale:
//   softmax               d_e = p_e (dw_e - sum_j dw_j p_j)   (dw_e = 0 unless taken)
//   softmax, renormalised the same over the taken experts alone
//   sigmoid               d_e = dw_e s_e (1 - s_e)
//   sigmoid, renormalised d_e = (dw_e - sum_j dw_j p_j) / total * s_e (1 - s_e)
// Every lane stores its columns of the row (zeros but for the first form),
// then lanes j < k overwrite the taken columns.
template <typename T, int VPL>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) route_backward_kernel(RouteParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp;
  pdl_wait();
  pdl_launch_dependents();
  if (t >= p.T) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.stride0;
  T* drow = static_cast<T*>(p.d_logits) + t * p.d_stride0;
  int64_t id = -1;
  float dw = 0.0f, lv = -INFINITY;
  if (lane < p.k) {
    id = load_id(p.ids, p.ids64, t * p.k + lane);
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) {
      dw = p.d_weights[t * p.k + lane] * p.scale;
      lv = to_f32(row[id]);
    }
  }
  float d = 0.0f;
  if (!p.sigmoid && !p.renorm) {
    float l[VPL], z = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 32 + lane;
      l[i] = e < p.E ? to_f32(row[e]) : -INFINITY;
      top = max(top, order_key(l[i]));
    }
    const float m = warp_max_key(top);
    exp_row<VPL>(l, m);
#pragma unroll
    for (int i = 0; i < VPL; ++i) z += l[i];
    z = warp_sum(z);
    const float inv = z > 0.0f ? 1.0f / z : 0.0f;
    const float w = id >= 0 ? exp_rel(lv, m) * inv : 0.0f;
    const float mean = warp_sum(dw * w);
    d = w * (dw - mean);
    const float base = -(inv * mean);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 32 + lane;
      if (e < p.E) drow[e] = from_f32<T>(l[i] * base);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 32 + lane;
      if (e < p.E) drow[e] = from_f32<T>(0.0f);
    }
    if (p.sigmoid) {
      const float s = id >= 0 ? sigmoid(lv) : 0.0f;
      float up = dw;
      if (p.renorm) {
        const float total = warp_sum(s) + 1e-20f;
        up = (dw - warp_sum(dw * (s / total))) / total;
      }
      d = up * s * (1.0f - s);
    } else {
      const float m = warp_max(lv);
      const float x = id >= 0 ? exp_rel(lv, m) : 0.0f;
      const float w = x / fmaxf(warp_sum(x), 1e-20f);
      d = w * (dw - warp_sum(dw * w));
    }
  }
  __syncwarp();  // the row's stores come before those of the taken columns
  if (id >= 0) drow[id] = from_f32<T>(d);
}

}  // namespace moe

namespace moe_host {

using moe::RouteParams;

template <typename T, int VPL>
static moe_status_t launch_one(const RouteParams& p, bool backward, cudaStream_t s) {
  const dim3 grid((unsigned)((p.T + moe::ROUTE_WARPS - 1) / moe::ROUTE_WARPS));
  const dim3 block(moe::ROUTE_WARPS * 32);
  if (backward)
    return launched(launch_pdl(moe::route_backward_kernel<T, VPL>, grid, block, 0, s, p),
                    "route backward");
  const size_t smem = p.groups > 1 ? (size_t)moe::ROUTE_WARPS * p.E * 4 : 0;  // <= 32 KB
  if (p.score_key)
    return launched(launch_pdl(moe::route_kernel<T, VPL, true>, grid, block, smem, s, p), "route");
  return launched(launch_pdl(moe::route_kernel<T, VPL, false>, grid, block, smem, s, p), "route");
}

static moe_status_t launch_any(const RouteParams& p, int32_t dtype, bool backward,
                               cudaStream_t s) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    // keys a lane: the smallest power of two that holds the experts, unused ones costing
    // issue slots
    if (p.E <= 32) return launch_one<T, 1>(p, backward, s);
    if (p.E <= 64) return launch_one<T, 2>(p, backward, s);
    if (p.E <= 128) return launch_one<T, 4>(p, backward, s);
    if (p.E <= 256) return launch_one<T, 8>(p, backward, s);
    if (p.E <= 512) return launch_one<T, 16>(p, backward, s);
    return launch_one<T, 32>(p, backward, s);
  });
}

}  // namespace moe_host

using namespace moe_host;

static moe_status_t check_route(int64_t T, int64_t E, int64_t k, int32_t dtype, int32_t scoring,
                                int32_t ids_dtype) {
  if (T < 0 || E < 0 || k < 0) return set_error(MOE_ERR_INVALID_ARGUMENT, "negative size");
  if (!dtype_ok(dtype)) return set_error(MOE_ERR_INVALID_ARGUMENT, "bad logits_dtype %d", dtype);
  const int32_t form = scoring & ~MOE_SCORE_BIAS_ON_SCORE;
  if (form != MOE_SCORE_SOFTMAX && form != MOE_SCORE_SIGMOID)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "bad scoring %d", scoring);
  if (ids_dtype != MOE_IDS_INT32 && ids_dtype != MOE_IDS_INT64)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "bad topk_ids_dtype");
  if (k < 1 || k > E)
    return set_error(MOE_ERR_SHAPE, "top_k %lld outside [1, %lld experts]", (long long)k,
                     (long long)E);
  if (E > 1024 || k > 32)
    return set_error(MOE_ERR_UNSUPPORTED, "routing supports at most 1024 experts and top_k 32");
  if (T > ((int64_t)1 << 33)) return set_error(MOE_ERR_UNSUPPORTED, "too many tokens");
  return MOE_OK;
}

extern "C" {

moe_status_t moe_route(const moe_route_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  moe_status_t st = check_route(a->num_tokens, a->num_experts, a->top_k, a->logits_dtype,
                                a->scoring, a->topk_ids_dtype);
  if (st != MOE_OK) return st;
  if (a->num_groups < 1 || a->num_experts % a->num_groups != 0 || a->top_groups < 1 ||
      a->top_groups > a->num_groups ||
      a->top_k > a->top_groups * (a->num_experts / a->num_groups))
    return set_error(MOE_ERR_SHAPE, "bad groups: %lld of %lld over %lld experts, top_k %lld",
                     (long long)a->top_groups, (long long)a->num_groups,
                     (long long)a->num_experts, (long long)a->top_k);
  if (a->num_groups > 32) return set_error(MOE_ERR_UNSUPPORTED, "at most 32 groups");
  if (a->num_tokens == 0) return MOE_OK;
  if (!a->logits || !a->topk_ids || !a->topk_weights)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if (a->num_tokens > 1 && a->logits_stride0 < a->num_experts)
    return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
  RouteParams p{};
  p.T = a->num_tokens;
  p.E = (int)a->num_experts;
  p.k = (int)a->top_k;
  p.logits = a->logits;
  p.stride0 = a->logits_stride0;
  p.bias = a->bias;
  p.is_padding = a->is_padding;
  p.sigmoid = (a->scoring & ~MOE_SCORE_BIAS_ON_SCORE) == MOE_SCORE_SIGMOID;
  p.renorm = a->renormalize != 0;
  p.score_key = !p.sigmoid && p.bias != nullptr && (a->scoring & MOE_SCORE_BIAS_ON_SCORE) != 0;
  p.scale = a->scale;
  p.groups = (int)a->num_groups;
  p.top_groups = (int)a->top_groups;
  p.ids = a->topk_ids;
  p.ids64 = a->topk_ids_dtype == MOE_IDS_INT64;
  p.weights = a->topk_weights;
  return launch_any(p, a->logits_dtype, false, static_cast<cudaStream_t>(stream));
}

moe_status_t moe_route_backward(const moe_route_backward_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  moe_status_t st = check_route(a->num_tokens, a->num_experts, a->top_k, a->logits_dtype,
                                a->scoring, a->topk_ids_dtype);
  if (st != MOE_OK) return st;
  if (a->num_tokens == 0) return MOE_OK;
  if (!a->logits || !a->topk_ids || !a->d_weights || !a->d_logits)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if (a->num_tokens > 1 &&
      (a->logits_stride0 < a->num_experts || a->d_logits_stride0 < a->num_experts))
    return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
  RouteParams p{};
  p.T = a->num_tokens;
  p.E = (int)a->num_experts;
  p.k = (int)a->top_k;
  p.logits = a->logits;
  p.stride0 = a->logits_stride0;
  p.sigmoid = (a->scoring & ~MOE_SCORE_BIAS_ON_SCORE) == MOE_SCORE_SIGMOID;
  p.renorm = a->renormalize != 0;
  p.scale = a->scale;
  p.groups = p.top_groups = 1;
  p.ids = const_cast<void*>(a->topk_ids);
  p.ids64 = a->topk_ids_dtype == MOE_IDS_INT64;
  p.d_weights = a->d_weights;
  p.d_logits = a->d_logits;
  p.d_stride0 = a->d_logits_stride0;
  return launch_any(p, a->logits_dtype, true, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
