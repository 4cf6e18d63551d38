// Router: top-k ids and weights of logits, and the gradient of the logits.
//
// One warp per token; lane i holds logits i, i + 32, i + 64, ... in registers,
// so a row is read once and coalesced.  Selection compares order-preserving
// 32-bit integers of the keys: k rounds, each a warp maximum of the lanes' best
// keys (redux.sync) and a warp minimum of the index among equal ones.  Without
// a bias the key is the logit itself (softmax and sigmoid are monotone), so the
// choice does not depend on how exp rounds.  With a sigmoid and a bias the key
// is 1/(1+expf(-l)) + bias with IEEE division and no contraction, the value that
// elementary fp32 tensor operations give.
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

__device__ __forceinline__ int64_t load_id(const void* ids, int ids64, int64_t i) {
  return ids64 ? static_cast<const int64_t*>(ids)[i] : (int64_t)static_cast<const int32_t*>(ids)[i];
}

// Clears the keys of experts outside the best top_groups groups.  The keys go
// through shared memory; lanes_per_group lanes share a group, each starting at
// an offset of its own so that the groups' lanes fall into different banks.
template <int VPL>
__device__ __forceinline__ void limit_groups(const RouteParams& p, uint32_t (&key)[VPL],
                                             uint32_t* sk, int lane) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    if (e < p.E) sk[e] = key[i];
  }
  __syncwarp();
  const int size = p.E / p.groups;
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
  uint32_t gk = k1;
  if (p.bias != nullptr && k1 != 0) gk = order_key(key_value(k1) + (k2 ? key_value(k2) : 0.0f));
  if (g >= p.groups) gk = 0;
  // a group stays when fewer than top_groups others come before it
  int before = 0;
  for (int o = 0; o < p.groups; ++o) {
    const uint32_t v = __shfl_sync(0xFFFFFFFFu, gk, o << shift);
    before += (v > gk || (v == gk && o < g)) ? 1 : 0;
  }
  const bool stays = g < p.groups && gk != 0 && before < p.top_groups;
  const uint32_t kept = __ballot_sync(0xFFFFFFFFu, stays);  // bit g << shift
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    if (e < p.E && !((kept >> ((e / size) << shift)) & 1u)) key[i] = 0;
  }
}

template <typename T, int VPL>
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
  if (!p.sigmoid && !p.renorm) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) m_all = fmaxf(m_all, l[i]);
    m_all = warp_max(m_all);
#pragma unroll
    for (int i = 0; i < VPL; ++i) z_all += l[i] > -INFINITY ? exp_rel(l[i], m_all) : 0.0f;
    z_all = warp_sum(z_all);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    float v = l[i];
    if (p.bias != nullptr && e < p.E) v = __fadd_rn(p.sigmoid ? sigmoid(v) : v, __ldg(p.bias + e));
    key[i] = e < p.E ? order_key(v) : 0u;
  }
  if (p.groups > 1) limit_groups<VPL>(p, key, smem_keys + warp * p.E, lane);
  const bool padding = p.is_padding != nullptr && p.is_padding[t] != 0;

  uint32_t bk = 0;
  int bi = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (key[i] > bk) bk = key[i], bi = i;
  int my_id = -1;
  for (int j = 0; j < p.k && !padding; ++j) {
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, bk);
    if (m == 0) break;
    const uint32_t win = __reduce_min_sync(0xFFFFFFFFu, bk == m ? (uint32_t)(bi * 32 + lane) : 0x7FFFFFFFu);
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
    float l[VPL], m = -INFINITY, z = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 32 + lane;
      l[i] = e < p.E ? to_f32(row[e]) : -INFINITY;
      m = fmaxf(m, l[i]);
    }
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      l[i] = l[i] > -INFINITY ? exp_rel(l[i], m) : 0.0f;
      z += l[i];
    }
    z = warp_sum(z);
    const float w = id >= 0 ? exp_rel(lv, m) / z : 0.0f;
    const float mean = warp_sum(dw * w);
    d = w * (dw - mean);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 32 + lane;
      if (e < p.E) drow[e] = from_f32<T>(z > 0.0f ? -(l[i] / z) * mean : 0.0f);
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
  return launched(launch_pdl(moe::route_kernel<T, VPL>, grid, block, smem, s, p), "route");
}

static moe_status_t launch_any(const RouteParams& p, int32_t dtype, bool backward,
                               cudaStream_t s) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
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
  if (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID)
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
  p.sigmoid = a->scoring == MOE_SCORE_SIGMOID;
  p.renorm = a->renormalize != 0;
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
  p.sigmoid = a->scoring == MOE_SCORE_SIGMOID;
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
