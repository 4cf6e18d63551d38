// Rows sorted by expert and back with the routing weights applied, and the
// gradients of both.
//
// moe_sort_routes is a stable counting sort: a route's row is the number of
// routes to lower experts plus that of earlier routes to its own.  Blocks take
// consecutive routes and the warps of a block consecutive segments; in a warp
// __match_any_sync gives the rank among 32 routes and a shared table of counts
// per (warp, expert) the ranks across its segment.  Up to kSortOneBlock routes
// one block does it all; above, a first launch counts each block's routes per
// expert and a second one places them, every block summing the counts of the
// blocks before it.  No atomics on results, so rows are the same every time.
//
// The row kernels move each routed row once: moe_permute reads a token's row
// once and writes it to its k rows, moe_unpermute reads k rows and writes one,
// the gradient of the weights comes from the same reads that scale d_out.
// All are bound by HBM.  Measured at 8192 tokens x 8 routes x 7168 bf16 (1.06 GB each
// way): permute 178 us, 5.9 TB/s; unpermute 155 us, 6.8 TB/s; at 2051 x 6 x 4096 fp16 the
// gradient of unpermute 32 us, permute and unpermute 19 and 20 us.
#include "block_common.cuh"

namespace moe {

constexpr int SORT_WARPS = 16;
constexpr int SORT_THREADS = SORT_WARPS * 32;
constexpr int SORT_MAX_EXPERTS = 1024;
constexpr int SORT_BLOCKS = 128;          // while their shares stay within
constexpr int SORT_MAX_PER_BLOCK = 32768;  // (ranks in a block are 16 bits)

struct SortParams {
  const void* ids;
  int ids64;
  int none_last;  // ids outside [0, E - 1) count as E - 1 (adapters: tokens without one)
  int align;       // experts begin at multiples of this, the rows between are -1
  int32_t R, E, blocks, per_block;  // per_block: a multiple of SORT_THREADS
  int32_t rows;    // length of row_route
  int32_t* offsets;
  int32_t* route_row;
  int32_t* row_route;
  int32_t* hist;  // [E, hist_row]: an expert's counts by block
  int hist_row;   // blocks, up to a multiple of four
  uint32_t* status;
};

// Expert of route r, or -1.
__device__ __forceinline__ int route_expert(const SortParams& p, int r, bool* bad) {
  const int64_t id = p.ids64 ? static_cast<const int64_t*>(p.ids)[r]
                             : (int64_t)static_cast<const int32_t*>(p.ids)[r];
  if (p.none_last) return id >= 0 && id < p.E ? (int)id : p.E - 1;
  if (id >= p.E) *bad = true;
  return id >= 0 && id < p.E ? (int)id : -1;
}

__global__ void __launch_bounds__(SORT_THREADS) sort_count_kernel(SortParams p) {
  __shared__ int cnt[SORT_MAX_EXPERTS];
  for (int e = threadIdx.x; e < p.E; e += SORT_THREADS) cnt[e] = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const int r0 = blockIdx.x * p.per_block, r1 = min(p.R, r0 + p.per_block);
  bool bad = false;
  for (int r = r0 + threadIdx.x; r < r1; r += SORT_THREADS) {
    const int e = route_expert(p, r, &bad);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  if (bad) set_status(p.status, MOE_DEV_BAD_EXPERT);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += SORT_THREADS) p.hist[e * p.hist_row + blockIdx.x] = cnt[e];
}

__global__ void __launch_bounds__(SORT_THREADS) sort_place_kernel(SortParams p) {
  // count of (warp, expert), then the rank in the block of the warp's next route:
  // at most per_block < 65536
  __shared__ uint16_t table[SORT_WARPS][SORT_MAX_EXPERTS];
  __shared__ int base[SORT_MAX_EXPERTS];  // first row of this block's routes of an expert
  __shared__ int warp_total[SORT_WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int e = lane; e < p.E; e += 32) table[warp][e] = 0;  // each warp its own row
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const int per_warp = p.per_block / SORT_WARPS;
  const int w0 = min((int64_t)p.R, (int64_t)blockIdx.x * p.per_block + (int64_t)warp * per_warp);
  const int w1 = min((int64_t)p.R, (int64_t)w0 + per_warp);
  bool bad = false;
  for (int r0 = w0; r0 < w1; r0 += 32) {
    const int r = r0 + lane;
    const int e = r < w1 ? route_expert(p, r, &bad) : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    if (e >= 0 && (same & lanemask_lt()) == 0) table[warp][e] += (uint16_t)__popc(same);
    __syncwarp();
  }
  if (bad && p.blocks == 1) set_status(p.status, MOE_DEV_BAD_EXPERT);
  __syncthreads();
  // per expert: the counts become exclusive prefixes over the warps; the rows
  // before this block's are those of all blocks to lower experts (scanned
  // below) and of earlier blocks to the same expert
  int carry = 0;
  for (int e0 = 0; e0 < p.E; e0 += SORT_THREADS) {
    const int e = e0 + tid;
    int mine = 0, all = 0, before = 0;
    if (e < p.E) {
      for (int w = 0; w < SORT_WARPS; ++w) {
        const int c = table[w][e];
        table[w][e] = (uint16_t)mine;
        mine += c;
      }
      if (p.blocks == 1) {
        all = mine;
      } else {
        // sixteen blocks' counts in flight; what lies past the last block is not used
        const int4* row = reinterpret_cast<const int4*>(p.hist + e * p.hist_row);
        for (int b0 = 0; b0 < p.blocks; b0 += 16) {
          int4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = b0 + 4 * i < p.hist_row ? __ldcg(row + b0 / 4 + i) : make_int4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int b = b0 + 4 * i + j;
              if (b < p.blocks) all += c[j];
              if (b < (int)blockIdx.x) before += c[j];
            }
          }
        }
      }
    }
    const int room = (all + p.align - 1) / p.align * p.align;
    int incl = room;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    int below = carry;
    for (int w = 0; w < SORT_WARPS; ++w) {
      if (w < warp) below += warp_total[w];
      carry += warp_total[w];
    }
    if (e < p.E) {
      const int start = below + incl - room;
      base[e] = start + before;
      if (blockIdx.x == 0) {
        p.offsets[e] = start;
        for (int r = start + all; r < start + room; ++r) p.row_route[r] = -1;
      }
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) p.offsets[p.E] = carry;
  for (int r0 = w0; r0 < w1; r0 += 32) {
    const int r = r0 + lane;
    bool unused = false;
    const int e = r < w1 ? route_expert(p, r, &unused) : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    int row = -1;
    if (e >= 0) {
      row = base[e] + table[warp][e] + __popc(same & lanemask_lt());
      p.row_route[row] = r;
    }
    if (r < w1) p.route_row[r] = row;
    __syncwarp();
    if (e >= 0 && (same & lanemask_lt()) == 0) table[warp][e] += (uint16_t)__popc(same);
    __syncwarp();
  }
  for (int64_t r = (int64_t)carry + (int64_t)blockIdx.x * SORT_THREADS + tid; r < p.rows;
       r += (int64_t)gridDim.x * SORT_THREADS)
    p.row_route[r] = -1;
}

struct RowParams {
  int64_t T, K, num_rows;
  int k;
  const int32_t* route_row;
  const float* w;         // nullable
  const int32_t* offsets;  // [E + 1]
  int64_t E;
  const void* x;  // token rows read
  int64_t x_stride;
  const void* rows;  // expert rows read
  int64_t rows_stride;
  void* out;  // token rows written
  int64_t out_stride;
  void* out_rows;  // expert rows written
  int64_t out_rows_stride;
  float* d_w;
};

// A warp's way over (token, chunk) tasks, nwarps apart, without a division each.
struct Walk {
  int64_t t, dt;
  int c, dc, chunks;
  __device__ __forceinline__ Walk(int64_t first, int64_t step, int n)
      : t(first / n), dt(step / n), c((int)(first % n)), dc((int)(step % n)), chunks(n) {}
  __device__ __forceinline__ void next() {
    t += dt;
    c += dc;
    if (c >= chunks) c -= chunks, ++t;
  }
};

// Row of route (t, lane) for lane < k, or -1.
__device__ __forceinline__ int lane_row(const RowParams& p, int64_t t, int lane) {
  const int r = lane < p.k ? p.route_row[t * p.k + lane] : -1;
  return r >= 0 && r < p.num_rows ? r : -1;
}

// One warp per (token, PERMUTE_VECS * 32 packs of the row): the packs are read
// once and written to the k rows.  Tasks past the tokens clear the rows past
// the last routed one.
constexpr int PERMUTE_VECS = 4;

template <typename T, int VEC>
__global__ void __launch_bounds__(256) permute_kernel(RowParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t gwarp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  constexpr int chunk = PERMUTE_VECS * 32 * VEC;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t used = min(max((int64_t)p.offsets[p.E], (int64_t)0), p.num_rows);
  const int64_t rows_and_rest = p.T + p.num_rows - used;
  T* rows = static_cast<T*>(p.out_rows);
  for (Walk w(gwarp, nwarps, (int)((p.K + chunk - 1) / chunk)); w.t < rows_and_rest; w.next()) {
    const int64_t t = w.t;
    const int64_t c0 = (int64_t)w.c * chunk + lane * VEC;
    Pack<T, VEC> v[PERMUTE_VECS];
    if (t >= p.T) {
      T* dst = rows + (used + t - p.T) * p.out_rows_stride;
      const Pack<T, VEC> zero = zero_pack<T, VEC>();
#pragma unroll
      for (int i = 0; i < PERMUTE_VECS; ++i)
        if (c0 + i * 32 * VEC < p.K) store_pack<T, VEC>(dst + c0 + i * 32 * VEC, zero);
      continue;
    }
    const int my_row = lane_row(p, t, lane);
    const T* src = static_cast<const T*>(p.x) + t * p.x_stride;
#pragma unroll
    for (int i = 0; i < PERMUTE_VECS; ++i)
      if (c0 + i * 32 * VEC < p.K) v[i] = load_pack_stream<T, VEC>(src + c0 + i * 32 * VEC);
    for (int j = 0; j < p.k; ++j) {
      const int row = __shfl_sync(0xFFFFFFFFu, my_row, j);
      if (row < 0) continue;
      T* dst = rows + (int64_t)row * p.out_rows_stride;
#pragma unroll
      for (int i = 0; i < PERMUTE_VECS; ++i)
        if (c0 + i * 32 * VEC < p.K) store_pack<T, VEC>(dst + c0 + i * 32 * VEC, v[i]);
    }
  }
}

// One warp per (token, CH times 32 packs): KB routes' packs are read at a time, KB
// CH = 8 of them in flight a lane (loads that a branch guards are not in flight
// together, so absent rows are selected afterwards: 8192 x 8 routes there and back 352 us,
// guarded 474), and summed in fp32 in ascending j.
template <typename T, int VEC, int KB>
__global__ void __launch_bounds__(256) unpermute_kernel(RowParams p) {
  constexpr int CH = 8 / KB, chunk = CH * 32 * VEC;
  const int lane = threadIdx.x & 31;
  const int64_t gwarp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const T* rows = static_cast<const T*>(p.rows);
  for (Walk w(gwarp, nwarps, (int)((p.K + chunk - 1) / chunk)); w.t < p.T; w.next()) {
    const int64_t t = w.t;
    const int64_t c0 = (int64_t)w.c * chunk + lane * VEC;
    const int my_row = lane_row(p, t, lane);
    const float my_w = my_row >= 0 ? (p.w != nullptr ? p.w[t * p.k + lane] : 1.0f) : 0.0f;
    float acc[CH][VEC];
#pragma unroll
    for (int h = 0; h < CH; ++h)
#pragma unroll
      for (int q = 0; q < VEC; ++q) acc[h][q] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += KB) {
      Pack<T, VEC> v[KB][CH];
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        // routes past the last read as absent: lanes >= k hold none
        const int row = j0 + i < 32 ? __shfl_sync(0xFFFFFFFFu, my_row, j0 + i) : -1;
#pragma unroll
        for (int h = 0; h < CH; ++h)
          v[i][h] = row >= 0 && c0 + h * 32 * VEC < p.K
                        ? load_pack_stream<T, VEC>(rows + (int64_t)row * p.rows_stride + c0 +
                                                   h * 32 * VEC)
                        : zero_pack<T, VEC>();
      }
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        const float wt = __shfl_sync(0xFFFFFFFFu, my_w, (j0 + i) & 31);
        if (j0 + i >= p.k) break;
#pragma unroll
        for (int h = 0; h < CH; ++h) {
          float f[VEC];
          v[i][h].get(f);
#pragma unroll
          for (int q = 0; q < VEC; ++q) acc[h][q] = fmaf(wt, f[q], acc[h][q]);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      if (c0 + h * 32 * VEC >= p.K) break;
      Pack<T, VEC> o;
      o.set(acc[h]);
      store_pack<T, VEC>(static_cast<T*>(p.out) + t * p.out_stride + c0 + h * 32 * VEC, o);
    }
  }
}

// One block per token: each thread takes packs of d_out and, for eight routes
// at a time, reads their rows' packs (for the weights' gradients) and writes
// w * d_out in their place.  Tasks past the tokens clear the unused rows.
constexpr int BACK_THREADS = 256;

template <typename T, int VEC>
__global__ void __launch_bounds__(BACK_THREADS) unpermute_backward_kernel(RowParams p) {
  __shared__ float part[BACK_THREADS / 32][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t used = min(max((int64_t)p.offsets[p.E], (int64_t)0), p.num_rows);
  const int64_t tasks = p.T + p.num_rows - used;
  const T* rows = static_cast<const T*>(p.rows);
  T* d_rows = static_cast<T*>(p.out_rows);
  for (int64_t t = blockIdx.x; t < tasks; t += gridDim.x) {
    if (t >= p.T) {
      T* dst = d_rows + (used + t - p.T) * p.out_rows_stride;
      for (int64_t c = (int64_t)tid * VEC; c < p.K; c += BACK_THREADS * VEC)
        store_pack<T, VEC>(dst + c, zero_pack<T, VEC>());
      continue;
    }
    const int my_row = lane_row(p, t, lane);
    const float my_w = lane < p.k ? p.w[t * p.k + lane] : 0.0f;
    const T* up = static_cast<const T*>(p.x) + t * p.x_stride;
    for (int j0 = 0; j0 < p.k; j0 += 8) {
      int row[8];
      float w[8], dot[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        row[i] = __shfl_sync(0xFFFFFFFFu, my_row, (j0 + i) & 31);
        if (j0 + i >= p.k) row[i] = -1;
        w[i] = __shfl_sync(0xFFFFFFFFu, my_w, (j0 + i) & 31);
        dot[i] = 0.0f;
      }
      for (int64_t c = (int64_t)tid * VEC; c < p.K; c += BACK_THREADS * VEC) {
        float g[VEC];
        load_pack<T, VEC>(up + c).get(g);
        Pack<T, VEC> v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (row[i] >= 0)
            v[i] = load_pack_stream<T, VEC>(rows + (int64_t)row[i] * p.rows_stride + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (row[i] < 0) continue;
          float f[VEC], wg[VEC];
          v[i].get(f);
#pragma unroll
          for (int q = 0; q < VEC; ++q) {
            dot[i] = fmaf(g[q], f[q], dot[i]);
            wg[q] = w[i] * g[q];
          }
          Pack<T, VEC> o;
          o.set(wg);
          store_pack<T, VEC>(d_rows + (int64_t)row[i] * p.out_rows_stride + c, o);
        }
      }
      __syncthreads();  // the sums of the routes before have been read
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dot[i] = warp_sum(dot[i]);
        if (lane == 0) part[warp][i] = dot[i];
      }
      __syncthreads();
      if (tid < 8 && j0 + tid < p.k) {
        float sum = 0.0f;
        for (int v = 0; v < BACK_THREADS / 32; ++v) sum += part[v][tid];
        p.d_w[t * p.k + j0 + tid] = sum;
      }
    }
  }
}

}  // namespace moe

namespace moe_host {

using moe::RowParams;
using moe::SortParams;

// Up to this many routes one block sorts them in one launch: at 2048 7 us against 9.6 for
// two launches, at 4096 11 us against 9.6.
constexpr int64_t kSortOneBlock = 2048;

static void sort_split(int64_t R, int32_t* blocks, int32_t* per_block) {
  int64_t per = 1024;
  if (R <= kSortOneBlock)
    per = kSortOneBlock;
  else if (R > per * moe::SORT_BLOCKS)
    per = ((R + moe::SORT_BLOCKS - 1) / moe::SORT_BLOCKS + 511) / 512 * 512;
  if (per > moe::SORT_MAX_PER_BLOCK) per = moe::SORT_MAX_PER_BLOCK;
  *per_block = (int32_t)per;
  *blocks = (int32_t)((R + per - 1) / per);
}

static int32_t hist_row(int32_t blocks) { return (blocks + 3) / 4 * 4; }

// Most blocks that R routes or fewer are split among: grows with R, unlike sort_split's
// (128 at 131,072 routes, 86 at one more), so that a workspace serves fewer routes too.
static int32_t most_blocks(int64_t R) {
  if (R <= kSortOneBlock) return 1;
  int64_t blocks = (R + 1023) / 1024;
  if (blocks > moe::SORT_BLOCKS) blocks = moe::SORT_BLOCKS;
  const int64_t full = (R + moe::SORT_MAX_PER_BLOCK - 1) / moe::SORT_MAX_PER_BLOCK;
  return (int32_t)(blocks > full ? blocks : full);
}

static size_t sort_workspace(int64_t R, int64_t E) {
  return R <= kSortOneBlock ? 0 : (size_t)hist_row(most_blocks(R)) * E * 4;
}

static moe_status_t launch_sort(const SortParams& p, cudaStream_t s) {
  if (p.blocks > 1) {
    moe_status_t st = launched(launch_pdl(moe::sort_count_kernel, dim3(p.blocks),
                                          dim3(moe::SORT_THREADS), 0, s, p), "sort count");
    if (st != MOE_OK) return st;
  }
  return launched(launch_pdl(moe::sort_place_kernel, dim3(p.blocks), dim3(moe::SORT_THREADS), 0,
                             s, p), "sort place");
}

// Tokens in the order of their adapters, those without one last: order[rows],
// each adapter from a multiple of `align` on, -1 in between and at the end;
// rows >= T + (align - 1) (S + 1).  Scratch: token_order_scratch() words, of which
// scratch[S + 1] is then the number of places taken.
size_t token_order_scratch(int64_t T, int64_t S) {
  const int32_t blocks = most_blocks(T);
  return (size_t)((blocks > 1 ? hist_row(blocks) * (S + 1) + 3 : 0) + (S + 2) + T);
}

moe_status_t launch_token_order(const int32_t* adapter_ids, int64_t T, int64_t S, int align,
                                int32_t* order, int64_t rows, int32_t* scratch, cudaStream_t s) {
  SortParams p{};
  p.ids = adapter_ids;
  p.none_last = 1;
  p.align = align;
  p.R = (int32_t)T;
  p.E = (int32_t)S + 1;
  p.rows = (int32_t)rows;
  sort_split(T, &p.blocks, &p.per_block);
  p.offsets = scratch;
  p.route_row = scratch + S + 2;
  p.row_route = order;
  p.hist = scratch + (S + 2 + T + 3) / 4 * 4;  // scratch is 16-byte aligned
  p.hist_row = hist_row(p.blocks);
  return launch_sort(p, s);
}

template <typename K>
static dim3 one_wave(K kernel, int64_t blocks, int threads) {
  const int64_t cap =
      (int64_t)num_sms() * resident_blocks(reinterpret_cast<const void*>(kernel), threads);
  return dim3((unsigned)(blocks < 1 ? 1 : (blocks > cap ? cap : blocks)));
}

static moe_status_t check_rows(int64_t T, int64_t K, int64_t k, int64_t num_rows, int32_t dtype) {
  if (T < 0 || K < 0 || k < 0 || num_rows < 0)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "negative size");
  if (!dtype_ok(dtype)) return set_error(MOE_ERR_INVALID_ARGUMENT, "bad dtype %d", dtype);
  if (k > 32) return set_error(MOE_ERR_UNSUPPORTED, "at most 32 routes a token");
  if (num_rows >= ((int64_t)1 << 31))
    return set_error(MOE_ERR_UNSUPPORTED, "num_rows must be below 2^31");
  return MOE_OK;
}

// 16-byte packs where every row of every tensor of the call starts on a
// 16-byte boundary and K fills whole packs, else element by element.
static bool packs16(int64_t K, size_t elem) { return (K * (int64_t)elem) % 16 == 0; }

}  // namespace moe_host

using namespace moe_host;

extern "C" {

size_t moe_sort_workspace_size(int64_t num_tokens, int64_t top_k, int64_t num_experts) {
  if (num_tokens <= 0 || top_k <= 0 || num_experts <= 0) return 0;
  return sort_workspace(num_tokens * top_k, num_experts);
}

moe_status_t moe_sort_routes(const moe_sort_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t num_tokens = a->num_tokens, top_k = a->top_k, num_experts = a->num_experts;
  if (num_tokens < 0 || top_k < 0) return set_error(MOE_ERR_INVALID_ARGUMENT, "negative size");
  if (a->topk_ids_dtype != MOE_IDS_INT32 && a->topk_ids_dtype != MOE_IDS_INT64)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "bad topk_ids_dtype");
  if (num_experts < 1) return set_error(MOE_ERR_SHAPE, "num_experts must be >= 1");
  if (num_experts > moe::SORT_MAX_EXPERTS)
    return set_error(MOE_ERR_UNSUPPORTED, "at most %d experts", moe::SORT_MAX_EXPERTS);
  if (top_k > 0 && num_tokens > ((int64_t)1 << 26) / top_k)
    return set_error(MOE_ERR_UNSUPPORTED, "num_tokens * top_k must be at most 2^26");
  const int64_t R = num_tokens * top_k;
  if (!a->expert_offsets || (R > 0 && (!a->topk_ids || !a->route_row || !a->row_route)))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  SortParams p{};
  p.ids = a->topk_ids;
  p.ids64 = a->topk_ids_dtype == MOE_IDS_INT64;
  p.align = 1;
  p.R = p.rows = (int32_t)R;
  p.E = (int32_t)num_experts;
  sort_split(R > 0 ? R : 1, &p.blocks, &p.per_block);
  p.offsets = a->expert_offsets;
  p.route_row = a->route_row;
  p.row_route = a->row_route;
  p.hist = static_cast<int32_t*>(a->workspace);
  p.hist_row = hist_row(p.blocks);
  p.status = a->device_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.blocks > 1) {
    const size_t need = sort_workspace(R, num_experts);
    if (a->workspace == nullptr || a->workspace_bytes < need)
      return set_error(MOE_ERR_WORKSPACE, "sorting needs %zu bytes of workspace, got %zu", need,
                       a->workspace_bytes);
    if ((reinterpret_cast<uintptr_t>(a->workspace) & 15u) != 0)
      return set_error(MOE_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  }
  return launch_sort(p, s);
}

moe_status_t moe_permute(const moe_permute_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t hidden_size = a->hidden_size, top_k = a->top_k, num_rows = a->num_rows;
  moe_status_t st = check_rows(a->num_tokens, hidden_size, top_k, num_rows, a->dtype);
  if (st != MOE_OK) return st;
  // tokens without routes have nothing to copy and their x, which may be NULL, is not read
  const int64_t num_tokens = top_k > 0 ? a->num_tokens : 0;
  if (a->num_experts < 0) return set_error(MOE_ERR_INVALID_ARGUMENT, "negative size");
  if (num_rows == 0 || hidden_size == 0) return MOE_OK;
  if (!a->rows || !a->expert_offsets || (num_tokens > 0 && (!a->x || !a->route_row)))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if ((num_tokens > 1 && a->x_stride0 < hidden_size) ||
      (num_rows > 1 && a->rows_stride0 < hidden_size))
    return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
  RowParams p{};
  p.T = num_tokens;
  p.K = hidden_size;
  p.num_rows = num_rows;
  p.k = (int)top_k;
  p.route_row = a->route_row;
  p.offsets = a->expert_offsets;
  p.E = a->num_experts;
  p.x = a->x;
  p.x_stride = a->x_stride0;
  p.out_rows = a->rows;
  p.out_rows_stride = a->rows_stride0;
  return with_dtype(a->dtype, [&](auto v) {
    using T = decltype(v);
    constexpr int V = 16 / sizeof(T);
    const bool wide = packs16(hidden_size, sizeof(T)) &&
                      rows_aligned16(a->x, a->x_stride0, sizeof(T), num_tokens) &&
                      rows_aligned16(a->rows, a->rows_stride0, sizeof(T), num_rows);
    auto go = [&](auto kernel, int vec) {
      const int64_t chunk = (int64_t)moe::PERMUTE_VECS * 32 * vec;
      const int64_t warps = (num_tokens + num_rows) * ((hidden_size + chunk - 1) / chunk);
      return launched(launch_pdl(kernel, one_wave(kernel, (warps + 7) / 8, 256), dim3(256), 0,
                                 static_cast<cudaStream_t>(stream), p), "permute");
    };
    return wide ? go(moe::permute_kernel<T, V>, V) : go(moe::permute_kernel<T, 1>, 1);
  });
}

moe_status_t moe_unpermute(const moe_unpermute_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t num_tokens = a->num_tokens, hidden_size = a->hidden_size;
  const int64_t top_k = a->top_k, num_rows = a->num_rows;
  moe_status_t st = check_rows(num_tokens, hidden_size, top_k, num_rows, a->dtype);
  if (st != MOE_OK) return st;
  if (num_tokens == 0 || hidden_size == 0) return MOE_OK;
  if (!a->out || (num_rows > 0 && !a->rows) || (top_k > 0 && !a->route_row))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if ((num_tokens > 1 && a->out_stride0 < hidden_size) ||
      (num_rows > 1 && a->rows_stride0 < hidden_size))
    return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
  RowParams p{};
  p.T = num_tokens;
  p.K = hidden_size;
  p.num_rows = num_rows;
  p.k = (int)top_k;
  p.route_row = a->route_row;
  p.w = a->topk_weights;
  p.rows = a->rows;
  p.rows_stride = a->rows_stride0;
  p.out = a->out;
  p.out_stride = a->out_stride0;
  return with_dtype(a->dtype, [&](auto v) {
    using T = decltype(v);
    constexpr int V = 16 / sizeof(T);
    const bool wide = packs16(hidden_size, sizeof(T)) &&
                      rows_aligned16(a->rows, a->rows_stride0, sizeof(T), num_rows) &&
                      rows_aligned16(a->out, a->out_stride0, sizeof(T), num_tokens);
    auto go = [&](auto kernel, int vec, int kb) {
      const int64_t chunk = (int64_t)(8 / kb) * 32 * vec;
      const int64_t warps = num_tokens * ((hidden_size + chunk - 1) / chunk);
      return launched(launch_pdl(kernel, one_wave(kernel, (warps + 7) / 8, 256), dim3(256), 0,
                                 static_cast<cudaStream_t>(stream), p), "unpermute");
    };
    // as many routes at a time as there are, up to eight
    if (wide)
      return top_k > 4   ? go(moe::unpermute_kernel<T, V, 8>, V, 8)
             : top_k > 2 ? go(moe::unpermute_kernel<T, V, 4>, V, 4)
                         : go(moe::unpermute_kernel<T, V, 2>, V, 2);
    return top_k > 4   ? go(moe::unpermute_kernel<T, 1, 8>, 1, 8)
           : top_k > 2 ? go(moe::unpermute_kernel<T, 1, 4>, 1, 4)
                       : go(moe::unpermute_kernel<T, 1, 2>, 1, 2);
  });
}

moe_status_t moe_unpermute_backward(const moe_unpermute_backward_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t num_tokens = a->num_tokens, hidden_size = a->hidden_size;
  const int64_t top_k = a->top_k, num_rows = a->num_rows;
  moe_status_t st = check_rows(num_tokens, hidden_size, top_k, num_rows, a->dtype);
  if (st != MOE_OK) return st;
  if (a->num_experts < 0) return set_error(MOE_ERR_INVALID_ARGUMENT, "negative size");
  if (num_tokens * top_k == 0 && num_rows == 0) return MOE_OK;
  if ((num_rows > 0 && hidden_size > 0 && (!a->rows || !a->d_rows)) || !a->expert_offsets ||
      (num_tokens * top_k > 0 &&
       (!a->route_row || !a->topk_weights || !a->d_weights || (hidden_size > 0 && !a->d_out))))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if ((num_tokens > 1 && a->d_out_stride0 < hidden_size) ||
      (num_rows > 1 && (a->rows_stride0 < hidden_size || a->d_rows_stride0 < hidden_size)))
    return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
  RowParams p{};
  p.T = num_tokens;
  p.K = hidden_size;
  p.num_rows = num_rows;
  p.k = (int)top_k;
  p.route_row = a->route_row;
  p.w = a->topk_weights;
  p.offsets = a->expert_offsets;
  p.E = a->num_experts;
  p.x = a->d_out;
  p.x_stride = a->d_out_stride0;
  p.rows = a->rows;
  p.rows_stride = a->rows_stride0;
  p.out_rows = a->d_rows;
  p.out_rows_stride = a->d_rows_stride0;
  p.d_w = a->d_weights;
  return with_dtype(a->dtype, [&](auto v) {
    using T = decltype(v);
    constexpr int V = 16 / sizeof(T);
    const bool wide = packs16(hidden_size, sizeof(T)) &&
                      rows_aligned16(a->d_out, a->d_out_stride0, sizeof(T), num_tokens) &&
                      rows_aligned16(a->rows, a->rows_stride0, sizeof(T), num_rows) &&
                      rows_aligned16(a->d_rows, a->d_rows_stride0, sizeof(T), num_rows);
    auto go = [&](auto kernel) {
      return launched(launch_pdl(kernel, one_wave(kernel, num_tokens + num_rows, moe::BACK_THREADS),
                                 dim3(moe::BACK_THREADS), 0, static_cast<cudaStream_t>(stream), p),
                      "unpermute backward");
    };
    return wide ? go(moe::unpermute_backward_kernel<T, V>)
                : go(moe::unpermute_backward_kernel<T, 1>);
  });
}

}  // extern "C"
