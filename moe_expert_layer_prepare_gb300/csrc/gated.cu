// The gated projection of a feed-forward block and its gradients:
//   g = x Wg^T, u = x Wu^T, out = act(g) u;
//   d_g = d_out u act'(g), d_u = d_out act(g), d_x = [d_g d_u] W, d_W = [d_g d_u]^T x.
//
// Three products on tcgen05 of one shape, D[m, n] = sum_k A[m, k] B[n, k]:
//   forward   m tokens, n features, k the columns of x;
//   d_x       m tokens, n the columns of x, k the rows of W;
//   d_W       m the rows of W, n the columns of x, k tokens.
// Operands are read as they lie in memory, k along their rows or across them (the MMA takes
// either), so nothing is transposed.  The forward's tile takes as many gate rows as up rows
// of W, so that one thread has both values of an output and the activation costs no pass.
//
//   Few tokens (gated_split_kernel): W is streamed, so HBM bounds it.  Features are the
//   rows of the accumulator (64 gate, 64 up), tokens its columns, and with few tiles the
//   K slabs are dealt out to the CTAs of a cluster.
//   Many (gated_pair_kernel): the tensor cores bound it.  CTA pairs keep 256 x 256 tiles
//   and two accumulators, one in use while the other is written out.  Where the forward
//   has few tiles and a long K, two pairs share a tile (gated_cluster_kernel).
//
// d_g and d_u are a pass of their own over d_out and gate_up (12 us of the 4096 tokens
// below, at HBM's rate), rounded to the tensors' type as the MMA takes them: d_x and d_W are
// then off by 1.2 times what their own rounding makes.
//
// Measured, 7168 -> 2048 bf16: one token 12.4 us (59 MB, 4.7 TB/s), 512 tokens 24 us, 4096
// tokens 129 us (1.86 PFLOP/s) and their gradients 292 (1.65), 8192 tokens 250 (1.92); 64
// tokens 4096 -> 14336 39 us (6.0 TB/s).
#include <mutex>
#include <type_traits>

#include "activation.cuh"
#include "block_common.cuh"
#include "tc_common.cuh"

namespace moe {
namespace gated {

using namespace tc;

enum Mode { FORWARD = 0, D_X = 1, D_W = 2 };

struct Params {
  int64_t T, K, N;
  int act;
  void* out;  // out, d_x or d_weight
  int64_t out_stride;
  void* gate_up;  // nullable
  int64_t gate_up_stride;
  int out_wide, gate_up_wide;  // rows start on 32 bytes (2), 16 (1), or not (0)
  float* partials;              // pieces of tiles; nullptr: no tile is cut
  int half;                     // outputs of a tile of the forward
  int pairs, splits;
  uint32_t* status;
};

// 16 values a lane to neighbouring columns of its row, the warp's rows from `first` on, of
// which `rows` and `left` exist.  Rows that do not start on 16 bytes, and a last tile's columns,
// go through shared memory, so that a store covers two rows' 32 bytes and not two of 32 rows
// (1031 tokens, 2056 -> 1403, with gate_up: 73 us by single stores).  Of the others a lane stores
// whole sectors where it can: d_weight [28672, 4096] of 9 tokens, all stores, takes 73 us, by 16
// bytes 101, and by lines of 128 bytes of four rows through shared memory 81.
constexpr int STORE_PITCH = 18;
template <typename T>
__device__ __forceinline__ void store16(T* first, int64_t stride, int64_t rows, const float (&v)[16],
                                        int64_t left, int wide, T* buf) {
  const int lane = threadIdx.x & 31;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack2<T>(make_float2(v[2 * i], v[2 * i + 1]));
  if (wide > 0 && left >= 16) {
    if (lane >= rows) return;
    T* p = first + lane * stride;
    if (wide == 2) return st_v8(p, w);
    st_v4(p, make_uint4(w[0], w[1], w[2], w[3]));
    st_v4(p + 8, make_uint4(w[4], w[5], w[6], w[7]));
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) reinterpret_cast<uint32_t*>(buf + lane * STORE_PITCH)[i] = w[i];
  __syncwarp();
  const int c = lane & 15;
  if (c < left)
#pragma unroll
    for (int r = 0; r < 32; r += 2) {
      const int row = r + (lane >> 4);
      if (row < rows) first[row * stride + c] = buf[row * STORE_PITCH + c];
    }
  __syncwarp();
}

// ------------------------------------------------------------- few tokens
// At 128 tokens this path takes 16 us (7168 -> 2048) and two pairs a tile 22; at 512 36 us and
// 25, into 14336 features 175 and 82. From 65 tokens on, where more than every second pair has a
// tile of its own, the pairs are faster: 128 tokens, 7168 -> 4872 33 us against 39, -> 14336 71
// against 87. They lose where K is small and a second round is short (1024 -> 9600 11.8, 10.9).
constexpr int SPLIT_TOKENS = 128;
constexpr int SM_ROWS = 128;     // of a tile: 64 gate rows of W, 64 up rows
constexpr int SM_FEATURES = 64;  // outputs of a tile
constexpr int SM_A_BYTES = SM_ROWS * 128;
constexpr int SM_THREADS = 256;
constexpr int SM_MAX_STAGES = 5;
constexpr int sm_stages(int nt) { return nt <= 32 ? 5 : 4; }
constexpr int sm_smem(int nt) { return 1024 + sm_stages(nt) * (SM_A_BYTES + nt * 128) + 256; }

// Four neighbouring outputs of a token, of which some may not exist.
template <typename T>
__device__ __forceinline__ void store4(const Params& p, int64_t t, int64_t n, float4 g, float4 u) {
  const float gv[4] = {g.x, g.y, g.z, g.w}, uv[4] = {u.x, u.y, u.z, u.w};
  float o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = act_value(p.act, gv[e]) * uv[e];
  auto put = [&](T* dst, const float (&v)[4], int wide) {
    if (wide > 0 && n + 4 <= p.N) {
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack2<T>(make_float2(v[0], v[1])), pack2<T>(make_float2(v[2], v[3])));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N) dst[e] = from_f32<T>(v[e]);
    }
  };
  put(static_cast<T*>(p.out) + t * p.out_stride + n, o, p.out_wide);
  if (p.gate_up == nullptr) return;
  T* gu = static_cast<T*>(p.gate_up) + t * p.gate_up_stride + n;
  put(gu, gv, p.gate_up_wide);
  put(gu + p.N, uv, p.gate_up_wide);
}

// Stores the CTA's share of the tile's tokens from the cluster's sums in rank order.
template <typename T, int SPLITS>
__device__ __forceinline__ void join_tokens(const Params& p, const float* sums, int64_t t0,
                                            int64_t n0, int c0, int share) {
  const uint32_t at0 = smem_u32(sums);
  for (int i = threadIdx.x; i < share * (SM_FEATURES / 4); i += SM_THREADS) {
    const int c = c0 + i / (SM_FEATURES / 4), f = (i % (SM_FEATURES / 4)) * 4;
    const int64_t t = t0 + c, n = n0 + f;
    if (t >= p.T || n >= p.N) continue;
    float4 g[SPLITS], u[SPLITS];
#pragma unroll
    for (int r = 0; r < SPLITS; ++r) {
      const float* s = sums + c * SM_ROWS + f;
      g[r] = SPLITS == 1 ? *reinterpret_cast<const float4*>(s)
                         : ld_cluster4(at0 + (uint32_t)(c * SM_ROWS + f) * 4, r);
      u[r] = SPLITS == 1 ? *reinterpret_cast<const float4*>(s + SM_FEATURES)
                         : ld_cluster4(at0 + (uint32_t)(c * SM_ROWS + SM_FEATURES + f) * 4, r);
    }
#pragma unroll
    for (int r = 1; r < SPLITS; ++r) {
      g[0].x += g[r].x, g[0].y += g[r].y, g[0].z += g[r].z, g[0].w += g[r].w;
      u[0].x += u[r].x, u[0].y += u[r].y, u[0].z += u[r].z, u[0].w += u[r].w;
    }
    store4<T>(p, t, n, g[0], u[0]);
  }
}

template <typename T, int NT>
__global__ void __launch_bounds__(SM_THREADS, NT <= 64 ? 2 : 1)
    gated_split_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tmG,
                       const __grid_constant__ CUtensorMap tmU,
                       const __grid_constant__ CUtensorMap tmX) {
  constexpr int STAGES = sm_stages(NT), STAGE_BYTES = SM_A_BYTES + NT * 128;
  constexpr uint32_t IDESC = f16_idesc(std::is_same<T, __nv_bfloat16>::value, SM_ROWS, NT);
  constexpr uint32_t TMEM_COLS = NT < 32 ? 32 : NT;
  static_assert(NT * SM_ROWS * 4 <= STAGES * STAGE_BYTES, "the sums fit the ring");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
  // full[STAGES], empty[STAGES], done
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * SM_MAX_STAGES + 1);
  int* s_abort = reinterpret_cast<int*>(tmem_holder + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = s_abort;
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + SM_MAX_STAGES);
  const uint32_t done_bar = smem_u32(bars + 2 * SM_MAX_STAGES);

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(done_bar, 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    prefetch_map(&tmG);
    prefetch_map(&tmU);
    prefetch_map(&tmX);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_holder)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait();
  pdl_launch_dependents();

  const int rank = p.splits > 1 ? (int)(blockIdx.x % (unsigned)p.splits) : 0;
  const int64_t n0 = (int64_t)(blockIdx.x / (unsigned)p.splits) * SM_FEATURES;
  const int64_t t0 = (int64_t)blockIdx.y * NT;
  const int slabs = (int)((p.K + 63) / 64);
  const int per = (slabs + p.splits - 1) / p.splits;
  const int kb0 = rank * per, kb1 = min(slabs, kb0 + per);

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
#ifdef MOE_TEST_WITHHOLD_STAGE
      // Failure-detection test builds only: CTA 0 issues neither its second
      // slab nor anything after it, and the MMA warp's wait runs out.
      if (blockIdx.x == 0 && blockIdx.y == 0 && kb > kb0) break;
#endif
      if (!warp_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.status)) break;
      if (elect_one()) {
        const uint32_t bar = full0 + 8 * stage, s = smem_u32(smem + stage * STAGE_BYTES);
        mbar_expect_tx(bar, STAGE_BYTES);
        tma_load_2d(s, &tmG, kb * 64, (int)n0, bar);
        tma_load_2d(s + SM_A_BYTES / 2, &tmU, kb * 64, (int)n0, bar);
        tma_load_2d(s + SM_A_BYTES, &tmX, kb * 64, (int)t0, bar);
      }
      __syncwarp();
      issued |= 1u << stage;
      issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
      if (++stage == STAGES) stage = 0, phase ^= 1u;
    }
    for (int s = 0; s < STAGES; ++s)  // every copy has landed before exit
      if (issued & (1u << s)) {
        volatile int never = 0;
        mbar_wait(full0 + 8 * s, (issued_phase >> s) & 1u, &never, p.status);
      }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    int stage = 0;
    uint32_t phase = 0, accumulate = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!warp_wait(full0 + 8 * stage, phase, abort_flag, p.status)) break;
      fence_after();
      const uint32_t s = smem_u32(smem + stage * STAGE_BYTES);
      const uint64_t ad = sw128_desc(s), bd = sw128_desc(s + SM_A_BYTES);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16(tmem, ad + 2 * k, bd + 2 * k, IDESC, accumulate | (k > 0));
        mma_commit(empty0 + 8 * stage);
      }
      __syncwarp();
      accumulate = 1;
      if (++stage == STAGES) stage = 0, phase ^= 1u;
    }
    if (accumulate) {  // all MMAs complete before the sums are read or TMEM is freed
      if (elect_one()) mma_commit(done_bar);
      __syncwarp();
      volatile int never = 0;
      mbar_wait(done_bar, 0, &never, p.status);
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ sums
    // done is also signalled after a wait ran out; the sums are then not whole
    if (warp_wait(done_bar, 0, abort_flag, p.status) && *abort_flag == 0) {
      fence_after();
      const int nl = (warp & 3) * 32 + lane;
      const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      float* red = reinterpret_cast<float*>(smem);  // the ring is no longer in use
#pragma unroll 1
      for (int c = 0; c < NT; c += 16) {
        uint32_t v[16];
        tmem_ld16(lanes + c, v);
        tmem_wait16(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) red[(c + j) * SM_ROWS + nl] = __uint_as_float(v[j]);
      }
      fence_before();
    }
  }
  __syncwarp();
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  // Each CTA finishes its share of the tile's tokens.
  if (*abort_flag == 0) {
    const float* sums = reinterpret_cast<const float*>(smem);
    const int share = NT / p.splits, c0 = rank * share;
    if (p.splits == 1)
      join_tokens<T, 1>(p, sums, t0, n0, c0, share);
    else if (p.splits == 2)
      join_tokens<T, 2>(p, sums, t0, n0, c0, share);
    else if (p.splits == 4)
      join_tokens<T, 4>(p, sums, t0, n0, c0, share);
    else
      join_tokens<T, 8>(p, sums, t0, n0, c0, share);
  }
  __syncwarp();
  if (p.splits > 1) cluster_sync();  // no CTA leaves while its sums are read
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS)
                 : "memory");
  }
}

// ------------------------------------------------------------ many tokens
constexpr int TILE = 256;  // rows and columns of a pair's accumulator
constexpr int HALF = 128;  // of them one CTA's operands
constexpr int STAGES = 6;
constexpr int OPERAND = HALF * 128;  // bytes of one CTA's A or B in a stage
constexpr int STAGE_BYTES = 2 * OPERAND;
constexpr int EPI_WARPS = 8;  // two for each 32 rows of the accumulator
constexpr int THREADS = (2 + EPI_WARPS) * 32;
constexpr int STORE_BYTES = 32 * STORE_PITCH * 2;  // of a warp
constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + 256 + EPI_WARPS * STORE_BYTES;
constexpr int MIN_SLABS = 8;                    // of a piece of a tile
constexpr int64_t PIECE = (int64_t)TILE * TILE;  // its sums

// The work of the pairs: whole tiles dealt out in rounds, and the tiles of a last round
// that would leave pairs idle cut along k, so that each pair has a piece.
struct Work {
  int m_tiles, n_tiles, units, slabs, full, parts, items, per;
  __host__ __device__ Work(Mode mode, int64_t T, int64_t K, int64_t N, int pairs, bool cut, int half) {
    const int64_t m = mode == D_W ? 2 * N : T, n = mode == FORWARD ? 2 * N : K;
    const int64_t k = mode == FORWARD ? K : (mode == D_X ? 2 * N : T);
    m_tiles = (int)((m + TILE - 1) / TILE);
    // a tile of the forward has `half` gate rows and as many up rows
    n_tiles = mode == FORWARD ? (int)((N + half - 1) / half) : (int)((n + TILE - 1) / TILE);
    units = m_tiles * n_tiles;
    slabs = (int)((k + 63) / 64);
    const int rest = units % pairs;
    parts = 1;
    if (cut && rest > 0) {
      parts = pairs / rest < slabs / MIN_SLABS ? pairs / rest : slabs / MIN_SLABS;
      if (parts < 2) parts = 1;
    }
    per = (slabs + parts - 1) / parts;
    parts = (slabs + per - 1) / per;  // every piece has slabs
    full = parts > 1 ? units - rest : units;
    items = full + (units - full) * parts;
  }
};
struct Item {
  int unit, kb0, kb1, piece;  // piece: -1, a whole tile; else its place among the pieces
};
__device__ __forceinline__ Item work_item(const Work& w, int i) {
  if (i < w.full) return Item{i, 0, w.slabs, -1};
  const int j = i - w.full, part = j % w.parts;
  return Item{w.full + j / w.parts, part * w.per, min(w.slabs, (part + 1) * w.per), j};
}

// A persistent pair of CTAs; CTA r has rows [128 r, 128 r + 128) of a tile's A and B and
// those rows of its sums.  The first CTA issues the MMAs of both; its full[] barriers count
// both CTAs' copies, and each commit reaches both.
template <typename T, Mode MODE>
__global__ void __launch_bounds__(THREADS, 1)
    gated_pair_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmB2) {
  constexpr bool A_MN = MODE == D_W, B_MN = MODE != FORWARD;
  constexpr uint32_t IDESC_FULL = f16_idesc(std::is_same<T, __nv_bfloat16>::value, TILE, TILE) |
                             (A_MN ? IDESC_A_MN : 0u) | (B_MN ? IDESC_B_MN : 0u);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
  // full[STAGES], empty[STAGES], tfull[2], tempty[2]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 4);
  int* s_abort = reinterpret_cast<int*>(tmem_holder + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = s_abort;
  const uint32_t rank = cluster_rank();
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + STAGES);
  const uint32_t tfull0 = smem_u32(bars + 2 * STAGES), tempty0 = tfull0 + 16;

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 2 * EPI_WARPS);
    }
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    prefetch_map(&tmA);
    prefetch_map(&tmB);
    prefetch_map(&tmB2);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_holder)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are set up
  fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait();
  pdl_launch_dependents();

  const Work work(MODE, p.T, p.K, p.N, p.pairs, p.partials != nullptr, p.half);
  const int first = (int)(blockIdx.x >> 1), stride = (int)(gridDim.x >> 1);

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_phase = 0;
    bool ok = true;
    const uint32_t bytes = MODE == FORWARD ? 2 * (OPERAND + p.half * 128) : 2 * STAGE_BYTES;
    for (int i = first; ok && i < work.items; i += stride) {
      const Item item = work_item(work, i);
      const int m0 = item.unit / work.n_tiles * TILE + (int)rank * HALF;
      const int n0 = item.unit % work.n_tiles * (MODE == FORWARD ? p.half : TILE) +
                     (MODE == FORWARD ? 0 : (int)rank * HALF);
      for (int kb = item.kb0; kb < item.kb1; ++kb) {
#ifdef MOE_TEST_WITHHOLD_STAGE
        if (blockIdx.x < 2 && kb > item.kb0) {  // as above: the first pair stops here
          ok = false;
          break;
        }
#endif
        ok = warp_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.status);
        if (!ok) break;
        const uint32_t bar = cluster_address(full0 + 8 * stage, 0);
        const uint32_t s = smem_u32(smem + stage * STAGE_BYTES);
        if (elect_one()) {
          if (rank == 0) mbar_expect_tx(full0 + 8 * stage, bytes);
          if (A_MN) {
            tma_load_2d_pair(s, &tmA, m0, kb * 64, bar);
            tma_load_2d_pair(s + MN_BOX, &tmA, m0 + 64, kb * 64, bar);
          } else {
            tma_load_2d_pair(s, &tmA, kb * 64, m0, bar);
          }
          if (B_MN) {
            tma_load_2d_pair(s + OPERAND, &tmB, n0, kb * 64, bar);
            tma_load_2d_pair(s + OPERAND + MN_BOX, &tmB, n0 + 64, kb * 64, bar);
          } else {
            tma_load_2d_pair(s + OPERAND, rank == 0 ? &tmB : &tmB2, kb * 64, n0, bar);
          }
        }
        __syncwarp();
        issued |= 1u << stage;
        issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) stage = 0, phase ^= 1u;
      }
    }
    if (rank == 0)  // both CTAs' copies have landed before either leaves
      for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s)) {
          volatile int never = 0;
          mbar_wait(full0 + 8 * s, (issued_phase >> s) & 1u, &never, p.status);
        }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------- MMA (the first CTA's)
    const uint32_t idesc = MODE == FORWARD ? IDESC_FULL - ((uint32_t)((HALF - p.half) >> 2) << 17) : IDESC_FULL;
    constexpr uint32_t A_STEP = A_MN ? 128 : 2, B_STEP = B_MN ? 128 : 2;  // 16 of k, in 16 bytes
    int stage = 0, ab = 0;
    uint32_t phase = 0, aphase = 0;
    bool ok = rank == 0;
    for (int i = first; ok && i < work.items; i += stride) {
      const Item item = work_item(work, i);
      ok = warp_wait(tempty0 + 8 * ab, aphase ^ 1u, abort_flag, p.status);
      const uint32_t d = tmem + (uint32_t)(ab * TILE);
      for (int kb = item.kb0; kb < item.kb1 && ok; ++kb) {
        ok = warp_wait(full0 + 8 * stage, phase, abort_flag, p.status);
        if (!ok) break;
        fence_after();
        const uint32_t s = smem_u32(smem + stage * STAGE_BYTES);
        const uint64_t ad = A_MN ? sw128_mn_desc(s) : sw128_desc(s);
        const uint64_t bd = B_MN ? sw128_mn_desc(s + OPERAND) : sw128_desc(s + OPERAND);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_pair(d, ad + A_STEP * k, bd + B_STEP * k, idesc, kb > item.kb0 || k > 0);
          mma_commit_pair(empty0 + 8 * stage);
        }
        __syncwarp();
        if (++stage == STAGES) stage = 0, phase ^= 1u;
      }
      if (elect_one()) mma_commit_pair(tfull0 + 8 * ab);
      __syncwarp();
      ab ^= 1;
      if (ab == 0) aphase ^= 1u;
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int row0 = (int)rank * HALF + (warp & 3) * 32;  // of the tile, this warp's first
    const int64_t rows = MODE == D_W ? 2 * p.N : p.T;
    const int part_of = (warp - 2) >> 2;  // which half of the columns
    T* buf = reinterpret_cast<T*>(smem + STAGES * STAGE_BYTES + 256 + (warp - 2) * STORE_BYTES);
    int ab = 0;
    uint32_t aphase = 0;
    for (int i = first; i < work.items; i += stride) {
      const Item item = work_item(work, i);
      const int64_t m = (int64_t)(item.unit / work.n_tiles) * TILE + row0, rows_left = rows - m;
      if (!warp_wait(tfull0 + 8 * ab, aphase, abort_flag, p.status) || *abort_flag != 0) break;
      fence_after();
      const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(ab * TILE);
      if constexpr (MODE == FORWARD) {
        const int64_t n0 = (int64_t)(item.unit % work.n_tiles) * p.half;
        T* out = static_cast<T*>(p.out) + m * p.out_stride + n0;
        T* gu = static_cast<T*>(p.gate_up) + m * p.gate_up_stride + n0;
#pragma unroll 1
        for (int c = part_of * 16; c < p.half; c += EPI_WARPS * 4) {
          uint32_t vg[16], vu[16];
          tmem_ld16(lanes + c, vg);
          tmem_ld16(lanes + p.half + c, vu);
          tmem_wait16(vg);
          tmem_wait16(vu);
          float o[16], g[16], u[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            g[j] = __uint_as_float(vg[j]), u[j] = __uint_as_float(vu[j]);
            o[j] = act_value(p.act, g[j]) * u[j];
          }
          const int64_t left = p.N - n0 - c;
          if (rows_left <= 0 || left <= 0) continue;
          store16<T>(out + c, p.out_stride, rows_left, o, left, p.out_wide, buf);
          if (p.gate_up != nullptr) {
            store16<T>(gu + c, p.gate_up_stride, rows_left, g, left, p.gate_up_wide, buf);
            store16<T>(gu + p.N + c, p.gate_up_stride, rows_left, u, left, p.gate_up_wide, buf);
          }
        }
      } else {
        const int64_t n0 = (int64_t)(item.unit % work.n_tiles) * TILE;
        T* out = static_cast<T*>(p.out) + m * p.out_stride + n0;
        float* part = p.partials + item.piece * PIECE + (row0 + lane) * TILE;
#pragma unroll 1
        for (int c = part_of * 16; c < TILE; c += EPI_WARPS * 4) {
          uint32_t v[16];
          tmem_ld16(lanes + c, v);
          tmem_wait16(v);
          if (item.piece >= 0) {
#pragma unroll
            for (int j = 0; j < 16; j += 8) {
              const uint32_t w[8] = {v[j],     v[j + 1], v[j + 2], v[j + 3],
                                     v[j + 4], v[j + 5], v[j + 6], v[j + 7]};
              st_v8(part + c + j, w);
            }
            continue;
          }
          float f[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(v[j]);
          const int64_t left = p.K - n0 - c;
          if (rows_left > 0 && left > 0)
            store16<T>(out + c, p.out_stride, rows_left, f, left, p.out_wide, buf);
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_address(tempty0 + 8 * ab, 0));
      ab ^= 1;
      if (ab == 0) aphase ^= 1u;
    }
  }
  __syncwarp();
  fence_before();
  cluster_sync();  // both CTAs' copies, MMAs and reads are done
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// One tile of the forward for a cluster of `splits` pairs, each with a share of the K slabs:
// where there are fewer tiles than pairs.  A CTA's sums go to its own shared memory, the
// ring's, and each of the CTAs that have the same rows finishes a share of the outputs from
// all of theirs in the order of the pairs.
constexpr int SUM_PITCH = TILE + 4;  // floats: lanes' rows lie in different banks
static_assert(HALF * SUM_PITCH * 4 <= STAGES * STAGE_BYTES, "the sums fit the ring");

template <typename T, int SPLITS>
__global__ void __launch_bounds__(THREADS, 1)
    gated_cluster_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tmX,
                         const __grid_constant__ CUtensorMap tmG,
                         const __grid_constant__ CUtensorMap tmU) {
  constexpr uint32_t IDESC = f16_idesc(std::is_same<T, __nv_bfloat16>::value, TILE, TILE);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
  // full[STAGES], empty[STAGES], done
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 1);
  int* s_abort = reinterpret_cast<int*>(tmem_holder + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = s_abort;
  const uint32_t cta = cluster_rank(), rank = cta & 1, leader = cta & ~1u;
  const int share = (int)(cta >> 1);
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + STAGES);
  const uint32_t done_bar = smem_u32(bars + 2 * STAGES);
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(done_bar, 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    prefetch_map(&tmX);
    prefetch_map(&tmG);
    prefetch_map(&tmU);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_holder)),
                 "r"(TILE)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers are set up
  fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait();
  pdl_launch_dependents();

  const int n_tiles = (int)((p.N + HALF - 1) / HALF), unit = (int)blockIdx.x / (2 * SPLITS);
  const int m0 = unit / n_tiles * TILE + (int)rank * HALF, n0 = unit % n_tiles * HALF;
  const int slabs = (int)((p.K + 63) / 64), per = (slabs + SPLITS - 1) / SPLITS;
  const int kb0 = share * per, kb1 = min(slabs, kb0 + per);  // every share has slabs

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
#ifdef MOE_TEST_WITHHOLD_STAGE
      if (blockIdx.x < 2 && kb > kb0) break;  // as above: the first pair stops here
#endif
      if (!warp_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.status)) break;
      const uint32_t bar = cluster_address(full0 + 8 * stage, leader);
      const uint32_t s = smem_u32(smem + stage * STAGE_BYTES);
      if (elect_one()) {
        if (rank == 0) mbar_expect_tx(full0 + 8 * stage, 2 * STAGE_BYTES);
        tma_load_2d_pair(s, &tmX, kb * 64, m0, bar);
        tma_load_2d_pair(s + OPERAND, rank == 0 ? &tmG : &tmU, kb * 64, n0, bar);
      }
      __syncwarp();
      issued |= 1u << stage;
      issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
      if (++stage == STAGES) stage = 0, phase ^= 1u;
    }
    if (rank == 0)  // both CTAs' copies have landed before either goes on
      for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s)) {
          volatile int never = 0;
          mbar_wait(full0 + 8 * s, (issued_phase >> s) & 1u, &never, p.status);
        }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------- MMA (the pair's first CTA's)
    int stage = 0;
    uint32_t phase = 0, accumulate = 0;
    for (int kb = kb0; kb < kb1 && rank == 0; ++kb) {
      if (!warp_wait(full0 + 8 * stage, phase, abort_flag, p.status)) break;
      fence_after();
      const uint32_t s = smem_u32(smem + stage * STAGE_BYTES);
      const uint64_t ad = sw128_desc(s), bd = sw128_desc(s + OPERAND);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_pair(tmem, ad + 2 * k, bd + 2 * k, IDESC, accumulate | (k > 0));
        mma_commit_pair(empty0 + 8 * stage, leader);
      }
      __syncwarp();
      accumulate = 1;
      if (++stage == STAGES) stage = 0, phase ^= 1u;
    }
    if (rank == 0) {  // done also when a wait ran out; the sums are then not whole
      if (elect_one()) mma_commit_pair(done_bar, leader);
      __syncwarp();
    }
    volatile int never = 0;
    mbar_wait(done_bar, 0, &never, p.status);  // no MMA is left that reads or writes
    __syncwarp();
  } else if (warp_wait(done_bar, 0, abort_flag, p.status)) {
    // ------------------------------------------------------------------ sums
    fence_after();
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    float* red = reinterpret_cast<float*>(smem) + row * SUM_PITCH;  // the ring is no longer in use
#pragma unroll 1
    for (int c = ((warp - 2) >> 2) * 16; c < TILE; c += EPI_WARPS * 4) {
      uint32_t v[16];
      tmem_ld16(lanes + c, v);
      tmem_wait16(v);
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<uint4*>(red + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
    fence_before();
  }
  __syncwarp();
  cluster_sync();
  bool whole = true;  // no CTA of the cluster gave up
  for (int r = 0; r < 2 * SPLITS; ++r) {
    int gave_up;
    asm volatile("ld.shared::cluster.s32 %0, [%1];"
                 : "=r"(gave_up)
                 : "r"(cluster_address(smem_u32(s_abort), r))
                 : "memory");
    whole = whole && gave_up == 0;
  }
  constexpr int LANES = HALF / SPLITS / 4;  // of a row's share of outputs, four a lane
  const uint32_t sums = smem_u32(smem);
  for (int i = tid; whole && i < HALF * LANES; i += THREADS) {
    const int row = i / LANES, c = share * (HALF / SPLITS) + i % LANES * 4;
    const int64_t t = m0 + row, n = n0 + c;
    if (t >= p.T || n >= p.N) continue;
    float4 g[SPLITS], u[SPLITS];
    const uint32_t at = sums + (uint32_t)(row * SUM_PITCH + c) * 4;
#pragma unroll
    for (int r = 0; r < SPLITS; ++r) {
      g[r] = ld_cluster4(at, 2 * r + rank);
      u[r] = ld_cluster4(at + HALF * 4, 2 * r + rank);
    }
#pragma unroll
    for (int r = 1; r < SPLITS; ++r) {
      g[0].x += g[r].x, g[0].y += g[r].y, g[0].z += g[r].z, g[0].w += g[r].w;
      u[0].x += u[r].x, u[0].y += u[r].y, u[0].z += u[r].z, u[0].w += u[r].w;
    }
    store4<T>(p, t, n, g[0], u[0]);
  }
  __syncwarp();
  fence_before();
  cluster_sync();  // no CTA leaves while its sums are read
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TILE)
                 : "memory");
  }
}

// Sums the pieces of the tiles that were cut, in their order, and stores them: a block
// JOIN_ROWS rows of a tile, a thread four columns of two of them.
constexpr int JOIN_ROWS = 8;

template <typename T, Mode MODE>
__global__ void __launch_bounds__(256) gated_join_kernel(Params p) {
  pdl_wait();
  pdl_launch_dependents();
  const Work work(MODE, p.T, p.K, p.N, p.pairs, true, HALF);
  const int u = work.full + blockIdx.y;
  const int64_t rows = MODE == D_W ? 2 * p.N : p.T;
  const int f = (threadIdx.x & 63) * 4;
  const int64_t n = (int64_t)(u % work.n_tiles) * TILE + f;
  const float* from = p.partials + (int64_t)blockIdx.y * work.parts * PIECE + f;
  for (int r = blockIdx.x * JOIN_ROWS + (threadIdx.x >> 6); r < (blockIdx.x + 1) * JOIN_ROWS; r += 4) {
    const int64_t m = (int64_t)(u / work.n_tiles) * TILE + r;
    if (m >= rows) continue;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int q0 = 0; q0 < work.parts; q0 += 4) {
      float4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[q] = q0 + q < work.parts
                   ? __ldcg(reinterpret_cast<const float4*>(from + (q0 + q) * PIECE + r * TILE))
                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sum.x += v[q].x, sum.y += v[q].y, sum.z += v[q].z, sum.w += v[q].w;
    }
    const float w[4] = {sum.x, sum.y, sum.z, sum.w};
    T* out = static_cast<T*>(p.out) + m * p.out_stride + n;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.K) out[e] = from_f32<T>(w[e]);
  }
}

// ------------------------------------------------- gradients of gate and up
// [d_g d_u] of VEC neighbouring columns a thread, rounded to the tensors' type, as which
// they enter both products.
struct SlopeParams {
  int64_t T, N;
  int act;
  const void *d_out, *gate_up;
  int64_t d_out_stride, gate_up_stride, d_stride;
  void* d_gate_up;
};

template <typename T, int VEC>
__global__ void __launch_bounds__(256) gated_slope_kernel(SlopeParams p) {
  constexpr int U = VEC == 1 ? 4 : 1;  // packs in flight
  pdl_wait();
  pdl_launch_dependents();
  const int N = (int)p.N;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const T* gu = static_cast<const T*>(p.gate_up) + t * p.gate_up_stride;
    const T* d_out = static_cast<const T*>(p.d_out) + t * p.d_out_stride;
    T* dst = static_cast<T*>(p.d_gate_up) + t * p.d_stride;
    for (int n0 = (blockIdx.y * U * 256 + threadIdx.x) * VEC; n0 < N; n0 += gridDim.y * U * 256 * VEC) {
      Pack<T, VEC> pg[U], pu[U], pd[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int n = min(n0 + k * 256 * VEC, N - VEC);
        pg[k] = load_pack<T, VEC>(gu + n);
        pu[k] = load_pack<T, VEC>(gu + N + n);
        pd[k] = load_pack<T, VEC>(d_out + n);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int n = n0 + k * 256 * VEC;
        if (n >= N) break;
        float g[VEC], u[VEC], d[VEC];
        pg[k].get(g), pu[k].get(u), pd[k].get(d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float2 a = act_slope(p.act, g[e]);
          g[e] = d[e] * u[e] * a.y;
          u[e] = d[e] * a.x;
        }
        Pack<T, VEC> o;
        o.set(g);
        store_pack<T, VEC>(dst + n, o);
        o.set(u);
        store_pack<T, VEC>(dst + N + n, o);
      }
    }
  }
}

}  // namespace gated
}  // namespace moe

namespace moe_host {

namespace gated = moe::gated;

// 2 where rows of 16-bit values start on 32 bytes, 1 on 16, else 0.
static int row_width(const void* p, int64_t stride0, int64_t rows) {
  const uint64_t bits = reinterpret_cast<uintptr_t>(p) | (rows > 1 ? (uint64_t)stride0 * 2 : 0);
  return bits % 32 == 0 ? 2 : (bits % 16 == 0 ? 1 : 0);
}

// How many clusters of 2, 4 or 8 CTAs, each on an SM of its own, the GPU runs at once.  Of four
// it is 36, not 38, of eight 15: some of the chip's partitions leave SMs over.
static int clusters_at_once(int ctas) {
  constexpr auto kernel = gated::gated_cluster_kernel<__nv_bfloat16, 2>;
  static_assert(2 * gated::SMEM > kMaxSmem, "one CTA an SM");
  static std::mutex mu;
  static int known[64][9] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (allow_smem<kernel>(gated::SMEM) != MOE_OK) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev][ctas] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(gated::THREADS);
    cfg.dynamicSmemBytes = (size_t)gated::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    known[dev][ctas] = n;
  }
  return known[dev][ctas];
}

// A cluster shares a tile's K while all the clusters run at once.  Up to 64 tokens two CTAs fit
// an SM: then a cluster of eight takes four SMs and two of four share them.  (Measured: of 37
// and 38 tiles in eighths, of 75 and 76 in quarters some wait; one token of 7168 -> 2432 18.8
// us, in quarters 14.2; -> 4864 30.6, in halves 24.8.  73 and 74 in quarters would still fit,
// 64 tokens -> 4672 25.4 against 26.8.  128 tokens -> 1024, an SM each: eighths 20.9, quarters
// 13.8.)  The sums' exchange grows with the tokens: for 17 or more a share on a second CTA of
// an SM has to be eight slabs (64 tokens, 2048 -> 2048 7.3 us, with four 8.5; 32 tokens 6.6
// and 7.3; but one token, 2048 -> 1024, 4.7 and 4.4).
template <int NT>
static int splits_of(int64_t K, int64_t N) {
  const int64_t tiles = (N + gated::SM_FEATURES - 1) / gated::SM_FEATURES;
  const int64_t slabs = (K + 63) / 64;
  int splits = 1;
  while (splits < 8) {
    const int more = 2 * splits;
    const int64_t per = (slabs + more - 1) / more;
    if (per < 4 || per * (more - 1) >= slabs) break;  // every share has slabs
    const bool two = NT <= 64 && per >= (NT <= 16 ? 4 : 8);
    const int64_t fit = !two ? clusters_at_once(more)
                             : (more == 2 ? num_sms() : clusters_at_once(4) * 8 / more);
    if (tiles > fit) break;
    splits = more;
  }
  return splits;
}

template <typename T, int NT>
static moe_status_t launch_gated_split(gated::Params p, const CUtensorMap& g, const CUtensorMap& u,
                                       const CUtensorMap& x, cudaStream_t s) {
  constexpr auto kernel = gated::gated_split_kernel<T, NT>;
  static_assert(gated::sm_smem(NT) <= kMaxSmem, "shared memory of one CTA");
  moe_status_t st = allow_smem<kernel>(gated::sm_smem(NT));
  if (st != MOE_OK) return st;
  p.splits = splits_of<NT>(p.K, p.N);
  const dim3 grid((unsigned)((p.N + gated::SM_FEATURES - 1) / gated::SM_FEATURES * p.splits),
                  (unsigned)((p.T + NT - 1) / NT));
  return launched(launch_cluster(kernel, grid, gated::SM_THREADS, p.splits,
                                 (size_t)gated::sm_smem(NT), s, p, g, u, x),
                  "gated projection");
}

template <typename T, gated::Mode MODE>
static moe_status_t launch_gated_pair(const gated::Params& p, const CUtensorMap& a,
                                      const CUtensorMap& b, const CUtensorMap& b2, cudaStream_t s) {
  constexpr auto kernel = gated::gated_pair_kernel<T, MODE>;
  static_assert(gated::SMEM <= kMaxSmem, "shared memory of one CTA");
  moe_status_t st = allow_smem<kernel>(gated::SMEM);
  if (st != MOE_OK) return st;
  const gated::Work work(MODE, p.T, p.K, p.N, p.pairs, p.partials != nullptr, p.half);
  const int pairs = work.items < p.pairs ? work.items : p.pairs;
  st = launched(launch_cluster(kernel, dim3((unsigned)(2 * pairs)), gated::THREADS, 2,
                               (size_t)gated::SMEM, s, p, a, b, b2),
                "gated projection");
  if (st != MOE_OK || work.full == work.units) return st;
  if constexpr (MODE != gated::FORWARD)
    st = launched(launch_pdl(gated::gated_join_kernel<T, MODE>,
                             dim3(gated::TILE / gated::JOIN_ROWS, (unsigned)(work.units - work.full)),
                             dim3(256), 0, s, p),
                  "gated projection join");
  return st;
}

template <typename T, int SPLITS>
static moe_status_t launch_gated_cluster(const gated::Params& p, int units, const CUtensorMap& x,
                                         const CUtensorMap& g, const CUtensorMap& u, cudaStream_t s) {
  constexpr auto kernel = gated::gated_cluster_kernel<T, SPLITS>;
  moe_status_t st = allow_smem<kernel>(gated::SMEM);
  if (st != MOE_OK) return st;
  return launched(launch_cluster(kernel, dim3((unsigned)(units * 2 * SPLITS)), gated::THREADS,
                                 2 * SPLITS, (size_t)gated::SMEM, s, p, x, g, u),
                  "gated projection");
}

// Outputs of a forward tile: narrower ones where they leave fewer pairs idle in the last
// round (4096 tokens, 7168 -> 2048: 3.4 rounds of 128, exactly 4 of 112).  A tile costs its
// columns and, as x is read for fewer of them, some more.
static int best_half(const gated::Params& p) {
  int best = gated::HALF;
  int64_t least = INT64_MAX;
  for (int half = gated::HALF; half >= 64; half -= 16) {
    const gated::Work w(gated::FORWARD, p.T, p.K, p.N, p.pairs, false, half);
    const int64_t cost = (int64_t)((w.units + p.pairs - 1) / p.pairs) * (half + 24);
    if (cost < least) best = half, least = cost;
  }
  return best;
}

template <typename T>
static moe_status_t launch_gated(const moe_gated_linear_args_t* a, gated::Params p, cudaStream_t s) {
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const int64_t x_stride = p.T > 1 ? a->x_stride0 : p.K;
  const T* up = static_cast<const T*>(a->weight) + p.N * p.K;
  const gated::Work whole(gated::FORWARD, p.T, p.K, p.N, p.pairs, false, gated::HALF);
  const bool split = p.T <= 64 || (p.T <= gated::SPLIT_TOKENS && whole.units * 2 <= p.pairs);
  // smallest tile that holds the batch
  const int nt = p.T <= 16 ? 16 : (p.T <= 32 ? 32 : (p.T <= 64 ? 64 : 128));
  // Two pairs a tile where all the clusters run at once (256 tokens, 7168 -> 4608 29.3 us and
  // alone 31.6; with two clusters more 49 and 32) and the K that a second pair takes over is
  // worth the sums' exchange (256 tokens -> 2048 features of 1024 8.6 us, alone 7.1; of 4096
  // 15.7 and 17.5, -> 4096 19.0 and 19.2).
  const bool shared = !split && whole.slabs >= 56 && whole.units <= clusters_at_once(4);
  if (!split && !shared) p.half = best_half(p);
  const int rows = split ? gated::SM_FEATURES : p.half;
  CUtensorMap g, u, x;
  if (!make_map16(&g, bf16, a->weight, p.N, p.K, p.K, rows) ||
      !make_map16(&u, bf16, up, p.N, p.K, p.K, rows) ||
      !make_map16(&x, bf16, a->x, p.T, p.K, x_stride, split ? nt : gated::HALF))
    return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed for the gated projection");
  // (Four, in clusters of eight CTAs, of which not sixteen fit the GPU at once: 256 tokens of
  // 7168 -> 2048 34 us, two 23.)
  if (shared) return launch_gated_cluster<T, 2>(p, whole.units, x, g, u, s);
  if (!split) return launch_gated_pair<T, gated::FORWARD>(p, x, g, u, s);
  switch (nt) {
    case 16: return launch_gated_split<T, 16>(p, g, u, x, s);
    case 32: return launch_gated_split<T, 32>(p, g, u, x, s);
    case 64: return launch_gated_split<T, 64>(p, g, u, x, s);
    default: return launch_gated_split<T, 128>(p, g, u, x, s);
  }
}

// Workspace of the gradient: [T][d_stride] gradients of gate and up, then pieces of tiles.
static int64_t d_gate_up_stride(int64_t N) { return (2 * N + 7) / 8 * 8; }
static int64_t d_gate_up_bytes(int64_t T, int64_t N) {
  return (T * d_gate_up_stride(N) * 2 + 255) / 256 * 256;
}

template <typename T>
static moe_status_t launch_gated_backward(const moe_gated_linear_backward_args_t* a,
                                          gated::Params p, cudaStream_t s) {
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const int64_t ds = d_gate_up_stride(p.N);
  gated::SlopeParams sp{};
  sp.T = p.T;
  sp.N = p.N;
  sp.act = p.act;
  sp.d_out = a->d_out;
  sp.d_out_stride = a->d_out_stride0;
  sp.gate_up = a->gate_up;
  sp.gate_up_stride = a->gate_up_stride0;
  sp.d_gate_up = a->workspace;
  sp.d_stride = ds;
  const bool wide = p.N % 8 == 0 && rows_aligned16(a->d_out, a->d_out_stride0, 2, p.T) &&
                    rows_aligned16(a->gate_up, a->gate_up_stride0, 2, p.T);
  const int64_t cap = 8 * (int64_t)num_sms();
  // a row a block, of few rows its parts
  const int64_t parts = (p.N + (wide ? 2048 : 1024) - 1) / (wide ? 2048 : 1024);
  const int64_t spread = cap / p.T < 1 ? 1 : cap / p.T;
  const dim3 grid((unsigned)(p.T < cap ? p.T : cap), (unsigned)(parts < spread ? parts : spread));
  moe_status_t st = launched(wide ? launch_pdl(gated::gated_slope_kernel<T, 8>, grid, dim3(256), 0, s, sp)
                                  : launch_pdl(gated::gated_slope_kernel<T, 1>, grid, dim3(256), 0, s, sp),
                             "gated slope");
  if (st != MOE_OK) return st;
  // on 32 bytes, as sums are stored
  p.partials = reinterpret_cast<float*>(
      (reinterpret_cast<uintptr_t>(a->workspace) + d_gate_up_bytes(p.T, p.N) + 31) & ~(uintptr_t)31);
  CUtensorMap ma, mb;
  if (a->d_x != nullptr) {
    if (!make_map16(&ma, bf16, a->workspace, p.T, 2 * p.N, ds, gated::HALF) ||
        !make_map16(&mb, bf16, a->weight, 2 * p.N, p.K, p.K, 64))
      return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed for d_x");
    p.out = a->d_x;
    p.out_stride = a->d_x_stride0;
    p.out_wide = row_width(a->d_x, a->d_x_stride0, p.T);
    st = launch_gated_pair<T, gated::D_X>(p, ma, mb, mb, s);
    if (st != MOE_OK) return st;
  }
  if (a->d_weight != nullptr) {
    const int64_t x_stride = p.T > 1 ? a->x_stride0 : p.K;
    if (!make_map16(&ma, bf16, a->workspace, p.T, 2 * p.N, ds, 64) ||
        !make_map16(&mb, bf16, a->x, p.T, p.K, x_stride, 64))
      return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed for d_weight");
    p.out = a->d_weight;
    p.out_stride = p.K;
    p.out_wide = row_width(a->d_weight, p.K, 2 * p.N);
    st = launch_gated_pair<T, gated::D_W>(p, ma, mb, mb, s);
  }
  return st;
}

static moe_status_t check_gated(int64_t T, int64_t K, int64_t N, int32_t dtype, int32_t act) {
  if (T < 0 || K < 0 || N < 0) return set_error(MOE_ERR_INVALID_ARGUMENT, "negative size");
  if (!dtype_ok(dtype)) return set_error(MOE_ERR_INVALID_ARGUMENT, "bad dtype %d", dtype);
  if (act < MOE_ACT_SILU || act > MOE_ACT_NONE)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "bad activation %d", act);
  if (act == MOE_ACT_NONE)
    return set_error(MOE_ERR_UNSUPPORTED, "a gated projection has an activation");
  if (dtype == MOE_DTYPE_FP32)
    return set_error(MOE_ERR_UNSUPPORTED, "the projection takes bf16 or fp16");
  if (T >= ((int64_t)1 << 22) || K >= ((int64_t)1 << 28) || N >= ((int64_t)1 << 28))
    return set_error(MOE_ERR_UNSUPPORTED, "problem too large for 32-bit tile coordinates");
  return MOE_OK;
}

// x and weight as TMA reads them.
static moe_status_t check_gated_operands(const void* x, int64_t x_stride, const void* weight,
                                         int64_t T, int64_t K) {
  if (K % 8 != 0 || !rows_aligned16(x, x_stride, 2, T) || !rows_aligned16(weight, K, 2, 2))
    return set_error(MOE_ERR_ALIGNMENT, "rows of x and weight must start on 16-byte boundaries");
  return MOE_OK;
}

}  // namespace moe_host

using namespace moe_host;

extern "C" {

moe_status_t moe_gated_linear(const moe_gated_linear_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t T = a->num_tokens, K = a->in_features, N = a->out_features;
  moe_status_t st = check_gated(T, K, N, a->dtype, a->activation);
  if (st != MOE_OK) return st;
  if (T == 0 || N == 0) return MOE_OK;
  if (K < 1) return set_error(MOE_ERR_SHAPE, "in_features must be >= 1");
  if (!a->x || !a->weight || !a->out)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if (T > 1 && (a->x_stride0 < K || a->out_stride0 < N ||
                (a->gate_up != nullptr && a->gate_up_stride0 < 2 * N)))
    return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
  st = check_gated_operands(a->x, a->x_stride0, a->weight, T, K);
  if (st != MOE_OK) return st;
  gated::Params p{};
  p.T = T;
  p.K = K;
  p.N = N;
  p.act = a->activation;
  p.out = a->out;
  p.out_stride = a->out_stride0;
  p.out_wide = row_width(a->out, a->out_stride0, T);
  p.gate_up = a->gate_up;
  p.gate_up_stride = a->gate_up_stride0;
  {  // both halves of a row
    const int width = row_width(a->gate_up, a->gate_up_stride0, T);
    p.gate_up_wide = N % 16 == 0 ? width : (N % 8 == 0 && width > 0);
  }
  p.pairs = num_sms() / 2;
  p.half = gated::HALF;
  p.splits = 1;
  p.status = a->device_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a->dtype == MOE_DTYPE_BF16 ? launch_gated<__nv_bfloat16>(a, p, s)
                                    : launch_gated<__half>(a, p, s);
}

size_t moe_gated_linear_workspace_size(int64_t num_tokens, int64_t in_features,
                                       int64_t out_features) {
  if (num_tokens <= 0 || in_features <= 0 || out_features <= 0) return 0;
  return (size_t)(d_gate_up_bytes(num_tokens, out_features) + 32 +
                  (int64_t)(num_sms() / 2) * gated::PIECE * 4);
}

moe_status_t moe_gated_linear_backward(const moe_gated_linear_backward_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t T = a->num_tokens, K = a->in_features, N = a->out_features;
  moe_status_t st = check_gated(T, K, N, a->dtype, a->activation);
  if (st != MOE_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) return MOE_OK;
  if (T == 0 || N == 0) {  // sums of nothing
    cudaError_t e = cudaSuccess;
    if (T == 0 && N > 0 && a->d_weight != nullptr)
      e = cudaMemsetAsync(a->d_weight, 0, (size_t)(2 * N * K) * 2, s);
    if (N == 0 && T > 0 && a->d_x != nullptr) {
      if (T > 1 && a->d_x_stride0 < K)
        return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
      e = cudaMemset2DAsync(a->d_x, (size_t)(T > 1 ? a->d_x_stride0 : K) * 2, 0, (size_t)K * 2,
                            (size_t)T, s);
    }
    if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "memset: %s", cudaGetErrorString(e));
    return MOE_OK;
  }
  if (!a->d_out || !a->x || !a->weight || !a->gate_up)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if (T > 1 && (a->x_stride0 < K || a->d_out_stride0 < N || a->gate_up_stride0 < 2 * N ||
                (a->d_x != nullptr && a->d_x_stride0 < K)))
    return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
  st = check_gated_operands(a->x, a->x_stride0, a->weight, T, K);
  if (st != MOE_OK) return st;
  if (a->d_x == nullptr && a->d_weight == nullptr) return MOE_OK;
  const size_t need = moe_gated_linear_workspace_size(T, K, N);
  if (a->workspace == nullptr || a->workspace_bytes < need)
    return set_error(MOE_ERR_WORKSPACE, "the gradients need %zu bytes of workspace, got %zu", need,
                     a->workspace_bytes);
  if ((reinterpret_cast<uintptr_t>(a->workspace) & 15u) != 0)
    return set_error(MOE_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  gated::Params p{};
  p.T = T;
  p.K = K;
  p.N = N;
  p.act = a->activation;
  p.pairs = num_sms() / 2;
  p.half = gated::HALF;
  p.splits = 1;
  p.status = a->device_status;
  return a->dtype == MOE_DTYPE_BF16 ? launch_gated_backward<__nv_bfloat16>(a, p, s)
                                    : launch_gated_backward<__half>(a, p, s);
}

}  // extern "C"
