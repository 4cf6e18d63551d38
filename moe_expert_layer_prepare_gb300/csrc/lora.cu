// A projection shared by all tokens plus each token's own low-rank adapter:
//   out = x W^T + s_a (x A_a^T) B_a^T.
//
// The shrink gives h = x A_a^T as fp32 sums per share of K.  It reads A and the rows of
// x, a few flops a byte; blocks take (64 or 128 tokens, share of K, share of the adapters
// among them) and copy only the rows of an adapter's own tokens, so the copies are
// cp.async.  Up to 128 tokens (lora_shrink_kernel) on mma.sync, above
// (lora_shrink_long_kernel) on tcgen05.
//
// The projection is on tcgen05, features by tokens: the accumulator's rows are
// features (the MMA's A operand is a weight tile) and its columns tokens, so that
// a single token costs a 16-column tile.  K slabs of 64 come by TMA through a ring
// of shared-memory stages.
//
//   Up to SPLIT_TOKENS tokens (lora_split_kernel): W is streamed once or a few
//   times, so HBM bounds it.  With few tiles the K slabs are dealt out to the CTAs of
//   a cluster and the sums joined through distributed shared memory in rank order.
//   The adapters' second product is done meanwhile by warps that have no part in the
//   main loop, on mma.sync tiles of 16 features by 8 tokens of one adapter.
//
//   Above (lora_pair_kernel): the tensor cores bound it.  CTA pairs keep 256 x 256
//   tiles and two accumulators, one in use while the other is written out.  Tokens
//   are taken in the order of their adapters (a counting sort of the ids), every
//   adapter from a multiple of RUN tokens on: rows that lie together in x are read
//   there, others from a copy that the shrink writes in that order.  A tile's
//   columns are then runs of one adapter each, and the second product enters the
//   accumulator as further K steps on the columns of a run alone: B_a's rows as the A
//   operand, s_a h as the B operand.
//
// In both an adapter's values reach its own tokens only (a non-finite weight stays
// with them), and as the MMA takes 16-bit operands, s_a h enters as its rounding and
// the rounded remainder: 16 bits of its significand in bf16, 22 in fp16, where the output
// keeps 8 and 11.  What fp16's exponents do not hold is added in fp32 (wide_piece).
//
// The projection's launch starts while the shrink still runs and waits for it only
// where h is read.
//
// Measured, 7168 -> 4096 bf16: one token of rank 16 14.2 us (59 MB, 4.2 TB/s); 512 tokens,
// 16 adapters of rank 64, 56 us; 8192 tokens in order 313 us (1.58 PFLOP/s, the pairs alone
// 1.8), without adapters 250 us (1.92 PFLOP/s).  2048 -> 7168 fp16, 64 tokens that name 36
// adapters of rank 32: 20.3 us (59 MB).
#include <mutex>

#include "block_common.cuh"
#include "tc_common.cuh"

namespace moe {

using namespace tc;

constexpr int LORA_MAX_RANK = 128;
constexpr int LORA_MAX_ADAPTERS = 1023;  // the counting sort's bins, less one
constexpr int RUN = 32;  // an adapter's tokens begin at multiples of this: the pair MMA's N step

struct LoraParams {
  int64_t T, N, K, S, R;
  const void* x;
  int64_t x_stride;
  const void* a;
  const void* b;
  const int32_t* ids;
  const int32_t* order;  // nullable: tokens in the order of their adapters, -1 between
  const int32_t* places;  // of order, in use (device)
  void* xs;               // x's rows in that order, where they do not lie together in x
  const float* scale;
  void* out;
  int64_t out_stride;
  float* partials;  // pair, nullable: pieces of tiles, [pairs][2][LP_TILE tokens][LP_HALF]
  int pairs;        // of CTAs
  float* h;        // [shares][T][R]
  uint32_t* wide;  // pair, fp16: whether any piece of s h is wide, then from word 4 on which
  int shares;      // of K in the shrink
  int share_k;     // K of one share, a multiple of 64
  int splits;      // cluster size of the projection
  int wait_first;  // no shrink was launched: wait for the stream's predecessor at once
  uint32_t* status;
};

__device__ __forceinline__ int adapter_of(const LoraParams& p, int64_t t, bool* bad) {
  const int a = t >= 0 && t < p.T ? p.ids[t] : -1;
  if (a >= p.S) *bad = true;
  return a >= 0 && a < p.S ? a : -1;
}

// The distinct ids >= 0 among id[0, n), n <= blockDim.x, in ascending order, by a
// bitmap; list and its length.  All threads of the block call it.
__device__ __forceinline__ int distinct_adapters(const int16_t* id, int16_t* list, uint32_t* bits,
                                                 int* count, int n) {
  const int tid = threadIdx.x;
  if (tid < 32) bits[tid] = 0;
  __syncthreads();
  if (tid < n && id[tid] >= 0) atomicOr(&bits[id[tid] >> 5], 1u << (id[tid] & 31));
  __syncthreads();
  if (tid < 32) {
    uint32_t w = bits[tid];
    int incl = __popc(w);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (tid >= o) incl += v;
    }
    if (tid == 31) *count = incl;
    for (int at = incl - __popc(w); w != 0; w &= w - 1) list[at++] = (int16_t)(tid * 32 + __ffs(w) - 1);
  }
  __syncthreads();
  return *count;
}

// ------------------------------------------------------------------ shrink
constexpr int SH_THREADS = 256;
constexpr int SH_STAGES = 4;
constexpr int SH_TOK = 64, SH_LONG = 128;  // tokens of a block

// Shared memory of a block of `tok` tokens.
__host__ __device__ constexpr int sh_smem(int tok, int r16) {
  return SH_STAGES * (tok + r16) * 128 + (tok == SH_LONG ? 1024 : 0);  // 1024: alignment
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <typename T>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether a piece of a token's s h (N neighbouring ranks: four in short batches, eight in
// long ones) is wide: beyond fp16's exponents, with a value above 65504 or not finite, or
// all of them below its normal range, where the remainder's step of 2^-24 would show in
// the output's 11 bits.  It goes into the MMA as zeros and is added in fp32: 2048 -> 7168,
// 64 tokens of rank 32 20 us, all pieces wide 44; 7168 -> 4096, 1024 tokens of rank 64 112
// and 434.
template <typename T, int N>
__device__ __forceinline__ bool wide_piece(const float (&f)[N]) {
  if constexpr (!std::is_same<T, __half>::value) return false;
  float m = 0.0f;
  bool fits = true;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    fits = fits && fabsf(f[e]) <= 65504.0f;
    m = fmaxf(m, fabsf(f[e]));
  }
  return !fits || (m > 0.0f && m < 0x1p-14f);
}

// Two values of s h as their roundings and rounded remainders; an infinity has none.
template <typename T>
__device__ __forceinline__ void split_pair(float2 f, uint32_t& hi, uint32_t& low) {
  hi = pack2<T>(f);
  const float2 h = unpack2<T>(hi);
  low = pack2<T>(make_float2(fabsf(h.x) < INFINITY ? f.x - h.x : 0.0f,
                             fabsf(h.y) < INFINITY ? f.y - h.y : 0.0f));
}

// Byte offset of 16-byte piece `piece` of row `row` in a tile of 128-byte rows,
// permuted so that eight rows' same pieces lie in different banks.
__device__ __forceinline__ uint32_t tile_at(int row, int piece) {
  return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4));
}

// Whether the RUN places of a group, one a lane (-1: no token), hold tokens that
// follow one another, so that one copy fetches their rows.
__device__ __forceinline__ bool group_together(int tok) {
  const int first = __shfl_sync(0xFFFFFFFFu, tok, 0);
  return __all_sync(0xFFFFFFFFu, tok < 0 || tok == first + (int)(threadIdx.x & 31));
}

// Up to 128 tokens in all, SH_TOK a block as they come, on mma.sync: eight warps as
// four rows of 16 tokens by two shares of the ranks, each warp up to NT16 times 16 of
// them.  Block z has the adapters z, z + gridDim.z, ... of its tokens.
template <typename T, int NT16>
__global__ void __launch_bounds__(SH_THREADS, 2) lora_shrink_kernel(LoraParams p) {
  constexpr int XP = SH_TOK / 32;                        // a thread's pieces of x
  constexpr int NSPLIT = 2;                              // shares of the ranks
  constexpr int AP = (NT16 * NSPLIT * 16 + 31) / 32;     // a thread's pieces of A
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int16_t s_id[SH_TOK], s_list[SH_TOK];
  __shared__ uint32_t s_bits[32];
  __shared__ int s_n;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t0 = (int64_t)blockIdx.x * SH_TOK;
  bool bad = false;
  if (tid < SH_TOK) s_id[tid] = (int16_t)adapter_of(p, t0 + tid, &bad);
  if (bad) set_status(p.status, MOE_DEV_BAD_ADAPTER);
  __syncthreads();
  const int n_list = distinct_adapters(s_id, s_list, s_bits, &s_n, SH_TOK);
  const int64_t k0 = (int64_t)blockIdx.y * p.share_k;
  const int64_t k1 = min(p.K, k0 + p.share_k);
  const int slabs = k1 > k0 ? (int)((k1 - k0 + 63) / 64) : 0;
  const int R = (int)p.R, r16 = (R + 15) & ~15;
  const uint32_t base = smem_u32(smem);
  const uint32_t stage_bytes = (SH_TOK + r16) * 128;
  const T* x = static_cast<const T*>(p.x);
  const int m0 = (warp % 4) * 16, nh = warp / 4;

  // a thread's pieces: 16-byte piece c of rows row, row + 32, ...
  const int row = tid >> 3, c = tid & 7;
  const uint32_t at = base + tile_at(row, c);
  // a lane's addresses for ldmatrix: row of the tile, and the permuted piece of
  // each 16-wide K step (rows eight apart have the same permutation)
  const uint32_t xrow = (uint32_t)(m0 + (lane & 15)) * 128;
  const uint32_t arow = (uint32_t)(SH_TOK + nh * 16 + (lane & 7) + ((lane >> 4) << 3)) * 128;
  uint32_t xk[4], ak[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    xk[k] = xrow + (((uint32_t)(k * 2 + (lane >> 4)) ^ (lane & 7)) << 4);
    ak[k] = arow + (((uint32_t)(k * 2 + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
  }
  for (int d = blockIdx.z; d < n_list; d += gridDim.z) {
    const int a = s_list[d];
    const T* A = static_cast<const T*>(p.a) + (int64_t)a * R * p.K;
    const T *xp[XP], *ap[AP];
    uint32_t take = 0;
#pragma unroll
    for (int j = 0; j < XP; ++j) {
      const bool t = s_id[row + 32 * j] == a;
      xp[j] = t ? x + (t0 + row + 32 * j) * p.x_stride + k0 + c * 8 : x;
      take |= (uint32_t)t << j;
    }
#pragma unroll
    for (int j = 0; j < AP; ++j) {
      const bool t = row + 32 * j < R;
      ap[j] = t ? A + (int64_t)(row + 32 * j) * p.K + k0 + c * 8 : A;
      take |= (uint32_t)t << (XP + j);
    }
    int fill = 0;  // stage of the next load
    int64_t left = k1 - k0 - c * 8;  // this thread's columns from the next load on
    auto load = [&] {
      const uint32_t s = at + (uint32_t)fill * stage_bytes;
      const uint32_t t = left > 0 ? take : 0u;
#pragma unroll
      for (int j = 0; j < XP; ++j) {
        cp_async16(s + j * 4096, xp[j], (t >> j) & 1u);
        xp[j] += (t >> j) & 1u ? 64 : 0;
      }
#pragma unroll
      for (int j = 0; j < AP; ++j)
        if (row + 32 * j < r16) {
          cp_async16(s + SH_TOK * 128 + j * 4096, ap[j], (t >> (XP + j)) & 1u);
          ap[j] += (t >> (XP + j)) & 1u ? 64 : 0;
        }
      left -= 64;
      if (++fill == SH_STAGES) fill = 0;
    };
    float acc[NT16][2][4];
#pragma unroll
    for (int i = 0; i < NT16; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.0f;
    for (int s = 0; s < SH_STAGES - 1; ++s) {
      if (s < slabs) load();
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    uint32_t st = base;
    for (int s = 0; s < slabs; ++s) {
      asm volatile("cp.async.wait_group %0;" ::"n"(SH_STAGES - 2) : "memory");
      __syncthreads();
      if (s + SH_STAGES - 1 < slabs) load();
      asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t av[4];
        ldmatrix4(av, st + xk[k]);
#pragma unroll
        for (int i = 0; i < NT16; ++i) {
          if ((i * NSPLIT + nh) * 16 >= r16) break;
          uint32_t bv[4];
          ldmatrix4(bv, st + ak[k] + i * NSPLIT * 2048);
          mma_16816<T>(acc[i][0], av, bv[0], bv[1]);
          mma_16816<T>(acc[i][1], av, bv[2], bv[3]);
        }
      }
      st += stage_bytes;
      if (st == base + SH_STAGES * stage_bytes) st = base;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the stages are free for the next adapter
    float* h = p.h + (int64_t)blockIdx.y * p.T * R;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = m0 + (lane >> 2) + half * 8;
      if (s_id[r] != a) continue;
#pragma unroll
      for (int i = 0; i < NT16; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int n = (i * NSPLIT + nh) * 16 + j * 8 + (lane & 3) * 2;
          if (n < R)
            *reinterpret_cast<float2*>(h + (t0 + r) * R + n) =
                make_float2(acc[i][j][half * 2], acc[i][j][half * 2 + 1]);
        }
    }
  }
}

// More tokens, SH_LONG a block as they come or in their order, on tcgen05: a tile of the
// accumulator has a token a lane and a rank a column, and the cp.async stages have the
// 128-byte swizzle that the MMA reads.  In the tokens' order block z has the adapter of
// group z, unless an earlier group has it, and copies the rows of that group that do
// not lie together.
template <typename T>
__global__ void __launch_bounds__(SH_THREADS, 2) lora_shrink_long_kernel(LoraParams p) {
  constexpr int XP = SH_LONG / 32, AP = LORA_MAX_RANK / 32;  // a thread's pieces of x and A
  extern __shared__ uint8_t smem_raw[];
  __shared__ int16_t s_id[SH_LONG], s_list[SH_LONG];
  __shared__ int32_t s_tok[SH_LONG];
  __shared__ uint32_t s_bits[32];
  __shared__ int s_n, s_abort;
  __shared__ uint32_t s_tmem;
  __shared__ __align__(8) uint64_t s_bars[SH_STAGES];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t0 = (int64_t)blockIdx.x * SH_LONG;
  if (p.wide != nullptr && blockIdx.x + blockIdx.y + blockIdx.z == 0 && tid == 0) *p.wide = 0;
  if (p.order != nullptr && t0 >= *p.places) return;
  bool bad = false;
  if (tid < SH_LONG) {
    int64_t t = t0 + tid;
    if (p.order != nullptr) t = t < *p.places ? p.order[t] : -1;
    s_tok[tid] = (int32_t)t;
    s_id[tid] = (int16_t)adapter_of(p, t, &bad);
  }
  if (bad) set_status(p.status, MOE_DEV_BAD_ADAPTER);
  __syncthreads();
  int n_list;
  if (p.order == nullptr) {
    n_list = distinct_adapters(s_id, s_list, s_bits, &s_n, SH_LONG);
  } else {
    const int z = blockIdx.z;
    bool mine = s_id[z * RUN] >= 0;
    for (int g = 0; g < z; ++g) mine = mine && s_id[g * RUN] != s_id[z * RUN];
    if (tid == 0) s_list[z] = s_id[z * RUN];
    n_list = mine ? z + 1 : 0;
    __syncthreads();
  }
  const int64_t k0 = (int64_t)blockIdx.y * p.share_k;
  const int64_t k1 = min(p.K, k0 + p.share_k);
  const int slabs = (int)((k1 - k0 + 63) / 64);  // every share has some
  const int R = (int)p.R, r16 = (R + 15) & ~15;
  const T* x = static_cast<const T*>(p.x);

  if (p.order != nullptr) {
    // of group z's rows, where the projection cannot fetch them as they lie in x,
    // this share of K: 16-byte pieces, four in flight a thread
    const int g0 = blockIdx.z * RUN;
    if (!group_together(s_tok[g0 + lane])) {
      T* xs = static_cast<T*>(p.xs);
      const int pieces = (int)((k1 - k0) / 8);
      for (int i0 = tid; i0 < RUN * pieces; i0 += 4 * SH_THREADS) {
        Pack<T, 8> v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * SH_THREADS, r = i / pieces;
          if (i < RUN * pieces && s_tok[g0 + r] >= 0)
            v[u] = load_pack<T, 8>(x + s_tok[g0 + r] * p.x_stride + k0 + (i - r * pieces) * 8);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * SH_THREADS, r = i / pieces;
          if (i < RUN * pieces && s_tok[g0 + r] >= 0)
            store_pack<T, 8>(xs + (t0 + g0 + r) * p.K + k0 + (i - r * pieces) * 8, v[u]);
        }
      }
    }
  }

  if ((int)blockIdx.z >= n_list) return;
  const uint32_t cols = r16 <= 32 ? 32 : (r16 <= 64 ? 64 : 128);
  const uint32_t bars = smem_u32(s_bars);
  volatile int* abort_flag = &s_abort;
  if (tid == 0) {
    for (int s = 0; s < SH_STAGES; ++s) mbar_init(bars + 8 * s, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t stage_bytes = (SH_LONG + r16) * 128;
  const uint32_t idesc = f16_idesc(std::is_same<T, __nv_bfloat16>::value, SH_LONG, r16);
  // a thread's pieces: 16-byte piece c of rows row, row + 32, ...
  const int row = tid >> 3, c = tid & 7;
  const uint32_t at = base + tile_at(row, c);
  uint32_t seq = 0;  // slabs of all adapters so far; slab i has stage i % SH_STAGES
  bool ok = true;
  for (int d = blockIdx.z; d < n_list; d += gridDim.z) {
    const int a = s_list[d];
    const T* A = static_cast<const T*>(p.a) + (int64_t)a * R * p.K;
    const T *xp[XP], *ap[AP];
    uint32_t take = 0;
#pragma unroll
    for (int j = 0; j < XP; ++j) {
      const bool t = s_id[row + 32 * j] == a;
      xp[j] = t ? x + s_tok[row + 32 * j] * p.x_stride + k0 + c * 8 : x;
      take |= (uint32_t)t << j;
    }
#pragma unroll
    for (int j = 0; j < AP; ++j) {
      const bool t = row + 32 * j < R;
      ap[j] = t ? A + (int64_t)(row + 32 * j) * p.K + k0 + c * 8 : A;
      take |= (uint32_t)t << (XP + j);
    }
    uint32_t fill = seq % SH_STAGES;  // stage of the next load
    int64_t left = k1 - k0 - c * 8;   // this thread's columns from the next load on
    auto load = [&] {
      const uint32_t s = at + fill * stage_bytes;
      const uint32_t t = left > 0 ? take : 0u;
#pragma unroll
      for (int j = 0; j < XP; ++j) {
        cp_async16(s + j * 4096, xp[j], (t >> j) & 1u);
        xp[j] += (t >> j) & 1u ? 64 : 0;
      }
#pragma unroll
      for (int j = 0; j < AP; ++j)
        if (row + 32 * j < r16) {
          cp_async16(s + SH_LONG * 128 + j * 4096, ap[j], (t >> (XP + j)) & 1u);
          ap[j] += (t >> (XP + j)) & 1u ? 64 : 0;
        }
      left -= 64;
      if (++fill == SH_STAGES) fill = 0;
    };
    for (int s = 0; s < SH_STAGES - 1; ++s) {
      if (s < slabs) load();
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    bool failed = false;
    for (int s = 0; s < slabs; ++s, ++seq) {
      asm volatile("cp.async.wait_group %0;" ::"n"(SH_STAGES - 2) : "memory");
      fence_async_smem();  // each thread's own copies, before the MMA reads them
      failed = __syncthreads_or(!ok);
      if (failed) break;
      const uint32_t stage = seq % SH_STAGES;
      if (warp == 0) {
        const uint32_t st = base + stage * stage_bytes;
        const uint64_t ad = sw128_desc(st), bd = sw128_desc(st + SH_LONG * 128);
        if (elect_one()) {
          fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16(tmem, ad + 2 * k, bd + 2 * k, idesc, (s > 0 || k > 0) ? 1u : 0u);
          mma_commit(bars + 8 * stage);
        }
        __syncwarp();
      }
      if (s + SH_STAGES - 1 < slabs) {  // over the stage of the slab before
        if (s > 0) ok = mbar_wait(bars + 8 * ((seq - 1) % SH_STAGES),
                                  ((seq - 1) / SH_STAGES) & 1u, abort_flag, p.status);
        if (ok) load();
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (seq > 0) {  // the last MMAs issued; those before them are done too
      volatile int never = 0;
      ok = mbar_wait(bars + 8 * ((seq - 1) % SH_STAGES), ((seq - 1) / SH_STAGES) & 1u, &never,
                     p.status) && ok;
    }
    if (__syncthreads_or(!ok || failed)) break;
    fence_after();
    const int r = (warp & 3) * 32 + lane;  // lane of the sums, its token
    const bool mine = s_id[r] == a;
    float* h = p.h + ((int64_t)blockIdx.y * p.T + (mine ? s_tok[r] : 0)) * R;
    for (int n = (warp >> 2) * 16; n < r16; n += 32) {
      uint32_t v[16];
      tmem_ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + n, v);
      tmem_wait16(v);
#pragma unroll
      for (int q = 0; q < 16; q += 4)
        if (mine && n + q < R)
          *reinterpret_cast<float4*>(h + n + q) =
              make_float4(__uint_as_float(v[q]), __uint_as_float(v[q + 1]),
                          __uint_as_float(v[q + 2]), __uint_as_float(v[q + 3]));
      __syncwarp();
    }
    fence_before();
    __syncthreads();  // stages and sums are free for the next adapter
    fence_after();
  }
  fence_before();
  __syncthreads();
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                 : "memory");
  }
}

// ------------------------------------------------- projection, few tokens
// At 512 tokens this path takes 56 us and the pairs 81 (two more launches for the order);
// at 1024 the pairs take 113 us, and W would pass eight times here.
constexpr int SPLIT_TOKENS = 512;
constexpr int LG_M = 128;  // features of a tile
constexpr int LG_A_BYTES = LG_M * 128;
constexpr int LG_THREADS = 256;
constexpr int LG_SIDE = 192;  // warps 2..7 prepare the adapters' part
constexpr int LG_MAX_STAGES = 5;

// Stages of the ring for a tile of NT tokens: two CTAs share an SM up to NT = 64.
constexpr int lg_stages(int nt) { return nt <= 32 ? 5 : 4; }
constexpr int lg_ring(int nt) { return lg_stages(nt) * (LG_A_BYTES + nt * 128); }
// Shared memory: ring; of this CTA's share of the tokens s h (rounding, remainder)
// and the adapters' part; barriers, ids, order, chunks, wide pieces.
__host__ __device__ inline int lg_smem(int nt, int splits, int R) {
  return 1024 + lg_ring(nt) + (R > 0 ? nt / splits * (R + LG_M) * 4 : 0) + 512 + nt * 12;
}

// Tokens of one adapter, neighbours in the order, at most 8: one MMA tile.
struct Chunk {
  int16_t pos, count, adapter, unused;
};

// The adapters' part of a share of the tokens, add[token][LG_M features], with
// mma.sync: 16 features by 8 tokens a task, dealt out to the warps, U tasks in
// flight.  Any order of the ranks serves as long as both operands have the same:
// lane q of four takes ranks 8 q .. 8 q + 7 of every 32 for two K steps, so a
// feature's row of B comes in 16-byte loads, end to end over the four lanes.
// hs: s h of the share, [token][R] its rounding, then the same of the remainder.
template <typename T, int RS, int U>  // RS: K of the tasks, 32 ranks each
__device__ __forceinline__ void expand_tokens(const LoraParams& p, const Chunk* chunks, int n,
                                              const T* hs, int share, float* add, int64_t n0,
                                              int warp, int warps) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int R = (int)p.R;
  const T* B = static_cast<const T*>(p.b) + n0 * R;
  const T* low = hs + share * R;
  const int tasks = n * (LG_M / 16);
  for (int k0 = warp * U; k0 < tasks; k0 += warps * U) {
    uint4 b[U][RS][2];  // rows g and g + 8
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = min(k0 + u, tasks - 1), f = (k % (LG_M / 16)) * 16 + g;
      const int a = chunks[k / (LG_M / 16)].adapter;
#pragma unroll
      for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = s * 32 + q * 8;
          b[u][s][e] = make_uint4(0, 0, 0, 0);
          if (a >= 0 && r < R && n0 + f + e * 8 < p.N)
            b[u][s][e] = __ldg(reinterpret_cast<const uint4*>(
                B + ((int64_t)a * p.N + f + e * 8) * R + r));
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u >= tasks) break;
      const Chunk c = chunks[(k0 + u) / (LG_M / 16)];
      const int f = ((k0 + u) % (LG_M / 16)) * 16 + g;
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        const int r = s * 32 + q * 8;
        uint4 h[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (c.adapter >= 0 && g < c.count && r < R) {  // token g of the chunk
          h[0] = *reinterpret_cast<const uint4*>(hs + (c.pos + g) * R + r);
          h[1] = *reinterpret_cast<const uint4*>(low + (c.pos + g) * R + r);
        }
        const uint4 b0 = b[u][s][0], b1 = b[u][s][1];
        const uint32_t a0[4] = {b0.x, b1.x, b0.y, b1.y}, a1[4] = {b0.z, b1.z, b0.w, b1.w};
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          mma_16816<T>(acc, a0, h[part].x, h[part].y);
          mma_16816<T>(acc, a1, h[part].z, h[part].w);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // feature f (+ 8), token 2 q (+ 1)
        const int t = q * 2 + (e & 1);
        if (t < c.count) add[(c.pos + t) * LG_M + f + (e >> 1) * 8] = acc[e];
      }
    }
  }
}

// The wide pieces, in fp32: feature f a thread, piece after piece, bit i of `wide` ranks
// 4 i, ... of the share's s h.  Where a piece's rounding and remainder were, hs has its
// four floats by now.
template <typename T>
__device__ __forceinline__ void add_wide_tokens(const LoraParams& p, const uint32_t* wide,
                                                const T* hs, const int16_t* id,
                                                const int16_t* order, int share, float* add,
                                                int64_t n0, int f) {
  const int R = (int)p.R, q4 = R / 4;
  for (int w = 0; w * 32 < share * q4; ++w)
    for (uint32_t m = wide[w]; m != 0;) {
      constexpr int U = 4;  // rows of B in flight
      int piece[U];
      uint2 b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = m != 0 ? w * 32 + __ffs(m) - 1 : -1, k = i / q4;
        m &= m - 1;
        piece[u] = i;
        b[u] = make_uint2(0, 0);
        if (i >= 0 && n0 + f < p.N)
          b[u] = __ldg(reinterpret_cast<const uint2*>(
              static_cast<const T*>(p.b) +
              ((int64_t)id[order[k]] * p.N + n0 + f) * R + (i - k * q4) * 4));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (piece[u] < 0) break;
        const float2 b0 = unpack2<T>(b[u].x), b1 = unpack2<T>(b[u].y);
        const float2 h0 = reinterpret_cast<const float2*>(hs)[piece[u]];
        const float2 h1 = reinterpret_cast<const float2*>(hs + share * R)[piece[u]];
        float& sum = add[piece[u] / q4 * LG_M + f];
        sum = fmaf(b0.x, h0.x, fmaf(b0.y, h0.y, fmaf(b1.x, h1.x, fmaf(b1.y, h1.y, sum))));
      }
    }
}

// Stores the share's tokens: the cluster's sums in rank order and the adapters' part.
template <typename T, int SPLITS>
__device__ __forceinline__ void join_tokens(const LoraParams& p, const float* sums,
                                            const float* add, const int16_t* order, int64_t t0,
                                            int64_t n0, int pos0, int share) {
  const uint32_t at0 = smem_u32(sums);
  const bool pairs = (p.out_stride % 2 == 0) && (reinterpret_cast<uintptr_t>(p.out) & 3u) == 0;
  for (int i = threadIdx.x; i < share * (LG_M / 4); i += LG_THREADS) {
    const int k = i / (LG_M / 4), c = order[pos0 + k], f = (i % (LG_M / 4)) * 4;
    if (t0 + c >= p.T) continue;
    float4 v[SPLITS];
#pragma unroll
    for (int r = 0; r < SPLITS; ++r)
      v[r] = SPLITS == 1 ? *reinterpret_cast<const float4*>(sums + c * LG_M + f)
                         : ld_cluster4(at0 + (uint32_t)(c * LG_M + f) * 4, r);
#pragma unroll
    for (int r = 1; r < SPLITS; ++r)
      v[0].x += v[r].x, v[0].y += v[r].y, v[0].z += v[r].z, v[0].w += v[r].w;
    if (add != nullptr) {
      const float4 u = *reinterpret_cast<const float4*>(add + k * LG_M + f);
      v[0].x += u.x, v[0].y += u.y, v[0].z += u.z, v[0].w += u.w;
    }
    T* out = static_cast<T*>(p.out) + (t0 + c) * p.out_stride + n0 + f;
    if (pairs && n0 + f + 4 <= p.N) {
      reinterpret_cast<uint32_t*>(out)[0] = pack2<T>(make_float2(v[0].x, v[0].y));
      reinterpret_cast<uint32_t*>(out)[1] = pack2<T>(make_float2(v[0].z, v[0].w));
    } else {
      const float w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n0 + f + e < p.N) out[e] = from_f32<T>(w[e]);
    }
  }
}

template <typename T, int NT>
__global__ void __launch_bounds__(LG_THREADS, NT <= 64 ? 2 : 1)
    lora_split_kernel(const __grid_constant__ LoraParams p, const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmX) {
  constexpr int STAGES = lg_stages(NT), STAGE_BYTES = LG_A_BYTES + NT * 128;
  constexpr uint32_t IDESC = f16_idesc(std::is_same<T, __nv_bfloat16>::value, LG_M, NT);
  constexpr uint32_t TMEM_COLS = NT < 32 ? 32 : NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int share = NT / p.splits;
  T* hs = reinterpret_cast<T*>(smem + STAGES * STAGE_BYTES);  // [2][share][R]
  float* add = reinterpret_cast<float*>(hs + 2 * share * p.R);  // [share][LG_M]
  uint64_t* bars = reinterpret_cast<uint64_t*>(add + (p.S > 0 ? share * LG_M : 0));
  // full[STAGES], empty[STAGES], done
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * LG_MAX_STAGES + 1);
  int* s_abort = reinterpret_cast<int*>(tmem_holder + 1);
  int* s_chunks = s_abort + 1;
  int* s_any_wide = s_chunks + 1;
  Chunk* chunks = reinterpret_cast<Chunk*>(reinterpret_cast<uint8_t*>(bars) + 256);  // [NT]
  int16_t* s_id = reinterpret_cast<int16_t*>(chunks + NT);
  int16_t* s_order = s_id + NT;
  uint32_t* s_wide = reinterpret_cast<uint32_t*>(s_order + NT);  // [64]: NT R / 4 bits, R <= 64
                                                                 // above 64 tokens
  constexpr bool half = std::is_same<T, __half>::value;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = s_abort;
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + LG_MAX_STAGES);
  const uint32_t done_bar = smem_u32(bars + 2 * LG_MAX_STAGES);

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(done_bar, 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    prefetch_map(&tmW);
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
  // Behind a shrink launch everything before it has completed when this
  // kernel starts (it lets its dependents start after its own wait), so x, W
  // and ids may be read; h only after pdl_wait.
  if (p.wait_first) pdl_wait();
  pdl_launch_dependents();

  const int rank = p.splits > 1 ? (int)(blockIdx.x % (unsigned)p.splits) : 0;
  const int64_t n0 = (int64_t)(blockIdx.x / (unsigned)p.splits) * LG_M;
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
        tma_load_2d(s, &tmW, kb * 64, (int)n0, bar);
        tma_load_2d(s + LG_A_BYTES, &tmX, kb * 64, (int)t0, bar);
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
      const uint64_t ad = sw128_desc(s), bd = sw128_desc(s + LG_A_BYTES);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f16(tmem, ad + 2 * k, bd + 2 * k, IDESC, accumulate | (k > 0));
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
  } else {
    // -------------------------------------- tokens' order, s h; then the sums
    const int st = tid - 64;
    auto side_sync = [] { asm volatile("bar.sync 1, 192;" ::: "memory"); };
    if (p.S > 0) {
      bool bad = false;
      for (int i = st; i < NT; i += LG_SIDE) s_id[i] = (int16_t)adapter_of(p, t0 + i, &bad);
      side_sync();
      for (int i = st; i < NT; i += LG_SIDE) {
        int before = 0;
        for (int j = 0; j < NT; ++j)
          before += s_id[j] < s_id[i] || (s_id[j] == s_id[i] && j < i);
        s_order[before] = (int16_t)i;
      }
      side_sync();
      // chunks of the share: runs of an adapter, cut every 8 tokens; the rows of B
      // that they will read start towards L2
      const int pos0 = rank * share;
      auto adapter = [&](int i) { return (int)s_id[s_order[pos0 + i]]; };
      auto run_begin = [&](int i) {
        int j = i;
        while (j > 0 && adapter(j - 1) == adapter(i)) --j;
        return j;
      };
      if (st == 0) *s_chunks = *s_any_wide = 0;
      for (int i = st; half && i < 64; i += LG_SIDE) s_wide[i] = 0;
      side_sync();
      for (int i = st; i < share; i += LG_SIDE) {
        const int a = adapter(i), begin = run_begin(i);
        if ((i - begin) % 8 != 0) continue;
        int count = 1;
        while (count < 8 && i + count < share && adapter(i + count) == a) ++count;
        chunks[atomicAdd(s_chunks, 1)] = Chunk{(int16_t)i, (int16_t)count, (int16_t)a, 0};
        if (a >= 0 && i == begin)
          prefetch_l2(static_cast<const T*>(p.b) + ((int64_t)a * p.N + n0) * p.R,
                      (uint32_t)(min((int64_t)LG_M, p.N - n0) * p.R * 2));
      }
      if (!p.wait_first) pdl_wait();
      // s h of the share, four ranks a thread: their roundings and remainders, or, where
      // `floats` and the piece is wide, the values themselves
      auto gather = [&](bool floats) {
        const int q4 = (int)p.R / 4;
        for (int i = st; i < share * q4; i += LG_SIDE) {
          const int k = i / q4, c = s_order[pos0 + k], a = s_id[c];
          if (a < 0) continue;
          float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          const float* src = p.h + (t0 + c) * p.R + (i - k * q4) * 4;
          for (int s0 = 0; s0 < p.shares; s0 += 8) {  // eight shares' sums in flight
            float4 u[8];
#pragma unroll
            for (int s = 0; s < 8; ++s)
              u[s] = s0 + s < p.shares
                         ? __ldcg(reinterpret_cast<const float4*>(src + (s0 + s) * p.T * p.R))
                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int s = 0; s < 8; ++s)
              sum.x += u[s].x, sum.y += u[s].y, sum.z += u[s].z, sum.w += u[s].w;
          }
          const float scale = __ldg(p.scale + a);
          const float f[4] = {scale * sum.x, scale * sum.y, scale * sum.z, scale * sum.w};
          uint2 hi, low;
          if (half && wide_piece<T>(f)) {
            atomicOr(s_wide + i / 32, 1u << (i & 31));
            *s_any_wide = 1;
            hi = low = make_uint2(0, 0);
            if (floats) {
              hi = make_uint2(__float_as_uint(f[0]), __float_as_uint(f[1]));
              low = make_uint2(__float_as_uint(f[2]), __float_as_uint(f[3]));
            }
          } else {
            split_pair<T>(make_float2(f[0], f[1]), hi.x, low.x);
            split_pair<T>(make_float2(f[2], f[3]), hi.y, low.y);
          }
          reinterpret_cast<uint2*>(hs)[i] = hi;
          reinterpret_cast<uint2*>(hs + share * p.R)[i] = low;
        }
        side_sync();
      };
      gather(false);
      const int n = *s_chunks, w = warp - 2;
      if (p.R <= 32)
        expand_tokens<T, 1, 4>(p, chunks, n, hs, share, add, n0, w, LG_SIDE / 32);
      else if (p.R <= 64)
        expand_tokens<T, 2, 2>(p, chunks, n, hs, share, add, n0, w, LG_SIDE / 32);
      else
        expand_tokens<T, 4, 1>(p, chunks, n, hs, share, add, n0, w, LG_SIDE / 32);
      if (half && *s_any_wide != 0) {
        side_sync();  // the MMAs' part is there, and hs free
        gather(true);
        if (st < LG_M)
          add_wide_tokens<T>(p, s_wide, hs, s_id, s_order + pos0, share, add, n0, st);
      }
    } else {
      for (int i = st; i < NT; i += LG_SIDE) s_id[i] = -1, s_order[i] = (int16_t)i;
    }
    // done is also signalled after a wait ran out; the sums are then not whole
    if (warp >= 4 && warp_wait(done_bar, 0, abort_flag, p.status) && *abort_flag == 0) {
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
        for (int j = 0; j < 16; ++j) red[(c + j) * LG_M + nl] = __uint_as_float(v[j]);
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
    const float* part = p.S > 0 ? add : nullptr;
    const int pos0 = rank * share;
    if (p.splits == 1)
      join_tokens<T, 1>(p, sums, part, s_order, t0, n0, pos0, share);
    else if (p.splits == 2)
      join_tokens<T, 2>(p, sums, part, s_order, t0, n0, pos0, share);
    else if (p.splits == 4)
      join_tokens<T, 4>(p, sums, part, s_order, t0, n0, pos0, share);
    else
      join_tokens<T, 8>(p, sums, part, s_order, t0, n0, pos0, share);
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

// ------------------------------------------------ projection, many tokens
constexpr int LP_TILE = 256;    // features and tokens of a pair's tile
constexpr int LP_HALF = 128;    // of them one CTA's
constexpr int LP_STAGES = 6;
constexpr int LP_STAGE_BYTES = 2 * LP_HALF * 128;  // a CTA's part: W rows, x rows
constexpr int LP_H_BYTES = LP_HALF * 128;
constexpr int LP_THREADS = 384;
constexpr int LP_EPI_WARP0 = 8;                    // warps 8..11: epilogue
constexpr int LP_BUILD_WARPS = 6;                  // warps 2..7: tiles of s h
constexpr int LP_BUILDERS = LP_BUILD_WARPS * 32;
constexpr int LP_SMEM = 1024 + LP_STAGES * LP_STAGE_BYTES + 2 * LP_H_BYTES + 256 + LP_HALF * 8;
constexpr int LP_GROUPS = LP_TILE / RUN;

// The runs of a tile, the same in every warp that asks: lane g < LP_GROUPS has
// the adapter of columns [RUN g, RUN g + RUN), and bit g of `starts` is set where
// a run of an adapter begins, of `ends` where a run or a gap ends.
struct Runs {
  int adapter;
  uint32_t starts, ends;
};
__device__ __forceinline__ Runs tile_runs(const LoraParams& p, int64_t pos0, int64_t places,
                                          int lane) {
  Runs r;
  const int64_t pos = pos0 + lane * RUN;
  bool bad = false;
  r.adapter = -1;
  if (lane < LP_GROUPS && pos < places) r.adapter = adapter_of(p, p.order[pos], &bad);
  const int before = __shfl_up_sync(0xFFFFFFFFu, r.adapter, 1);
  const bool begins = lane < LP_GROUPS && (lane == 0 || before != r.adapter);
  r.starts = __ballot_sync(0xFFFFFFFFu, begins && r.adapter >= 0);
  r.ends = __ballot_sync(0xFFFFFFFFu, begins) >> 1 | 1u << (LP_GROUPS - 1);
  return r;
}
// Last group of the run that begins at g.
__device__ __forceinline__ int run_end(const Runs& r, int g) { return __ffs(r.ends >> g) - 1 + g; }

// The work of the pairs: whole tiles dealt out in rounds, and the tiles of a last
// round that would leave pairs idle cut along K, so that each pair has a piece (1024
// tokens 113 us, uncut 132; 8192 324 against 328).
constexpr int LP_MIN_SLABS = 8;  // of a piece
constexpr int64_t LP_PIECE = 2 * LP_TILE * LP_HALF;  // its sums
struct Work {
  int units, pairs, full, parts, items, per, slabs;
  __device__ __forceinline__ Work(int n_units, int n_pairs, int n_slabs, bool cut)
      : units(n_units), pairs(n_pairs), slabs(n_slabs) {
    const int rest = n_units % n_pairs;
    parts = cut && rest > 0 ? min(n_pairs / rest, n_slabs / LP_MIN_SLABS) : 1;
    if (parts < 2) parts = 1;
    per = (n_slabs + parts - 1) / parts;
    parts = (n_slabs + per - 1) / per;  // every piece has slabs
    full = parts > 1 ? n_units - rest : n_units;
    items = full + (n_units - full) * parts;
  }
};
struct Item {
  int unit, kb0, kb1, piece;  // piece: -1, a whole tile; else its place among the pieces
  bool adapters;              // the adapters' part goes with the first piece
};
__device__ __forceinline__ Item work_item(const Work& w, int i) {
  if (i < w.full) return Item{i, 0, w.slabs, -1, true};
  const int j = i - w.full, part = j % w.parts;
  return Item{w.full + j / w.parts, part * w.per, min(w.slabs, (part + 1) * w.per), j, part == 0};
}

// Adds the wide pieces of a group's tokens, lane l's tok (-1: none), all of adapter a, to
// this lane's sums, v[j >> 4][j & 15] of token j and feature n.
template <typename T>
__device__ __forceinline__ void add_wide(const LoraParams& p, int a, int tok, int64_t n,
                                         uint32_t (&v)[2][16]) {
  const int R = (int)p.R;
  uint4 flags = make_uint4(0, 0, 0, 0);  // of pieces, a byte each
  if (tok >= 0) flags = __ldcg(reinterpret_cast<const uint4*>(p.wide + 4) + tok);
  for (int r = 0; r < R; r += 8) {
    const uint32_t word = r < 32 ? flags.x : (r < 64 ? flags.y : (r < 96 ? flags.z : flags.w));
    const bool mine = tok >= 0 && ((word >> (r & 31)) & 0xFFu) != 0;
    const uint32_t which = __ballot_sync(0xFFFFFFFFu, mine);
    if (which == 0) continue;
    float f[8] = {};
    if (mine) {
      for (int s = 0; s < p.shares; ++s) {
        const float4* src = reinterpret_cast<const float4*>(p.h + (s * p.T + tok) * R + r);
        const float4 u0 = __ldcg(src), u1 = __ldcg(src + 1);
        f[0] += u0.x, f[1] += u0.y, f[2] += u0.z, f[3] += u0.w;
        f[4] += u1.x, f[5] += u1.y, f[6] += u1.z, f[7] += u1.w;
      }
      const float scale = __ldg(p.scale + a);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= scale;
    }
    float b[8] = {};
    if (n < p.N)
      load_pack<T, 8>(static_cast<const T*>(p.b) + (a * p.N + n) * R + r).get(b);
#pragma unroll
    for (int j = 0; j < 32; ++j) {  // no branch a token: their chains overlap
      const float before = __uint_as_float(v[j >> 4][j & 15]);
      float sum = before;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(b[e], __shfl_sync(0xFFFFFFFFu, f[e], j), sum);
      v[j >> 4][j & 15] = __float_as_uint((which >> j) & 1u ? sum : before);
    }
  }
}

// A persistent pair of CTAs; CTA r of the pair has features [128 r, 128 r + 128)
// and tokens [128 r, ...) of a tile's operands, and those features' sums for all
// 256 tokens.  The first CTA issues the MMAs of both; its full[] and hfull
// barriers count both CTAs' copies and tiles, and each commit reaches both.
template <typename T>
__global__ void __launch_bounds__(LP_THREADS, 1)
    lora_pair_kernel(const __grid_constant__ LoraParams p, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ CUtensorMap tmXs,
                     const __grid_constant__ CUtensorMap tmB) {
  constexpr uint32_t IDESC = f16_idesc(std::is_same<T, __nv_bfloat16>::value, LP_TILE, LP_TILE);
  constexpr uint32_t IDESC_RUN = f16_idesc(std::is_same<T, __nv_bfloat16>::value, LP_TILE, RUN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* hbuf = smem + LP_STAGES * LP_STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(hbuf + 2 * LP_H_BYTES);
  // full[STAGES], empty[STAGES], hfull[2], hempty[2], tfull[2], tempty[2]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * LP_STAGES + 8);
  int* s_abort = reinterpret_cast<int*>(tmem_holder + 1);
  int* s_go = s_abort + 1;
  int32_t* s_tok = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(bars) + 256);  // [128]
  int32_t* s_row = s_tok + LP_HALF;  // adapter of a row of the tile of s h

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = s_abort;
  const uint32_t rank = cluster_rank();
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + LP_STAGES);
  const uint32_t hfull0 = smem_u32(bars + 2 * LP_STAGES), hempty0 = hfull0 + 16;
  const uint32_t tfull0 = hfull0 + 32, tempty0 = hfull0 + 48;

  if (tid == 0) {
    for (int s = 0; s < LP_STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(hfull0 + 8 * b, 2 * LP_BUILD_WARPS);
      mbar_init(hempty0 + 8 * b, 1);
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 2 * 4);
    }
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    prefetch_map(&tmW);
    prefetch_map(&tmX);
    prefetch_map(&tmXs);
    prefetch_map(&tmB);
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
  if (p.wait_first) pdl_wait();  // else as in lora_split_kernel; order too is complete
  pdl_launch_dependents();

  const bool adapters = p.S > 0;
  const int64_t places = adapters ? *p.places : p.T;
  const int n_tiles = (int)((p.N + LP_TILE - 1) / LP_TILE);
  const int units = n_tiles * (int)((places + LP_TILE - 1) / LP_TILE);
  const int first = (int)(blockIdx.x >> 1), stride = (int)(gridDim.x >> 1);
  const Work work(units, stride, (int)((p.K + 63) / 64), p.partials != nullptr);
  const int r16 = (int)((p.R + 15) & ~15);
  const int rchunks = (r16 + 63) / 64;
  const bool one_part = 2 * r16 <= 64;  // rounding and remainder fit one tile
  const int builds = adapters ? rchunks * (one_part ? 1 : 2) : 0;  // tiles of s h of a unit

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_phase = 0;
    auto advance = [&] {
      issued |= 1u << stage;
      issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
      if (++stage == LP_STAGES) stage = 0, phase ^= 1u;
    };
    bool ok = true;
    for (int i = first; ok && i < work.items; i += stride) {
      const Item item = work_item(work, i);
      const int u = item.unit;
      const int n0 = (u % n_tiles) * LP_TILE + (int)rank * LP_HALF;
      const int64_t t0 = (int64_t)(u / n_tiles) * LP_TILE;
      // this CTA's four groups: first row in x where their tokens follow one
      // another, else ~place in the rows that the shrink has put in order
      int from[LP_GROUPS / 2];
      bool sorted_rows = false;
#pragma unroll
      for (int i = 0; i < LP_GROUPS / 2; ++i) {
        const int64_t place = t0 + rank * LP_HALF + i * RUN;
        from[i] = (int)place;
        if (!adapters) continue;
        const int tok = place + lane < places ? p.order[place + lane] : -1;
        const bool together = group_together(tok);
        const int row0 = __shfl_sync(0xFFFFFFFFu, tok, 0);
        from[i] = place >= places ? 0 : (together ? row0 : ~(int)place);
        sorted_rows = sorted_rows || from[i] < 0;
      }
      if (sorted_rows) pdl_wait();
      for (int kb = item.kb0; kb < item.kb1 && ok; ++kb) {
#ifdef MOE_TEST_WITHHOLD_STAGE
        if (blockIdx.x < 2 && kb > item.kb0) {  // as in lora_split_kernel: the first pair stops here
          ok = false;
          break;
        }
#endif
        ok = warp_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.status);
        if (!ok) break;
        const uint32_t bar = cluster_address(full0 + 8 * stage, 0);
        const uint32_t s = smem_u32(smem + stage * LP_STAGE_BYTES);
        if (elect_one()) {
          if (rank == 0) mbar_expect_tx(full0 + 8 * stage, 2 * LP_STAGE_BYTES);
          tma_load_2d_pair(s, &tmW, kb * 64, n0, bar);
#pragma unroll
          for (int i = 0; i < LP_GROUPS / 2; ++i) {
            const uint32_t dst = s + LP_HALF * 128 + i * RUN * 128;
            if (from[i] >= 0)
              tma_load_2d_pair(dst, &tmX, kb * 64, from[i], bar);
            else
              tma_load_2d_pair(dst, &tmXs, kb * 64, ~from[i], bar);
          }
        }
        __syncwarp();
        advance();
      }
      if (!adapters || !item.adapters || !ok) continue;
      const Runs runs = tile_runs(p, t0, places, lane);
      for (int b = 0; b < builds && ok; ++b) {
        const int rc = (one_part ? b : b >> 1) * 64;
        for (uint32_t m = runs.starts; m != 0 && ok; m &= m - 1) {
          const int a = __shfl_sync(0xFFFFFFFFu, runs.adapter, __ffs(m) - 1);
          ok = warp_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.status);
          if (!ok) break;
          if (elect_one()) {
            if (rank == 0) mbar_expect_tx(full0 + 8 * stage, 2 * LP_HALF * 128);
            tma_load_2d_pair(smem_u32(smem + stage * LP_STAGE_BYTES), &tmB, rc,
                             (int)(a * p.N + n0), cluster_address(full0 + 8 * stage, 0));
          }
          __syncwarp();
          advance();
        }
      }
    }
    if (rank == 0)  // both CTAs' copies have landed before either leaves
      for (int s = 0; s < LP_STAGES; ++s)
        if (issued & (1u << s)) {
          volatile int never = 0;
          mbar_wait(full0 + 8 * s, (issued_phase >> s) & 1u, &never, p.status);
        }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------- MMA (the first CTA's)
    int stage = 0, ab = 0, hs = 0;
    uint32_t phase = 0, hphase = 0, aphase = 0;
    bool ok = rank == 0;
    for (int i = first; ok && i < work.items; i += stride) {
      const Item item = work_item(work, i);
      const int u = item.unit;
      ok = warp_wait(tempty0 + 8 * ab, aphase ^ 1u, abort_flag, p.status);
      const uint32_t d = tmem + (uint32_t)(ab * LP_TILE);
      for (int kb = item.kb0; kb < item.kb1 && ok; ++kb) {
        ok = warp_wait(full0 + 8 * stage, phase, abort_flag, p.status);
        if (!ok) break;
        fence_after();
        const uint32_t s = smem_u32(smem + stage * LP_STAGE_BYTES);
        const uint64_t ad = sw128_desc(s), bd = sw128_desc(s + LP_HALF * 128);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f16_pair(d, ad + 2 * k, bd + 2 * k, IDESC,
                         kb > item.kb0 || k > 0);
          mma_commit_pair(empty0 + 8 * stage);
        }
        __syncwarp();
        if (++stage == LP_STAGES) stage = 0, phase ^= 1u;
      }
      Runs runs{};
      if (adapters && item.adapters)
        runs = tile_runs(p, (int64_t)(u / n_tiles) * LP_TILE, places, lane);
      if (runs.starts != 0) {
        for (int b = 0; b < builds && ok; ++b) {
          const int steps = min(4, r16 / 16 - (one_part ? b : b >> 1) * 4);
          ok = warp_wait(hfull0 + 8 * hs, hphase, abort_flag, p.status);
          const uint8_t* hb = hbuf + hs * LP_H_BYTES;
          for (uint32_t m = runs.starts; m != 0 && ok; m &= m - 1) {
            const int g = __ffs(m) - 1, len = run_end(runs, g) - g + 1;
            ok = warp_wait(full0 + 8 * stage, phase, abort_flag, p.status);
            if (!ok) break;
            fence_after();
            // the run's columns alone; each CTA has half of its tokens in hbuf
            const uint32_t dr = d + (uint32_t)(g * RUN);
            const uint32_t idesc = IDESC_RUN + ((uint32_t)((len - 1) * (RUN >> 3)) << 17);
            const uint64_t ad = sw128_desc(smem_u32(smem + stage * LP_STAGE_BYTES));
            const uint64_t bd = sw128_desc(smem_u32(hb + g * (RUN / 2) * 128));
            if (elect_one()) {
              for (int k = 0; k < steps; ++k) {
                mma_f16_pair(dr, ad + 2 * k, bd + 2 * k, idesc, 1);
                if (one_part) mma_f16_pair(dr, ad + 2 * k, bd + 2 * (steps + k), idesc, 1);
              }
              mma_commit_pair(empty0 + 8 * stage);
            }
            __syncwarp();
            if (++stage == LP_STAGES) stage = 0, phase ^= 1u;
          }
          if (elect_one()) mma_commit_pair(hempty0 + 8 * hs);
          __syncwarp();
          hs ^= 1;
          if (hs == 0) hphase ^= 1u;
        }
      }
      if (elect_one()) mma_commit_pair(tfull0 + 8 * ab);
      __syncwarp();
      ab ^= 1;
      if (ab == 0) aphase ^= 1u;
    }
  } else if (warp < LP_EPI_WARP0) {
    // ---------------------------------------------------------- tiles of s h
    const int bt = tid - 64;
    auto build_sync = [] { asm volatile("bar.sync 1, 192;" ::: "memory"); };
    int hs = 0;
    uint32_t hphase = 0;
    bool ok = true, waited = p.wait_first != 0;
    const int R = (int)p.R;
    for (int i = first; adapters && i < work.items; i += stride) {
      const Item item = work_item(work, i);
      if (!item.adapters) continue;
      const int u = item.unit;
      // one warp decides for all whether to go on, so that the barriers match
      if (bt == 0) *s_go = ok && *abort_flag == 0;
      build_sync();
      if (*s_go == 0) break;
      const int64_t t0 = (int64_t)(u / n_tiles) * LP_TILE;
      const Runs runs = tile_runs(p, t0, places, lane);
      if (runs.starts == 0) {
        build_sync();
        continue;
      }
      // row j of this CTA's tile: of a run of `len` groups from g on, the first
      // half of its tokens lies in the first CTA's rows, the second in the other's
      if (warp < 6) {
        const int j = bt, grp = j / (RUN / 2);
        const int g = 31 - __clz(runs.starts & ((2u << grp) - 1u));  // -1: no run before
        int tok = -1, a = -1;
        const int end = g >= 0 ? run_end(runs, g) : -1;
        if (g >= 0 && grp <= end) {
          const int len = end - g + 1;
          tok = p.order[t0 + g * RUN + (int)rank * len * (RUN / 2) + j - g * (RUN / 2)];
        }
        a = __shfl_sync(0xFFFFFFFFu, runs.adapter, g >= 0 ? g : 0);
        s_tok[j] = tok;
        s_row[j] = a;
      }
      build_sync();
      if (!waited) pdl_wait();
      waited = true;
      // hi: the rounding of s h, low: the rounded remainder.  With one_part both
      // go to one tile, side by side; else to two tiles, from one reading of h.
      constexpr int U = 2, SH = 4;  // pieces and shares' sums in flight
      auto values = [&](const int (&t)[U], const int (&r)[U], Pack<T, 8> (&hi)[U],
                        Pack<T, 8> (&low)[U]) {
        float4 u0[U], u1[U];
        const int64_t step = p.T * R;
#pragma unroll
        for (int k = 0; k < U; ++k) u0[k] = u1[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int s0 = 0; s0 < p.shares; s0 += SH) {
          float4 v0[U][SH], v1[U][SH];
#pragma unroll
          for (int k = 0; k < U; ++k)
#pragma unroll
            for (int s = 0; s < SH; ++s) {
              v0[k][s] = v1[k][s] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              if (t[k] >= 0 && s_tok[t[k]] >= 0 && r[k] < R && s0 + s < p.shares) {
                const float4* src = reinterpret_cast<const float4*>(
                    p.h + (int64_t)s_tok[t[k]] * R + r[k] + (s0 + s) * step);
                v0[k][s] = __ldcg(src);
                v1[k][s] = __ldcg(src + 1);
              }
            }
#pragma unroll
          for (int k = 0; k < U; ++k)
#pragma unroll
            for (int s = 0; s < SH; ++s) {
              u0[k].x += v0[k][s].x, u0[k].y += v0[k][s].y;
              u0[k].z += v0[k][s].z, u0[k].w += v0[k][s].w;
              u1[k].x += v1[k][s].x, u1[k].y += v1[k][s].y;
              u1[k].z += v1[k][s].z, u1[k].w += v1[k][s].w;
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const float scale = t[k] >= 0 && s_row[t[k]] >= 0 ? __ldg(p.scale + s_row[t[k]]) : 0.0f;
          float f[8] = {scale * u0[k].x, scale * u0[k].y, scale * u0[k].z, scale * u0[k].w,
                        scale * u1[k].x, scale * u1[k].y, scale * u1[k].z, scale * u1[k].w};
          if constexpr (std::is_same<T, __half>::value) {
            const bool wide = wide_piece<T>(f);
            if (t[k] >= 0 && s_tok[t[k]] >= 0 && r[k] < R) {
              reinterpret_cast<uint8_t*>(p.wide + 4)[(int64_t)s_tok[t[k]] * 16 + r[k] / 8] = wide;
              if (wide) *p.wide = 1;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = wide ? 0.0f : f[e];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t h, l;
            split_pair<T>(make_float2(f[2 * e], f[2 * e + 1]), h, l);
            hi[k].set_word(e, h), low[k].set_word(e, l);
          }
        }
      };
      auto ready = [&] {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_address(hfull0 + 8 * hs, 0));
        hs ^= 1;
        if (hs == 0) hphase ^= 1u;
      };
      for (int rc = 0; rc < r16 && ok; rc += 64) {
        ok = warp_wait(hempty0 + 8 * hs, hphase ^ 1u, abort_flag, p.status);
        if (!one_part) ok = ok && warp_wait(hempty0 + 8, hphase ^ 1u, abort_flag, p.status);
        if (!ok) break;
        uint8_t* to = hbuf + hs * LP_H_BYTES;
        const int pieces = min(8, (r16 - rc) / 8);  // of a row, those that the MMAs read
        for (int e = bt; e < LP_HALF * pieces; e += U * LP_BUILDERS) {
          int t[U], r[U];
          Pack<T, 8> hi[U], low[U];
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const int j = e + k * LP_BUILDERS;
            t[k] = j < LP_HALF * pieces ? j / pieces : -1;
            r[k] = rc + (j % pieces) * 8;
          }
          values(t, r, hi, low);
#pragma unroll
          for (int k = 0; k < U; ++k) {
            if (t[k] < 0) continue;
            const int c = (r[k] - rc) / 8;
            *reinterpret_cast<uint4*>(to + tile_at(t[k], c)) = hi[k].w;
            *reinterpret_cast<uint4*>(one_part ? to + tile_at(t[k], pieces + c)
                                               : to + LP_H_BYTES + tile_at(t[k], c)) = low[k].w;
          }
        }
        ready();
        if (!one_part) ready();
      }
    }
    if (!waited) pdl_wait();
  } else {
    // -------------------------------------------------------------- epilogue
    constexpr bool half = std::is_same<T, __half>::value;
    const int nl = (warp & 3) * 32 + lane;
    int ab = 0;
    uint32_t aphase = 0;
    for (int i = first; i < work.items; i += stride) {
      const Item item = work_item(work, i);
      const int u = item.unit;
      const int64_t n = (int64_t)(u % n_tiles) * LP_TILE + rank * LP_HALF + nl;
      const int64_t t0 = (int64_t)(u / n_tiles) * LP_TILE;
      Runs runs{};
      if (half && adapters && item.adapters) runs = tile_runs(p, t0, places, lane);
      if (!warp_wait(tfull0 + 8 * ab, aphase, abort_flag, p.status) || *abort_flag != 0) break;
      fence_after();
      // the builders of both CTAs have set the flag before their tiles went into the MMAs
      const bool wide = half && runs.starts != 0 && __ldcg(p.wide) != 0;
      const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(ab * LP_TILE);
      T* out = static_cast<T*>(p.out) + n;
      float* part = p.partials + item.piece * LP_PIECE + rank * (LP_TILE * LP_HALF) + nl;
#pragma unroll 1
      for (int c = 0; c < LP_TILE; c += 32) {
        uint32_t v[2][16];
        tmem_ld16(lanes + c, v[0]);
        tmem_ld16(lanes + c + 16, v[1]);
        // lane l holds the token of column c + l
        const int64_t mine = t0 + c + lane;
        const int tok = mine < places ? (adapters ? p.order[mine] : (int)mine) : -1;
        tmem_wait16(v[0]);
        tmem_wait16(v[1]);
        if constexpr (half) {
          const int a = __shfl_sync(0xFFFFFFFFu, runs.adapter, c / RUN);
          if (wide && a >= 0) add_wide<T>(p, a, tok, n, v);
        }
        if (item.piece >= 0) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            part[(c + j) * LP_HALF] = __uint_as_float(v[j >> 4][j & 15]);
          continue;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int t = __shfl_sync(0xFFFFFFFFu, tok, j);
          if (t >= 0 && n < p.N)
            out[t * p.out_stride] = from_f32<T>(__uint_as_float(v[j >> 4][j & 15]));
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

// Sums the pieces of the tiles that were cut, in their order, and stores them: a
// block eight tokens of a tile, a thread four features of two of them.
constexpr int JOIN_TOKENS = 8;

template <typename T>
__global__ void __launch_bounds__(256) lora_join_kernel(LoraParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t places = *p.places;
  const int n_tiles = (int)((p.N + LP_TILE - 1) / LP_TILE);
  const Work work(n_tiles * (int)((places + LP_TILE - 1) / LP_TILE), p.pairs,
                  (int)((p.K + 63) / 64), true);
  const int u = work.full + blockIdx.y;
  if (u >= work.units) return;
  const int f = (threadIdx.x & 63) * 4;  // feature of the tile
  const int64_t n = (int64_t)(u % n_tiles) * LP_TILE + f;
  const float* from = p.partials + (int64_t)blockIdx.y * work.parts * LP_PIECE +
                      (f / LP_HALF) * (LP_TILE * LP_HALF) + f % LP_HALF;
  for (int c = blockIdx.x * JOIN_TOKENS + (threadIdx.x >> 6); c < (blockIdx.x + 1) * JOIN_TOKENS;
       c += 4) {
    const int64_t place = (int64_t)(u / n_tiles) * LP_TILE + c;
    const int t = place < places ? p.order[place] : -1;
    if (t < 0) continue;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int q0 = 0; q0 < work.parts; q0 += 4) {
      float4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[q] = q0 + q < work.parts
                   ? __ldcg(reinterpret_cast<const float4*>(from + (q0 + q) * LP_PIECE + c * LP_HALF))
                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sum.x += v[q].x, sum.y += v[q].y, sum.z += v[q].z, sum.w += v[q].w;
    }
    const float w[4] = {sum.x, sum.y, sum.z, sum.w};
    T* out = static_cast<T*>(p.out) + t * p.out_stride + n;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) out[e] = from_f32<T>(w[e]);
  }
}

}  // namespace moe

namespace moe_host {

using moe::LoraParams;

size_t token_order_scratch(int64_t T, int64_t S);
moe_status_t launch_token_order(const int32_t* adapter_ids, int64_t T, int64_t S, int align,
                                int32_t* order, int64_t rows, int32_t* scratch, cudaStream_t s);

// Sizes of one call; the same for the workspace query and the launch.
struct LoraPlan {
  bool pair;                        // lora_pair_kernel
  int64_t places;                   // most places of the tokens' order (pair)
  int64_t order_words;              // of the workspace: order and the sort's scratch
  int64_t copy_words;               // of the workspace: x in that order
  int64_t part_words;               // of the workspace: pieces of tiles (pair)
  int64_t wide_words;               // of the workspace: which pieces of s h are wide (pair)
  int tok, tiles, shares, share_k, zs;  // shrink: tokens a block
  int nt, splits;                   // lora_split_kernel
};

// Blocks of the shrink that an SM is given: four of 64 tokens by 32 ranks (62
// registers a thread; 64 tokens of 36 adapters: 20.3 us against 22.5 with two), else two.
static int shrink_fill(int tok, int64_t R) { return tok == moe::SH_TOK && R <= 32 ? 4 : 2; }

static LoraPlan lora_plan(int64_t T, int64_t K, int64_t N, int64_t S, int64_t R) {
  LoraPlan q{};
  const int64_t sms = num_sms();
  q.pair = T > moe::SPLIT_TOKENS;
  q.places = T;
  if (q.pair && S > 0) {
    q.places = (T + (moe::RUN - 1) * (S + 1) + 127) / 128 * 128;
    q.order_words = (q.places + (int64_t)token_order_scratch(T, S) + 3) / 4 * 4;
    q.copy_words = (q.places * K / 2 + 3) / 4 * 4;
    q.part_words = sms / 2 * moe::LP_PIECE;
    q.wide_words = 4 + 4 * T;
  }
  // Shrink: 64 tokens, from 129 on 128 (they read A_a once for twice the tokens, and
  // fill the tcgen05 tile: 512 tokens 56 us against 72, 256 37 against 43), as they come
  // or in their order, and a block for each adapter that these may have (in the order a group of
  // RUN has one).  A block whose tokens have fewer ends at once, so K is dealt out, in
  // shares at least 128 wide, by the number of adapters that they have on average.
  q.tok = T > 128 ? moe::SH_LONG : moe::SH_TOK;
  q.tiles = (int)((q.places + q.tok - 1) / q.tok);
  const int64_t groups = q.pair ? q.tok / moe::RUN : (T < q.tok ? T : q.tok);
  q.zs = (int)(S < groups ? (S < 1 ? 1 : S) : groups);
  if (q.pair) q.zs = (int)groups;  // block z copies group z's rows too
  double live = q.pair ? 1.0 + (double)S * q.tok / (double)T : q.zs;
  if (live > q.zs) live = q.zs;
  int64_t shares = (int64_t)(shrink_fill(q.tok, R) * sms / (q.tiles * live));
  if (shares > (K + 127) / 128) shares = (K + 127) / 128;
  if (shares > 16) shares = 16;
  if (shares < 1) shares = 1;
  q.share_k = (int)(((K + shares - 1) / shares + 63) / 64 * 64);
  q.shares = (int)((K + q.share_k - 1) / q.share_k);
  // Split projection: the smallest tile that holds the batch, up to 128 tokens; a
  // cluster shares a tile's K while tiles leave CTA slots empty; eight CTAs for the
  // smallest tiles only where each has an SM, joining eight sums being most of their
  // work otherwise (16 tokens, 4096 x 7168: 15.1 us against 16.7).
  // (Shared memory holds the adapters' part of 128 tokens up to rank 64.)
  q.nt = T <= 16 ? 16 : (T <= 32 ? 32 : (T <= 64 || R > 64 ? 64 : 128));
  const int64_t tiles = (N + moe::LG_M - 1) / moe::LG_M * ((T + q.nt - 1) / q.nt);
  const int64_t slots = q.nt <= 64 ? 2 * sms : sms;
  const int64_t slabs = (K + 63) / 64;
  q.splits = 1;
  while (q.splits < 8 && tiles * q.splits * 2 <= (q.splits < 4 || q.nt > 16 ? slots : sms)) {
    const int64_t per = (slabs + 2 * q.splits - 1) / (2 * q.splits);
    if (per < 4 || per * (2 * q.splits - 1) >= slabs) break;  // every share has slabs
    q.splits *= 2;
  }
  return q;
}

// The sums of the shrink come last: shares * T <= 16 T, and as tiles * shares is at
// most shrink_fill blocks an SM, shares * T <= that * SMs * (tokens of a tile) unless
// shares is 1.
// Bounded so, the size grows with T: a workspace serves every shorter batch too.
static size_t lora_workspace(const LoraPlan& q, int64_t T, int64_t R) {
  int64_t rows = shrink_fill(q.tok, R) * (int64_t)num_sms() * q.tok;
  if (rows > 16 * T) rows = 16 * T;
  if (rows < T) rows = T;
  return (size_t)((q.order_words + q.copy_words + q.part_words + q.wide_words + rows * R) * 4);
}

// Dynamic shared memory limit of a kernel, raised once per device.
template <auto Kernel>
static moe_status_t allow_smem(int bytes) {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return set_error(MOE_ERR_CUDA, "no current device");
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev]) return MOE_OK;
  cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "shared memory attribute: %s", cudaGetErrorString(e));
  done[dev] = true;
  return MOE_OK;
}

template <typename... KArgs, typename... Args>
static cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, int threads, int cluster,
                                  size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int kMaxSmem = 232448;

template <auto Kernel>
static moe_status_t launch_shrink(const LoraPlan& q, const LoraParams& p, cudaStream_t s) {
  moe_status_t st = allow_smem<Kernel>(moe::sh_smem(q.tok, moe::LORA_MAX_RANK));
  if (st != MOE_OK) return st;
  const int r16 = (int)((p.R + 15) & ~15);
  return launched(launch_pdl(Kernel, dim3((unsigned)q.tiles, (unsigned)q.shares, (unsigned)q.zs),
                             dim3(moe::SH_THREADS), (size_t)moe::sh_smem(q.tok, r16), s, p),
                  "adapter");
}

template <typename T, int NT>
static moe_status_t launch_split(const LoraParams& p, const CUtensorMap& w, const CUtensorMap& x,
                                 cudaStream_t s) {
  const int smem = moe::lg_smem(NT, p.splits, (int)p.R);  // <= kMaxSmem
  moe_status_t st = allow_smem<moe::lora_split_kernel<T, NT>>(kMaxSmem);
  if (st != MOE_OK) return st;
  const dim3 grid((unsigned)((p.N + moe::LG_M - 1) / moe::LG_M * p.splits),
                  (unsigned)((p.T + NT - 1) / NT));
  return launched(launch_cluster(moe::lora_split_kernel<T, NT>, grid, moe::LG_THREADS, p.splits,
                                 smem, s, p, w, x), "projection");
}

template <typename T>
static moe_status_t launch_pair(const LoraParams& p, int64_t places, const CUtensorMap& w,
                                const CUtensorMap& x, const CUtensorMap& xs, const CUtensorMap& b,
                                cudaStream_t s) {
  static_assert(moe::LP_SMEM <= kMaxSmem, "shared memory of one CTA");
  moe_status_t st = allow_smem<moe::lora_pair_kernel<T>>(moe::LP_SMEM);
  if (st != MOE_OK) return st;
  const int64_t units = (p.N + moe::LP_TILE - 1) / moe::LP_TILE *
                        ((places + moe::LP_TILE - 1) / moe::LP_TILE);
  const int64_t pairs = num_sms() / 2;  // with adapters few tiles are cut to give all a piece
  const dim3 grid((unsigned)(2 * (units < pairs && p.partials == nullptr ? units : pairs)));
  st = launched(launch_cluster(moe::lora_pair_kernel<T>, grid, moe::LP_THREADS, 2, moe::LP_SMEM,
                               s, p, w, x, xs, b), "projection");
  if (st != MOE_OK || p.partials == nullptr) return st;
  return launched(launch_pdl(moe::lora_join_kernel<T>,
                             dim3(moe::LP_TILE / moe::JOIN_TOKENS, (unsigned)(pairs / 2)), dim3(256),
                             0, s, p), "projection join");
}

template <typename T>
static moe_status_t launch_lora(const moe_lora_args_t* a, const LoraPlan& q, LoraParams p,
                                cudaStream_t s) {
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const bool adapters = p.S > 0;
  p.wait_first = !adapters;
  CUtensorMap w, x, xs, b;
  const int64_t x_stride = p.T > 1 ? p.x_stride : p.K;
  if (!make_map16(&w, bf16, a->weight, p.N, p.K, p.K, moe::LG_M) ||
      !make_map16(&x, bf16, a->x, p.T, p.K, x_stride, q.pair ? moe::RUN : q.nt))
    return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed for the projection");
  b = xs = x;
  if (adapters) {
    if (q.pair) {
      p.xs = static_cast<int32_t*>(a->workspace) + q.order_words;
      p.partials = static_cast<float*>(a->workspace) + q.order_words + q.copy_words;
      p.pairs = num_sms() / 2;
      if (!bf16) p.wide = reinterpret_cast<uint32_t*>(p.partials + q.part_words);
      if (!make_map16(&b, bf16, a->lora_b, p.S * p.N, p.R, p.R, moe::LP_HALF) ||
          !make_map16(&xs, bf16, p.xs, q.places, p.K, p.K, moe::RUN))
        return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed for the adapters");
      int32_t* order = static_cast<int32_t*>(a->workspace);
      int32_t* scratch = order + q.places;
      moe_status_t st =
          launch_token_order(p.ids, p.T, p.S, moe::RUN, order, q.places, scratch, s);
      if (st != MOE_OK) return st;
      p.order = order;
      p.places = scratch + p.S + 1;
    }
    moe_status_t st;
    if (q.tok == moe::SH_LONG)
      st = launch_shrink<moe::lora_shrink_long_kernel<T>>(q, p, s);
    else if (p.R <= 32)
      st = launch_shrink<moe::lora_shrink_kernel<T, 1>>(q, p, s);
    else if (p.R <= 64)
      st = launch_shrink<moe::lora_shrink_kernel<T, 2>>(q, p, s);
    else
      st = launch_shrink<moe::lora_shrink_kernel<T, 4>>(q, p, s);
    if (st != MOE_OK) return st;
  }
  if (q.pair) return launch_pair<T>(p, q.places, w, x, xs, b, s);
  switch (q.nt) {
    case 16: return launch_split<T, 16>(p, w, x, s);
    case 32: return launch_split<T, 32>(p, w, x, s);
    case 64: return launch_split<T, 64>(p, w, x, s);
    default: return launch_split<T, 128>(p, w, x, s);
  }
}

}  // namespace moe_host

using namespace moe_host;

extern "C" {

size_t moe_lora_workspace_size(int64_t num_tokens, int64_t in_features, int64_t out_features,
                               int64_t num_adapters, int64_t rank) {
  if (num_tokens <= 0 || in_features <= 0 || out_features <= 0 || num_adapters <= 0 || rank <= 0)
    return 0;
  return lora_workspace(lora_plan(num_tokens, in_features, out_features, num_adapters, rank),
                        num_tokens, rank);
}

moe_status_t moe_lora_linear(const moe_lora_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t T = a->num_tokens, K = a->in_features, N = a->out_features;
  const int64_t S = a->num_adapters, R = a->rank;
  if (T < 0 || K < 0 || N < 0 || S < 0 || R < 0)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "negative size");
  if (!dtype_ok(a->dtype)) return set_error(MOE_ERR_INVALID_ARGUMENT, "bad dtype %d", a->dtype);
  if (a->dtype == MOE_DTYPE_FP32)
    return set_error(MOE_ERR_UNSUPPORTED, "the projection takes bf16 or fp16");
  if (T == 0 || N == 0) return MOE_OK;
  if (K < 1 || (S > 0 && R < 1)) return set_error(MOE_ERR_SHAPE, "in_features and rank must be >= 1");
  if (R > moe::LORA_MAX_RANK || S > moe::LORA_MAX_ADAPTERS)
    return set_error(MOE_ERR_UNSUPPORTED, "at most rank %d and %d adapters", moe::LORA_MAX_RANK,
                     moe::LORA_MAX_ADAPTERS);
  if (!a->x || !a->weight || !a->out ||
      (S > 0 && (!a->lora_a || !a->lora_b || !a->adapter_ids || !a->lora_scale)))
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if (T > 1 && (a->x_stride0 < K || a->out_stride0 < N))
    return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
  auto al = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
  if (K % 8 != 0 || (T > 1 && a->x_stride0 % 8 != 0) || !al(a->x) || !al(a->weight) ||
      (S > 0 && (R % 8 != 0 || !al(a->lora_a) || !al(a->lora_b))))
    return set_error(MOE_ERR_ALIGNMENT,
                     "rows of x, weight, lora_a and lora_b must start on 16-byte boundaries");
  if (T >= ((int64_t)1 << 22) || K >= ((int64_t)1 << 31) || N >= ((int64_t)1 << 28) ||
      S * N >= ((int64_t)1 << 31))
    return set_error(MOE_ERR_UNSUPPORTED, "problem too large for 32-bit tile coordinates");
  const LoraPlan q = lora_plan(T, K, N, S, R);
  if (S > 0) {
    const size_t need = lora_workspace(q, T, R);
    if (a->workspace == nullptr || a->workspace_bytes < need)
      return set_error(MOE_ERR_WORKSPACE, "the adapters need %zu bytes of workspace, got %zu", need,
                       a->workspace_bytes);
    if (!al(a->workspace))
      return set_error(MOE_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  }
  LoraParams p{};
  p.T = T;
  p.N = N;
  p.K = K;
  p.S = S;
  p.R = S > 0 ? R : 0;
  p.x = a->x;
  p.x_stride = a->x_stride0;
  p.a = a->lora_a;
  p.b = a->lora_b;
  p.ids = a->adapter_ids;
  p.scale = a->lora_scale;
  p.out = a->out;
  p.out_stride = a->out_stride0;
  p.h = static_cast<float*>(a->workspace) + q.order_words + q.copy_words + q.part_words +
        q.wide_words;
  p.shares = q.shares;
  p.share_k = q.share_k;
  p.splits = q.splits;
  p.status = a->device_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a->dtype == MOE_DTYPE_BF16 ? launch_lora<__nv_bfloat16>(a, q, p, s)
                                    : launch_lora<__half>(a, q, p, s);
}

}  // extern "C"
