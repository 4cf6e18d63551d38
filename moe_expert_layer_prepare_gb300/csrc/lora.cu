// A projection shared by all tokens plus each token's own low-rank adapter:
//   out = x W^T + s_a (x A_a^T) B_a^T.
//
// Two launches.  The first, lora_shrink_kernel, gives h = x A_a^T as fp32 sums
// per share of K.  It reads A and the rows of x, a few flops a byte, so it
// runs on mma.sync tiles fed by cp.async; blocks take (64 tokens, share of K,
// share of the adapters among these tokens).
//
// The second, lora_gemm_kernel, is the projection on tcgen05, features by
// tokens: the accumulator's 128 rows are features (the MMA's A operand is a
// weight tile) and its columns a tile of tokens, so that a single token costs a
// 16-column tile and a decode batch streams W once.  K slabs of 64 come by TMA
// through a ring of shared-memory stages.  After them the adapters of the tile's
// tokens enter the same accumulator, one K step of the MMA per 16 ranks: B_a's
// rows by TMA as the A operand, and as the B operand a tile of s_a h with zeros
// in the rows of tokens that have another adapter, which the warps that later
// run the epilogue write during the main loop.  h is in fp32; as the MMA takes 16-bit operands
// s_a h enters as its rounding and the rounded remainder, which keeps the
// adapters' part as exact as the rest.
//
// With few tiles (decode) the K slabs are dealt out to the CTAs of a cluster and
// their sums joined through distributed shared memory in rank order.  The second
// launch starts while the first still runs and waits for it only where h is read.
#include <mutex>

#include "block_common.cuh"
#include "tc_common.cuh"

namespace moe {

using namespace tc;

constexpr int LORA_MAX_RANK = 128;
constexpr int LORA_MAX_ADAPTERS = 4096;

struct LoraParams {
  int64_t T, N, K, S, R;
  const void* x;
  int64_t x_stride;
  const void* a;
  const int32_t* ids;
  const float* scale;
  void* out;
  int64_t out_stride;
  float* h;        // [shares][T][R]
  int shares;      // of K in the shrink
  int share_k;     // K of one share, a multiple of 64
  int splits;      // cluster size of the projection
  int wait_first;  // no shrink was launched: wait for the stream's predecessor at once
  uint32_t* status;
};

__device__ __forceinline__ int adapter_of(const LoraParams& p, int64_t t, bool* bad) {
  const int a = t < p.T ? p.ids[t] : -1;
  if (a >= p.S) *bad = true;
  return a >= 0 && a < p.S ? a : -1;
}

// Distinct values >= 0 of id[0, n) in order of first appearance: list and its
// length.  All `threads` threads call it, n <= threads or strided; sync() is
// their barrier.
template <typename Sync>
__device__ __forceinline__ int distinct_adapters(const int16_t* id, int16_t* first, int16_t* list,
                                                 int n, int tid, int threads, Sync sync) {
  for (int i = tid; i < n; i += threads) {
    bool is = id[i] >= 0;
    for (int j = 0; j < i && is; ++j) is = id[j] != id[i];
    first[i] = is;
  }
  sync();
  int count = 0;
  for (int i = tid; i < n; i += threads) {
    int rank = 0;
    for (int j = 0; j < i; ++j) rank += first[j];
    if (first[i]) list[rank] = id[i];
  }
  for (int j = 0; j < n; ++j) count += first[j];
  sync();
  return count;
}

// ------------------------------------------------------------------ shrink
constexpr int SH_TOK = 64;
constexpr int SH_THREADS = 256;
constexpr int SH_STAGES = 4;
constexpr int SH_X_BYTES = SH_TOK * 128;

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

// Byte offset of 16-byte piece `piece` of row `row` in a tile of 128-byte rows,
// permuted so that eight rows' same pieces lie in different banks.
__device__ __forceinline__ uint32_t tile_at(int row, int piece) {
  return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4));
}

template <typename T>
__global__ void __launch_bounds__(SH_THREADS) lora_shrink_kernel(LoraParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int16_t s_id[SH_TOK], s_first[SH_TOK], s_list[SH_TOK];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t0 = (int64_t)blockIdx.x * SH_TOK;
  bool bad = false;
  if (tid < SH_TOK) s_id[tid] = (int16_t)adapter_of(p, t0 + tid, &bad);
  if (bad) set_status(p.status, MOE_DEV_BAD_ADAPTER);
  __syncthreads();
  const int n_list = distinct_adapters(s_id, s_first, s_list, SH_TOK, tid, SH_THREADS,
                                       [] { __syncthreads(); });
  const int64_t k0 = (int64_t)blockIdx.y * p.share_k;
  const int64_t k1 = min(p.K, k0 + p.share_k);
  const int slabs = k1 > k0 ? (int)((k1 - k0 + 63) / 64) : 0;
  const int R = (int)p.R, r16 = (R + 15) & ~15;
  const uint32_t base = smem_u32(smem);
  const uint32_t stage_bytes = SH_X_BYTES + r16 * 128;
  const T* x = static_cast<const T*>(p.x);
  const int m0 = (warp & 3) * 16, nh = warp >> 2;

  for (int d = blockIdx.z; d < n_list; d += gridDim.z) {
    const int a = s_list[d];
    const T* A = static_cast<const T*>(p.a) + (int64_t)a * R * p.K;
    auto load = [&](int slab) {
      const uint32_t s = base + (slab % SH_STAGES) * stage_bytes;
      const int64_t k = k0 + (int64_t)slab * 64;
      for (int i = tid; i < SH_TOK * 8; i += SH_THREADS) {
        const int r = i >> 3, c = i & 7;
        const bool take = s_id[r] == a && k + c * 8 < k1;
        cp_async16(s + tile_at(r, c), take ? x + (t0 + r) * p.x_stride + k + c * 8 : x, take);
      }
      for (int i = tid; i < r16 * 8; i += SH_THREADS) {
        const int r = i >> 3, c = i & 7;
        const bool take = r < R && k + c * 8 < k1;
        cp_async16(s + SH_X_BYTES + tile_at(r, c), take ? A + (int64_t)r * p.K + k + c * 8 : A,
                   take);
      }
    };
    float acc[4][2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.0f;
    for (int s = 0; s < SH_STAGES - 1; ++s) {
      if (s < slabs) load(s);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    for (int s = 0; s < slabs; ++s) {
      asm volatile("cp.async.wait_group %0;" ::"n"(SH_STAGES - 2) : "memory");
      __syncthreads();
      if (s + SH_STAGES - 1 < slabs) load(s + SH_STAGES - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      const uint32_t xs = base + (s % SH_STAGES) * stage_bytes, as = xs + SH_X_BYTES;
#pragma unroll
      for (int k16 = 0; k16 < 4; ++k16) {
        uint32_t av[4];
        ldmatrix4(av, xs + tile_at(m0 + (lane & 15), k16 * 2 + (lane >> 4)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n0 = (i * 2 + nh) * 16;
          if (n0 >= r16) break;
          uint32_t bv[4];
          ldmatrix4(bv, as + tile_at(n0 + (lane & 7) + ((lane >> 4) << 3),
                                     k16 * 2 + ((lane >> 3) & 1)));
          mma_16816<T>(acc[i][0], av, bv[0], bv[1]);
          mma_16816<T>(acc[i][1], av, bv[2], bv[3]);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the stages are free for the next adapter
    float* h = p.h + (int64_t)blockIdx.y * p.T * R;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = m0 + (lane >> 2) + half * 8;
      if (s_id[r] != a) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int n = (i * 2 + nh) * 16 + j * 8 + (lane & 3) * 2;
          if (n < R)
            *reinterpret_cast<float2*>(h + (t0 + r) * R + n) =
                make_float2(acc[i][j][half * 2], acc[i][j][half * 2 + 1]);
        }
    }
  }
}

// -------------------------------------------------------------- projection
constexpr int LG_M = 128;  // features of a tile
constexpr int LG_A_BYTES = LG_M * 128;
constexpr int LG_THREADS = 256;
constexpr int LG_BUILDERS = 192;  // warps 2..7 write the tiles of s h
constexpr int LG_MAX_STAGES = 6;

// Stages of the ring and buffers of s h for a tile of NT tokens: two CTAs
// share an SM up to NT = 64, one has it from NT = 128 on.
constexpr int lg_stages(int nt) { return nt <= 32 ? 5 : (nt <= 64 ? 4 : (nt <= 128 ? 5 : 4)); }
constexpr int lg_hbufs(int nt) { return nt <= 32 || nt == 128 ? 2 : 1; }
constexpr int lg_smem(int nt) {
  return 1024 + lg_stages(nt) * (LG_A_BYTES + nt * 128) + lg_hbufs(nt) * nt * 128 + 256 + nt * 6;
}

template <typename T, int NT>
__global__ void __launch_bounds__(LG_THREADS)
    lora_gemm_kernel(const __grid_constant__ LoraParams p, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ CUtensorMap tmB) {
  constexpr int STAGES = lg_stages(NT), HB = lg_hbufs(NT);
  constexpr int H_BYTES = NT * 128, STAGE_BYTES = LG_A_BYTES + NT * 128;
  constexpr uint32_t IDESC = f16_idesc(std::is_same<T, __nv_bfloat16>::value, LG_M, NT);
  constexpr uint32_t TMEM_COLS = NT < 32 ? 32 : NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* hbuf = smem + STAGES * STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(hbuf + HB * H_BYTES);
  // full[STAGES], empty[STAGES], hfull[HB], hempty[HB], list, done
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * LG_MAX_STAGES + 6);
  int* s_abort = reinterpret_cast<int*>(tmem_holder + 1);
  int* s_count = s_abort + 1;
  int16_t* s_id = reinterpret_cast<int16_t*>(reinterpret_cast<uint8_t*>(bars) + 256);
  int16_t* s_first = s_id + NT;
  int16_t* s_list = s_first + NT;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = s_abort;
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + LG_MAX_STAGES);
  const uint32_t hfull0 = smem_u32(bars + 2 * LG_MAX_STAGES);
  const uint32_t hempty0 = smem_u32(bars + 2 * LG_MAX_STAGES + 2);
  const uint32_t list_bar = smem_u32(bars + 2 * LG_MAX_STAGES + 4);
  const uint32_t done_bar = smem_u32(bars + 2 * LG_MAX_STAGES + 5);

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int s = 0; s < HB; ++s) {
      mbar_init(hfull0 + 8 * s, LG_BUILDERS);
      mbar_init(hempty0 + 8 * s, 1);
    }
    mbar_init(list_bar, LG_BUILDERS);
    mbar_init(done_bar, 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    prefetch_map(&tmW);
    prefetch_map(&tmX);
    prefetch_map(&tmB);
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
  const int r16 = (int)((p.R + 15) & ~15);
  const int rchunks = (r16 + 63) / 64;
  const bool one_part = 2 * r16 <= 64;  // rounding and remainder fit one tile
  const bool adapters = p.S > 0;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_phase = 0;
    auto next = [&](auto&& issue) {
      if (!warp_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.status)) return false;
      if (elect_one()) issue(full0 + 8 * stage, smem_u32(smem + stage * STAGE_BYTES));
      __syncwarp();
      issued |= 1u << stage;
      issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
      if (++stage == STAGES) stage = 0, phase ^= 1u;
      return true;
    };
    bool ok = true;
    for (int kb = kb0; kb < kb1 && ok; ++kb)
#ifdef MOE_TEST_WITHHOLD_STAGE
      // Failure-detection test builds only: CTA 0 issues neither its second
      // slab nor anything after it, and the MMA warp's wait runs out.
      if (blockIdx.x == 0 && blockIdx.y == 0 && kb > kb0) {
        ok = false;
      } else
#endif
      ok = next([&](uint32_t bar, uint32_t s) {
        mbar_expect_tx(bar, STAGE_BYTES);
        tma_load_2d(s, &tmW, kb * 64, (int)n0, bar);
        tma_load_2d(s + LG_A_BYTES, &tmX, kb * 64, (int)t0, bar);
      });
    if (adapters && ok) ok = warp_wait(list_bar, 0, abort_flag, p.status);
    if (adapters && ok) {
      const int n = *s_count * rchunks;
      for (int q = rank; q < n && ok; q += p.splits)
        ok = next([&](uint32_t bar, uint32_t s) {
          mbar_expect_tx(bar, LG_A_BYTES);
          tma_load_2d(s, &tmB, (q % rchunks) * 64, (int)(s_list[q / rchunks] * p.N + n0), bar);
        });
    }
    for (int s = 0; s < STAGES; ++s)  // every copy has landed before exit
      if (issued & (1u << s)) {
        volatile int never = 0;
        mbar_wait(full0 + 8 * s, (issued_phase >> s) & 1u, &never, p.status);
      }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    int stage = 0, slot = 0;
    uint32_t phase = 0, hphase = 0, accumulate = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = warp_wait(full0 + 8 * stage, phase, abort_flag, p.status);
      if (!ok) break;
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
    if (adapters && ok) ok = warp_wait(list_bar, 0, abort_flag, p.status);
    if (adapters && ok) {
      const int n = *s_count * rchunks;
      for (int q = rank; q < n && ok; q += p.splits) {
        ok = warp_wait(full0 + 8 * stage, phase, abort_flag, p.status);
        const uint64_t ad = sw128_desc(smem_u32(smem + stage * STAGE_BYTES));
        const int steps = min(4, r16 / 16 - (q % rchunks) * 4);
        for (int part = 0; part < (one_part ? 1 : 2) && ok; ++part) {
          ok = warp_wait(hfull0 + 8 * slot, hphase, abort_flag, p.status);
          if (!ok) break;
          fence_after();
          const uint64_t bd = sw128_desc(smem_u32(hbuf + slot * H_BYTES));
          if (elect_one()) {
            for (int k = 0; k < steps; ++k) {
              mma_f16(tmem, ad + 2 * k, bd + 2 * k, IDESC, accumulate | (k > 0));
              if (one_part) mma_f16(tmem, ad + 2 * k, bd + 2 * (steps + k), IDESC, 1);
            }
            mma_commit(hempty0 + 8 * slot);
          }
          __syncwarp();
          accumulate = 1;
          if (++slot == HB) slot = 0, hphase ^= 1u;
        }
        if (ok && elect_one()) mma_commit(empty0 + 8 * stage);
        __syncwarp();
        if (++stage == STAGES) stage = 0, phase ^= 1u;
      }
    }
    if (accumulate) {  // all MMAs complete before the sums are read or TMEM is freed
      if (elect_one()) mma_commit(done_bar);
      __syncwarp();
      volatile int never = 0;
      mbar_wait(done_bar, 0, &never, p.status);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------- tiles of s h, epilogue
    const int bt = tid - 64;
    auto builders_sync = [] { asm volatile("bar.sync 1, 192;" ::: "memory"); };
    if (adapters) {
      bool bad = false;
      for (int i = bt; i < NT; i += LG_BUILDERS) s_id[i] = (int16_t)adapter_of(p, t0 + i, &bad);
      builders_sync();
      const int count =
          distinct_adapters(s_id, s_first, s_list, NT, bt, LG_BUILDERS, builders_sync);
      if (bt == 0) *s_count = count;
      mbar_arrive(list_bar);
      if (!p.wait_first) pdl_wait();
      int slot = 0;
      uint32_t hphase = 0;
      bool ok = true;
      const int R = (int)p.R, n = count * rchunks;
      for (int q = rank; q < n && ok; q += p.splits) {
        const int a = s_list[q / rchunks], rc = (q % rchunks) * 64;
        const float scale = __ldg(p.scale + a);
        for (int part = 0; part < (one_part ? 1 : 2) && ok; ++part) {
          ok = warp_wait(hempty0 + 8 * slot, hphase ^ 1u, abort_flag, p.status);
          if (!ok) break;
          uint8_t* dst = hbuf + slot * H_BYTES;
          for (int i = bt; i < NT * 8; i += LG_BUILDERS) {
            const int t = i >> 3, c = i & 7;
            // columns of the tile: the rounding, then (one_part) the remainder
            const bool low = one_part ? c * 8 >= r16 : part == 1;
            const int r = rc + (one_part && low ? c * 8 - r16 : c * 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (s_id[t] == a && r < R) {
              float hv[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) hv[e] = 0.0f;
              const float* src = p.h + (t0 + t) * R + r;
              for (int s = 0; s < p.shares; ++s, src += p.T * R) {
                const float4 u0 = __ldcg(reinterpret_cast<const float4*>(src));
                const float4 u1 = __ldcg(reinterpret_cast<const float4*>(src) + 1);
                hv[0] += u0.x, hv[1] += u0.y, hv[2] += u0.z, hv[3] += u0.w;
                hv[4] += u1.x, hv[5] += u1.y, hv[6] += u1.z, hv[7] += u1.w;
              }
              T o[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float sh = scale * hv[e];
                o[e] = from_f32<T>(sh);
                if (low) o[e] = from_f32<T>(sh - to_f32(o[e]));
              }
              memcpy(&v, o, 16);
            }
            *reinterpret_cast<uint4*>(dst + tile_at(t, c)) = v;
          }
          fence_async_smem();
          mbar_arrive(hfull0 + 8 * slot);
          if (++slot == HB) slot = 0, hphase ^= 1u;
        }
      }
    } else if (!p.wait_first) {
      pdl_wait();
    }
    // done is also signalled after a wait ran out; the sums are then not whole
    if (warp >= 4 && warp_wait(done_bar, 0, abort_flag, p.status) && *abort_flag == 0) {
      fence_after();
      const int nl = (warp & 3) * 32 + lane;
      const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      T* out = static_cast<T*>(p.out) + n0 + nl;
      float* red = reinterpret_cast<float*>(smem);  // the ring is no longer in use
#pragma unroll 1
      for (int c = 0; c < NT; c += 16) {
        uint32_t v[16];
        tmem_ld16(lanes + c, v);
        tmem_wait16(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (p.splits > 1)
            red[(c + j) * LG_M + nl] = __uint_as_float(v[j]);
          else if (t0 + c + j < p.T && n0 + nl < p.N)
            out[(t0 + c + j) * p.out_stride] = from_f32<T>(__uint_as_float(v[j]));
        }
      }
      fence_before();
    }
  }
  __syncwarp();
  if (p.splits > 1) {
    // each CTA joins its share of the tile's tokens, partial sums in rank order
    cluster_sync();
    const int share = NT / p.splits;
    const uint32_t red0 = smem_u32(smem);
    if (*abort_flag == 0) {
      for (int i = tid; i < share * LG_M; i += LG_THREADS) {
        const int c = rank * share + i / LG_M, nl = i % LG_M;
        if (t0 + c >= p.T || n0 + nl >= p.N) continue;
        float sum = 0.0f;
        for (int r = 0; r < p.splits; ++r) sum += ld_cluster(red0 + (c * LG_M + nl) * 4, r);
        static_cast<T*>(p.out)[(t0 + c) * p.out_stride + n0 + nl] = from_f32<T>(sum);
      }
    }
    cluster_sync();  // no CTA leaves while its sums are read
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS)
                 : "memory");
  }
}

}  // namespace moe

namespace moe_host {

using moe::LoraParams;

struct LoraPlan {
  int tiles, shares, share_k, zs;  // shrink
  int nt, splits;                  // projection
};

static LoraPlan lora_plan(int64_t T, int64_t K, int64_t N, int64_t S) {
  LoraPlan q{};
  const int64_t sms = num_sms();
  // Shrink: shares of K until about two blocks an SM, at least 256 wide.
  q.tiles = (int)((T + moe::SH_TOK - 1) / moe::SH_TOK);
  int64_t z = S < moe::SH_TOK ? S : moe::SH_TOK;
  if (T < z) z = T;
  if (z < 1) z = 1;
  const int64_t most = q.tiles >= sms ? 1 : (2 * sms + q.tiles - 1) / q.tiles;
  q.zs = (int)(z < most ? z : most);
  if (q.tiles >= 32) q.zs = 1;  // long batches: a tile's tokens share few adapters
  int64_t shares = (2 * sms) / ((int64_t)q.tiles * q.zs);
  if (shares > (K + 255) / 256) shares = (K + 255) / 256;
  if (shares > 16) shares = 16;
  if (shares < 1) shares = 1;
  q.share_k = (int)(((K + shares - 1) / shares + 63) / 64 * 64);
  q.shares = (int)((K + q.share_k - 1) / q.share_k);
  // Projection: the smallest tile that holds the batch, up to 256 tokens; a
  // cluster shares a tile's K while tiles leave CTA slots empty.
  q.nt = T <= 16 ? 16 : (T <= 32 ? 32 : (T <= 64 ? 64 : (T <= 128 ? 128 : 256)));
  const int64_t tiles = (N + moe::LG_M - 1) / moe::LG_M * ((T + q.nt - 1) / q.nt);
  const int64_t slots = q.nt <= 64 ? 2 * sms : sms;
  const int64_t slabs = (K + 63) / 64;
  q.splits = 1;
  while (q.splits < 8 && tiles * q.splits * 2 <= slots) {
    const int64_t per = (slabs + 2 * q.splits - 1) / (2 * q.splits);
    if (per < 4 || per * (2 * q.splits - 1) >= slabs) break;  // every share has slabs
    q.splits *= 2;
  }
  return q;
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

template <typename T, int NT>
static moe_status_t launch_gemm(const LoraParams& p, const CUtensorMap& w, const CUtensorMap& x,
                                const CUtensorMap& b, cudaStream_t s) {
  auto kernel = moe::lora_gemm_kernel<T, NT>;
  constexpr int smem = moe::lg_smem(NT);
  static_assert(smem <= 232448, "shared memory of one CTA");
  moe_status_t st = allow_smem<moe::lora_gemm_kernel<T, NT>>(smem);
  if (st != MOE_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.N + moe::LG_M - 1) / moe::LG_M * p.splits),
                     (unsigned)((p.T + NT - 1) / NT));
  cfg.blockDim = dim3(moe::LG_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return launched(cudaLaunchKernelEx(&cfg, kernel, p, w, x, b), "projection");
}

template <typename T>
static moe_status_t launch_lora(const moe_lora_args_t* a, const LoraPlan& q, LoraParams p,
                                cudaStream_t s) {
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const bool adapters = p.S > 0;
  p.wait_first = !adapters;
  CUtensorMap w, x, b;
  const int64_t x_stride = p.T > 1 ? p.x_stride : p.K;
  if (!make_map16(&w, bf16, a->weight, p.N, p.K, p.K, moe::LG_M) ||
      !make_map16(&x, bf16, a->x, p.T, p.K, x_stride, q.nt))
    return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed for the projection");
  b = w;
  if (adapters) {
    if (!make_map16(&b, bf16, a->lora_b, p.S * p.N, p.R, p.R, moe::LG_M))
      return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed for lora_b");
    auto kernel = moe::lora_shrink_kernel<T>;
    const int r16 = (int)((p.R + 15) & ~15);
    const size_t smem = (size_t)moe::SH_STAGES * (moe::SH_X_BYTES + r16 * 128);
    moe_status_t st = allow_smem<moe::lora_shrink_kernel<T>>(
        moe::SH_STAGES * (moe::SH_X_BYTES + moe::LORA_MAX_RANK * 128));
    if (st != MOE_OK) return st;
    st = launched(
        launch_pdl(kernel, dim3((unsigned)q.tiles, (unsigned)q.shares, (unsigned)q.zs),
                   dim3(moe::SH_THREADS), smem, s, p), "adapter");
    if (st != MOE_OK) return st;
  }
  switch (q.nt) {
    case 16: return launch_gemm<T, 16>(p, w, x, b, s);
    case 32: return launch_gemm<T, 32>(p, w, x, b, s);
    case 64: return launch_gemm<T, 64>(p, w, x, b, s);
    case 128: return launch_gemm<T, 128>(p, w, x, b, s);
    default: return launch_gemm<T, 256>(p, w, x, b, s);
  }
}

}  // namespace moe_host

using namespace moe_host;

extern "C" {

size_t moe_lora_workspace_size(int64_t num_tokens, int64_t in_features, int64_t out_features,
                               int64_t num_adapters, int64_t rank) {
  if (num_tokens <= 0 || in_features <= 0 || out_features <= 0 || num_adapters <= 0 || rank <= 0)
    return 0;
  const LoraPlan q = lora_plan(num_tokens, in_features, out_features, num_adapters);
  return (size_t)q.shares * num_tokens * rank * 4;
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
  const LoraPlan q = lora_plan(T, K, N, S);
  if (S > 0) {
    const size_t need = (size_t)q.shares * T * R * 4;
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
  p.ids = a->adapter_ids;
  p.scale = a->lora_scale;
  p.out = a->out;
  p.out_stride = a->out_stride0;
  p.h = static_cast<float*>(a->workspace);
  p.shares = q.shares;
  p.share_k = q.share_k;
  p.splits = q.splits;
  p.status = a->device_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a->dtype == MOE_DTYPE_BF16 ? launch_lora<__nv_bfloat16>(a, q, p, s)
                                    : launch_lora<__half>(a, q, p, s);
}

}  // extern "C"
