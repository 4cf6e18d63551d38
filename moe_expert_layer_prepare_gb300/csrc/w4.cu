// Products with 4-bit weights and group scales, for few rows:
//   y[r, n] = sum over groups j of s[n, j] sum_{k in j} (q[n, k] - z[n, j]) x[r, k],
// of one matrix, or of the matrix of each row's expert; with an activation the first half
// of the rows n is a gate and y = act(gate) up.
//
// The codes are the bytes that count, each read once for up to 8 NT rows, so HBM is the
// bound and the work around a code has to stay under some three instructions.  Codes
// become 16-bit numbers without rounding (an integer by its bits behind a power of two
// that holds all sixteen, then minus that power and the zero point; e2m1 by its bits as
// sign, exponent and mantissa of a number 2^126 or 2^14 times too small), the products of
// a group are summed by mma.sync tiles in fp32, and the scale multiplies the group's sum.
//
// A unit is 16 rows of a matrix (gated: 8 gate rows and their 8 up rows, so that both
// values of an output meet in one thread's reach) by all of K for up to 8 NT rows of x.
// Its K blocks of 256 codes are dealt out to the eight warps of a block, each with a ring
// of cp.async stages of its own that runs ahead across units; the warps' sums are joined
// in their order.  The k of a tile may come in any order that both operands share: lane c
// of four takes the codes 8 c .. 8 c + 7 of 32, one word, and the same of x.
#include <mutex>
#include <type_traits>

#include "activation.cuh"
#include "block_common.cuh"

namespace moe {
namespace w4 {

constexpr int WARPS = 8, THREADS = WARPS * 32;
constexpr int ROWS = 16;           // of a unit
constexpr int BLOCK_K = 256;       // codes of a row in a stage: 128 bytes
constexpr int STAGE = ROWS * 128;  // bytes
constexpr int STAGES = 5;
constexpr int MAX_ROUTES = 1024, MAX_EXPERTS = 1024;

struct Params {
  int64_t T, K, N;  // N: rows of a matrix
  int64_t n_out;    // columns of out
  int E, top_k, routes;
  const void* x;
  int64_t x_stride;
  const uint8_t* w;
  const void* scales;
  const uint8_t* zeros;  // nullable
  const void* ids;       // nullable: one matrix for all rows
  int ids64;
  int act;
  bool wide_scales;  // a block's scales of a row may be read at once
  void* out;
  int64_t out_stride;
  uint32_t* status;
};

struct Chunk {  // rows of x that share a matrix
  int16_t expert, first, count;
};

template <typename T, bool E2M1>
struct Codes;
// Pair i of a word: codes i and i + 4 as two 16-bit numbers, the lower first.
template <typename T>
struct Codes<T, false> {
  static constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  static constexpr uint32_t BASE = BF16 ? 0x43004300u : 0x64006400u;  // 128 or 1024 in both halves
  // what the numbers have too much: the base and the zero point
  static __device__ __forceinline__ uint32_t offset(uint32_t zero) { return BASE + zero * 0x10001u; }
  static __device__ __forceinline__ uint32_t pair(uint32_t w, int i, uint32_t off) {
    const uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | BASE;
    if constexpr (BF16) {
      const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                       *reinterpret_cast<const __nv_bfloat162*>(&off));
      return *reinterpret_cast<const uint32_t*>(&d);
    } else {
      const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v),
                                *reinterpret_cast<const __half2*>(&off));
      return *reinterpret_cast<const uint32_t*>(&d);
    }
  }
};
template <typename T>
struct Codes<T, true> {
  static constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  static constexpr int UP = BF16 ? 6 : 9;  // place of the mantissa's bit
  static __device__ __forceinline__ uint32_t offset(uint32_t) { return 0; }
  static __device__ __forceinline__ uint32_t pair(uint32_t w, int i, uint32_t) {
    const int up = UP - 4 * i;
    const uint32_t v = ((up >= 0 ? w << (up & 31) : w >> (-up & 31)) & (0x00070007u << UP)) |
                       ((w << (12 - 4 * i)) & 0x80008000u);
    if constexpr (BF16) {
      const uint32_t f = 0x7E807E80u;  // 2^126
      const __nv_bfloat162 d = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                       *reinterpret_cast<const __nv_bfloat162*>(&f));
      return *reinterpret_cast<const uint32_t*>(&d);
    } else {
      const uint32_t f = 0x74007400u;  // 2^14
      const __half2 d =
          __hmul2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&f));
      return *reinterpret_cast<const uint32_t*>(&d);
    }
  }
};

// 16 rows by 16 of k times 16 of k by 8 columns, added to d.
template <typename T>
__device__ __forceinline__ void mma_tile(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The scales of a K block of two rows (a lane's): 8 / SPG a row, of T or as exponents.
template <typename T, bool E2M1, int SPG>
struct Scales {
  static constexpr int COUNT = 8 / SPG;
  static constexpr int BYTES = COUNT * (E2M1 ? 1 : 2);
  static constexpr int WORDS = (BYTES + 3) / 4;
  uint32_t s[2][WORDS], z[2][2];

  __device__ __forceinline__ float scale(int row, int j) const {
    if constexpr (E2M1) {
      const uint32_t e = (s[row][j / 4] >> (8 * (j % 4))) & 0xFFu;
      // 2^-127 is subnormal; the largest byte is not a number
      return e == 0 ? __uint_as_float(0x00400000u)
                    : __uint_as_float(e == 255u ? 0x7FC00000u : e << 23);
    } else {
      const float2 v = unpack2<T>(s[row][j / 2]);
      return j % 2 == 0 ? v.x : v.y;
    }
  }
  __device__ __forceinline__ uint32_t zero(int row, int j) const {
    return (z[row][j / 4] >> (8 * (j % 4))) & 15u;
  }

  // of block kb of the rows at `at` (in groups; < 0: no such row)
  __device__ __forceinline__ void load(const Params& p, const int64_t (&at)[2], int kb) {
    const int groups = (int)(p.K / (32 * SPG)), g0 = kb * COUNT;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int i = 0; i < WORDS; ++i) s[r][i] = 0;
      z[r][0] = z[r][1] = 0x08080808u;
      if (at[r] < 0) continue;
      const uint8_t* src = static_cast<const uint8_t*>(p.scales) + (at[r] + g0) * (E2M1 ? 1 : 2);
      const uint8_t* zsrc = p.zeros + (at[r] + g0);
      if (p.wide_scales) {
        if constexpr (BYTES == 16) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
          s[r][0] = v.x, s[r][1] = v.y, s[r][2] = v.z, s[r][3] = v.w;
        } else if constexpr (BYTES == 8) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
          s[r][0] = v.x, s[r][1] = v.y;
        } else {
          s[r][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
        }
        if (!E2M1 && p.zeros != nullptr) {
          if constexpr (COUNT == 8) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(zsrc));
            z[r][0] = v.x, z[r][1] = v.y;
          } else if constexpr (COUNT == 4) {
            z[r][0] = __ldg(reinterpret_cast<const uint32_t*>(zsrc));
          } else {
            z[r][0] = __ldg(reinterpret_cast<const uint16_t*>(zsrc));
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < COUNT; ++j) {
          if (g0 + j >= groups) break;
          if constexpr (E2M1)
            s[r][j / 4] |= (uint32_t)__ldg(src + j) << (8 * (j % 4));
          else
            s[r][j / 2] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(src) + j) << (16 * (j % 2));
          if (!E2M1 && p.zeros != nullptr)
            z[r][j / 4] = (z[r][j / 4] & ~(0xFFu << (8 * (j % 4)))) |
                          (uint32_t)__ldg(zsrc + j) << (8 * (j % 4));
        }
      }
    }
  }
};

// Routes by expert: s_route in the order of the experts, chunks of at most `most`.  Routes
// without an expert get zeros in out.  All threads of the block call it.
template <typename T>
__device__ __forceinline__ int sort_routes(const Params& p, int most, int* s_count, int* s_first,
                                           uint16_t* s_route, Chunk* s_chunk, int* s_part) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto id_of = [&](int r) {
    return p.ids64 ? static_cast<const int64_t*>(p.ids)[r]
                   : (int64_t) static_cast<const int32_t*>(p.ids)[r];
  };
  for (int e = tid; e < p.E; e += THREADS) s_count[e] = 0;
  __syncthreads();
  for (int r = tid; r < p.routes; r += THREADS) {
    const int64_t e = id_of(r);
    if (e >= 0 && e < p.E)
      atomicAdd(s_count + e, 1);
    else if (e >= p.E)
      set_status(p.status, MOE_DEV_BAD_EXPERT);
  }
  for (int r = blockIdx.x; r < p.routes; r += gridDim.x) {
    const int64_t e = id_of(r);
    if (e >= 0 && e < p.E) continue;
    T* out = static_cast<T*>(p.out) + r * p.out_stride;
    for (int64_t n = tid; n < p.n_out; n += THREADS) out[n] = from_f32<T>(0.0f);
  }
  __syncthreads();
  // routes and chunks before each expert: four experts a thread, packed into one sum
  constexpr int PER = MAX_EXPERTS / THREADS;
  int mine[PER], total = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i, n = e < p.E ? s_count[e] : 0;
    mine[i] = n | ((n + most - 1) / most) << 16;
    total += mine[i];
  }
  int before = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) s_part[warp] = before;
  __syncthreads();
  int chunks = 0;
  before -= total;
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += s_part[w];
    chunks += s_part[w] >> 16;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    if (e < p.E) {
      const int n = mine[i] & 0xFFFF, first = before & 0xFFFF;
      s_first[e] = first;
      for (int c = 0; c * most < n; ++c)
        s_chunk[(before >> 16) + c] = Chunk{(int16_t)e, (int16_t)(first + c * most),
                                            (int16_t)min(most, n - c * most)};
    }
    before += mine[i];
  }
  __syncthreads();
  // in the order of the routes, the same in every block: an expert's chunks are in several
  if (warp == 0) {
    for (int r0 = 0; r0 < p.routes; r0 += 32) {
      const int r = r0 + lane;
      const int64_t id = r < p.routes ? id_of(r) : -1;
      const int e = id >= 0 && id < p.E ? (int)id : -1;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
      const int at = e >= 0 ? s_first[e] : 0;
      __syncwarp();
      if (e >= 0) {
        s_route[at + __popc(same & lanemask_lt())] = (uint16_t)r;
        if (lane == __ffs(same) - 1) s_first[e] = at + __popc(same);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  return chunks;
}

__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

constexpr int red_bytes(int nt) { return 2 * WARPS * ROWS * 8 * nt * 4; }
constexpr int smem_bytes(int nt, bool experts) {
  return WARPS * STAGES * STAGE + red_bytes(nt) +
         (experts ? 2 * MAX_EXPERTS * 4 + MAX_ROUTES * (2 + 6) + 64 : 0);
}

template <typename T, bool E2M1, int SPG, int NT, bool EXPERTS>
__global__ void __launch_bounds__(THREADS, 2) w4_kernel(Params p) {
  using C = Codes<T, E2M1>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  float* red = reinterpret_cast<float*>(smem + WARPS * STAGES * STAGE);
  pdl_wait();
  pdl_launch_dependents();

  constexpr int COLS = 8 * NT;
  Chunk* s_chunk = nullptr;
  uint16_t* s_route = nullptr;
  int chunks = (int)((p.T + COLS - 1) / COLS);
  if constexpr (EXPERTS) {
    int* s_count = reinterpret_cast<int*>(smem + WARPS * STAGES * STAGE + red_bytes(NT));
    int* s_first = s_count + MAX_EXPERTS;
    int* s_part = s_first + MAX_EXPERTS;
    s_route = reinterpret_cast<uint16_t*>(s_part + 16);
    s_chunk = reinterpret_cast<Chunk*>(s_route + MAX_ROUTES);
    chunks = sort_routes<T>(p, COLS, s_count, s_first, s_route, s_chunk, s_part);
  }
  const bool gated = p.act != MOE_ACT_NONE;
  const int tile_out = gated ? ROWS / 2 : ROWS;
  const int tiles = (int)((p.n_out + tile_out - 1) / tile_out);
  const int64_t units = (int64_t)chunks * tiles;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  if (u0 == u1) return;
  const int blocks = (int)((p.K + BLOCK_K - 1) / BLOCK_K);
  const int64_t pitch = p.K / 2;  // bytes of a row

  // Row r of unit u as a row of all matrices, -1 where there is none.
  auto row_of = [&](int64_t u, int r) -> int64_t {
    const int chunk = (int)(u / tiles);
    const int64_t n0 = (u - (int64_t)chunk * tiles) * tile_out;
    const int64_t base = EXPERTS ? (int64_t)s_chunk[chunk].expert * p.N : 0;
    if (!gated) return n0 + r < p.N ? base + n0 + r : -1;
    if (n0 + (r & 7) >= p.n_out) return -1;
    return base + n0 + (r & 7) + (r >= 8 ? p.n_out : 0);
  };

  // This warp's blocks: every WARPS-th of the sequence (unit, block) of the CTA's units.
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * STAGES * STAGE;
  struct Place {
    int64_t u;
    int kb;
  };
  auto next = [&](Place& q) {
    q.kb += WARPS;
    while (q.kb >= blocks) q.kb -= blocks, ++q.u;
  };
  Place ahead{u0, warp};
  while (ahead.kb >= blocks) ahead.kb -= blocks, ++ahead.u;
  Place at = ahead;
  auto fetch = [&](int stage) {
    if (ahead.u < u1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 4 + (lane >> 3), j = lane & 7;
        const int64_t row = row_of(ahead.u, r);
        const int64_t byte = (int64_t)ahead.kb * 128 + j * 16;
        const bool there = row >= 0 && byte < pitch;
        copy16_or_zero(ring + stage * STAGE + r * 128 + ((j ^ (r & 7)) << 4),
                       there ? p.w + row * pitch + byte : p.w, there);
      }
      next(ahead);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(s);

  const int groups = (int)(p.K / (32 * SPG));
  auto scale_rows = [&](const Place& q, int64_t (&rows)[2]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t row = q.u < u1 ? row_of(q.u, g + 8 * r) : -1;
      rows[r] = row < 0 ? -1 : row * groups;
    }
  };
  Scales<T, E2M1, SPG> sc;
  {
    int64_t rows[2];
    scale_rows(at, rows);
    sc.load(p, rows, at.kb);
  }

  int stage = 0, buf = 0;
  for (int64_t u = u0; u < u1; ++u, buf ^= 1) {
    const int chunk = (int)(u / tiles);
    int first = chunk * COLS, count = (int)min((int64_t)COLS, p.T - first);
    if constexpr (EXPERTS) first = s_chunk[chunk].first, count = s_chunk[chunk].count;
    const T* xr[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int col = t * 8 + g;
      xr[t] = nullptr;
      if (col < count) {
        int row = first + col;
        if constexpr (EXPERTS) row = s_route[row] / p.top_k;
        xr[t] = static_cast<const T*>(p.x) + row * p.x_stride + c * 8;
      }
    }
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = 0.0f;

    while (at.u == u) {
      const int kb = at.kb;
      next(at);
      Scales<T, E2M1, SPG> sc_next;
      {
        int64_t rows[2];
        scale_rows(at, rows);
        sc_next.load(p, rows, at.kb);
      }
      fetch((stage + STAGES - 1) % STAGES);
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
      __syncwarp();
      const uint32_t base = ring + stage * STAGE;
      const int steps = min(8, (int)((p.K - (int64_t)kb * BLOCK_K) / 32));
      float part[NT][4];
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        if (s >= steps) break;
        const int j = s / SPG;
        if (s % SPG == 0) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[t][e] = 0.0f;
        }
        // words of rows g and g + 8
        uint32_t w0, w1;
        {
          const int r = lane & 15;
          const uint32_t addr = base + r * 128 + ((s ^ (r & 7)) << 4);
          asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];"
                       : "=r"(w0), "=r"(w1)
                       : "r"(addr)
                       : "memory");
        }
        const uint32_t o0 = C::offset(sc.zero(0, j)), o1 = C::offset(sc.zero(1, j));
        const uint32_t a0[4] = {C::pair(w0, 0, o0), C::pair(w1, 0, o1), C::pair(w0, 1, o0),
                                C::pair(w1, 1, o1)};
        const uint32_t a1[4] = {C::pair(w0, 2, o0), C::pair(w1, 2, o1), C::pair(w0, 3, o0),
                                C::pair(w1, 3, o1)};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (xr[t] != nullptr)
            v = __ldg(reinterpret_cast<const uint4*>(xr[t] + kb * BLOCK_K + s * 32));
          mma_tile<T>(part[t], a0, __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632));
          mma_tile<T>(part[t], a1, __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        }
        if (s % SPG == SPG - 1) {
          const float s0 = sc.scale(0, j), s1 = sc.scale(1, j);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            acc[t][0] = fmaf(s0, part[t][0], acc[t][0]);
            acc[t][1] = fmaf(s0, part[t][1], acc[t][1]);
            acc[t][2] = fmaf(s1, part[t][2], acc[t][2]);
            acc[t][3] = fmaf(s1, part[t][3], acc[t][3]);
          }
        }
      }
      sc = sc_next;
      __syncwarp();  // the stage is free
      if (++stage == STAGES) stage = 0;
    }

    // sums of the warps, [warp][column][row]
    float* mine = red + (buf * WARPS + warp) * (ROWS * COLS);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int col = t * 8 + 2 * c;
      mine[col * ROWS + g] = acc[t][0];
      mine[(col + 1) * ROWS + g] = acc[t][1];
      mine[col * ROWS + g + 8] = acc[t][2];
      mine[(col + 1) * ROWS + g + 8] = acc[t][3];
    }
    __syncthreads();
    const float* all = red + buf * WARPS * (ROWS * COLS);
    const int64_t n0 = (u - (int64_t)chunk * tiles) * tile_out;
    for (int i = tid; i < tile_out * count; i += THREADS) {
      const int col = i / tile_out, r = i % tile_out;
      float v = 0.0f, up = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        v += all[(w * COLS + col) * ROWS + r];
        if (gated) up += all[(w * COLS + col) * ROWS + r + 8];
      }
      if (gated) v = act_value(p.act, v) * up;
      int row = first + col;
      if constexpr (EXPERTS) row = s_route[row];
      if (n0 + r < p.n_out)
        (static_cast<T*>(p.out) + row * p.out_stride)[n0 + r] = from_f32<T>(v);
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

}  // namespace w4
}  // namespace moe

namespace moe_host {

namespace w4 = moe::w4;

template <typename T, bool E2M1, int SPG, int NT, bool EXPERTS>
static moe_status_t launch_w4(const w4::Params& p, cudaStream_t s) {
  constexpr auto kernel = w4::w4_kernel<T, E2M1, SPG, NT, EXPERTS>;
  constexpr int smem = w4::smem_bytes(NT, EXPERTS);
  static std::mutex mu;
  static int resident[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return set_error(MOE_ERR_CUDA, "no current device");
  {
    std::lock_guard<std::mutex> lock(mu);
    if (resident[dev] == 0) {
      int n = 0;
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, w4::THREADS, smem);
      if (e != cudaSuccess || n < 1)
        return set_error(MOE_ERR_CUDA, "4-bit products: %s", cudaGetErrorString(e));
      resident[dev] = n;
    }
  }
  const int tile = p.act == MOE_ACT_NONE ? w4::ROWS : w4::ROWS / 2;
  const int64_t tiles = (p.n_out + tile - 1) / tile;
  const int64_t cap = (int64_t)num_sms() * resident[dev];
  // with experts at most a chunk a route
  int64_t units = tiles * (EXPERTS ? p.routes : (p.T + 8 * NT - 1) / (8 * NT));
  const unsigned grid = (unsigned)(units < cap ? units : cap);
  return launched(launch_pdl(kernel, dim3(grid), dim3(w4::THREADS), (size_t)smem, s, p),
                  "4-bit products");
}

template <typename T, bool E2M1, int SPG>
static moe_status_t run_w4(const w4::Params& p, cudaStream_t s) {
  if (p.ids != nullptr) {
    // most experts of a short batch have one or two of its routes
    if (p.routes <= 8 * p.E) return launch_w4<T, E2M1, SPG, 1, true>(p, s);
    return launch_w4<T, E2M1, SPG, 2, true>(p, s);
  }
  if (p.T <= 8) return launch_w4<T, E2M1, SPG, 1, false>(p, s);
  return launch_w4<T, E2M1, SPG, 2, false>(p, s);
}

template <typename T>
static moe_status_t run_w4_format(const w4::Params& p, int format, int64_t group, cudaStream_t s) {
  if (format == MOE_W4_E2M1) return run_w4<T, true, 1>(p, s);
  if (group == 32) return run_w4<T, false, 1>(p, s);
  if (group == 64) return run_w4<T, false, 2>(p, s);
  return run_w4<T, false, 4>(p, s);
}

}  // namespace moe_host

using namespace moe_host;

extern "C" {

moe_status_t moe_w4_linear(const moe_w4_linear_args_t* a, void* stream) {
  clear_error();
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARGUMENT, "args is NULL");
  const int64_t T = a->num_tokens, K = a->in_features, N = a->matrix_rows;
  const int64_t E = a->num_experts, G = a->group_size;
  if (T < 0 || K < 0 || N < 0 || E < 0 || a->top_k < 0)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "negative size");
  if (!dtype_ok(a->dtype)) return set_error(MOE_ERR_INVALID_ARGUMENT, "bad dtype %d", a->dtype);
  if (a->format != MOE_W4_INT4 && a->format != MOE_W4_E2M1)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "bad format %d", a->format);
  if (a->activation < MOE_ACT_SILU || a->activation > MOE_ACT_NONE)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "bad activation %d", a->activation);
  if (a->dtype == MOE_DTYPE_FP32)
    return set_error(MOE_ERR_UNSUPPORTED, "4-bit products take bf16 or fp16");
  if (G != 32 && ((G != 64 && G != 128) || a->format == MOE_W4_E2M1))
    return set_error(MOE_ERR_UNSUPPORTED, "groups of 32, 64 or 128 integers, or of 32 e2m1 values");
  if (a->format == MOE_W4_E2M1 && a->zeros != nullptr)
    return set_error(MOE_ERR_UNSUPPORTED, "e2m1 values have no zero points");
  const bool experts = a->topk_ids != nullptr;
  if (experts && a->topk_ids_dtype != MOE_IDS_INT32 && a->topk_ids_dtype != MOE_IDS_INT64)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "bad topk_ids_dtype %d", a->topk_ids_dtype);
  const bool gated = a->activation != MOE_ACT_NONE;
  if (gated && N % 2 != 0) return set_error(MOE_ERR_SHAPE, "as many gate rows as up rows are needed");
  const int64_t rows = experts ? T * a->top_k : T, n_out = gated ? N / 2 : N;
  if (rows == 0 || N == 0) return MOE_OK;
  if (K < 1 || K % G != 0)
    return set_error(MOE_ERR_SHAPE, "in_features must be a positive multiple of group_size");
  if (experts && E < 1) return set_error(MOE_ERR_SHAPE, "topk_ids without experts");
  if (experts && (rows > w4::MAX_ROUTES || E > w4::MAX_EXPERTS))
    return set_error(MOE_ERR_UNSUPPORTED, "at most %d routes to %d experts", w4::MAX_ROUTES,
                     w4::MAX_EXPERTS);
  if (!experts && T > w4::MAX_ROUTES)
    return set_error(MOE_ERR_UNSUPPORTED, "at most %d rows", w4::MAX_ROUTES);
  if (K >= ((int64_t)1 << 28) || N >= ((int64_t)1 << 28))
    return set_error(MOE_ERR_UNSUPPORTED, "matrix too large");
  if (!a->x || !a->weight || !a->scales || !a->out)
    return set_error(MOE_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if ((T > 1 && a->x_stride0 < K) || (rows > 1 && a->out_stride0 < n_out))
    return set_error(MOE_ERR_SHAPE, "row stride smaller than the row");
  if (!rows_aligned16(a->x, a->x_stride0, 2, T) || !rows_aligned16(a->weight, 0, 1, 1))
    return set_error(MOE_ERR_ALIGNMENT, "rows of x and weight must start on 16-byte boundaries");
  w4::Params p{};
  p.T = T;
  p.K = K;
  p.N = N;
  p.n_out = n_out;
  p.E = experts ? (int)E : 0;
  p.top_k = (int)a->top_k;
  p.routes = (int)rows;
  p.x = a->x;
  p.x_stride = a->x_stride0;
  p.w = static_cast<const uint8_t*>(a->weight);
  p.scales = a->scales;
  p.zeros = static_cast<const uint8_t*>(a->zeros);
  p.ids = a->topk_ids;
  p.ids64 = a->topk_ids_dtype == MOE_IDS_INT64;
  p.act = a->activation;
  p.wide_scales = K % w4::BLOCK_K == 0 && rows_aligned16(a->scales, 0, 1, 1) &&
                  (a->zeros == nullptr || (reinterpret_cast<uintptr_t>(a->zeros) & 7u) == 0);
  p.out = a->out;
  p.out_stride = a->out_stride0;
  p.status = a->device_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a->dtype == MOE_DTYPE_BF16 ? run_w4_format<__nv_bfloat16>(p, a->format, G, s)
                                    : run_w4_format<__half>(p, a->format, G, s);
}

}  // extern "C"
