// Products with 4-bit weights and group scales, for few rows:
//   y[r, n] = sum over groups j of s[n, j] sum_{k in j} (q[n, k] - z[n, j]) x[r, k],
// of one matrix, or of the matrix of each row's expert; with an activation the first half
// of the rows n is a gate and y = act(gate) up.
//
// The codes are the bytes that count, each read once for as many rows as there is room for,
// 8 NT at most (16 at K = 4096, 9 at 7168, 5 at 14336), so HBM is the bound as long as a
// code costs few instructions: an SM does 64 integer operations a clock and HBM gives it 46
// codes. Codes become fp16 numbers without rounding: an integer by a mask alone, its bits
// being those of a subnormal number, q 2^-24 or q 2^-20, and the zero point taken off it;
// e2m1 by the conversion instruction. So x is brought to fp16 too, each row times a power of
// two that puts its largest value in [2^14, 2^15): a bf16 value keeps all its bits down to
// 2^-31 of that, an fp16 value to 2^-28, and what is smaller is off by half a step of 2^-24
// at most, 2^-39 of the largest, far below the error of the fp32 sums. The products of a
// group are summed by mma.sync tiles in fp32; its scale times the row's power multiplies the
// group's sum.
//
// A unit is 16 rows of a matrix (gated: 8 gate rows and their 8 up rows, so that one lane
// has both values of an output) by all of K for up to 8 NT rows of x, which a CTA keeps
// in shared memory in the order of the codes.  The K blocks of the CTA's units
// are one sequence, cut into a run for each warp, all equal to a block; a warp stores the
// units that are all its own, and those cut between warps are joined in the warps' order.
// So no warp waits for another on the way, each with a ring of cp.async stages of its own.
// The k of a tile may come in any order that both operands share: lane c of four takes the
// codes 8 c .. 8 c + 7 of 32, one word, and the same of x.
//
// Measured: one token 7168 -> 4096, integers of groups of 128, 7.0 us (15 MB: launch, x and
// the join are 5 of them); through the gate and up rows, 7168 -> 2 x 2048, of eight e2m1
// experts 27 us (123 MB, 4.6 TB/s, bound by issue slots); 128 routes 2048 -> 7168 135 us (818
// MB, 6.1 TB/s); 16 tokens 4096 -> 2 x 14336 with zero points 28 us (64 MB: the second eight
// columns take 6 of them, the zero points 5).
#include <mutex>
#include <type_traits>

#include "activation.cuh"
#include "block_common.cuh"
#include "tc_common.cuh"

namespace moe {
namespace w4 {

constexpr int ROWS = 16;   // of a unit, an MMA tile
constexpr int WARPS = 16;  // they fill the register file
// A warp's block: 512 codes of the 16 rows, in a stage two parts of 16 rows by 128 bytes; or
// 256, one part, where the rows of x take the room.  A part's scales and zero points (16 and
// 8 bytes a row) stand behind the codes.  64 or 32 KB are on their way to an SM.
constexpr int PART = ROWS * 128;
constexpr int STAGES = 2;
constexpr int block_k(int parts) { return 256 * parts; }
constexpr int scales_at(int parts) { return parts * PART; }
constexpr int zeros_at(int parts) { return scales_at(parts) + parts * ROWS * 16; }
constexpr int stage_bytes(int parts) { return zeros_at(parts) + parts * ROWS * 8; }
constexpr int MAX_ROUTES = 1024, MAX_EXPERTS = 1024, MAX_K = 32768;

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
  int most, room;    // rows of a chunk, and in shared memory
  int tiles;         // units of a chunk
  int blocks;        // K blocks of a unit, and 2^32 / blocks rounded up
  uint32_t blocks_inverse;
  int scale_unit, zero_unit;  // see copy_groups
  void* out;
  int64_t out_stride;
  uint32_t* status;
};

struct Chunk {  // rows of x that share a matrix
  int16_t expert, first, count;
};

enum Format { INT4 = 0, INT4_ZEROS = 1, E2M1 = 2 };

// The eight codes of a word as fp16 numbers in pairs.
template <Format F>
struct Codes {
  // Pair i: codes i and i + 4 less their zero point, times 2^-20.  Those of even i come out of the
  // mask 2^-4 as large, which the instruction that takes the zero point off makes up for.
  static __device__ __forceinline__ void pairs(uint32_t w, uint32_t minus, uint32_t (&d)[4]) {
    const uint32_t v[4] = {w & 0x000F000Fu, w & 0x00F000F0u, (w >> 8) & 0x000F000Fu,
                           (w >> 8) & 0x00F000F0u};
    const __half2 o = *reinterpret_cast<const __half2*>(&minus);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 c = *reinterpret_cast<const __half2*>(&v[i]);
      const __half2 n = i % 2 == 0 ? __hfma2(c, __float2half2_rn(16.0f), o) : __hadd2(c, o);
      d[i] = *reinterpret_cast<const uint32_t*>(&n);
    }
  }
  static constexpr int UNIT = 20;  // the codes are 2^-20 as large as they should be
  // x's eight values in the same order
  static __device__ __forceinline__ uint4 order(float2 a, float2 b, float2 c, float2 d, float up) {
    return make_uint4(pack2<__half>(make_float2(a.x * up, c.x * up)), pack2<__half>(make_float2(a.y * up, c.y * up)),
                      pack2<__half>(make_float2(b.x * up, d.x * up)), pack2<__half>(make_float2(b.y * up, d.y * up)));
  }
};
// e2m1: neighbouring codes a pair.
template <>
struct Codes<E2M1> {
  static __device__ __forceinline__ void pairs(uint32_t w, uint32_t, uint32_t (&d)[4]) {
    asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4;"
        " cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b;"
        " cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d; }"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(w));
  }
  static constexpr int UNIT = 0;
  static __device__ __forceinline__ uint4 order(float2 a, float2 b, float2 c, float2 d, float up) {
    return make_uint4(pack2<__half>(make_float2(a.x * up, a.y * up)), pack2<__half>(make_float2(b.x * up, b.y * up)),
                      pack2<__half>(make_float2(c.x * up, c.y * up)), pack2<__half>(make_float2(d.x * up, d.y * up)));
  }
};

// 16 rows by 16 of k times 16 of k by 8 columns, added to d, or the first of a sum.
__device__ __forceinline__ void mma_tile(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, bool first) {
  if (first)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The scales of 256 codes of a row, 8 / SPG of T or exponents, and its zero points.
template <typename T, Format F, int SPG>
struct Scales {
  static constexpr int COUNT = 8 / SPG;
  static constexpr int ITEM = F == E2M1 ? 1 : 2;
  static constexpr int BYTES = COUNT * ITEM;
  uint32_t s[BYTES / 4], z[2];

  // from where a row's stand in a stage
  __device__ __forceinline__ void read(const uint8_t* at, const uint8_t* zat) {
    if constexpr (BYTES == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(at);
      s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
    } else if constexpr (BYTES == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(at);
      s[0] = v.x, s[1] = v.y;
    } else {
      s[0] = *reinterpret_cast<const uint32_t*>(at);
    }
    if constexpr (F == INT4_ZEROS) {
      if constexpr (COUNT == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(zat);
        z[0] = (v.x & 0x0F0F0F0Fu) << 4, z[1] = (v.y & 0x0F0F0F0Fu) << 4;
      } else if constexpr (COUNT == 4) {
        z[0] = (*reinterpret_cast<const uint32_t*>(zat) & 0x0F0F0F0Fu) << 4;
      } else {
        z[0] = (*reinterpret_cast<const uint16_t*>(zat) & 0x0F0Fu) << 4;
      }
    }
  }
  // scales 2 i and 2 i + 1
  __device__ __forceinline__ float2 scales(int i) const {
    if constexpr (F == E2M1) {
      uint32_t d;  // exponents are bf16 numbers too, 2^-127 a subnormal one and 255 none
      if (i % 2 == 0)
        asm("{ .reg .b16 a, b; mov.b32 {a, b}, %1; cvt.rn.bf16x2.ue8m0x2 %0, a; }" : "=r"(d) : "r"(s[i / 2]));
      else
        asm("{ .reg .b16 a, b; mov.b32 {a, b}, %1; cvt.rn.bf16x2.ue8m0x2 %0, b; }" : "=r"(d) : "r"(s[i / 2]));
      return unpack2<__nv_bfloat16>(d);
    }
    return unpack2<T>(s[i]);
  }
  // What a pair of codes of group j has too much, negative: the zero point times 2^-20, a
  // subnormal number like the codes.  (Positive and subtracted: 16 tokens with zero points 1%
  // faster, one token 8% slower, 4096 -> 28672 in groups of 64: the registers.)
  __device__ __forceinline__ uint32_t minus(int j) const {
    if constexpr (F != INT4_ZEROS) return 0x80808080u;
    return __byte_perm(z[j / 4], 0x80u, (j % 4) * 0x0101 + 0x4040);
  }
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// Copies BYTES of a row's scales or zero points, of which `left` exist, with zeros behind the
// last: every group needs a number.  Rows start on multiples of `unit` bytes: 16 (or all of
// BYTES), 4, or less.
template <int BYTES, int ITEM>
__device__ __forceinline__ void copy_groups(uint8_t* dst, const uint8_t* src, int left, int unit) {
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
  if (unit == 16 && left >= BYTES) {
    if constexpr (BYTES == 32) {
      copy_async<16>(to, src);
      copy_async<16>(to + 16, src + 16);
    } else {
      copy_async<BYTES>(to, src);
    }
  } else if (unit >= 4) {
#pragma unroll
    for (int j = 0; j < BYTES; j += 4) {
      if (j < left)
        copy_async<4>(to + j, src + j);
      else
        *reinterpret_cast<uint32_t*>(dst + j) = 0;
    }
  } else {
    for (int j = 0; j < BYTES; j += ITEM) {
      if constexpr (ITEM == 2)
        *reinterpret_cast<uint16_t*>(dst + j) = j < left ? __ldg(reinterpret_cast<const uint16_t*>(src + j)) : 0;
      else
        dst[j] = j < left ? __ldg(src + j) : 0;
    }
  }
}

// Routes by expert: s_route in the order of the experts, chunks of at most `most`.  Routes
// without an expert get zeros in out.  All threads of the block call it.
template <typename T>
__device__ __forceinline__ int sort_routes(const Params& p, int most, int* s_count, int* s_first,
                                           uint16_t* s_route, Chunk* s_chunk, int* s_part) {
  constexpr int THREADS = WARPS * 32;
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
  // routes and chunks before each expert, packed into one sum
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

// The same for at most 32 routes, a lane each of one warp; chunks in the order of their
// first routes.
template <typename T>
__device__ __forceinline__ int sort_few_routes(const Params& p, int most, uint16_t* s_route,
                                               Chunk* s_chunk, int* s_part) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) {
    const int64_t id = lane >= p.routes ? -1
                       : p.ids64        ? static_cast<const int64_t*>(p.ids)[lane]
                                        : (int64_t) static_cast<const int32_t*>(p.ids)[lane];
    const int e = id >= 0 && id < p.E ? (int)id : -1;
    if (id >= p.E) set_status(p.status, MOE_DEV_BAD_EXPERT);
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    const int rank = __popc(same & lanemask_lt()), count = __popc(same);
    const uint32_t leaders = __ballot_sync(0xFFFFFFFFu, e >= 0 && rank % most == 0);
    // experts in the order of their first routes: behind all routes and chunks of those before
    int first = 0, chunk = rank / most;
    for (uint32_t m = __ballot_sync(0xFFFFFFFFu, e >= 0 && rank == 0); m != 0; m &= m - 1) {
      const int l = __ffs(m) - 1, n = __shfl_sync(0xFFFFFFFFu, count, l);
      if (l < __ffs(same) - 1) first += n, chunk += (n + most - 1) / most;
    }
    if (e >= 0) s_route[first + rank] = (uint16_t)lane;
    if (e >= 0 && rank % most == 0)
      s_chunk[chunk] = Chunk{(int16_t)e, (int16_t)(first + rank), (int16_t)min(most, count - rank)};
    const uint32_t without = __ballot_sync(0xFFFFFFFFu, lane < p.routes && e < 0);
    if (lane == 0) s_part[0] = __popc(leaders), s_part[1] = (int)without;
  }
  __syncthreads();
  for (uint32_t m = (uint32_t)s_part[1]; m != 0; m &= m - 1) {
    const int r = __ffs(m) - 1;
    if ((unsigned)r % gridDim.x != blockIdx.x) continue;
    T* out = static_cast<T*>(p.out) + r * p.out_stride;
    for (int64_t n = tid; n < p.n_out; n += WARPS * 32) out[n] = from_f32<T>(0.0f);
  }
  return s_part[0];
}

// Bytes of a row of x in shared memory: zeros up to a whole block, and 64 bytes so that two
// rows' neighbouring 64 bytes lie in different banks.
__host__ __device__ constexpr int64_t x_pitch(int64_t K) {
  return (K + 511) / 512 * 1024 + 64;
}

constexpr int ring_bytes(int parts) { return WARPS * STAGES * stage_bytes(parts); }
constexpr int red_bytes(int nt) { return WARPS * 32 * 16 * nt; }
// s_part, then of each route its place and perhaps a chunk, then two words an expert
__host__ __device__ constexpr int route_bytes(int routes) {
  return routes == 0 ? 0 : 64 + (routes + 1) / 2 * 16 + (routes <= 32 ? 0 : 2 * MAX_EXPERTS * 4);
}
constexpr int MAX_ROOM = 16;  // rows of x in shared memory
constexpr int fixed_bytes(int nt, int parts, int routes) {  // beside x
  return ring_bytes(parts) + red_bytes(nt) + route_bytes(routes) + 2 * MAX_ROOM * 4 + WARPS * 4;
}

template <typename T, Format F, int SPG, int NT, int PARTS, bool EXPERTS>
__global__ void __launch_bounds__(WARPS * 32, 1) w4_kernel(Params p) {
  using C = Codes<F>;
  using S = Scales<T, F, SPG>;
  constexpr int BLOCK_K = block_k(PARTS), STAGE = stage_bytes(PARTS);
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int routes = EXPERTS ? p.routes : 0;
  float4* red = reinterpret_cast<float4*>(smem + ring_bytes(PARTS));
  uint8_t* routing = reinterpret_cast<uint8_t*>(red) + red_bytes(NT);
  float* s_power = reinterpret_cast<float*>(routing + route_bytes(routes));  // [MAX_ROOM]
  float* s_rest = s_power + MAX_ROOM;                                         // [MAX_ROOM]
  uint32_t* s_amax = reinterpret_cast<uint32_t*>(s_rest + MAX_ROOM);         // [WARPS]
  uint8_t* s_x = reinterpret_cast<uint8_t*>(s_amax + WARPS);
  pdl_wait();
  pdl_launch_dependents();

  Chunk* s_chunk = nullptr;
  uint16_t* s_route = nullptr;
  int chunks = (int)((p.T + p.most - 1) / p.most);
  if constexpr (EXPERTS) {
    int* s_part = reinterpret_cast<int*>(routing);
    s_route = reinterpret_cast<uint16_t*>(s_part + 16);
    s_chunk = reinterpret_cast<Chunk*>(s_route + (routes + 1) / 2 * 2);
    if (routes <= 32) {
      chunks = sort_few_routes<T>(p, p.most, s_route, s_chunk, s_part);
    } else {
      int* s_count = reinterpret_cast<int*>(routing + route_bytes(routes)) - 2 * MAX_EXPERTS;
      chunks = sort_routes<T>(p, p.most, s_count, s_count + MAX_EXPERTS, s_route, s_chunk, s_part);
    }
  }
  const bool gated = p.act != MOE_ACT_NONE;
  const int tile_out = gated ? ROWS / 2 : ROWS;  // outputs of a unit
  const int tiles = p.tiles, units = chunks * tiles, blocks = p.blocks;
  const int pitch = (int)(p.K / 2);  // bytes of a row
  const int xp = (int)x_pitch(p.K);
  const int even = units / (int)gridDim.x, odd = units % (int)gridDim.x, cta = (int)blockIdx.x;
  const int u0 = even * cta + min(cta, odd), u1 = u0 + even + (cta < odd);
  if (u0 == u1) return;

  // The CTA's units lie in one or a few chunks.  As many chunks as there is room for the
  // rows of are a batch: their blocks are dealt out to the warps in runs.
  const int chunk1 = (u1 - 1) / tiles;
  auto chunk_rows = [&](int chunk, int& first, int& count) {
    first = chunk * p.most, count = (int)min((int64_t)p.most, p.T - first);
    if constexpr (EXPERTS) first = s_chunk[chunk].first, count = s_chunk[chunk].count;
  };
  struct Batch {
    int chunk0, chunk1, u0, u1;  // chunks and units, those behind the last
  };
  auto batch_from = [&](int chunk) {
    Batch q{chunk, chunk, max(u0, chunk * tiles), 0};
    for (int rows = 0; q.chunk1 <= chunk1; ++q.chunk1) {
      int first, count;
      chunk_rows(q.chunk1, first, count);
      rows += count;
      if (rows > p.room) break;
    }
    q.u1 = min(u1, q.chunk1 * tiles);
    return q;
  };
  struct Run {
    int chunk, tile, kb, left;  // next block, blocks left of the run
    int after;                  // first chunk of the next batch
  };
  // Begin of warp w's run in a batch, in its blocks.
  auto run_begin = [&](const Batch& q, int w) { return (uint32_t)((q.u1 - q.u0) * blocks) * w / WARPS; };
  auto run_of = [&](const Batch& q) {
    const uint32_t begin = run_begin(q, warp), end = run_begin(q, warp + 1);
    // begin / blocks, exact as begin * blocks is below 2^32: blocks are at most 2^7, and a batch
    // has 2^16 tiles a row of x at most and as many rows as shared memory holds (3 of 2^7 blocks)
    const int unit = blocks == 1 ? (int)begin : (int)__umulhi(begin, p.blocks_inverse);
    Run r{q.chunk0, q.u0 - q.chunk0 * tiles + unit, (int)begin - unit * blocks, (int)(end - begin), q.chunk1};
    while (r.tile >= tiles) r.tile -= tiles, ++r.chunk;
    return r;
  };
  auto settle = [&](Run& q) {  // on to a batch in which this warp has a block
    while (q.left == 0 && q.after <= chunk1) q = run_of(batch_from(q.after));
  };
  // One block on; whether its rows are others (or there is none).
  auto step = [&](Run& q) {
    ++q.kb;
    if (--q.left == 0) {
      settle(q);
      return true;
    }
    if (q.kb < blocks) return false;
    q.kb = 0;
    if (++q.tile == tiles) q.tile = 0, ++q.chunk;
    return true;
  };
  // Row r of a unit as a row of all matrices; past the last one the last, whose results are
  // computed again and not stored.
  auto row_of = [&](const Run& q, int r) -> int64_t {
    const int64_t base = EXPERTS ? (int64_t)s_chunk[q.chunk].expert * p.N : 0;
    const int64_t n = (int64_t)q.tile * tile_out + (gated ? r & 7 : r);
    return base + min(n, p.n_out - 1) + (gated && r >= 8 ? p.n_out : 0);
  };

  // Rows of a batch in the order of its chunks: with experts they are neighbours in s_route.
  auto batch_rows = [&](const Batch& q, int& first, int& count) {
    int f, n;
    chunk_rows(q.chunk0, first, n);
    chunk_rows(q.chunk1 - 1, f, n);
    count = f + n - first;
  };
  auto row_of_x = [&](int row) {
    if constexpr (EXPERTS) row = s_route[row] / p.top_k;
    return static_cast<const T*>(p.x) + row * p.x_stride;
  };
  // A batch's rows of x come as they are, each with the warps that there are for one, and
  // are brought to fp16 in place, each piece by the thread that copied it.
  const int pieces = blocks * (BLOCK_K / 8), real = (int)(p.K / 8);
  auto warps_a_row = [&](int count) {
    int per = WARPS;
    while (per > 1 && per * count > WARPS) per >>= 1;
    return per;
  };
  auto copy_x = [&](const Batch& q) {
    int first, count;
    batch_rows(q, first, count);
    const int per = warps_a_row(count), lane0 = (warp % per) * 32 + lane;
    for (int col = warp / per; col < count; col += WARPS / per) {
      const T* src = row_of_x(first + col);
      uint4* dst = reinterpret_cast<uint4*>(s_x + col * xp);
      for (int i = lane0; i < pieces; i += per * 32) {
        if (i < real)
          copy_async<16>((uint32_t)__cvta_generic_to_shared(dst + i), src + i * 8);
        else
          dst[i] = make_uint4(0, 0, 0, 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  Batch batch = batch_from(u0 / tiles);
  copy_x(batch);  // before the weights, behind which it would queue

  // Weights and scales one block ahead.
  uint8_t* const ring_at = smem + warp * STAGES * STAGE;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(ring_at);
  const int groups = (int)(p.K / (32 * SPG));
  Run ahead = run_of(batch);
  settle(ahead);
  const uint8_t* from[4];  // this lane's 16 bytes of four rows
  int64_t groups_at = 0;   // this lane's row of scales (lanes 0 to 15) or zero points, in groups
  auto aim = [&] {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      from[i] = p.w + row_of(ahead, i * 4 + (lane >> 3)) * pitch + (lane & 7) * 16;
    groups_at = row_of(ahead, lane & 15) * groups;
  };
  const uint32_t to = ring + (lane >> 3) * 128;
  uint32_t at_piece[2];  // rows r and r + 4 differ in the permutation
#pragma unroll
  for (int i = 0; i < 2; ++i) at_piece[i] = to + (((lane & 7) ^ (((lane >> 3) + 4 * i) & 7)) << 4);
  // Of two zero points a block a word is copied, of a pair of blocks.
  constexpr bool ZERO_PAIRS = PARTS == 1 && S::COUNT == 2;
  auto fetch = [&](int stage) {
    if (ahead.left > 0) {
      const int byte = ahead.kb * (BLOCK_K / 2), group = ahead.kb * (PARTS * S::COUNT);
#pragma unroll
      for (int h = 0; h < PARTS; ++h)
        if (byte + h * 128 + (lane & 7) * 16 < pitch) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            copy_async<16>(at_piece[i & 1] + stage * STAGE + h * PART + i * 512, from[i] + byte + h * 128);
        }
      uint8_t* to_groups = ring_at + stage * STAGE;
      if (lane < 16) {
        copy_groups<PARTS * S::BYTES, S::ITEM>(to_groups + scales_at(PARTS) + lane * (PARTS * 16),
                                               static_cast<const uint8_t*>(p.scales) + (groups_at + group) * S::ITEM,
                                               (groups - group) * S::ITEM, p.scale_unit);
      } else if constexpr (F == INT4_ZEROS) {
        const int first = ZERO_PAIRS ? group & ~3 : group;
        copy_groups<ZERO_PAIRS ? 4 : PARTS * S::COUNT, 1>(to_groups + zeros_at(PARTS) + (lane - 16) * (PARTS * 8),
                                                          p.zeros + (groups_at + first), groups - first, p.zero_unit);
      }
      if (step(ahead) && ahead.left > 0) aim();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // all but the newest group of copies are there
  auto arrived = [&] { asm volatile("cp.async.wait_group 1;" ::: "memory"); };
  if (ahead.left > 0) aim();
  fetch(0);

  // a lane's row of two 32-code pieces for ldmatrix
  const uint32_t lane_row = (lane & 15) * 128, lane_piece = ((lane >> 4) ^ (lane & 7)) << 4;
  int stage = 0;
  for (bool again = false;; again = true) {
    if (again) {
      if (batch.chunk1 > chunk1) break;
      batch = batch_from(batch.chunk1);
      __syncthreads();  // the last batch's rows are no longer read
      copy_x(batch);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
      arrived();
    }
    int batch_first, rows;
    batch_rows(batch, batch_first, rows);
    const int per = warps_a_row(rows), lane0 = (warp % per) * 32 + lane;
    for (int col0 = 0; col0 < rows; col0 += WARPS / per) {
      const int col = col0 + warp / per;
      uint4* row = reinterpret_cast<uint4*>(s_x + col * xp);
      // the row's largest value, by its bits; where it is not a finite one, the largest that is
      constexpr uint32_t INF = std::is_same<T, __nv_bfloat16>::value ? 0x7F80u : 0x7C00u;
      uint32_t two = 0;
      if (col < rows) {
#pragma unroll 4
        for (int i = lane0; i < pieces; i += per * 32) {
          const uint4 v = row[i];
          two = __vmaxu2(__vmaxu2(two, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu)),
                         __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
        }
      }
      uint32_t most = __reduce_max_sync(0xFFFFFFFFu, max(two & 0xFFFFu, two >> 16));
      if (most >= INF) {
        most = 0;
        for (int i = lane0; i < pieces; i += per * 32) {
          const uint4 v = row[i];
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
          for (int e = 0; e < 8; ++e) {
            const uint32_t m = (u[e / 2] >> (16 * (e & 1))) & 0x7FFFu;
            most = max(most, m < INF ? m : 0u);
          }
        }
        most = __reduce_max_sync(0xFFFFFFFFu, most);
      }
      if (per > 1) {
        if (lane == 0) s_amax[warp] = most;
        __syncthreads();
      }
      if (col < rows) {
        if (per > 1)
          for (int w = warp / per * per; w < (warp / per + 1) * per; ++w) most = max(most, s_amax[w]);
        const T big = *reinterpret_cast<const T*>(&most);
        // 2^(14 - e) of a largest value in [2^e, 2^(e + 1)); of those below 2^-112 2^126
        const int e = max((int)(__float_as_uint(to_f32(big)) >> 23) - 127, -112);
        const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
#pragma unroll 4
        for (int i = lane0; i < pieces; i += per * 32) {
          const uint4 v = row[i];
          row[i] = C::order(unpack2<T>(v.x), unpack2<T>(v.y), unpack2<T>(v.z), unpack2<T>(v.w), up);
        }
        if (lane0 == 0) {
          // What makes up for it: with the scales, which stay finite, where it is below one, else at the
          // end and in two steps.  So only an output that is not finite overflows.
          const int back = e - 14 + C::UNIT, late = (max(back, 0) + 1) / 2;
          s_power[col] = __uint_as_float((uint32_t)(127 + back - 2 * late) << 23);
          s_rest[col] = __uint_as_float((uint32_t)(127 + late) << 23);
        }
      }
      __syncthreads();
    }
    int first = 0, count = 0, chunk = -1;  // of the unit at work
    const uint8_t* xr[NT];
    float2 power[NT];
    auto take_chunk = [&](int next) {
      if (next == chunk) return;
      chunk = next;
      chunk_rows(chunk, first, count);
      const int row0 = first - batch_first;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        // columns without a row take the first one's; they are not stored
        const int col = t * 8 + g;
        xr[t] = s_x + (row0 + (col < count ? col : 0)) * xp + c * 16;
        const int of = t * 8 + 2 * c;
        power[t] = make_float2(s_power[row0 + (of < count ? of : 0)],
                               s_power[row0 + (of + 1 < count ? of + 1 : 0)]);
      }
    };

    // Stores a unit's outputs from its lanes' sums.
    auto store = [&](int tile, const float4 (&sums)[NT]) {
      const int64_t n0 = (int64_t)tile * tile_out;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float v[4] = {sums[t].x, sums[t].y, sums[t].z, sums[t].w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = t * 8 + 2 * c + e;
          if (col >= count) continue;
          int row = first + col;
          const float rest = s_rest[row - batch_first];
          const float low = v[e] * rest * rest, high = v[2 + e] * rest * rest;
          if constexpr (EXPERTS) row = s_route[row];
          T* out = static_cast<T*>(p.out) + row * p.out_stride + n0 + g;
          if (gated) {
            if (n0 + g < p.n_out) *out = from_f32<T>(act_value(p.act, low) * high);
          } else {
            if (n0 + g < p.n_out) out[0] = from_f32<T>(low);
            if (n0 + g + 8 < p.n_out) out[8] = from_f32<T>(high);
          }
        }
      }
    };

    // The sums of a unit that another warp began, [warp][NT][lane]; the one that began it
    // keeps its own and adds them.
    auto place = [&](int w) { return red + w * (32 * NT) + lane; };
    float4 tail[NT];
    Run run = run_of(batch);
    bool begun = false;  // whether this warp has begun a unit that others go on with
    while (run.left > 0) {
      take_chunk(run.chunk);
      const int kb0 = run.kb, kb1 = min(blocks, run.kb + run.left);
      float2 acc[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = both(0.0f);

      for (int kb = kb0; kb < kb1; ++kb) {
        fetch(stage ^ 1);
        arrived();
        __syncwarp();
        const uint8_t* at = ring_at + stage * STAGE;
#pragma unroll
        for (int h = 0; h < PARTS; ++h) {
          S sc[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r;
            sc[r].read(at + scales_at(PARTS) + row * (PARTS * 16) + h * S::BYTES,
                       at + zeros_at(PARTS) + row * (PARTS * 8) + (ZERO_PAIRS ? (kb & 1) * 2 : h * S::COUNT));
          }
          const uint32_t base = ring + stage * STAGE + h * PART + lane_row;
          float part[NT][4];
          float2 s0, s1;
#pragma unroll
          for (int s = 0; s < 8; s += 2) {
            uint32_t w[4];  // words of rows g and g + 8 of 32 codes, then of the next 32
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(base + (lane_piece ^ (s << 4))));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int j = (s + i) / SPG;
              uint32_t d0[4], d1[4];
              C::pairs(w[2 * i], sc[0].minus(j), d0);
              C::pairs(w[2 * i + 1], sc[1].minus(j), d1);
              const uint32_t a0[4] = {d0[0], d1[0], d0[1], d1[1]};
              const uint32_t a1[4] = {d0[2], d1[2], d0[3], d1[3]};
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                const uint4 v = *reinterpret_cast<const uint4*>(xr[t] + kb * (BLOCK_K * 2) +
                                                                (h * 8 + s + i) * 64);
                mma_tile(part[t], a0, v.x, v.y, (s + i) % SPG == 0);
                mma_tile(part[t], a1, v.z, v.w, false);
              }
              if ((s + i) % SPG == SPG - 1) {
                if (j % 2 == 0) s0 = sc[0].scales(j / 2), s1 = sc[1].scales(j / 2);
                const float2 f0 = both(j % 2 == 0 ? s0.x : s0.y), f1 = both(j % 2 == 0 ? s1.x : s1.y);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                  acc[t][0] = fma2(mul2(f0, power[t]), make_float2(part[t][0], part[t][1]), acc[t][0]);
                  acc[t][1] = fma2(mul2(f1, power[t]), make_float2(part[t][2], part[t][3]), acc[t][1]);
                }
              }
            }
          }
        }
        __syncwarp();  // the stage is free
        stage ^= 1;
      }

      float4 sums[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) sums[t] = make_float4(acc[t][0].x, acc[t][0].y, acc[t][1].x, acc[t][1].y);
      if (kb1 - kb0 == blocks) {
        store(run.tile, sums);
      } else {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (kb0 > 0)
            place(warp)[t * 32] = sums[t];
          else
            tail[t] = sums[t];
        }
        begun = kb0 == 0;
      }
      run.left -= kb1 - kb0;
      if (run.left > 0) {
        run.kb = 0;
        if (++run.tile == tiles) run.tile = 0, ++run.chunk;
      }
    }
    __syncthreads();
    if (begun) {  // the rest of the unit is with the next warps, up to the one that ends it
      const uint32_t end = (uint32_t)(run.chunk * tiles + run.tile + 1 - batch.u0) * blocks;
      for (int w0 = warp + 1; w0 < WARPS && run_begin(batch, w0) < end; w0 += 4) {
        float4 o[4][NT];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int w = w0 + k;
          const bool has = w < WARPS && run_begin(batch, w) < end && run_begin(batch, w) < run_begin(batch, w + 1);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            o[k][t] = has ? place(w)[t * 32] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            tail[t].x += o[k][t].x, tail[t].y += o[k][t].y, tail[t].z += o[k][t].z, tail[t].w += o[k][t].w;
      }
      store(run.tile, tail);
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

}  // namespace w4
}  // namespace moe

namespace moe_host {

namespace w4 = moe::w4;

constexpr int kW4Smem = 232448 - 1024;

// Rows of x that a CTA has room for: always one beside blocks of one part; beside those of two
// perhaps none, where rows are long and routes many (1024 routes and K above 25,088, 33 routes
// and K above 29,184).
constexpr int w4_room(int nt, int parts, int routes, int64_t K) {
  const int64_t n = (kW4Smem - w4::fixed_bytes(nt, parts, routes)) / w4::x_pitch(K);
  return (int)(n < w4::MAX_ROOM ? n : w4::MAX_ROOM);
}
static_assert(w4_room(2, 1, w4::MAX_ROUTES, w4::MAX_K) >= 1, "a row of x has room");

template <typename T, w4::Format F, int SPG, int NT, int PARTS, bool EXPERTS>
static moe_status_t launch_w4(w4::Params p, cudaStream_t s) {
  constexpr auto kernel = w4::w4_kernel<T, F, SPG, NT, PARTS, EXPERTS>;
  moe_status_t st = allow_smem<kernel>(kW4Smem);
  if (st != MOE_OK) return st;
  const int routes = EXPERTS ? p.routes : 0;
  const int64_t rows = EXPERTS ? p.routes : p.T, ctas = num_sms();
  p.room = w4_room(NT, PARTS, routes, p.K);
  const int room = p.room < 8 * NT ? p.room : 8 * NT;
  const int64_t passes = (rows + room - 1) / room;
  p.most = EXPERTS ? (int)(rows < room ? rows : room) : (int)((rows + passes - 1) / passes);
  const int tile = p.act == MOE_ACT_NONE ? w4::ROWS : w4::ROWS / 2;
  const int64_t tiles = (p.n_out + tile - 1) / tile;
  const int64_t chunks = EXPERTS ? p.routes : passes, units = tiles * chunks;
  p.tiles = (int)tiles;
  p.blocks = (int)((p.K + w4::block_k(PARTS) - 1) / w4::block_k(PARTS));
  p.blocks_inverse = (uint32_t)(((uint64_t)1 << 32) / p.blocks + 1);  // of 1 it is not used
  // a CTA's units lie in few chunks where there are many units
  const int64_t likely = (EXPERTS && p.E < chunks ? p.E : chunks) / ctas + 2;
  if (p.room > p.most * likely) p.room = (int)(p.most * likely);
  const int64_t smem = w4::fixed_bytes(NT, PARTS, routes) + p.room * w4::x_pitch(p.K);
  return launched(launch_pdl(kernel, dim3((unsigned)(units < ctas ? units : ctas)), dim3(w4::WARPS * 32),
                             (size_t)smem, s, p),
                  "4-bit products");
}

// Blocks of two parts cost less beside the codes; of one they leave room for more rows of x,
// so that the weights pass fewer times.
template <typename T, w4::Format F, int SPG, bool EXPERTS>
static moe_status_t run_w4(const w4::Params& p, cudaStream_t s) {
  const int routes = EXPERTS ? p.routes : 0;
  // rows of a matrix: of a short batch's experts most have one or two
  const int64_t rows = EXPERTS ? (p.routes + p.E - 1) / p.E * 2 : p.T;
  auto passes = [&](int nt, int parts) {
    const int64_t n = w4_room(nt, parts, routes, p.K), m = n < 8 * nt ? n : 8 * nt;
    return m < 1 ? INT64_MAX : (rows + m - 1) / m;
  };
  if (passes(1, 2) <= passes(1, 1) && passes(1, 2) <= passes(2, 1))
    return launch_w4<T, F, SPG, 1, 2, EXPERTS>(p, s);
  if (passes(1, 1) <= passes(2, 1)) return launch_w4<T, F, SPG, 1, 1, EXPERTS>(p, s);
  return launch_w4<T, F, SPG, 2, 1, EXPERTS>(p, s);
}

template <typename T>
static moe_status_t run_w4_format(const w4::Params& p, int format, int64_t group, cudaStream_t s) {
  auto run = [&](auto f, auto spg) {
    constexpr w4::Format F = decltype(f)::value;
    constexpr int SPG = decltype(spg)::value;
    return p.ids != nullptr ? run_w4<T, F, SPG, true>(p, s) : run_w4<T, F, SPG, false>(p, s);
  };
  auto groups = [&](auto f) {
    if (group == 32) return run(f, std::integral_constant<int, 1>{});
    if (group == 64) return run(f, std::integral_constant<int, 2>{});
    return run(f, std::integral_constant<int, 4>{});
  };
  if (format == MOE_W4_E2M1)
    return run(std::integral_constant<w4::Format, w4::E2M1>{}, std::integral_constant<int, 1>{});
  if (p.zeros != nullptr) return groups(std::integral_constant<w4::Format, w4::INT4_ZEROS>{});
  return groups(std::integral_constant<w4::Format, w4::INT4>{});
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
  if (experts && a->top_k > 0 && T > INT64_MAX / a->top_k)
    return set_error(MOE_ERR_UNSUPPORTED, "at most %d routes to %d experts", w4::MAX_ROUTES,
                     w4::MAX_EXPERTS);
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
  if (K > w4::MAX_K || N >= ((int64_t)1 << 20))
    return set_error(MOE_ERR_UNSUPPORTED, "in_features above %d or 2^20 rows of a matrix", w4::MAX_K);
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
  auto unit = [&](const void* base, int64_t item) {
    const uint64_t row = (uint64_t)(K / G * item), block = (uint64_t)(512 / G * item);
    const uint64_t bits = row | reinterpret_cast<uintptr_t>(base);
    return bits % (block < 16 ? block : 16) == 0 ? 16 : (bits % 4 == 0 ? 4 : 1);
  };
  p.scale_unit = unit(a->scales, a->format == MOE_W4_E2M1 ? 1 : 2);
  p.zero_unit = unit(a->zeros, 1);
  p.out = a->out;
  p.out_stride = a->out_stride0;
  p.status = a->device_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a->dtype == MOE_DTYPE_BF16 ? run_w4_format<__nv_bfloat16>(p, a->format, G, s)
                                    : run_w4_format<__half>(p, a->format, G, s);
}

}  // extern "C"
