// int8 x int8 matrix product with a scale per token and per output channel,
// for any M, N and K and strided rows:
//   acc[m][n] = sum_k xq[m][k] wq[n][k]   (exact int32)
//   Y[m][n]   = ((acc * s_x[m]) * s_w[n]) * (1 / g) + bias[n], rounded once to
//               bf16, fp16 or fp32 (the epilogue order of the layers' GEMMs).
//
// Few tokens are bound by reading the weights once, many by the tensor cores,
// so there are three kernels:
//
// few_tokens_kernel   up to 32 tokens and small weights: a block takes tiles of 16
//   output channels, its warps split K.  Weights go from global memory straight into
//   the registers of mma.sync m16n8k32: a lane loads 16 consecutive codes of a
//   channel and of a token and uses them as the fragments of two products; both
//   operands see the same permutation of k, which the sum does not notice.  The
//   warps' int32 partials meet in shared memory.
//
// stream_kernel       few or small tiles: the weights are the 128-row operand of
//   tcgen05.mma kind::i8 (one CTA), the tokens its N.  Both come by TMA through a
//   ring of 108 KB, two CTAs per SM, so that one's weights stream while the other
//   starts or ends.  With few tiles K is split over a cluster and the int32
//   partials are summed through distributed shared memory.  A stage costs about
//   180 ns of TMA delivery (100 to 110 bytes per ns and SM) plus 23 ns per
//   product, in which the operands' shared-memory reads hold the copies up.
//
// tile_kernel         a cluster of two CTAs owns a 256 x BN tile and issues
//   tcgen05.mma kind::i8 in its pair form: each CTA holds 128 rows of A and
//   BN / 2 of B per stage, 128 bytes of k wide in the 128-byte swizzle that
//   TMA writes.  Two accumulators of BN columns in tensor memory let the epilogue
//   of one tile run under the products of the next.  8192 x 24576 x 8192: 1045 us
//   from a cool start, 1207 to 1275 in passes that last seconds (2590 to 2730 TOPS; the
//   power cap decides, and codes uniform over int8 take 1575); 4608 x 4096 x 4096: 53 us;
//   8192 x 4096 x 256, bound by its epilogues (3.1 us a tile; staged as int32 and scaled
//   on the way out they took 5.2): 25.6 us.  TMA fills what lies past M, N or K with zeros.
//     warp 0       TMA loads (both CTAs; both complete on the even CTA's
//                  barrier)
//     warp 1       MMA issue (even CTA)
//     warp 3       polls the barriers that the MMA warp depends on
//     warps 4-11   epilogue: tensor memory -> registers, a row per lane ->
//                  scaled and packed -> shared memory (32 rows of 128 bytes per
//                  warp) -> coalesced stores
//   SPLIT: too few tiles for the GPU; a cluster of 2 S CTAs owns one tile, pair
//   q takes a slice of K, and the int32 partials are summed exactly through
//   distributed shared memory, rows interleaved over the pairs.
// Every mbarrier wait is bounded; on timeout the kernel records an error in
// the device error word and runs to completion.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "plan_cache.h"
#include "tmap.h"

namespace w4a4 {

unsigned int* device_error_word();

namespace {

struct OutBf16 {
  using elem = __nv_bfloat16;
  static __device__ __forceinline__ elem from(float f) { return __float2bfloat16_rn(f); }
  static __device__ __forceinline__ float to(elem e) { return __bfloat162float(e); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
struct OutFp16 {
  using elem = __half;
  static __device__ __forceinline__ elem from(float f) { return __float2half_rn(f); }
  static __device__ __forceinline__ float to(elem e) { return __half2float(e); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
struct OutFp32 {
  using elem = float;
  static __device__ __forceinline__ elem from(float f) { return f; }
  static __device__ __forceinline__ float to(elem e) { return e; }
};

__device__ __forceinline__ float dequant(int acc, float sx, float sw, float inv_group, float bias, bool has_bias) {
  float y = __fmul_rn(__fmul_rn(__fmul_rn(__int2float_rn(acc), sx), sw), inv_group);
  return has_bias ? __fadd_rn(y, bias) : y;
}

// Four consecutive elements, n of them inside the row; vec: the address is
// aligned to their size.
template <class O>
__device__ __forceinline__ void store4(typename O::elem* p, int n, bool vec, const float (&y)[4]) {
  typename O::elem e[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) e[j] = O::from(y[j]);
  if (vec && n >= 4) {
    if constexpr (sizeof(typename O::elem) == 2) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(e);
    else *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(e);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[j] = e[j];
  }
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint16_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// ------------------------------------------------------------------ few tokens
constexpr int kFewWarps = 8;
constexpr int kFewRows = 16;     // output channels per block

// Plain (coherent) loads: this grid may have started while the kernel that wrote
// the operands still ran.
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Up to 16 codes at p (16-byte aligned) of which the row still has n, zeros behind
// them; nothing past the row is read.  Fewer come by four loads of falling size that
// do not wait for one another: one token, N = 175, K = 668 2.2 us, with a load per code
// 6.9.
__device__ __forceinline__ uint4 load_last_codes(const int8_t* p, int n) {
  uint4 whole = make_uint4(0u, 0u, 0u, 0u);
  if (n >= 16) whole = ldg_stream(p);
  const int r = n >= 16 ? 0 : max(n, 0);
  uint2 lo = make_uint2(0u, 0u);
  uint64_t b4 = 0, b2 = 0, b1 = 0;
  if (r & 8) lo = *reinterpret_cast<const uint2*>(p);
  if (r & 4) b4 = *reinterpret_cast<const uint32_t*>(p + (r & 8));
  if (r & 2) b2 = *reinterpret_cast<const uint16_t*>(p + (r & 12));
  if (r & 1) b1 = *reinterpret_cast<const uint8_t*>(p + (r & 14));
  const uint64_t t = b4 | b2 << (8 * (r & 4)) | b1 << (8 * (r & 6));
  const uint32_t t0 = (uint32_t)t, t1 = (uint32_t)(t >> 32);
  if (n >= 16) return whole;
  return r & 8 ? make_uint4(lo.x, lo.y, t0, t1) : make_uint4(t0, t1, 0u, 0u);
}

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// At most 8 NB tokens.  Bound by the latency of the loads: each warp has U k steps
// in flight, and a tile's weights are asked into L2 a tile ahead, the first one's
// before the wait for the previous kernel (a hint; the loads after the wait read
// memory as it then is).  Resident blocks take the tiles in turn: one token, K =
// 4096, replayed back to back, N = 4096 4.6 us (every load under its predicate 5.1, a
// block per tile 5.3, without the hint 6.1), N = 10240 8.8 (a block per tile 12.6).  Three blocks per SM (two from 9
// tokens on, whose fragments need the registers) leave room for the next kernel's
// blocks, whose hints then run under this one.  TAIL: K is not a multiple of 64 (a
// kernel of its own, as the last step's code costs the others 0.3 us of fetches and
// registers).
template <int NB, class O, bool TAIL>
__global__ void __launch_bounds__(kFewWarps * 32, NB == 1 ? 3 : 2) few_tokens_kernel(Matmul8Args p) {
  constexpr int U = NB <= 2 ? 4 : 2;   // k steps (64 codes) in flight per warp
  __shared__ int part[2][kFewWarps][8 * NB][kFewRows + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int64_t tiles = ((int64_t)p.N + kFewRows - 1) / kFewRows;
  auto hint = [&](int64_t tile) {
    const int64_t n = tile * kFewRows + (threadIdx.x & (kFewRows - 1));
    if (n < p.N)
      for (int k = (threadIdx.x / kFewRows) * 128; k < p.K; k += kFewWarps * 32 / kFewRows * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.B + n * p.ldb + k));
  };
  hint(blockIdx.x);
  grid_dependency_wait();
  grid_launch_dependents();
  const int steps = p.K / 64;      // whole ones
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  int buf = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    if (tile + gridDim.x < tiles) hint(tile + gridDim.x);
    const int64_t n0 = tile * kFewRows;
    // Channels and tokens past the ends read row 0 instead; their sums go nowhere.
    const int8_t* w0 = p.B + (n0 + g < p.N ? n0 + g : 0) * p.ldb + 16 * t;
    const int8_t* w1 = p.B + (n0 + g + 8 < p.N ? n0 + g + 8 : 0) * p.ldb + 16 * t;
    const int8_t* x[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) x[i] = p.A + (8 * i + g < p.M ? 8 * i + g : 0) * p.lda + 16 * t;
    int acc[NB][4] = {};
    auto round = [&](int s0, auto full) {              // steps s0, s0 + 8, ...: U of them, or those that there are
      uint4 a[U][2], b[U][NB];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool go = decltype(full)::value || s0 + u * kFewWarps < steps;
        const int k0 = (s0 + u * kFewWarps) * 64;
        a[u][0] = go ? ldg_stream(w0 + k0) : zero;
        a[u][1] = go ? ldg_stream(w1 + k0) : zero;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool go = decltype(full)::value || s0 + u * kFewWarps < steps;
        const int k0 = (s0 + u * kFewWarps) * 64;
#pragma unroll
        for (int i = 0; i < NB; ++i) b[u][i] = go ? *reinterpret_cast<const uint4*>(x[i] + k0) : zero;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          mma_s8(acc[i], a[u][0].x, a[u][1].x, a[u][0].y, a[u][1].y, b[u][i].x, b[u][i].y);
          mma_s8(acc[i], a[u][0].z, a[u][1].z, a[u][0].w, a[u][1].w, b[u][i].z, b[u][i].w);
        }
    };
    int s0 = warp;
    for (; s0 + (U - 1) * kFewWarps < steps; s0 += kFewWarps * U) round(s0, std::true_type{});
    if (s0 < steps) round(s0, std::false_type{});
    if (TAIL && warp == steps % kFewWarps) {
      const int n = p.K - steps * 64 - 16 * t;
      const uint4 a0 = load_last_codes(w0 + steps * 64, n), a1 = load_last_codes(w1 + steps * 64, n);
      uint4 b[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) b[i] = load_last_codes(x[i] + steps * 64, n);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        mma_s8(acc[i], a0.x, a1.x, a0.y, a1.y, b[i].x, b[i].y);
        mma_s8(acc[i], a0.z, a1.z, a0.w, a1.w, b[i].z, b[i].w);
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      part[buf][warp][8 * i + 2 * t][g] = acc[i][0];
      part[buf][warp][8 * i + 2 * t + 1][g] = acc[i][1];
      part[buf][warp][8 * i + 2 * t][g + 8] = acc[i][2];
      part[buf][warp][8 * i + 2 * t + 1][g + 8] = acc[i][3];
    }
    __syncthreads();
    // the buffer is written again two tiles on, behind the next tile's barrier
    const int c = threadIdx.x % kFewRows;
    const int64_t n = n0 + c;
    for (int m = threadIdx.x / kFewRows; m < min(p.M, 8 * NB) && n < p.N; m += kFewWarps * 32 / kFewRows) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) sum += part[buf][w][m][c];
      const auto* bias = static_cast<const typename O::elem*>(p.bias);
      const float y = dequant(sum, p.a_scale[m], p.b_scale[n], p.inv_group, bias ? O::to(bias[n]) : 0.0f, bias != nullptr);
      static_cast<typename O::elem*>(p.Y)[(int64_t)m * p.ldy + n] = O::from(y);
    }
  }
}

// ------------------------------------------------------------------ tiles
constexpr int BM = 128;              // A rows per CTA
constexpr int BK = 128;              // codes per k-block: one swizzle row
constexpr int kTileThreads = 384;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr int kIssueBar = 1;             // named barrier: MMA warp + the warp that waits for it
constexpr int kStagePitch = 128 + 16;                       // epilogue staging: 128 bytes of a row, bank-spread
constexpr int kStageBytes = 32 * kStagePitch + 1024;        // per epilogue warp: 32 rows; its columns' scales and bias
constexpr int kSmemLimit = 232448;

template <int BN>
struct TileCfg {
  static constexpr int kBRows = BN / 2;
  static constexpr int kABytes = BM * BK, kBBytes = kBRows * BK;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kEpi = kEpiWarps * kStageBytes;
  static constexpr int kBarBytes = 512;
  static constexpr int ST = (kSmemLimit - 1024 - kEpi - kBarBytes) / kStage;
  static constexpr int kRing = ST * kStage;
  static constexpr int kSmem = 1024 + kRing + kEpi + kBarBytes;
  static constexpr int kPartPitch = BN * 4 + 16;            // split: int32 partial row, bank-spread
  static constexpr int kTmemCols = 2 * BN;
  // k-blocks released to the MMA warp at a time: two narrow ones (256 x 128 x
  // 8192 alone: 290 -> 250 ns each), one wide one (its four products cover the
  // hand-off)
  static constexpr int kBatch = BN == 128 ? 2 : 1;
  static_assert(ST >= 4 && ST <= 12, "ring depth");
  static_assert(BM * kPartPitch <= kRing + kEpi, "partials fit where the ring was");
  static_assert(kSmem <= kSmemLimit, "shared memory budget");
};

// 32 rows of 128 bytes that a warp has staged, stored to y and ldy elements on;
// `rows` and `cols` of them are inside the matrix, rows of y are aligned to gran
// bytes.  16: four rows per store; else a row per store of 4 bytes per lane, or
// half of one of 2.
template <class E>
__device__ __forceinline__ void store_rows(uint32_t stg, E* y, int64_t ldy, int64_t rows, int64_t cols, int gran, int lane) {
  constexpr int kV = 16 / (int)sizeof(E), kW = 4 / (int)sizeof(E);
  using bits = typename std::conditional<sizeof(E) == 2, uint16_t, uint32_t>::type;
  bits* out = reinterpret_cast<bits*>(y);
  if (gran == 16) {
    const int c = (lane & 7) * kV;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int row = r * 4 + (lane >> 3);
      const uint4 a = ld_shared_v4(stg + (uint32_t)(row * kStagePitch + (lane & 7) * 16));
      if (row < rows && c < cols) {
        bits* to = out + row * ldy + c;
        if (c + kV <= cols) {
          *reinterpret_cast<uint4*>(to) = a;
        } else {
          const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int j = 0; j < kV - 1; ++j)
            if (c + j < cols) to[j] = (bits)(w[j / kW] >> (16 * (j % kW)));
        }
      }
    }
  } else if (gran == 4) {
    const int c = lane * kW;
#pragma unroll 8
    for (int row = 0; row < 32; ++row) {
      const uint32_t a = ld_shared_u32(stg + (uint32_t)(row * kStagePitch + lane * 4));
      if (row < rows && c < cols) {
        bits* to = out + row * ldy + c;
        if (c + kW <= cols) *reinterpret_cast<uint32_t*>(to) = a;
        else *to = (bits)a;
      }
    }
  } else if constexpr (sizeof(E) == 2) {
#pragma unroll 8
    for (int row = 0; row < 32; ++row)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint16_t a = ld_shared_u16(stg + (uint32_t)(row * kStagePitch + h * 64 + lane * 2));
        if (row < rows && h * 32 + lane < cols) out[row * ldy + h * 32 + lane] = a;
      }
  }
}

struct TileBars {
  uint64_t full[12], empty[12], acc_full[2], acc_empty[2];
  uint32_t tmem_base;
};
static_assert(sizeof(TileBars) <= 512, "barrier area");

// TMA load whose bytes complete on a barrier of either CTA of the pair (a
// shared::cluster address).  No multicast.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* tmap, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

struct TilePlan {
  int tiles_m, tiles_n, split;
};

// Tile t of a walk that goes down up to eight row tiles before it moves one
// column tile on, so that the pairs at work together share their operands in L2.
__device__ __forceinline__ void tile_at(int64_t t, const TilePlan& pl, int& tm, int& tn) {
  const int64_t per = (int64_t)8 * pl.tiles_n;
  const int band = (int)(t / per);
  const int rows = min(8, pl.tiles_m - 8 * band);
  const int64_t in = t - band * per;
  tn = (int)(in / rows);
  tm = 8 * band + (int)(in - (int64_t)tn * rows);
}

template <int BN, class O, bool SPLIT>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const Matmul8Args p, const TilePlan pl, const __grid_constant__ CUtensorMap tmA,
                const __grid_constant__ CUtensorMap tmB, unsigned int* err) {
  using C = TileCfg<BN>;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* gbase = raw + (base - smem_u32(raw));
  TileBars* bar = reinterpret_cast<TileBars*>(gbase + C::kRing + C::kEpi);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const uint32_t half = crank & 1u;                  // 0: the pair's even CTA
  const uint32_t lead = crank & ~1u;
  const uint16_t pmask = (uint16_t)(3u << lead);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(&bar->full[s], 1);
      mbar_init(&bar->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bar->acc_full[b], 1);
      mbar_init(&bar->acc_empty[b], 2 * kEpiWarps);
    }
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 2) {
    tmem_alloc_pair(&bar->tmem_base, C::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;

  // This pair's tiles and k-blocks.
  const int64_t tiles = (int64_t)pl.tiles_m * pl.tiles_n;
  const int nk = (p.K + BK - 1) / BK;
  int64_t t0, tstep;
  int kb0 = 0, kb1 = nk;
  if constexpr (SPLIT) {
    t0 = blockIdx.x / (2 * pl.split);
    tstep = tiles;                                   // one tile
    const int q = (int)(crank >> 1);
    kb0 = (int)((int64_t)q * nk / pl.split);
    kb1 = (int)((int64_t)(q + 1) * nk / pl.split);
  } else {
    t0 = blockIdx.x >> 1;
    tstep = gridDim.x >> 1;
  }

  // The next kernel of the stream may start where this one leaves SMs free, and
  // a split asks the first weights into L2 before it waits for the previous
  // kernel (a hint: the loads after the wait read memory as it then is).  256 x
  // 4096 x 12288 in thirds: 20.2 -> 19.7 -> 19.5 us; 333 x 1013 x 2995: 10.0 -> 9.4.
  if (SPLIT && warp == 3 && lane == 0) {
    int tm, tn;
    tile_at(t0, pl, tm, tn);
    for (int kb = kb0; kb < min(kb1, kb0 + 4); ++kb)
      prefetch_tile_l2(&tmB, kb * BK, tn * BN + (int)half * C::kBRows);
  }
  grid_dependency_wait();
  grid_launch_dependents();

  // SPLIT: this thread's columns in the final sum, their scales and bias loaded
  // while the products run
  constexpr int kG = SPLIT ? BN / 128 : 1;             // groups of four columns per lane
  int64_t sm0 = 0, sn0 = 0;
  float ssw[kG][4], sbs[kG][4];
  if constexpr (SPLIT) {
    int tm, tn;
    tile_at(t0, pl, tm, tn);
    sm0 = (int64_t)tm * 2 * BM + (int64_t)half * BM;
    sn0 = (int64_t)tn * BN + lane * 4;
#pragma unroll
    for (int c = 0; c < kG; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t n = sn0 + c * 128 + j;
        const auto* bias = static_cast<const typename O::elem*>(p.bias);
        ssw[c][j] = n < p.N ? p.b_scale[n] : 0.0f;
        sbs[c][j] = bias && n < p.N ? O::to(bias[n]) : 0.0f;
      }
  }

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    if (lane == 0) {
      int g = 0;
      bool ok = true;
      for (int64_t t = t0; t < tiles && ok; t += tstep) {
        int tm, tn;
        tile_at(t, pl, tm, tn);
        const int ya = tm * 2 * BM + (int)half * BM, yb = tn * BN + (int)half * C::kBRows;
        for (int kb = kb0; kb < kb1; ++kb, ++g) {
          const int s = g % C::ST;
          if (g >= C::ST && !mbar_wait_cluster(&bar->empty[s], (uint32_t)(g / C::ST - 1) & 1u)) {
            set_device_error(err, kDevErrTimeoutEmpty);
            ok = false;
            break;
          }
          if (half == 0) mbar_arrive_expect_tx(&bar->full[s], 2u * (uint32_t)C::kStage);
          const uint32_t fb = map_to_rank(smem_u32(&bar->full[s]), lead);
          const uint32_t dst = base + (uint32_t)(s * C::kStage);
          tma_load_2d_pair(dst, &tmA, kb * BK, ya, fb);
          tma_load_2d_pair(dst + C::kABytes, &tmB, kb * BK, yb, fb);
        }
      }
      // every stage given back: no copy, product or arrival is in flight
      // towards this CTA any more
      for (int s = 0; s < C::ST && ok; ++s) {
        const int uses = (g - s + C::ST - 1) / C::ST;
        if (uses > 0 && !mbar_wait_cluster(&bar->empty[s], (uint32_t)(uses - 1) & 1u)) {
          set_device_error(err, kDevErrTimeoutDrain);
          ok = false;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 && half == 0) {
    // ---------------------------------------------------------------- MMA
    // This warp never reads shared memory: a read whose result it uses would
    // queue behind the products it has issued.  Warp 3 polls the barriers in
    // the same order and releases each step through a named barrier.
    constexpr uint32_t idesc = idesc_i8(2 * BM, BN);
    const uint64_t da0 = smem_desc_kmajor_sw128(base), db0 = smem_desc_kmajor_sw128(base + C::kABytes);
    int s = 0, i = 0;
    for (int64_t t = t0; t < tiles; t += tstep, ++i) {
      const int b = i & 1;
      bool bad = false;
      for (int kb = kb0; kb < kb1;) {
        if ((bad = named_barrier_or(kIssueBar, 64, false))) break;
        if (kb == kb0) tc_fence_after();               // the epilogue has read this accumulator
        const int end = min(kb + C::kBatch, kb1);
        for (; kb < end; ++kb) {
          if (lane == 0) {
            const uint64_t off = (uint64_t)(s * (C::kStage >> 4));   // descriptors count 16 bytes
#pragma unroll
            for (int ks = 0; ks < BK / 32; ++ks)
              mma_i8_ss_pair(tmem + (uint32_t)(b * BN), da0 + off + 2 * ks, db0 + off + 2 * ks, idesc,
                             kb > kb0 || ks > 0 ? 1u : 0u);
            tc_commit_pair_mc(&bar->empty[s], pmask);
            if (kb == kb1 - 1) tc_commit_pair_mc(&bar->acc_full[b], pmask);
          }
          if (++s == C::ST) s = 0;
        }
        __syncwarp();
      }
      if (bad) break;
    }
  } else if (warp == 3 && half == 0) {
    // ---------------------------------------------------------------- waits for the MMA warp
    int s = 0, i = 0;
    uint32_t ph = 0;
    for (int64_t t = t0; t < tiles; t += tstep, ++i) {
      bool bad = false;
      for (int kb = kb0; kb < kb1;) {
        if (kb == kb0 && i >= 2) {
          if (!mbar_wait_cluster(&bar->acc_empty[i & 1], (uint32_t)(i / 2 - 1) & 1u)) {
            if (lane == 0) set_device_error(err, kDevErrTimeoutAcc);
            bad = true;
          }
          tc_fence_after();
          tc_fence_before();
        }
        const int end = min(kb + C::kBatch, kb1);
        for (; kb < end; ++kb) {
          if (!bad && !mbar_wait_cluster(&bar->full[s], ph)) {
            if (lane == 0) set_device_error(err, kDevErrTimeoutFull);
            bad = true;
          }
          if (++s == C::ST) {
            s = 0;
            ph ^= 1u;
          }
        }
        // a lane may have run out of time where the others did not: all agree
        if ((bad = named_barrier_or(kIssueBar, 64, bad))) break;
      }
      if (bad) break;
    }
  } else if (warp >= kEpiWarp0) {
    // ---------------------------------------------------------------- epilogue
    const int ew = warp - kEpiWarp0;
    const int quad = warp & 3, hc = ew >> 2;
    constexpr int kCols = BN / 2;                    // columns of a warp
    if constexpr (SPLIT) {
      if (__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&bar->acc_full[0], 0u))) {
        tc_fence_after();
        const uint32_t row = base + (uint32_t)((quad * 32 + lane) * C::kPartPitch + hc * kCols * 4);
#pragma unroll
        for (int ch = 0; ch < kCols / 32; ++ch) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(hc * kCols + ch * 32), v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row + (uint32_t)(ch * 128 + j * 16)),
                         "r"(v[4 * j]), "r"(v[4 * j + 1]), "r"(v[4 * j + 2]), "r"(v[4 * j + 3])
                         : "memory");
        }
      } else {
        set_device_error(err, kDevErrTimeoutAcc);
      }
    } else {
      // A lane owns a row: 32 sums from tensor memory (the next 32 under way),
      // scaled and packed, staged 128 bytes a row, then stored by rows.  The scales
      // and bias of the next tile are fetched a tile ahead.
      constexpr int kJ = kCols / 32;
      constexpr int kGroup = 4 / (int)sizeof(typename O::elem);        // chunks of 32 columns in 128 bytes
      const uint32_t stg = base + (uint32_t)(C::kRing + ew * kStageBytes), sc = stg + 32 * kStagePitch;
      const auto* bias = static_cast<const typename O::elem*>(p.bias);
      const uintptr_t at = reinterpret_cast<uintptr_t>(p.Y) | (uintptr_t)(p.ldy * (int64_t)sizeof(typename O::elem));
      const int gran = at % 16 == 0 ? 16 : at % 4 == 0 ? 4 : 2;
      float nsw[kJ], nbs[kJ], nsx;
      auto fetch = [&](int64_t t) {
        int tm, tn;
        tile_at(t, pl, tm, tn);
        const int64_t m = (int64_t)tm * 2 * BM + (int64_t)half * BM + quad * 32 + lane;
        nsx = m < p.M ? p.a_scale[m] : 0.0f;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const int64_t n = (int64_t)tn * BN + hc * kCols + j * 32 + lane;
          nsw[j] = n < p.N ? p.b_scale[n] : 0.0f;
          nbs[j] = bias && n < p.N ? O::to(bias[n]) : -0.0f;           // y + -0 is y
        }
      };
      if (t0 < tiles) fetch(t0);
      int i = 0;
      for (int64_t t = t0; t < tiles; t += tstep, ++i) {
        const int b = i & 1;
        int tm, tn;
        tile_at(t, pl, tm, tn);
        const int64_t m0 = (int64_t)tm * 2 * BM + (int64_t)half * BM + quad * 32;
        const int64_t n0 = (int64_t)tn * BN + hc * kCols;
        const float sx = nsx;
        __syncwarp();                                   // the last tile's scales are read
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          st_shared_f32(sc + (uint32_t)(j * 128 + lane * 4), nsw[j]);
          st_shared_f32(sc + (uint32_t)(512 + j * 128 + lane * 4), nbs[j]);
        }
        if (t + tstep < tiles) fetch(t + tstep);
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&bar->acc_full[b], (uint32_t)(i / 2) & 1u))) {
          set_device_error(err, kDevErrTimeoutAcc);
          break;
        }
        tc_fence_after();
        const uint32_t ta = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(b * BN + hc * kCols);
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(ta, v[0]);
#pragma unroll
        for (int ch = 0; ch < kJ; ++ch) {
          tmem_wait_ld_x32(v[ch & 1]);
          if (ch < kJ - 1) {
            tmem_ld_32x32b_x32(ta + (uint32_t)(32 * (ch + 1)), v[(ch + 1) & 1]);
          } else {                                      // the accumulator may be overwritten
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(&bar->acc_empty[b], lead);
          }
          if (ch % kGroup == 0) __syncwarp();           // the last rows are read
#pragma unroll
          for (int j = 0; j < 4; ++j) {                 // eight columns at a time
            float y[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t col = sc + (uint32_t)(ch * 128 + j * 32 + h * 16);
              const float4 w = ld_shared_f4(col), bb = ld_shared_f4(col + 512);
              const uint32_t* a = &v[ch & 1][8 * j + 4 * h];
              y[4 * h] = dequant((int)a[0], sx, w.x, p.inv_group, bb.x, true);
              y[4 * h + 1] = dequant((int)a[1], sx, w.y, p.inv_group, bb.y, true);
              y[4 * h + 2] = dequant((int)a[2], sx, w.z, p.inv_group, bb.z, true);
              y[4 * h + 3] = dequant((int)a[3], sx, w.w, p.inv_group, bb.w, true);
            }
            const uint32_t to = stg + (uint32_t)(lane * kStagePitch + (ch % kGroup * 32 + 8 * j) * (int)sizeof(typename O::elem));
            if constexpr (sizeof(typename O::elem) == 2) {
              st_shared_v4(to, make_uint4(O::pack(y[0], y[1]), O::pack(y[2], y[3]), O::pack(y[4], y[5]), O::pack(y[6], y[7])));
            } else {
              st_shared_v4(to, make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])));
              st_shared_v4(to + 16, make_uint4(__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]), __float_as_uint(y[7])));
            }
          }
          if (ch % kGroup == kGroup - 1) {
            __syncwarp();
            const int64_t n = n0 + (ch - kGroup + 1) * 32;
            store_rows<typename O::elem>(stg, static_cast<typename O::elem*>(p.Y) + m0 * p.ldy + n, p.ldy, p.M - m0, p.N - n, gran, lane);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if constexpr (SPLIT) {
    // Rows r = q, q + S, ... of this CTA's 128: the pairs' partials summed, a
    // lane per four columns.  128 columns keep two rows of remote loads in flight
    // (256 x 4096 x 12288 in halves 22.4 -> 21.3 us); 256 columns are bound by the
    // SM-to-SM network (2.4 TB/s) and gain nothing from it.
    constexpr int kRows = BN == 128 ? 2 : 1;
    const int64_t m0 = sm0, n0 = sn0;
    const int S = pl.split;
    const int step = (kTileThreads / 32) * S;
    uint32_t peer[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) peer[q] = map_to_rank(base, (uint32_t)(2 * (q < S ? q : 0)) + half);
    for (int r = (int)(crank >> 1) + warp * S; r < BM && m0 + r < p.M; r += kRows * step) {
      const bool two = kRows == 2 && r + step < BM && m0 + r + step < p.M;
      const float sx[2] = {p.a_scale[m0 + r], two ? p.a_scale[m0 + r + step] : 0.0f};
      uint4 v[kRows][4][kG];
#pragma unroll
      for (int h = 0; h < kRows; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int c = 0; c < kG; ++c)
            if (q < S && (h == 0 || two))
              v[h][q][c] = ld_cluster_v4(peer[q] + (uint32_t)((r + h * step) * C::kPartPitch + (c * 128 + lane * 4) * 4));
#pragma unroll
      for (int h = 0; h < kRows; ++h) {
        if (h == 1 && !two) break;
#pragma unroll
        for (int c = 0; c < kG; ++c) {
          int a[4] = {0, 0, 0, 0};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < S) {
              a[0] += (int)v[h][q][c].x;
              a[1] += (int)v[h][q][c].y;
              a[2] += (int)v[h][q][c].z;
              a[3] += (int)v[h][q][c].w;
            }
          const int64_t n = n0 + c * 128;
          if (n >= p.N) continue;
          const bool hb = p.bias != nullptr;
          float y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = dequant(a[j], sx[h], ssw[c][j], p.inv_group, sbs[c][j], hb);
          store4<O>(static_cast<typename O::elem*>(p.Y) + (m0 + r + h * step) * p.ldy + n, (int)min((int64_t)4, p.N - n),
                    p.vec_out, y);
        }
      }
    }
    cluster_sync();                                  // the partials stay readable until every CTA has summed
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::kTmemCols);
  }
}

// Codes [rows, K] as boxes of 128 codes x `box` rows; what lies past K or the
// rows reads as zero.
bool codes_tmap(CUtensorMap* tm, const int8_t* x, int rows, int K, int64_t ld, int box) {
  const uint64_t dims[2] = {(uint64_t)K, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)(rows == 1 ? (K + 15) / 16 * 16 : ld)};
  const uint32_t bx[2] = {BK, (uint32_t)box};
  return encode_tmap_nd(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, 2, dims, strides, bx, CU_TENSOR_MAP_SWIZZLE_128B);
}

// ------------------------------------------------------------------ streamed weights
constexpr int kStreamThreads = 256;
constexpr int kStreamRows = 128;          // output channels per tile: the MMA's M
constexpr int kStreamRing = 108 * 1024;   // two CTAs per SM

template <int NT>
struct StreamCfg {
  static constexpr int kW = kStreamRows * BK, kX = NT * BK;
  static constexpr int kStage = kW + kX;
  static constexpr int ST = kStreamRing / kStage;
  static constexpr int kRing = ST * kStage;
  static constexpr int kTmemCols = NT < 32 ? 32 : NT;
  static constexpr int kSmem = 1024 + kRing + 1024 + NT * 4;   // alignment, ring, barriers, token scales
  static constexpr int kPartPitch = kStreamRows * 4;           // a token's sums over the tile's channels
  static_assert(ST >= 2 && ST <= 8, "barrier arrays");
  static_assert(NT * kPartPitch <= kRing, "the sums fit where the ring was");
};

struct StreamBars {
  uint64_t full[8], empty[8], acc_full;
  uint32_t tmem_base;
};

// One tile of 128 output channels, or (split > 1, a cluster of that many CTAs)
// one slice of its K.  Warp 0 loads, warp 1 issues the products, warps 4 to 7
// leave the int32 sums in shared memory as [token][channel], and then all
// warps finish tokens in turn, a lane per four channels.
template <int NT, class O>
__global__ void __launch_bounds__(kStreamThreads, 2)
    stream_kernel(const Matmul8Args p, int split, int tiles_m, const __grid_constant__ CUtensorMap tmX,
                  const __grid_constant__ CUtensorMap tmW, unsigned int* err) {
  using C = StreamCfg<NT>;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* gbase = raw + (base - smem_u32(raw));
  StreamBars* bar = reinterpret_cast<StreamBars*>(gbase + C::kRing);
  float* sx = reinterpret_cast<float*>(gbase + C::kRing + 1024);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = split > 1 ? (int)cluster_ctarank() : 0;
  const int tile = (int)blockIdx.x / split / tiles_m;      // of channels; its token tiles are neighbours
  const int m0 = (int)blockIdx.x / split % tiles_m * NT;
  const int tokens = min(NT, p.M - m0);
  const int nk = (p.K + BK - 1) / BK;
  const int kb0 = (int)((int64_t)q * nk / split), kb1 = (int)((int64_t)(q + 1) * nk / split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(&bar->full[s], 1);
      mbar_init(&bar->empty[s], 1);
    }
    mbar_init(&bar->acc_full, 1);
    fence_mbar_init();
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmW);
  }
  if (warp == 2) {
    tmem_alloc(&bar->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  // A slice asks its first weights into L2 before the wait for the previous
  // kernel (a hint; the loads after the wait read memory as it then is): 16 x 4096
  // x 4096 in quarters 7.2 -> 6.7 us.  Whole tiles gain nothing (21.8, 21.9).
  if (split > 1 && warp == 3 && lane == 0)
    for (int kb = kb0; kb < min(kb1, kb0 + C::ST); ++kb) prefetch_tile_l2(&tmW, kb * BK, tile * kStreamRows);
  grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();                            // after this CTA has its tensor memory
  const uint32_t tmem = bar->tmem_base;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int g = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++g) {
        const int s = g % C::ST;
        if (g >= C::ST && !mbar_wait(&bar->empty[s], (uint32_t)(g / C::ST - 1) & 1u)) {
          set_device_error(err, kDevErrTimeoutEmpty);
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&bar->full[s], (uint32_t)C::kStage);
        const uint32_t dst = base + (uint32_t)(s * C::kStage);
        tma_load_2d(dst, &tmW, kb * BK, tile * kStreamRows, &bar->full[s]);
        tma_load_2d(dst + C::kW, &tmX, kb * BK, m0, &bar->full[s]);
      }
      for (int s = 0; s < C::ST && ok; ++s) {          // no copy or product is in flight any more
        const int uses = (g - s + C::ST - 1) / C::ST;
        if (uses > 0 && !mbar_wait(&bar->empty[s], (uint32_t)(uses - 1) & 1u)) {
          set_device_error(err, kDevErrTimeoutDrain);
          ok = false;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_i8(kStreamRows, NT);
      const uint64_t da0 = smem_desc_kmajor_sw128(base), db0 = smem_desc_kmajor_sw128(base + C::kW);
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&bar->full[s], ph)) {
          set_device_error(err, kDevErrTimeoutFull);
          ok = false;
          break;
        }
        const uint64_t off = (uint64_t)(s * (C::kStage >> 4));   // descriptors count 16 bytes
#pragma unroll
        for (int ks = 0; ks < BK / 32; ++ks)
          mma_i8_ss(tmem, da0 + off + 2 * ks, db0 + off + 2 * ks, idesc, kb > kb0 || ks > 0 ? 1u : 0u);
        tc_commit(&bar->empty[s]);
        if (++s == C::ST) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (ok) tc_commit(&bar->acc_full);
    }
    __syncwarp();
  }

  // What the final step needs from global memory, while the products run.
  const int64_t n = (int64_t)tile * kStreamRows + 4 * lane;
  const auto* bias = static_cast<const typename O::elem*>(p.bias);
  float sw[4], bs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sw[j] = n + j < p.N ? p.b_scale[n + j] : 0.0f;
    bs[j] = bias && n + j < p.N ? O::to(bias[n + j]) : 0.0f;
  }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + NT) {    // warps 2 to 5
    const int m = (int)threadIdx.x - 64;
    sx[m] = m < tokens ? p.a_scale[m0 + m] : 0.0f;
  }
  if (warp >= 4) {
    if (__all_sync(0xFFFFFFFFu, mbar_wait(&bar->acc_full, 0u))) {
      tc_fence_after();
      constexpr int CH = NT < 32 ? NT : 32;
      const int c = (warp - 4) * 32 + lane;            // this thread's channel of the tile
#pragma unroll
      for (int ch = 0; ch < NT / CH; ++ch) {
        if (ch * CH >= tokens) break;
        uint32_t v[CH];
        const uint32_t ta = tmem + ((uint32_t)((warp - 4) * 32) << 16) + (uint32_t)(ch * CH);
        if constexpr (CH == 16) tmem_ld_32x32b_x16(ta, v);
        else tmem_ld_32x32b_x32(ta, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < CH; ++j)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + (uint32_t)((ch * CH + j) * C::kPartPitch + c * 4)), "r"(v[j])
                       : "memory");
      }
    } else {
      set_device_error(err, kDevErrTimeoutAcc);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_sync();
  uint32_t peer[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) peer[r] = split > 1 && r < split ? map_to_rank(base, (uint32_t)r) : base;
  for (int m = q + warp * split; m < tokens; m += (kStreamThreads / 32) * split) {
    const uint32_t at = (uint32_t)(m * C::kPartPitch + 16 * lane);
    int a[4];
    if (split == 1) {
      const uint4 v = ld_shared_v4(base + at);
      a[0] = (int)v.x;
      a[1] = (int)v.y;
      a[2] = (int)v.z;
      a[3] = (int)v.w;
    } else {
      uint4 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < split) v[r] = ld_cluster_v4(peer[r] + at);
      a[0] = a[1] = a[2] = a[3] = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < split) {
          a[0] += (int)v[r].x;
          a[1] += (int)v[r].y;
          a[2] += (int)v[r].z;
          a[3] += (int)v[r].w;
        }
    }
    if (n < p.N) {
      const float s = sx[m];
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = dequant(a[j], s, sw[j], p.inv_group, bs[j], bias != nullptr);
      store4<O>(static_cast<typename O::elem*>(p.Y) + (int64_t)(m0 + m) * p.ldy + n, (int)min((int64_t)4, p.N - n),
                p.vec_out, y);
    }
  }
  if (split > 1) cluster_sync();                       // the sums stay readable until every CTA has taken them
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------ host side
template <int NT, class O>
cudaError_t launch_stream(const Matmul8Args& a, int split, int dev, cudaStream_t st) {
  using C = StreamCfg<NT>;
  auto kern = stream_kernel<NT, O>;
  static DeviceFlags configured;
  cudaError_t e;
  if (!configured.done(dev)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) != cudaSuccess)
      return e;
    configured.set(dev);
  }
  unsigned int* err = device_error_word();
  if (!err) return cudaErrorInvalidDevicePointer;
  CUtensorMap tX, tW;
  if (!codes_tmap(&tX, a.A, a.M, a.K, a.lda, NT) || !codes_tmap(&tW, a.B, a.N, a.K, a.ldb, kStreamRows))
    return cudaErrorInvalidValue;
  const int tiles_m = (int)(((int64_t)a.M + NT - 1) / NT);
  const int64_t tiles = ((int64_t)a.N + kStreamRows - 1) / kStreamRows * tiles_m;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split), 1, 1);
  cfg.blockDim = dim3(kStreamThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, split, tiles_m, tX, tW, err);
}

template <int NB, class O>
cudaError_t launch_few(const Matmul8Args& a, int sms, cudaStream_t st) {
  const int64_t tiles = ((int64_t)a.N + kFewRows - 1) / kFewRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(tiles, (int64_t)sms * (NB == 1 ? 3 : 2)), 1, 1);
  cfg.blockDim = dim3(kFewWarps * 32, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.K % 64 ? cudaLaunchKernelEx(&cfg, few_tokens_kernel<NB, O, true>, a)
                  : cudaLaunchKernelEx(&cfg, few_tokens_kernel<NB, O, false>, a);
}

// How many clusters of `size` CTAs of a kernel fit on the device at once (0
// when the runtime cannot say), asked once per device and size.
template <class Kernel>
int resident_clusters(Kernel kern, int threads, int smem, int size, int dev, std::atomic<int> (&cache)[64][9]) {
  std::atomic<int>* slot = dev >= 0 && dev < 64 ? &cache[dev][size] : nullptr;
  if (slot) {
    const int v = slot->load(std::memory_order_relaxed);
    if (v > 0) return v - 1;
  }
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)size, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = size;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return 0;
  if (slot) slot->store(n + 1, std::memory_order_relaxed);
  return n;
}

template <int BN, class O, bool SPLIT>
cudaError_t launch_tile(const Matmul8Args& a, const TilePlan& pl, int sms, int dev, cudaStream_t st) {
  using C = TileCfg<BN>;
  auto kern = tile_kernel<BN, O, SPLIT>;
  static DeviceFlags configured;
  cudaError_t e;
  if (!configured.done(dev)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) != cudaSuccess)
      return e;
    configured.set(dev);
  }
  unsigned int* err = device_error_word();
  if (!err) return cudaErrorInvalidDevicePointer;
  CUtensorMap tA, tB;
  if (!codes_tmap(&tA, a.A, a.M, a.K, a.lda, BM) || !codes_tmap(&tB, a.B, a.N, a.K, a.ldb, C::kBRows))
    return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)pl.tiles_m * pl.tiles_n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(SPLIT ? 2 * pl.split * tiles : 2 * std::min<int64_t>(tiles, sms / 2)), 1, 1);
  cfg.blockDim = dim3(kTileThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = SPLIT ? 2 * pl.split : 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, pl, tA, tB, err);
}

template <int BN, class O>
int resident_tiles(int split, int dev) {
  static std::atomic<int> cache[64][9];
  return resident_clusters(tile_kernel<BN, O, true>, kTileThreads, TileCfg<BN>::kSmem, 2 * split, dev, cache);
}
template <int NT, class O>
int resident_streams(int split, int dev) {
  static std::atomic<int> cache[64][9];
  return resident_clusters(stream_kernel<NT, O>, kStreamThreads, StreamCfg<NT>::kSmem, split, dev, cache);
}

// A form of the product and its modelled time in us.
enum FormKernel { kFew, kStream, kTile };
struct Form {
  FormKernel kernel;
  int width;     // few tokens and streamed: tokens per tile; pair tiles: their columns
  int split;
  float cost;
};

// How many clusters are resident at once: `given` for streams in clusters of 2, 4
// and 8 CTAs and pair tiles of 2, 3 and 4 pairs, or, null, what this device says.
template <int NT, class O>
int streams_at_once(int split, int dev, const int* given) {
  return given ? given[split == 2 ? 0 : split == 4 ? 1 : 2] : resident_streams<NT, O>(split, dev);
}
template <int BN, class O>
int tiles_at_once(int split, int dev, const int* given) {
  return given ? given[1 + split] : resident_tiles<BN, O>(split, dev);
}

// What every form moves at least, in us.
template <class O>
float memory_time(const Matmul8Args& a) {
  return ((float)a.N * (float)a.K + (float)a.M * (float)a.K + (float)a.M * (float)a.N * sizeof(typename O::elem)) * (1.0f / 6.5e6f);
}

// The streaming kernel.  A k-block costs 0.26 (16 to 64 tokens; with 64 1.15 times
// that where rows of 128 codes lie in two lines of memory) or 0.37 (128), 1.4 times
// that where SMs hold two CTAs; a launch 2.8 to 4 with its first loads and last step,
// a further wave 3 to 5.5 besides its k-blocks of 0.36 or 0.42; a split 0.8 for its
// cluster barriers and its sums' way between SMs at 3.5 MB per us.
template <int NT, class O>
void consider_streamed(const Matmul8Args& a, int sms, int dev, const int* given, Form& best) {
  constexpr float base = NT <= 32 ? 2.8f : NT == 64 ? 3.0f : 4.0f, wave = NT <= 32 ? 3.0f : NT == 64 ? 4.0f : 5.5f;
  const float lines = NT == 64 && (a.lda | a.ldb) % BK != 0 ? 1.15f : 1.0f;
  const float kb = lines * (NT <= 64 ? 0.26f : 0.37f), wave_kb = lines * (NT <= 64 ? 0.36f : 0.42f);
  const int64_t tiles = ((int64_t)a.N + kStreamRows - 1) / kStreamRows * (((int64_t)a.M + NT - 1) / NT);
  const int nk = (a.K + BK - 1) / BK;
  if (tiles > 0x7FFFFFFF / 8) return;
  for (int s = 1; s <= 8; s *= 2) {
    if (s > 1 && (nk < 2 * s || tiles * s > 2 * (int64_t)sms || tiles > streams_at_once<NT, O>(s, dev, given))) break;
    const int64_t ctas = tiles * s, waves = (ctas + 2 * sms - 1) / (2 * sms);
    const float per = (float)((nk + s - 1) / s);
    const float work = per * kb * (ctas > sms ? 1.4f : 1.0f) + (float)(waves - 1) * (wave + per * wave_kb);
    float cost = std::max(memory_time<O>(a), work) + base;
    if (s > 1) cost += 0.8f + (float)(ctas * NT * kStreamRows * 4 / s * (s - 1)) * (1.0f / 3.5e6f);
    if (cost < best.cost) best = Form{kStream, NT, s, cost};
  }
}

// The pair kernel.  A k-block costs 0.28 (256 x 128) or 0.30 (256 x 256), a launch
// 4.7 or 5.8, a split 1.75; whole tiles walk in rounds of SMs / 2, none of which is shorter
// than its epilogue: 1.75 or 3.1.  Clusters that are not all resident at once would
// cost a second round (256 x 4096 x 12288 in quarters 34 us, in thirds 20), so they
// are not considered.
template <int BN, class O>
void consider_tiled(const Matmul8Args& a, int sms, int dev, const int* given, Form& best) {
  constexpr float kb = BN == 256 ? 0.30f : 0.28f, base = BN == 256 ? 5.8f : 4.7f, epilogue = BN == 256 ? 3.1f : 1.75f;
  const int64_t tiles = (((int64_t)a.M + 2 * BM - 1) / (2 * BM)) * (((int64_t)a.N + BN - 1) / BN);
  const int nk = (a.K + BK - 1) / BK, pairs = sms / 2;
  for (int s = 1; s <= 4; ++s) {
    if (s > 1 && (nk < 2 * s || tiles * s > pairs)) break;
    if (s > 1 && tiles > tiles_at_once<BN, O>(s, dev, given)) continue;
    const int64_t rounds = s > 1 ? 1 : (tiles + pairs - 1) / pairs;
    const float per = (float)((nk + s - 1) / s) * kb;
    const float work = per + (float)(rounds - 1) * std::max(per, epilogue);
    const float cost = std::max(memory_time<O>(a), work) + base + (s > 1 ? 1.75f : 0.0f);
    if (cost < best.cost) best = Form{kTile, BN, s, cost};
  }
}

// The form with the least modelled time.  Over 186 sizes (9 to 8192 tokens, N 8 to
// 28672, K 16 to 16384) it is 2.3% above the best form measured on average, 21% at
// most but for one product of 10 channels; us measured: 16 tokens, 28672 x 4096
// streamed 22.1 (pair tiles 33); 64, 4096 x 4096 streamed in quarters 8.0 (11); 256,
// 1024 x 1024 streamed 5.1 (7.0); 333, 1013 x 2995 streamed 7.7 (9.3); 333, 4096 x
// 12288 pair tiles in halves 22.5 (streamed 27.5); 1000, 14336 x 4096 pair tiles 51
// (65); 7404, 18199 x 27 pair tiles 123 (180).
template <class O>
Form choose_form(const Matmul8Args& a, int sms, int dev, const int* given) {
  // Few tokens (us against the best streamed form).  Up to 8, with 52 MB of weights and
  // 8192 codes of k, or 16 MB and 16384, at most; 8 tokens: 4096 x 4096 5.1 (6.6), 12288 x
  // 4096 10.4 (12.4), 14336 x 4096 13.4 (13.2), 6144 x 8192 9.3 (12.9), 8192 x 8192 16.8
  // (14.5), 1024 x 16384 8.7 (9.0), 4096 x 12288 12.8 (11.4).  Up to 16, with 8192 codes and
  // every tile resident at once: 4096 x 4096 5.2 (6.7), 1024 x 1024 2.2 (4.0), 4736 x 8192
  // 8.8 (12.1), 14336 x 1024 6.4 (6.1).  Up to 32, with 4096 codes besides: 1024 x 1024 2.6
  // (4.3), 4096 x 4096 6.7 (6.9), 2048 x 8192 9.5 (7.5).
  const bool resident = a.N <= 2 * sms * kFewRows;
  if (a.M <= 8 && a.K <= 16384 && (int64_t)a.N * a.K <= (int64_t)(a.K <= 8192 ? 52 : 16) << 20) return Form{kFew, 8, 1, 0.0f};
  if (a.M <= 16 && a.K <= 8192 && resident) return Form{kFew, 16, 1, 0.0f};
  if (a.M <= 32 && a.K <= 4096 && resident) return Form{kFew, 32, 1, 0.0f};
  Form f{kTile, 0, 0, 1e30f};
  if (a.M <= 16) consider_streamed<16, O>(a, sms, dev, given, f);
  else if (a.M <= 32) consider_streamed<32, O>(a, sms, dev, given, f);
  else consider_streamed<64, O>(a, sms, dev, given, f);
  if (a.M > 64) consider_streamed<128, O>(a, sms, dev, given, f);
  consider_tiled<256, O>(a, sms, dev, given, f);
  consider_tiled<128, O>(a, sms, dev, given, f);
  return f;
}

template <class O>
cudaError_t launch_out(const Matmul8Args& a, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = device_sm_count(dev, &sms)) != cudaSuccess) return e;
  const Form f = choose_form<O>(a, sms, dev, nullptr);
  if (f.kernel == kFew) {
    if (f.width == 8) return launch_few<1, O>(a, sms, st);
    return f.width == 16 ? launch_few<2, O>(a, sms, st) : launch_few<4, O>(a, sms, st);
  }
  if (f.kernel == kStream) {
    switch (f.width) {
      case 16: return launch_stream<16, O>(a, f.split, dev, st);
      case 32: return launch_stream<32, O>(a, f.split, dev, st);
      case 64: return launch_stream<64, O>(a, f.split, dev, st);
      default: return launch_stream<128, O>(a, f.split, dev, st);
    }
  }
  const TilePlan pl{(int)(((int64_t)a.M + 2 * BM - 1) / (2 * BM)), (int)(((int64_t)a.N + f.width - 1) / f.width), f.split};
  if (f.width == 128) return f.split > 1 ? launch_tile<128, O, true>(a, pl, sms, dev, st) : launch_tile<128, O, false>(a, pl, sms, dev, st);
  return f.split > 1 ? launch_tile<256, O, true>(a, pl, sms, dev, st) : launch_tile<256, O, false>(a, pl, sms, dev, st);
}

}  // namespace

void plan_matmul8(const Matmul8Args& a, int dtype, int sms, int dev, const int* clusters, int out[3]) {
  const Form f = dtype == 0   ? choose_form<OutBf16>(a, sms, dev, clusters)
                 : dtype == 1 ? choose_form<OutFp16>(a, sms, dev, clusters)
                              : choose_form<OutFp32>(a, sms, dev, clusters);
  out[0] = (int)f.kernel;
  out[1] = f.width;
  out[2] = f.split;
}

cudaError_t launch_matmul8(const Matmul8Args& a, int dtype, cudaStream_t st) {
  if (dtype == 0) return launch_out<OutBf16>(a, st);
  if (dtype == 1) return launch_out<OutFp16>(a, st);
  return launch_out<OutFp32>(a, st);
}

}  // namespace w4a4
