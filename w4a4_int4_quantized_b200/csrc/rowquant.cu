// Row operators that end in int8 codes with one scale per row:
//   norm:  h = x + r,  y = (h / sqrt(mean(h^2) + eps)) gamma   (the residual's
//          addition and the root-mean-square norm before a projection)
//   silu:  y = (a / (1 + exp(-a))) b                           (the gate
//          between the two products of a gated MLP)
// then, per row and as in the rotate + quantize path: y <- H_g y per group of
// g (fp32 butterflies in the order h = 1, 2, 4, ...; g = 0: none), s =
// fl32(max |y| / 127), q = rint_half_even(y / s) with 1 / s within one rounding
// of fp32, codes 0 where s = 0.
//
// Everything between the loads and the codes is fp32 in registers: h is not
// rounded to the tensors' type before the norm (only the stored sum is), and
// y is not rounded before it is quantized.  A row that holds an infinity or a
// NaN, or whose y overflows, has the scale NaN and codes 0, so every value the
// codes stand for is NaN, as the formula gives.  A sum of squares that
// overflows fp32 on finite h (|h| past 1e18) is taken again with the row
// scaled by an exact power of two.
//
// Layout: a row belongs to `tpr` consecutive threads (a multiple of 32); chunk
// v * tpr + t of 8 consecutive elements to its thread t.  Rotation stages 1, 2
// and 4 stay in a thread, 8 .. g/2 are shuffles inside 8 or 16 lanes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "plan_cache.h"

#include <algorithm>

namespace w4a4 {

unsigned int* device_error_word();

namespace {

struct Bf16 {
  using word = uint16_t;
  static constexpr int kWords = 4;     // 32-bit words of 8 elements
  static __device__ __forceinline__ float one(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
  static __device__ __forceinline__ float2 two(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float2 f) {
    __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};
struct Fp16 {
  using word = uint16_t;
  static constexpr int kWords = 4;
  static __device__ __forceinline__ float one(uint16_t b) { return __half2float(__ushort_as_half(b)); }
  static __device__ __forceinline__ float2 two(uint32_t w) {
    return __half22float2(*reinterpret_cast<__half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float2 f) {
    __half2 h = __floats2half2_rn(f.x, f.y);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};
struct Fp32 {
  using word = uint32_t;
  static constexpr int kWords = 8;
  static __device__ __forceinline__ float one(uint32_t b) { return __uint_as_float(b); }
};

// Eight consecutive elements of a row, n of them inside it (the rest read as
// zero).  VEC: the address is 16-byte aligned and n is 8 or 0.
template <class T, bool VEC>
__device__ __forceinline__ void load8(const typename T::word* p, int n, float2 (&f)[4]) {
  if constexpr (VEC) {
    uint4 w[T::kWords / 4];
#pragma unroll
    for (int i = 0; i < T::kWords / 4; ++i)
      w[i] = n > 0 ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (T::kWords == 4) f[j] = T::two(u[j]);
      else f[j] = make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j].x = 2 * j < n ? T::one(p[2 * j]) : 0.0f;
      f[j].y = 2 * j + 1 < n ? T::one(p[2 * j + 1]) : 0.0f;
    }
  }
}

// Eight elements to a 16-byte aligned address where n > 0.
template <class T>
__device__ __forceinline__ void store8(typename T::word* p, int n, const float2 (&f)[4]) {
  if (n <= 0) return;
  uint32_t u[T::kWords];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (T::kWords == 4) {
      u[j] = T::pack(f[j]);
    } else {
      u[2 * j] = __float_as_uint(f[j].x);
      u[2 * j + 1] = __float_as_uint(f[j].y);
    }
  }
#pragma unroll
  for (int i = 0; i < T::kWords / 4; ++i)
    reinterpret_cast<uint4*>(p)[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
}

// The words of a window moved down by `bytes` (0 to 15, the same in the whole warp).
template <int IN, int OUT>
__device__ __forceinline__ void shift_words(const uint32_t (&w)[IN], uint32_t bytes, uint32_t (&out)[OUT]) {
  static_assert(IN >= OUT + 4, "a window of one 16-byte granule more");
  const uint32_t bits = (bytes & 3u) * 8u;
  switch (bytes >> 2) {
    case 0:
#pragma unroll
      for (int i = 0; i < OUT; ++i) out[i] = __funnelshift_r(w[i], w[i + 1], bits);
      break;
    case 1:
#pragma unroll
      for (int i = 0; i < OUT; ++i) out[i] = __funnelshift_r(w[i + 1], w[i + 2], bits);
      break;
    case 2:
#pragma unroll
      for (int i = 0; i < OUT; ++i) out[i] = __funnelshift_r(w[i + 2], w[i + 3], bits);
      break;
    default:
#pragma unroll
      for (int i = 0; i < OUT; ++i) out[i] = __funnelshift_r(w[i + 3], i + 4 < IN ? w[i + 4] : 0u, bits);
  }
}

// Eight consecutive elements at any element alignment, n of them inside the row,
// by the 16-byte granules that hold them, which bring up to 14 bytes of the row's
// neighbours along.  EDGE: rows near the operand's ends (lo, hi), where a granule
// that passes them is not read and the chunk goes element by element.
template <class T, bool EDGE>
__device__ __forceinline__ void load8_window(const typename T::word* p, int n, const void* lo, const void* hi,
                                             float2 (&f)[4]) {
  constexpr int NW = T::kWords;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uint32_t off = (uint32_t)(at & 15u);
  const int bytes = n > 0 ? (int)off + min(n, 8) * (int)sizeof(typename T::word) : 0;
  if (EDGE && n > 0 &&
      (at - off < reinterpret_cast<uintptr_t>(lo) || at - off + ((bytes + 15) & ~15) > reinterpret_cast<uintptr_t>(hi))) {
    load8<T, false>(p, n, f);
    return;
  }
  uint32_t w[NW + 4], u[NW];
#pragma unroll
  for (int i = 0; i < NW / 4 + 1; ++i) {
    const uint4 g = 16 * i < bytes ? reinterpret_cast<const uint4*>(at - off)[i] : make_uint4(0u, 0u, 0u, 0u);
    w[4 * i] = g.x;
    w[4 * i + 1] = g.y;
    w[4 * i + 2] = g.z;
    w[4 * i + 3] = g.w;
  }
  shift_words(w, off, u);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (NW == 4) f[j] = T::two(u[j]);
    else f[j] = make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
  }
  if (n < 8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (2 * j >= n) f[j].x = 0.0f;
      if (2 * j + 1 >= n) f[j].y = 0.0f;
    }
  }
}

// max(m, |a|, |b|) that keeps a NaN of any of them
__device__ __forceinline__ float max_abs(float m, float2 v) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(fabsf(v.x)), "f"(fabsf(v.y)));
  return d;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
// Largest of non-negative floats; the bits of a NaN rank above infinity's.
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v)));
}

// Sums and maxima over the warps of a row.  A buffer is not written again
// before another call's barrier, which every thread passes after it has read
// this one.
__device__ __forceinline__ float row_sum(float v, float* buf, int nwarps) {
  v = warp_sum(v);
  if (nwarps == 1) return v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  return warp_sum(lane < nwarps ? buf[lane] : 0.0f);
}
__device__ __forceinline__ float row_max(float v, float* buf, int nwarps) {
  v = warp_max(v);
  if (nwarps == 1) return v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  return warp_max(lane < nwarps ? buf[lane] : 0.0f);
}

// One thread's 8 elements through every stage of H_g, in the order h = 1, 2,
// 4 (in the thread), 8, 16, 32, 64 (lanes 1, 2, 4, 8 apart).  The lower index
// of a pair takes a + b, the upper a - b, formed as fma(b, -1, a).
__device__ __forceinline__ void rotate8(float2 (&f)[4], int group, int lane) {
  const float2 m1 = make_float2(-1.0f, -1.0f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = f[j].x, b = f[j].y;
    f[j] = make_float2(__fadd_rn(a, b), __fsub_rn(a, b));
  }
#pragma unroll
  for (int h = 1; h < 4; h <<= 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if ((j & h) == 0) {
        const float2 a = f[j], b = f[j + h];
        f[j] = __fadd2_rn(a, b);
        f[j + h] = __ffma2_rn(b, m1, a);
      }
    }
  }
  const int stages = group == 128 ? 4 : 3;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < stages) {
      const float sg = (lane >> k) & 1 ? -1.0f : 1.0f;
      const float2 s2 = make_float2(sg, sg);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 p;
        p.x = __shfl_xor_sync(0xFFFFFFFFu, f[j].x, 1 << k);
        p.y = __shfl_xor_sync(0xFFFFFFFFu, f[j].y, 1 << k);
        f[j] = __ffma2_rn(f[j], s2, p);
      }
    }
  }
}

// Codes of 8 elements: each times 1 / s (`inv`), rounded to the nearest integer
// by adding 1.5 * 2^23 in one fused operation.  inv is off by at most 1.01 * 2^-24
// of itself, so a quotient q within |q| * 1.01 * 2^-24 of a half may go to the
// other side; y itself is known no better than that.
__device__ __forceinline__ uint2 quantize8(const float2 (&f)[4], float inv) {
  const float2 mg = make_float2(kMagic, kMagic), iv = make_float2(inv, inv);
  uint32_t t[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = __ffma2_rn(f[j], iv, mg);
    t[2 * j] = __float_as_uint(a.x);
    t[2 * j + 1] = __float_as_uint(a.y);
  }
  return make_uint2(pack_bytes4(t[0], t[1], t[2], t[3]), pack_bytes4(t[4], t[5], t[6], t[7]));
}

// silu(a) b = a b / (1 + 2^(-a log2 e)).  With u = 2^-24: the exponent's two
// roundings put 1.5 |a| u into the power and ex2.approx 4 u, of which the share
// t / (1 + t) reaches the result (all of it for a far below 0, at most 0.3 |a| u
// above); 1 + t, rcp.approx and two products add 5 u.  For gates of -87 and above,
// where the power and its reciprocal stay in fp32's range.
__device__ __forceinline__ float2 silu_mul2(float2 a, float2 b) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float2 p = __fmul2_rn(a, make_float2(-kLog2e, -kLog2e));
  float2 t, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(p.x));   // a power flushed to 0 is lost in 1 + t anyway
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(p.y));
  const float2 d = __fadd2_rn(t, make_float2(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return __fmul2_rn(__fmul2_rn(a, r), b);
}

// How far into a row an element at e is: 8 or more where every chunk is whole.
template <bool FULL>
__device__ __forceinline__ int left(int K, int e) {
  return FULL ? 8 : K - e;
}

template <int VPT>
__device__ __forceinline__ float thread_max(const float2 (&f)[VPT][4]) {
  float m = 0.0f;
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max_abs(m, f[v][j]);
  return m;
}
template <int VPT>
__device__ __forceinline__ float thread_squares(const float2 (&f)[VPT][4]) {
  float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) s2 = __ffma2_rn(f[v][j], f[v][j], s2);
  return __fadd_rn(s2.x, s2.y);
}
template <int VPT>
__device__ __forceinline__ void scale_row(float2 (&f)[VPT][4], float k) {
  const float2 k2 = make_float2(k, k);
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) f[v][j] = __fmul2_rn(f[v][j], k2);
}

// 1 / sqrt(x): the hardware's estimate (2 ulp) and one Newton step
__device__ __forceinline__ float inv_sqrt(float x) {
  float r;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return fmaf(0.5f * r, fmaf(-x * r, r, 1.0f), r);
}

struct RowShared {
  float sum[32], max[2][32];
};

template <class T, int VPT, bool FULL>
__device__ __forceinline__ void store_sum(const float2 (&f)[VPT][4], const RowQuantArgs& p, int64_t row, int t,
                                          int tpr) {
  if (!p.H) return;
  auto* h = static_cast<typename T::word*>(p.H) + row * p.ldh;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int e = (v * tpr + t) * 8;
    store8<T>(h + e, left<FULL>(p.K, e), f[v]);
  }
}
template <class T, int VPT>
__device__ __forceinline__ void store_sum_elements(const float2 (&f)[VPT][4], const RowQuantArgs& p, int64_t row, int t,
                                                   int tpr) {
  if (!p.H) return;
  auto* h = static_cast<typename T::word*>(p.H) + row * p.ldh;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int e = (v * tpr + t) * 8, n = p.K - e;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t lo, hi;
      if constexpr (T::kWords == 4) {
        const uint32_t w = T::pack(f[v][j]);
        lo = w & 0xFFFFu;
        hi = w >> 16;
      } else {
        lo = __float_as_uint(f[v][j].x);
        hi = __float_as_uint(f[v][j].y);
      }
      if (2 * j < n) h[e + 2 * j] = (typename T::word)lo;
      if (2 * j + 1 < n) h[e + 2 * j + 1] = (typename T::word)hi;
    }
  }
}
template <int VPT>
__device__ __forceinline__ void rotate_row(float2 (&f)[VPT][4], int group) {
  if (group) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) rotate8(f[v], group, (int)threadIdx.x & 31);
  }
}
// Scale and codes of a row y in f whose max |y| is m.
template <int VPT, bool VEC, bool FULL>
__device__ __forceinline__ void quantize_row(float2 (&f)[VPT][4], const RowQuantArgs& p, int64_t row, int t, int tpr,
                                             float m) {
  const bool finite = m < __int_as_float(0x7F800000);
  const float s = finite ? __fdiv_rn(m, 127.0f) : __int_as_float(0x7FC00000);
  if (t == 0) p.x_scale[row] = s;
  // Codes are 0 in a row of zeros and in one whose scale is NaN.
  const bool some = s > 0.0f;
  const uint32_t keep = some ? 0xFFFFFFFFu : 0u;
  // The hardware's reciprocal (1 ulp, so codes next to a half by up to |q| 2^-23) and a
  // Newton step: r (1 + e) -> r (1 - e^2), then one rounding.  Per row and thread: norm
  // 16384 x 8192 bf16 157.1 -> 157.4 us, SiLU 8 x 14336 3.1 -> 3.2.
  const float div = some && s >= 0x1p-100f ? s : 1.0f;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(div));
  inv = fmaf(inv, fmaf(-div, inv, 1.0f), inv);
  if (some && s < 0x1p-100f) {     // too small for its reciprocal, and of few bits itself where it is subnormal
    scale_row(f, 0x1p80f);
    const float big = s * 0x1p80f, top = 127.0f * big;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f[v][j] = make_float2(fminf(fmaxf(f[v][j].x, -top), top), fminf(fmaxf(f[v][j].y, -top), top));
    inv = __frcp_rn(big);
  }
  int8_t* q = p.Xq + row * p.ldq;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int e = (v * tpr + t) * 8;
    const int n = left<FULL>(p.K, e);
    uint2 w = quantize8(f[v], inv);
    w.x &= keep;
    w.y &= keep;
    if (FULL || n >= 8) {
      *reinterpret_cast<uint2*>(q + e) = w;
    } else if (!VEC) {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < n) q[e + j] = (int8_t)((j < 4 ? w.x >> (8 * j) : w.y >> (8 * j - 32)) & 0xFFu);
    }
  }
}

__device__ __forceinline__ void times8(float2 (&f)[4], const float2 (&g)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = __fmul2_rn(f[j], g[j]);
}

// The norm of a row h in f, its rotation, scale and codes: a reduction for the
// sum of squares and one for max |y|, and two more with h scaled by a power of two
// where the squares pass fp32's range.  gamma(f) multiplies by the
// weights; taken() runs in every thread once all have their inputs in registers.
template <int VPT, bool VEC, bool FULL, class Gamma, class Taken>
__device__ __forceinline__ void norm_row(float2 (&f)[VPT][4], const RowQuantArgs& p, int64_t row, int t, int tpr,
                                         RowShared& sh, Gamma&& gamma, Taken&& taken) {
  const int nwarps = tpr >> 5;
  float eps = p.eps;
  float ss = row_sum(thread_squares(f), sh.sum, nwarps);
  taken();
  if (!(ss <= 3.4e38f)) {          // the same value in every thread of the row
    const float m = row_max(thread_max(f), sh.max[1], nwarps);
    // an infinity or a NaN stays one through all that follows
    const float k = m < __int_as_float(0x7F800000) ? exp2f(1.0f - (float)ilogbf(m)) : 1.0f;
    scale_row(f, k);
    ss = row_sum(thread_squares(f), sh.sum, nwarps);
    eps = eps * k * k;
  }
  scale_row(f, inv_sqrt(fmaf(ss, p.inv_k, eps)));
  if (p.gamma) gamma(f);
  rotate_row(f, p.group);
  const float m = row_max(thread_max(f), sh.max[0], nwarps);
  quantize_row<VPT, VEC, FULL>(f, p, row, t, tpr, m);
}

// The rotation, scale and codes of a row y in f: one reduction, so rows
// alternate between two buffers.
template <int VPT, bool VEC, bool FULL, class Taken>
__device__ __forceinline__ void plain_row(float2 (&f)[VPT][4], const RowQuantArgs& p, int64_t row, int t, int tpr,
                                          float* buf, Taken&& taken) {
  rotate_row(f, p.group);
  const float m = row_max(thread_max(f), buf, tpr >> 5);
  taken();
  quantize_row<VPT, VEC, FULL>(f, p, row, t, tpr, m);
}

// The weights of a thread's chunks, all loads before the first use.  VEC: aligned
// and whole; else whole chunks of aligned weights at once, so that no load waits
// behind a branch, and the rest element by element.
template <class T, int VPT, bool VEC>
__device__ __forceinline__ void load_gamma(const RowQuantArgs& p, int t, int tpr, float2 (&g)[VPT][4]) {
  const auto* w = static_cast<const typename T::word*>(p.gamma);
  const int whole = VEC || (reinterpret_cast<uintptr_t>(w) & 15u) == 0 ? p.K & ~7 : 0;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int e = (v * tpr + t) * 8;
    load8<T, true>(w + e, whole - e, g[v]);
  }
  if (!VEC && whole < p.K) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int e = (v * tpr + t) * 8;
      if (e >= whole && e < p.K) load8<T, false>(w + e, p.K - e, g[v]);
    }
  }
}

// A gate a < -87 and its b replaced by ones whose silu_mul2 is the same: there
// 1 + e^-a is e^-a to fp32's last bit, silu(a) b = a e^a b, and with v = e^(a / 4)
// (2 a v^2, b v^2) gives it, as silu(x) = x / 2 for |x| < 2^-54.  v twice on
// either side keeps every factor in range where the result is.  The exponent's
// two roundings put 1.22 |a| u into the result (1.5 |a| u bounds them above), four
// powers 16 u and the rest 11 u, together under (9 + 1.5 |a|) u from 87 on.
// The test for such gates costs SiLU 4096 x 28672 bf16 91.0 -> 93.6 us, 4608 x 12288 47.5 ->
// 48.4, the rest under 1%; counted as 0 they lost up to 1.2e-36 |b|.
constexpr float kDeepGate = -87.0f;
__device__ __forceinline__ void fold_deep_gate(float& a, float& b) {
  if (a < kDeepGate) {
    float v;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v) : "f"(a * (0.25f * 1.4426950408889634f)));
    a = 2.0f * ((a * v) * v);
    b = (b * v) * v;
  }
}

// The second operand into f: added (OP 0) or gated by it (OP 1).
template <int OP>
__device__ __forceinline__ void combine8(float2 (&f)[4], float2 (&g)[4]) {
  if constexpr (OP == 1) {
    float lo = 0.0f;                   // a NaN passes by: it goes through silu_mul2
#pragma unroll
    for (int j = 0; j < 4; ++j) lo = fminf(lo, fminf(f[j].x, f[j].y));
    if (lo < kDeepGate) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        fold_deep_gate(f[j].x, g[j].x);
        fold_deep_gate(f[j].y, g[j].y);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = OP == 0 ? __fadd2_rn(f[j], g[j]) : silu_mul2(f[j], g[j]);
}

// A row of the sum to global memory at any element alignment.  A whole chunk's
// thread writes the 16-byte granules that begin in it, filling the first with
// the end of the chunk before, which the lane below holds; what no such thread
// covers (the first bytes of a warp's first chunk, the last bytes before a warp
// or the row ends, a partial chunk) goes element by element.
template <class T, int VPT>
__device__ __forceinline__ void store_sum_shifted(const float2 (&f)[VPT][4], const RowQuantArgs& p, int64_t row, int t,
                                                  int tpr) {
  using W = typename T::word;
  constexpr int NW = T::kWords;
  if (!p.H) return;
  W* h = static_cast<W*>(p.H) + row * p.ldh;
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(h) & 15u);
  const int own = (int)((16u - off) / sizeof(W));       // elements of a chunk before its first granule begins
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int e = (v * tpr + t) * 8;
    const int n = p.K - e;
    uint32_t u[NW], w[NW + 4], g[NW];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (NW == 4) {
        u[j] = T::pack(f[v][j]);
      } else {
        u[2 * j] = __float_as_uint(f[v][j].x);
        u[2 * j + 1] = __float_as_uint(f[v][j].y);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __shfl_up_sync(0xFFFFFFFFu, u[NW - 4 + j], 1);
#pragma unroll
    for (int j = 0; j < NW; ++j) w[4 + j] = u[j];
    int lo = 0, hi = 0;                                  // elements [0, lo) and [hi, 8) are written one by one
    if (off == 0) {
      if (n >= 8) {
#pragma unroll
        for (int q = 0; q < NW / 4; ++q)
          reinterpret_cast<uint4*>(h + e)[q] = make_uint4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
        hi = 8;
      } else {
        lo = max(n, 0);
        hi = 8;
      }
    } else if (n < 8) {
      lo = max(n, 0);
      hi = 8;
    } else {
      // granules at h + e - off: the first holds the lane below's last `off` bytes
      shift_words(w, 16u - off, g);
      uint4* at = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(h + e) - off);
#pragma unroll
      for (int q = 0; q < NW / 4; ++q)
        if (q > 0 || lane > 0) at[q] = make_uint4(g[4 * q], g[4 * q + 1], g[4 * q + 2], g[4 * q + 3]);
      lo = lane > 0 ? 0 : own;
      hi = lane == 31 || n < 16 ? 8 - (int)(off / sizeof(W)) : 8;   // nobody's granule takes the end
    }
    if (lo > 0 || hi < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < lo || i >= hi) {
          if constexpr (NW == 4) h[e + i] = (W)((i & 1) ? u[i / 2] >> 16 : u[i / 2] & 0xFFFFu);
          else h[e + i] = u[i];
        }
    }
  }
}

// How the direct kernel reads and writes rows: at 16-byte alignment, by the
// granules around their chunks, or, rows of one warp, element by element (a SiLU of
// 8027 x 37 fp32 4.0 us, by granules 4.9; a norm of 16384 x 100 bf16 10.1 and 12.6;
// but 488 x 4993 18.2 and 10.5).
enum RowLoads { kAligned16, kWindows, kElements };

// OP 0: norm (A = x, B = residual or null, gamma, H or null); OP 1: silu (A =
// gate, B = up).  VPT: chunks of 8 per thread.  Rows straight from global
// memory: few or short rows, at any alignment, and rows whose inputs do not fit in
// shared memory.  One row per team of tpr threads, bound by the latency of its
// loads and two reductions: 1 x 4096 bf16 2.3 us, 517 x 2777 fp16 4.4 us.
template <class T, int OP, int VPT, int MAXT, RowLoads LOADS>
__global__ void __launch_bounds__(MAXT) row_quantize_kernel(RowQuantArgs p, int tpr) {
  using W = typename T::word;
  __shared__ RowShared sh;
  const int rpb = blockDim.x / tpr;            // > 1 only where a row is one warp
  const int t = threadIdx.x % tpr;
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr;
  if (row >= p.M) return;
  const W* a = static_cast<const W*>(p.A) + row * p.lda;
  const W* b = p.B ? static_cast<const W*>(p.B) + row * p.ldb : nullptr;
  float2 f[VPT][4];
  auto load = [&](auto read) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int e = (v * tpr + t) * 8;
      read(a + e, p.K - e, p.A, p.lda, f[v]);
    }
    if (b) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int e = (v * tpr + t) * 8;
        float2 g[4];
        read(b + e, p.K - e, p.B, p.ldb, g);
        combine8<OP>(f[v], g);
      }
    }
  };
  if constexpr (LOADS == kAligned16) {
    load([](const W* x, int n, const void*, int64_t, float2 (&y)[4]) { load8<T, true>(x, n, y); });
  } else if constexpr (LOADS == kElements) {
    load([](const W* x, int n, const void*, int64_t, float2 (&y)[4]) { load8<T, false>(x, n, y); });
  } else if (row > 0 && row < p.M - 1) {
    load([](const W* x, int n, const void*, int64_t, float2 (&y)[4]) { load8_window<T, false>(x, n, nullptr, nullptr, y); });
  } else {
    load([&](const W* x, int n, const void* lo, int64_t ld, float2 (&y)[4]) {
      load8_window<T, true>(x, n, lo, static_cast<const W*>(lo) + (int64_t)(p.M - 1) * ld + p.K, y);
    });
  }
  if constexpr (OP == 1) {
    plain_row<VPT, LOADS == kAligned16, false>(f, p, row, t, tpr, sh.max[0], [] {});
  } else {
    if constexpr (LOADS == kAligned16) store_sum<T, VPT, false>(f, p, row, t, tpr);
    else if constexpr (LOADS == kWindows) store_sum_shifted<T, VPT>(f, p, row, t, tpr);
    else store_sum_elements<T, VPT>(f, p, row, t, tpr);
    norm_row<VPT, LOADS == kAligned16, false>(
        f, p, row, t, tpr, sh,
        [&](float2 (&y)[VPT][4]) {
          float2 g[VPT][4];
          load_gamma<T, VPT, LOADS == kAligned16>(p, t, tpr, g);
#pragma unroll
          for (int v = 0; v < VPT; ++v) times8(y[v], g[v]);
        },
        [] {});
  }
}

// Bytes of a contiguous row into shared memory, completing on a barrier (16-byte
// aligned addresses and sizes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// 8 elements from shared memory (16-byte aligned), zeros where n <= 0.
template <class T>
__device__ __forceinline__ void smem8(uint32_t addr, int n, float2 (&f)[4]) {
  uint32_t u[T::kWords];
#pragma unroll
  for (int i = 0; i < T::kWords / 4; ++i) {
    u[4 * i] = u[4 * i + 1] = u[4 * i + 2] = u[4 * i + 3] = 0u;
    if (n > 0)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(u[4 * i]), "=r"(u[4 * i + 1]), "=r"(u[4 * i + 2]), "=r"(u[4 * i + 3])
                   : "r"(addr + 16 * i));
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (T::kWords == 4) f[j] = T::two(u[j]);
    else f[j] = make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
  }
}

// How the rows of a ring lie: every thread has whole chunks (kWhole), the last
// threads may have none (kAligned), or rows start off the 16-byte alignment or
// end inside a chunk (kShifted).
enum RowLayout { kWhole, kAligned, kShifted };

// The first n of 8 elements whose row begins `off` bytes into a 16-byte granule
// of shared memory; the rest are zero.  at: the granule that the first one lies
// in once `off` is added (the same `off` for every chunk of a row).
template <class T>
__device__ __forceinline__ void smem8_shifted(uint32_t at, uint32_t off, int n, float2 (&f)[4]) {
  constexpr int NW = T::kWords;
  uint32_t w[NW + 4], u[NW];
#pragma unroll
  for (int i = 0; i < NW / 4 + 1; ++i) {
    w[4 * i] = w[4 * i + 1] = w[4 * i + 2] = w[4 * i + 3] = 0u;
    if (n > 0)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "r"(at + 16 * i));
  }
  shift_words(w, off, u);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (NW == 4) f[j] = T::two(u[j]);
    else f[j] = make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
  }
  if (n < 8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (2 * j >= n) f[j].x = 0.0f;
      if (2 * j + 1 >= n) f[j].y = 0.0f;
    }
  }
}

// Where an operand's row lies in its slot of a stage: the bytes from the 16-byte
// granule of its first element to that of its last.
struct RowSpan {
  const uint8_t* from;
  uint32_t off, bytes;
};
__device__ __forceinline__ RowSpan row_span(const void* row, uint32_t row_bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(row);
  const uint32_t off = (uint32_t)(a & 15u);
  return RowSpan{reinterpret_cast<const uint8_t*>(a - off), off, (off + row_bytes + 15u) & ~15u};
}
// A slot holds any such span and the granule past it that a window may touch.
__host__ __device__ __forceinline__ uint32_t slot_bytes(uint32_t row_bytes, bool shifted) {
  return shifted ? ((row_bytes + 15u) & ~15u) + 32u : row_bytes;
}

// Many rows: persistent blocks, each row's inputs brought into a ring of
// `stages` rows in shared memory by bulk copies, so that the next rows arrive
// while one is worked on and no register holds a load in flight.  A team of tpr
// threads owns a ring; with rows of one warp a block has several.  Long rows run at
// HBM's rate: 16384 x 8192 bf16 norm with residual 157 us, 6.0 TB/s (91% of the copy
// rate); 4608 x 12288 bf16 gate 48 us, 5.9 TB/s.  The others are bound by latency, with
// a third of the warps resident and issue slots 46 to 59% active: 19 instructions per
// element of a norm (loads and the two reductions' barriers wait), 29 with the rotation
// (its shuffles), 14 and 23 of a gate (64 us rotated); and by the last round: 4608 rows
// over 888 rings are 5.2 rounds, run as 6.  kShifted
// copies whole 16-byte granules, so a row brings up to 14 bytes of its
// neighbours along; the first and the last row, which have none on one side,
// are read from global memory element by element.
constexpr int kRingStages = 4, kRingTeams = 4;
constexpr int kRingThreads = 768;          // threads of an SM (1024 where rows are too wide for fewer)

template <class T, int OP, int VPT, int MAXT, RowLayout LAY>
__global__ void __launch_bounds__(MAXT, MAXT < kRingThreads ? kRingThreads / MAXT : 1)
    row_ring_kernel(RowQuantArgs p, int tpr, int stages, unsigned int* err) {
  using W = typename T::word;
  constexpr bool FULL = LAY == kWhole;
  // The weights of a thread's elements are loaded once and held packed.  They do not all
  // fit beside the row in the 80 registers that 768 threads leave: bf16 rows of four
  // chunks spill 156 bytes a thread to the stack, fp16 56 (27 of the 158 row kernels spill).
  constexpr bool kHoldGamma = OP == 0 && T::kWords == 4 && MAXT < 1024 && LAY != kShifted;
  extern __shared__ __align__(128) uint8_t ring_raw[];
  __shared__ RowShared sh;
  __shared__ __align__(8) uint64_t full[kRingTeams][kRingStages];
  const int rpb = blockDim.x / tpr;
  const int team = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const uint32_t row_bytes = (uint32_t)p.K * sizeof(W);
  const uint32_t slot = slot_bytes(row_bytes, LAY == kShifted);
  const uint32_t stage_bytes = p.B ? 2 * slot : slot;
  const uint32_t ring = smem_u32(ring_raw) + (uint32_t)(team * stages) * stage_bytes;
  const int64_t row0 = (int64_t)blockIdx.x * rpb + team, step = (int64_t)gridDim.x * rpb;
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[team][s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  auto a_row = [&](int64_t row) { return static_cast<const W*>(p.A) + row * p.lda; };
  auto b_row = [&](int64_t row) { return static_cast<const W*>(p.B) + row * p.ldb; };
  auto at_end = [&](int64_t row) { return LAY == kShifted && (row == 0 || row == p.M - 1); };
  auto issue = [&](int64_t row, int s) {
    if (at_end(row)) {
      mbar_arrive(&full[team][s]);
      return;
    }
    const uint32_t dst = ring + (uint32_t)s * stage_bytes;
    if constexpr (LAY == kShifted) {
      const RowSpan a = row_span(a_row(row), row_bytes), b = row_span(p.B ? b_row(row) : a_row(row), row_bytes);
      mbar_arrive_expect_tx(&full[team][s], a.bytes + (p.B ? b.bytes : 0u));
      bulk_load(dst, a.from, a.bytes, &full[team][s]);
      if (p.B) bulk_load(dst + slot, b.from, b.bytes, &full[team][s]);
    } else {
      mbar_arrive_expect_tx(&full[team][s], stage_bytes);
      bulk_load(dst, a_row(row), row_bytes, &full[team][s]);
      if (p.B) bulk_load(dst + slot, b_row(row), row_bytes, &full[team][s]);
    }
  };
  if (t == 0)
    for (int s = 0; s < stages; ++s)
      if (row0 + s * step < p.M) issue(row0 + s * step, s);
  uint4 gw[kHoldGamma ? VPT : 1];
  if (kHoldGamma && p.gamma) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int e = (v * tpr + t) * 8;
      gw[v] = left<FULL>(p.K, e) > 0 ? *reinterpret_cast<const uint4*>(static_cast<const W*>(p.gamma) + e)
                                     : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  int s = 0, parity = 0;
  uint32_t ph = 0;
  for (int64_t row = row0; row < p.M; row += step, parity ^= 1) {
    if (!mbar_wait(&full[team][s], ph)) set_device_error(err, kDevErrTimeoutFull);
    const uint32_t src = ring + (uint32_t)s * stage_bytes;
    float2 f[VPT][4];
    const bool direct = at_end(row);
    const uint32_t oa = LAY == kShifted ? (uint32_t)(reinterpret_cast<uintptr_t>(a_row(row)) & 15u) : 0u;
    const uint32_t ob = LAY == kShifted && p.B ? (uint32_t)(reinterpret_cast<uintptr_t>(b_row(row)) & 15u) : 0u;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int e = (v * tpr + t) * 8;
      const int n = left<FULL>(p.K, e);
      const uint32_t at = src + (uint32_t)(e * sizeof(W));
      float2 g[4];
      if constexpr (LAY == kShifted) {
        if (direct) {
          load8<T, false>(a_row(row) + e, n, f[v]);
          if (p.B) load8<T, false>(b_row(row) + e, n, g);
        } else {
          smem8_shifted<T>(at, oa, n, f[v]);
          if (p.B) smem8_shifted<T>(at + slot, ob, n, g);
        }
      } else {
        smem8<T>(at, n, f[v]);
        if (p.B) smem8<T>(at + slot, n, g);
      }
      if (p.B) combine8<OP>(f[v], g);
    }
    // the row's sum or maximum depends on everything that its threads read
    // here, so once it is known the stage takes the row after next
    auto taken = [&] {
      if (t == 0 && row + stages * step < p.M) {
        fence_proxy_async_smem();
        issue(row + stages * step, s);
      }
    };
    if constexpr (OP == 1) {
      plain_row<VPT, LAY != kShifted, FULL>(f, p, row, t, tpr, sh.max[parity], taken);
    } else {
      if constexpr (LAY == kShifted) store_sum_shifted<T, VPT>(f, p, row, t, tpr);
      else store_sum<T, VPT, FULL>(f, p, row, t, tpr);
      norm_row<VPT, LAY != kShifted, FULL>(
          f, p, row, t, tpr, sh,
          [&](float2 (&y)[VPT][4]) {
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
              float2 g[4];
              if constexpr (kHoldGamma) {
                g[0] = T::two(gw[v].x);
                g[1] = T::two(gw[v].y);
                g[2] = T::two(gw[v].z);
                g[3] = T::two(gw[v].w);
              } else {
                const int e = (v * tpr + t) * 8;
                const W* w = static_cast<const W*>(p.gamma) + e;
                const int n = left<FULL>(p.K, e);
                if (LAY != kShifted || (n >= 8 && (reinterpret_cast<uintptr_t>(p.gamma) & 15u) == 0)) load8<T, true>(w, n, g);
                else load8<T, false>(w, n, g);
              }
              times8(y[v], g);
            }
          },
          taken);
    }
    if (++s == stages) {
      s = 0;
      ph ^= 1u;
    }
  }
}

// ------------------------------------------------------------------ host side
template <class Kernel, class... Args>
cudaError_t launch_rows(Kernel kern, int64_t grid, int threads, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(grid < 0x7FFFFFFF ? grid : 0x7FFFFFFF), 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

int threads_per_row(int chunks, int vpt) { return ((chunks + vpt - 1) / vpt + 31) / 32 * 32; }

// What a launch is chosen by.
struct RowShape {
  int M, K, op;
  size_t es;         // bytes of an element
  bool second;       // a residual, or up
  bool vec;          // rows and weights 16-byte aligned, K a multiple of 8
};
struct RowPlan {
  bool ring;
  int form;          // RowLayout of a ring, RowLoads of the direct kernel
  int vpt, tpr, rpb; // chunks per thread, threads per row, rows (or rings) per block
  int stages, per_sm;
};

// Chunks per thread of the direct kernel: one, the shortest chain, where there are
// at most two rows per SM or every row is resident at once, else two (norm of 600 x
// 768 bf16 2.7 us with one, 2.9 with two; off the alignment 3.3 and 4.4; 600 x 4096
// 7.5 and 5.6; 900 x 5120 gated 6.8 with two, 7.5 with four), four where one warp then
// has a row (2000 x 768 4.5 us, with two 4.9) or 1024 threads cannot hold it in two.
RowPlan plan_direct(const RowShape& r, int sms) {
  const int chunks = (r.K + 7) / 8;
  int vpt = r.M <= 2 * sms || (int64_t)r.M * threads_per_row(chunks, 1) <= (int64_t)1024 * sms ? 1 : r.vec && chunks <= 128 ? 4 : 2;
  while (vpt < 4 && (chunks + vpt - 1) / vpt > 1024) vpt *= 2;
  while (vpt > 1 && chunks <= 32 * (vpt / 2)) vpt /= 2;
  const int tpr = threads_per_row(chunks, vpt);
  const int form = r.vec ? kAligned16 : tpr == 32 ? kElements : kWindows;
  return RowPlan{false, form, vpt, tpr, tpr == 32 ? 4 : 1, 0, 0};
}

// An SM's shared memory for rings: 228 KB less 2 KB for each block (the runtime's
// share and the static variables).
constexpr int kSmemSm = 228 * 1024, kSmemBlock = 2 * 1024;
constexpr int kRingMax = 224 * 1024;

// Threads per row, rings and their depth for rows of `stage` bytes.  Four chunks
// per thread (its share of the two reductions is some 120 instructions), fewer
// where the rings that fit an SM's memory would then leave it under 512 threads
// (norm of 8192 x 5120 fp32 96 us with 320 threads, 91 with 640) or where more than 384
// threads hold four each in 64 registers (4096 x 16384 bf16 111 us, with two 81).
bool plan_ring(int K, size_t stage, RowPlan& pl) {
  const int chunks = (K + 7) / 8;
  int most = 0;
  for (int vpt = chunks <= 32 ? 1 : chunks <= 64 ? 2 : 4; vpt >= 1; vpt /= 2) {
    const int tpr = threads_per_row(chunks, vpt);
    if (tpr > 1024) break;
    if (vpt == 4 && tpr > 384 && chunks <= 2 * 1024) continue;
    const int rpb = tpr == 32 ? kRingTeams : 1;
    const int per_sm =
        (int)std::min<size_t>(kSmemSm / (2 * stage * rpb + kSmemBlock), std::max(1, kRingThreads / (tpr * rpb)));
    if (per_sm < 1 || 2 * stage * rpb > kRingMax) break;
    if (per_sm * tpr * rpb > most) {
      most = per_sm * tpr * rpb;
      const size_t room = std::min<size_t>(kSmemSm / per_sm - kSmemBlock, kRingMax);
      pl = RowPlan{true, 0, vpt, tpr, rpb, (int)std::min<size_t>(kRingStages, room / (stage * rpb)), per_sm};
    }
    if (most >= 512) break;
  }
  return most > 0;
}

size_t stage_bytes(const RowShape& r) { return slot_bytes((uint32_t)(r.K * r.es), !r.vec) * (r.second ? 2 : 1); }

// The ring pays where rows are long or many; us direct, ring.  Aligned: norm of 1200
// x 4096 bf16 9.4, 11.1, of 3000 x 4096 19.2, 20.1, of 4608 x 4096 31, 27, of 2000 x 8192
// 29.6, 26.0; SiLU of 2000 x 5120 12.7, 15.1, of 600 x 14336 15.7, 12.4.  Off the
// alignment, where the stored sum costs the ring more registers than it saves:
// norm of 1200 x 8195 28, 35, of 8192 x 4099 80, 95, of 13340 x 5222 168, 163, of 1623 x
// 14470 69, 55, without a residual of 16384 x 1030 fp32 36, 48, of 16384 x 5003 124, 101;
// SiLU, which stores none, of 1021 x 5461 fp32 18.0, 13.2, of 1500 x 6001
// 17.9, 16.5.  At most two rows per SM go direct; rows under 16 bytes have no granule
// of their own to copy.
RowPlan plan_rows(const RowShape& r, int sms) {
  const size_t slot = slot_bytes((uint32_t)(r.K * r.es), !r.vec), stage = stage_bytes(r);
  const bool much = !r.vec && r.op == 0 ? slot >= 24u * 1024u || (size_t)r.M * slot >= (size_t)80 << 20
                                        : stage >= 24u * 1024u || (size_t)r.M * stage >= (size_t)(r.vec ? 64 : 32) << 20;
  RowPlan pl;
  if (r.M <= 2 * sms || !much || r.K * r.es < 16 || !plan_ring(r.K, stage, pl)) return plan_direct(r, sms);
  pl.form = !r.vec ? kShifted : r.K == 8 * pl.vpt * pl.tpr ? kWhole : kAligned;
  return pl;
}

// Rows of one warp, four to a block.
template <class T, int OP, RowLoads LOADS>
cudaError_t launch_warp_rows(const RowQuantArgs& a, const RowPlan& pl, cudaStream_t st) {
  const int64_t blocks = ((int64_t)a.M + 3) / 4;
  if (pl.vpt == 1) return launch_rows(row_quantize_kernel<T, OP, 1, 128, LOADS>, blocks, 128, 0, st, a, 32);
  if (pl.vpt == 2) return launch_rows(row_quantize_kernel<T, OP, 2, 128, LOADS>, blocks, 128, 0, st, a, 32);
  if constexpr (LOADS == kAligned16) return launch_rows(row_quantize_kernel<T, OP, 4, 128, LOADS>, blocks, 128, 0, st, a, 32);
  else return cudaErrorInvalidConfiguration;           // plan_direct: four chunks in one warp only where aligned
}
template <class T, int OP, RowLoads LOADS>
cudaError_t launch_block_rows(const RowQuantArgs& a, const RowPlan& pl, cudaStream_t st) {
  if (pl.vpt == 1) return launch_rows(row_quantize_kernel<T, OP, 1, 1024, LOADS>, a.M, pl.tpr, 0, st, a, pl.tpr);
  if (pl.vpt == 2) return launch_rows(row_quantize_kernel<T, OP, 2, 1024, LOADS>, a.M, pl.tpr, 0, st, a, pl.tpr);
  return launch_rows(row_quantize_kernel<T, OP, 4, 1024, LOADS>, a.M, pl.tpr, 0, st, a, pl.tpr);
}

template <class T, int OP, int VPT, int MAXT, RowLayout LAY>
cudaError_t launch_ring_t(const RowQuantArgs& a, const RowPlan& pl, size_t stage, int sms, int dev, cudaStream_t st) {
  auto kern = row_ring_kernel<T, OP, VPT, MAXT, LAY>;
  static DeviceFlags configured;
  cudaError_t e;
  if (!configured.done(dev)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingMax)) != cudaSuccess) return e;
    configured.set(dev);
  }
  unsigned int* err = device_error_word();
  if (!err) return cudaErrorInvalidDevicePointer;
  const int64_t teams = ((int64_t)a.M + pl.rpb - 1) / pl.rpb;
  return launch_rows(kern, std::min<int64_t>(teams, (int64_t)sms * pl.per_sm), pl.tpr * pl.rpb,
                     stage * pl.rpb * pl.stages, st, a, pl.tpr, pl.stages, err);
}

template <class T, int OP, int VPT, int MAXT>
cudaError_t launch_ring(const RowQuantArgs& a, const RowPlan& pl, size_t stage, int sms, int dev, cudaStream_t st) {
  if (pl.form == kShifted) return launch_ring_t<T, OP, VPT, MAXT, kShifted>(a, pl, stage, sms, dev, st);
  if (pl.form == kWhole) {
    if constexpr (T::kWords == 8 && OP == 1 && VPT == 4) return cudaErrorInvalidConfiguration;   // see launch_op
    else return launch_ring_t<T, OP, VPT, MAXT, kWhole>(a, pl, stage, sms, dev, st);
  }
  return launch_ring_t<T, OP, VPT, MAXT, kAligned>(a, pl, stage, sms, dev, st);
}

template <class T, int OP>
cudaError_t launch_op(const RowQuantArgs& a, cudaStream_t st) {
  const size_t es = sizeof(typename T::word);
  auto rows16 = [&](const void* p, int64_t ld) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (a.M == 1 || (uint64_t)ld * es % 16 == 0));
  };
  const bool vec = a.K % 8 == 0 && rows16(a.A, a.lda) && rows16(a.B, a.ldb) && rows16(a.H, a.ldh) && rows16(a.gamma, 0);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = device_sm_count(dev, &sms)) != cudaSuccess) return e;
  const RowShape shape{a.M, a.K, OP, es, a.B != nullptr, vec};
  const RowPlan pl = plan_rows(shape, sms);
  if (!pl.ring) {
    if (pl.tpr == 32) return vec ? launch_warp_rows<T, OP, kAligned16>(a, pl, st) : launch_warp_rows<T, OP, kElements>(a, pl, st);
    return vec ? launch_block_rows<T, OP, kAligned16>(a, pl, st) : launch_block_rows<T, OP, kWindows>(a, pl, st);
  }
  const size_t stage = stage_bytes(shape);
  // What plan_ring gives: one chunk for more than 384 threads only in fp32, where the
  // rings of two inputs leave an SM too few threads with more; and four only up to
  // 384 threads and never whole where two fp32 rows are in a stage.
  constexpr bool kWide = T::kWords == 8, kTwoWide = kWide && OP == 1;
  if (pl.vpt == 1 && pl.tpr <= 384) return launch_ring<T, OP, 1, 384>(a, pl, stage, sms, dev, st);
  if constexpr (kWide)
    if (pl.vpt == 1) return launch_ring<T, OP, 1, 1024>(a, pl, stage, sms, dev, st);
  if (pl.vpt == 2 && pl.tpr <= 384) return launch_ring<T, OP, 2, 384>(a, pl, stage, sms, dev, st);
  if (pl.vpt == 2) return launch_ring<T, OP, 2, 1024>(a, pl, stage, sms, dev, st);
  if (pl.vpt == 4 && pl.tpr <= 384) return launch_ring<T, OP, 4, 384>(a, pl, stage, sms, dev, st);
  if constexpr (!kTwoWide)
    if (pl.vpt == 4) return launch_ring<T, OP, 4, 1024>(a, pl, stage, sms, dev, st);
  return cudaErrorInvalidConfiguration;
}

template <class T>
cudaError_t launch_type(const RowQuantArgs& a, bool silu, cudaStream_t st) {
  return silu ? launch_op<T, 1>(a, st) : launch_op<T, 0>(a, st);
}

}  // namespace

void plan_row_quantize(bool silu, bool second, bool aligned, int dtype, int M, int K, int sms, int out[5]) {
  const RowPlan pl = plan_rows(RowShape{M, K, silu ? 1 : 0, dtype == 2 ? 4u : 2u, second, aligned && K % 8 == 0}, sms);
  out[0] = pl.ring ? 3 + pl.form : pl.form;
  out[1] = pl.vpt;
  out[2] = pl.tpr;
  out[3] = pl.rpb;
  out[4] = pl.stages;
}

cudaError_t launch_row_quantize(const RowQuantArgs& a, bool silu, int dtype, cudaStream_t st) {
  if (dtype == 0) return launch_type<Bf16>(a, silu, st);
  if (dtype == 1) return launch_type<Fp16>(a, silu, st);
  return launch_type<Fp32>(a, silu, st);
}

}  // namespace w4a4
