// Row operators that end in int8 codes with one scale per row:
//   norm:  h = x + r,  y = (h / sqrt(mean(h^2) + eps)) gamma   (the residual's
//          addition and the root-mean-square norm before a projection)
//   silu:  y = (a / (1 + exp(-a))) b                           (the gate
//          between the two products of a gated MLP)
// then, per row and as in the rotate + quantize path: y <- H_g y per group of
// g (fp32 butterflies in the order h = 1, 2, 4, ...; g = 0: none), s =
// fl32(max |y| / 127), q = rint_half_even(fl32(y / s)), codes 0 where s = 0.
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

namespace w4a4 {

namespace {

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23

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

template <class T, bool VEC>
__device__ __forceinline__ void store8(typename T::word* p, int n, const float2 (&f)[4]) {
  if constexpr (VEC) {
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
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t lo, hi;
      if constexpr (T::kWords == 4) {
        const uint32_t w = T::pack(f[j]);
        lo = w & 0xFFFFu;
        hi = w >> 16;
      } else {
        lo = __float_as_uint(f[j].x);
        hi = __float_as_uint(f[j].y);
      }
      if (2 * j < n) p[2 * j] = (typename T::word)lo;
      if (2 * j + 1 < n) p[2 * j + 1] = (typename T::word)hi;
    }
  }
}

// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
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

// Sums and maxima over the warps of a row.  Each call has its own buffer of
// 32 floats: a buffer is written again only after another call's barrier,
// which every thread passes after it has read the first one.
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

__device__ __forceinline__ uint32_t pack_bytes4(uint32_t t0, uint32_t t1, uint32_t t2, uint32_t t3) {
  return __byte_perm(__byte_perm(t0, t1, 0x0040), __byte_perm(t2, t3, 0x0040), 0x5410);
}

// Codes of 8 elements.  Both ends of a bracket around 1 / s (2^-20 wide on
// each side) rounding to one integer prove that the IEEE quotient rounds to it
// too; otherwise, or where s is too small for its reciprocal, the quotient is
// taken.
__device__ __forceinline__ uint2 quantize8(const float2 (&f)[4], float s, float inv_lo, float inv_hi, bool exact) {
  const float2 mg = make_float2(kMagic, kMagic), ih = make_float2(inv_hi, inv_hi), il = make_float2(inv_lo, inv_lo);
  uint32_t t[8], bad = exact ? 1u : 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = __ffma2_rn(f[j], ih, mg), b = __ffma2_rn(f[j], il, mg);
    t[2 * j] = __float_as_uint(a.x);
    t[2 * j + 1] = __float_as_uint(a.y);
    bad |= (t[2 * j] ^ __float_as_uint(b.x)) | (t[2 * j + 1] ^ __float_as_uint(b.y));
  }
  if (bad) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t[2 * j] = (uint32_t)min(max(__float2int_rn(__fdiv_rn(f[j].x, s)), -127), 127);
      t[2 * j + 1] = (uint32_t)min(max(__float2int_rn(__fdiv_rn(f[j].y, s)), -127), 127);
    }
  }
  return make_uint2(pack_bytes4(t[0], t[1], t[2], t[3]), pack_bytes4(t[4], t[5], t[6], t[7]));
}

// silu(a) b with t = exp(-|a|) <= 1, so that neither side overflows before
// the result does.
__device__ __forceinline__ float silu_mul(float a, float b) {
  const float t = expf(-fabsf(a));
  return __fmul_rn(__fdividef(a >= 0.0f ? a : a * t, 1.0f + t), b);
}

// OP 0: norm (A = x, B = residual or null, gamma, H or null); OP 1: silu (A =
// gate, B = up).  VPT: chunks of 8 per thread; MAXT: most threads of a block.
template <class T, int OP, int VPT, int MAXT, bool VEC>
__global__ void __launch_bounds__(MAXT) row_quantize_kernel(RowQuantArgs p, int tpr) {
  using W = typename T::word;
  __shared__ float red[3][32];
  const int rpb = blockDim.x / tpr;            // > 1 only where a row is one warp
  const int nwarps = tpr >> 5;
  const int t = threadIdx.x % tpr;
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  for (int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr; row < p.M; row += (int64_t)gridDim.x * rpb) {
    const W* a = static_cast<const W*>(p.A) + row * p.lda;
    const W* b = p.B ? static_cast<const W*>(p.B) + row * p.ldb : nullptr;
    float2 f[VPT][4];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int e = (v * tpr + t) * 8;
      load8<T, VEC>(a + e, p.K - e, f[v]);
    }
    if (b) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int e = (v * tpr + t) * 8;
        float2 g[4];
        load8<T, VEC>(b + e, p.K - e, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (OP == 0) f[v][j] = __fadd2_rn(f[v][j], g[j]);
          else f[v][j] = make_float2(silu_mul(f[v][j].x, g[j].x), silu_mul(f[v][j].y, g[j].y));
        }
      }
    }
    if (OP == 0) {
      if (p.H) {
        W* h = static_cast<W*>(p.H) + row * p.ldh;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const int e = (v * tpr + t) * 8;
          store8<T, VEC>(h + e, p.K - e, f[v]);
        }
      }
      float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2 = __ffma2_rn(f[v][j], f[v][j], s2);
      float ss = row_sum(__fadd_rn(s2.x, s2.y), red[0], nwarps);
      float eps = p.eps;
      if (!(ss <= 3.4e38f)) {   // the same value in every thread of the row
        float m = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
          for (int j = 0; j < 4; ++j) m = max_nan(m, max_nan(fabsf(f[v][j].x), fabsf(f[v][j].y)));
        m = row_max(m, red[2], nwarps);
        // an infinity or a NaN stays one through all that follows
        const float k = m < __int_as_float(0x7F800000) ? exp2f(1.0f - (float)ilogbf(m)) : 1.0f;
        s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[v][j].x *= k;
            f[v][j].y *= k;
            s2 = __ffma2_rn(f[v][j], f[v][j], s2);
          }
        ss = row_sum(__fadd_rn(s2.x, s2.y), red[0], nwarps);
        eps = eps * k * k;
      }
      const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)p.K), eps)));
      const float2 r2 = make_float2(r, r);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int e = (v * tpr + t) * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j) f[v][j] = __fmul2_rn(f[v][j], r2);
        if (p.gamma) {
          float2 g[4];
          load8<T, VEC>(static_cast<const W*>(p.gamma) + e, p.K - e, g);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[v][j] = __fmul2_rn(f[v][j], g[j]);
        }
      }
    }
    if (p.group) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) rotate8(f[v], p.group, lane);
    }
    float m = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max_nan(m, max_nan(fabsf(f[v][j].x), fabsf(f[v][j].y)));
    m = row_max(m, red[1], nwarps);
    const bool finite = m < __int_as_float(0x7F800000);
    const float s = finite ? __fdiv_rn(m, 127.0f) : __int_as_float(0x7FC00000);
    if (t == 0) p.x_scale[row] = s;
    const bool some = s > 0.0f;               // false for a row of zeros and for a NaN
    const bool exact = s < 0x1p-100f;
    const float inv = __frcp_rn(exact || !some ? 1.0f : s);
    const float inv_hi = __fmul_rn(inv, 1.0f + 0x1p-20f), inv_lo = __fmul_rn(inv, 1.0f - 0x1p-20f);
    int8_t* q = p.Xq + row * p.ldq;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int e = (v * tpr + t) * 8;
      const int n = p.K - e;
      if (n <= 0) continue;
      uint2 w = some ? quantize8(f[v], s, inv_lo, inv_hi, exact) : make_uint2(0u, 0u);
      if (n >= 8) {
        *reinterpret_cast<uint2*>(q + e) = w;
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (j < n) q[e + j] = (int8_t)((j < 4 ? w.x >> (8 * j) : w.y >> (8 * j - 32)) & 0xFFu);
      }
    }
  }
}

template <class T, int OP, int VPT, int MAXT, bool VEC>
cudaError_t launch_t(const RowQuantArgs& a, int tpr, int rpb, int grid, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(tpr * rpb, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, row_quantize_kernel<T, OP, VPT, MAXT, VEC>, a, tpr);
}

template <class T, int OP, bool VEC>
cudaError_t launch_v(const RowQuantArgs& a, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = device_sm_count(dev, &sms)) != cudaSuccess) return e;
  const int chunks = (a.K + 7) / 8;
  // Few rows (at most two per SM): a chunk per thread, the shortest chain.
  // Otherwise up to four per thread.
  int vpt = a.M <= 2 * sms ? 1 : 4;
  while (vpt < 4 && (chunks + vpt - 1) / vpt > 1024) vpt *= 2;
  while (vpt > 1 && chunks <= 32 * (vpt / 2)) vpt /= 2;
  const int tpr = ((chunks + vpt - 1) / vpt + 31) / 32 * 32;
  const int rpb = tpr == 32 ? 4 : 1;
  const int64_t blocks = (a.M + rpb - 1) / rpb;
  const int grid = (int)(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF);
  if (vpt == 1) return launch_t<T, OP, 1, 1024, VEC>(a, tpr, rpb, grid, st);
  if (vpt == 2) return launch_t<T, OP, 2, 1024, VEC>(a, tpr, rpb, grid, st);
  if (tpr <= 512) return launch_t<T, OP, 4, 512, VEC>(a, tpr, rpb, grid, st);
  return launch_t<T, OP, 4, 1024, VEC>(a, tpr, rpb, grid, st);
}

template <class T>
cudaError_t launch_type(const RowQuantArgs& a, bool silu, cudaStream_t st) {
  const size_t es = sizeof(typename T::word);
  auto rows16 = [&](const void* p, int64_t ld) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (a.M == 1 || (uint64_t)ld * es % 16 == 0));
  };
  const bool vec = a.K % 8 == 0 && rows16(a.A, a.lda) && rows16(a.B, a.ldb) && rows16(a.H, a.ldh) && rows16(a.gamma, 0);
  if (silu) return vec ? launch_v<T, 1, true>(a, st) : launch_v<T, 1, false>(a, st);
  return vec ? launch_v<T, 0, true>(a, st) : launch_v<T, 0, false>(a, st);
}

}  // namespace

cudaError_t launch_row_quantize(const RowQuantArgs& a, bool silu, int dtype, cudaStream_t st) {
  if (dtype == 0) return launch_type<Bf16>(a, silu, st);
  if (dtype == 1) return launch_type<Fp16>(a, silu, st);
  return launch_type<Fp32>(a, silu, st);
}

}  // namespace w4a4
