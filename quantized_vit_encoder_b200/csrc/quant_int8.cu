// Row kernels of the INT8 path: one scale per row (token, or output channel of a
// weight), symmetric codes in [-127, 127]; plain, after LayerNorm, after GELU.
//
//   s = fl32(amax / 127),  amax = max_k |y[k]|,   q[k] = round_half_even(y[k] / s)
//
// with the exact quotient by the fp32 number s.  A zero s (amax 0, or below
// 127 * 2^-150) gives zero codes; a row holding an infinity or a NaN gets
// s = NaN and zero codes, so that its row of a product comes out NaN.
#include "internal.h"
#include "ptx.cuh"

#include <cuda_fp16.h>

namespace vitq {
namespace {

enum : int { kI8Plain = 0, kI8Ln = 1, kI8Gelu = 2 };

// ---------------------------------------------------------------- element types
// A chunk is 16 bytes of a row: 8 bf16 or fp16 values, or 4 fp32 values.
// kInf: the bit pattern from which a magnitude is infinite or NaN.
template <class T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static constexpr bool kMove = true;   // codes by the moved reciprocal
  static constexpr int PER = 8;
  static constexpr uint32_t kInf = 0x7F80u;
  static __device__ __forceinline__ float at(const uint4& u, int i) {
    const uint32_t w = (&u.x)[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  static __device__ __forceinline__ float of_mag(uint32_t m) { return __uint_as_float(m << 16); }
};
template <> struct Elem<__half> {
  static constexpr bool kMove = false;
  static constexpr int PER = 8;
  static constexpr uint32_t kInf = 0x7C00u;
  static __device__ __forceinline__ float at(const uint4& u, int i) {
    const uint32_t w = (&u.x)[i >> 1];
    return __half2float(__ushort_as_half((unsigned short)((i & 1) ? (w >> 16) : (w & 0xFFFFu))));
  }
  static __device__ __forceinline__ float of_mag(uint32_t m) { return __half2float(__ushort_as_half((unsigned short)m)); }
};
template <> struct Elem<float> {
  static constexpr bool kMove = false;
  static constexpr int PER = 4;
  static constexpr uint32_t kInf = 0x7F800000u;
  static __device__ __forceinline__ float at(const uint4& u, int i) { return __uint_as_float((&u.x)[i]); }
  static __device__ __forceinline__ float of_mag(uint32_t m) { return __uint_as_float(m); }
};

// Largest magnitude of a chunk as a bit pattern (magnitudes order like their bits).
template <class T>
__device__ __forceinline__ uint32_t chunk_mag(const uint4& u) {
  if (Elem<T>::PER == 4) {
    return max(max(u.x & 0x7FFFFFFFu, u.y & 0x7FFFFFFFu), max(u.z & 0x7FFFFFFFu, u.w & 0x7FFFFFFFu));
  } else {
    uint32_t m;
    asm("{.reg .b32 t0, t1; max.u16x2 t0, %1, %2; max.u16x2 t1, %3, %4; max.u16x2 %0, t0, t1;}"
        : "=r"(m)
        : "r"(u.x & 0x7FFF7FFFu), "r"(u.y & 0x7FFF7FFFu), "r"(u.z & 0x7FFF7FFFu), "r"(u.w & 0x7FFF7FFFu));
    return max(m & 0xFFFFu, m >> 16);
  }
}

// ---------------------------------------------------------------- codes of a row
// How the codes of a row come from its scale s.  With s >= 2^-107 the product
// p = y * r, r = fl32(1 / s), is within 2^-23 (relative) of y / s.  For bf16 values p
// rounds like y / s once r is moved by 2^-21 in the right direction: with the 8-bit
// significands Y of y and A of amax, amax / 127 against y / (k + 1/2) is a comparison
// of 254 Y 2^i with (2k + 1) A 2^j, integers below 2^16 times one power of two.
// Either they differ by 2^-16 of their size, which the move and the roundings cannot
// cross, or they are equal.  Equality needs 127 | A, and then s is a power of two, r
// and p are exact and p rounds ties to even itself; or 127 | 2k + 1, so |y| = amax / 2,
// and the sign of amax/2 - 63.5 s (one FMA, exact sign) says to which side of 63.5 the
// quotient falls and r moves.
// fp16 and fp32 values have more exact ties: where p lies within 2^-14 of one, the
// sign of y - h s decides.  Rows with a smaller scale (amax < 127 * 2^-107) divide in
// fp64.
struct RowScale {
  float s, r;
  int mode;   // 0: product, 1: fp64 quotient, 2: zero codes
};

template <class T>
__device__ __forceinline__ RowScale row_scale(uint32_t mag) {
  RowScale c;
  if (mag >= Elem<T>::kInf) {
    c.s = __uint_as_float(0x7FC00000u);
    c.r = 0.f;
    c.mode = 2;
    return c;
  }
  const float a = Elem<T>::of_mag(mag);
  c.s = __fdiv_rn(a, 127.0f);
  c.mode = c.s == 0.f ? 2 : (c.s < 0x1p-107f ? 1 : 0);
  c.r = c.mode == 0 ? __fdiv_rn(1.0f, c.s) : 0.f;
  if (Elem<T>::kMove) {
    const float side = __fmaf_rn(-63.5f, c.s, 0.5f * a);
    if (side > 0.f) c.r = __fmaf_rn(c.r, 0x1p-21f, c.r);
    if (side < 0.f) c.r = __fmaf_rn(c.r, -0x1p-21f, c.r);
  }
  return c;
}

// Nearest integer of |p| <= 128 (ties to even) in the low bits of the result.
__device__ __forceinline__ uint32_t rint_bits(float p) { return __float_as_uint(__fadd_rn(p, 12582912.0f)); }

// The code of one value near a tie, from the exact sign of y - h s.
__device__ __noinline__ uint32_t code_near_tie(float y, float s, float p) {
  const float f = floorf(p), h = f + 0.5f;
  const float side = __fmaf_rn(-h, s, y);
  const int fi = (int)f;
  const int k = side > 0.f ? fi + 1 : side < 0.f ? fi : fi + (fi & 1);
  return (uint32_t)max(-127, min(127, k));
}

__device__ __noinline__ uint32_t code_fp64(float y, float s) {
  const double q = rint((double)y / (double)s);
  return (uint32_t)(int)fmax(-127.0, fmin(127.0, q));
}

template <class T>
__device__ __forceinline__ uint32_t code_of(float y, const RowScale& c) {
  if (c.mode == 0) {
    const float p = __fmul_rn(y, c.r);
    if (Elem<T>::kMove) return rint_bits(p) & 0xFFu;
    const uint32_t b = rint_bits(p);
    const float k = __fsub_rn(__uint_as_float(b), 12582912.0f);
    if (fabsf(__fsub_rn(p, k)) > 0.5f - 0x1p-14f) return code_near_tie(y, c.s, p) & 0xFFu;
    return b & 0xFFu;
  }
  return c.mode == 1 ? code_fp64(y, c.s) & 0xFFu : 0u;
}

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Codes of one chunk at column col of a row with K columns.
template <class T>
__device__ __forceinline__ void store_codes(const uint4& u, const RowScale& c, int8_t* qr, int col, int K) {
  constexpr int PER = Elem<T>::PER;
  uint32_t w[PER / 4];
  if (Elem<T>::kMove && c.mode == 0) {   // two values a multiply and an add
    const uint64_t r = f2pack(c.r, c.r), magic = f2pack(12582912.0f, 12582912.0f);
#pragma unroll
    for (int g = 0; g < PER / 4; ++g) {
      const float2 a = f2unpack(fadd2(fmul2(f2pack(Elem<T>::at(u, 4 * g), Elem<T>::at(u, 4 * g + 1)), r), magic));
      const float2 b = f2unpack(fadd2(fmul2(f2pack(Elem<T>::at(u, 4 * g + 2), Elem<T>::at(u, 4 * g + 3)), r), magic));
      w[g] = pack4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    }
  } else {
#pragma unroll
  for (int g = 0; g < PER / 4; ++g)
    w[g] = pack4(code_of<T>(Elem<T>::at(u, 4 * g), c), code_of<T>(Elem<T>::at(u, 4 * g + 1), c),
                 code_of<T>(Elem<T>::at(u, 4 * g + 2), c), code_of<T>(Elem<T>::at(u, 4 * g + 3), c));
  }
  if (col + PER <= K) {
    if (PER == 8) *reinterpret_cast<uint2*>(qr + col) = make_uint2(w[0], w[PER / 4 - 1]);
    else *reinterpret_cast<uint32_t*>(qr + col) = w[0];
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (col + i < K) qr[col + i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// ---------------------------------------------------------------- loads
template <class T>
__device__ __forceinline__ uint4 load_chunk16(const T* xr, int col, int K) {
  constexpr int PER = Elem<T>::PER;
  if (col + PER <= K) return *reinterpret_cast<const uint4*>(xr + col);
  uint4 u = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (col + i < K) {
      if (PER == 8) (&u.x)[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(xr)[col + i] << (16 * (i & 1));
      else (&u.x)[i & 3] = reinterpret_cast<const uint32_t*>(xr)[col + i];
    }
  }
  return u;
}

// ---------------------------------------------------------------- row reductions
// Over the TPR threads that share a row (all of them take part).  TPR = 32: a warp;
// otherwise the whole CTA, through shared memory.
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* sh) {
  v = __reduce_max_sync(0xffffffffu, v);
  if (TPR > 32) {
    __syncthreads();   // sh may still be read from an earlier reduction
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < TPR / 32 ? sh[threadIdx.x & 31] : 0u;
    v = __reduce_max_sync(0xffffffffu, v);
  }
  return v;
}
template <int TPR>
__device__ __forceinline__ double row_sum(double v, double* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (TPR > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < TPR / 32 ? sh[threadIdx.x & 31] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// ---------------------------------------------------------------- LayerNorm, GELU
__device__ __forceinline__ uint32_t bf16_bits_fp64(double y) {
  const __nv_bfloat16 h = __double2bfloat16(y);
  return (uint32_t)__bfloat16_as_ushort(h);
}

// bf16 rounding of (x - mean) rstd gamma + beta in fp64.
__device__ __noinline__ uint32_t ln_fp64(float x, float g, float b, double mean, double rstd) {
  return bf16_bits_fp64(((double)x - mean) * rstd * (double)g + (double)b);
}

__device__ __forceinline__ uint32_t gelu_bits(uint32_t x) { return g_gelu_table[x & 0xFFFFu]; }

// ---------------------------------------------------------------- the row kernel
// TPR threads per row, the row held in registers as at most NC chunks per thread,
// read once.  Rows 16-byte aligned.
template <int OP, class T, int TPR, int NC>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR)
    rows_int8_kernel(const T* __restrict__ x, int ldx, int M, int K, int8_t* __restrict__ q, int ldq,
                     float* __restrict__ s) {
  constexpr int PER = Elem<T>::PER;
  __shared__ uint32_t sh_max[32];
  pdl_trigger();
  pdl_wait();
  const int row = TPR == 32 ? blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  const int t = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
  if (row >= M) return;   // whole warps (TPR = 32) or whole CTAs
  const T* xr = x + (size_t)row * ldx;
  uint4 u[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = (c * TPR + t) * PER;
    u[c] = col < K ? load_chunk16(xr, col, K) : make_uint4(0u, 0u, 0u, 0u);
  }
  if (OP == kI8Gelu) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) (&u[c].x)[j] = gelu_bits((&u[c].x)[j]) | (gelu_bits((&u[c].x)[j] >> 16) << 16);
  }
  uint32_t m = 0u;
#pragma unroll
  for (int c = 0; c < NC; ++c) m = max(m, chunk_mag<T>(u[c]));
  const RowScale sc = row_scale<T>(row_max<TPR>(m, sh_max));
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = (c * TPR + t) * PER;
    if (col < K) store_codes<T>(u[c], sc, q + (size_t)row * ldq, col, K);
  }
  if (t == 0) s[row] = sc.s;
}

// ---------------------------------------------------------------- LayerNorm
// TPR threads per row (a warp, or a CTA of 128), the row in registers (at most NC
// chunks of 8 columns a thread) and the next row's loads in flight; gamma and beta
// staged once per CTA as fp32.  Persistent over the rows.
//
// Statistics: exact fp64 sums of x and x^2 (bf16 -> fp64 is exact); where the mean is
// far above the spread (E[x^2] > 64 var), which would cost the difference its bits,
// the squares are summed again around the mean.
// y = (x - mean) rstd gamma + beta in fp32, mean as a sum of two fp32 numbers: x - mh,
// (x - mh) r - ml r, and the last FMA round once each and r = fl32(rstd) once, so
// |error| <= 3 2^-24 (|y| + |beta|) + 2^-24 |y| < (|y| + |beta|) 2^-21.  Where y minus and
// plus that bound round to the same bf16 value, that value is the rounding of the exact
// y; the other pairs (about 1 in 2^12) are evaluated in fp64.  Rows whose statistics are
// not finite, or whose rstd leaves 2^-100 .. 2^100, are evaluated in fp64 as a whole.
__device__ __noinline__ uint32_t ln_pair_exact(float x0, float x1, float g0, float g1, float b0, float b1, double mean,
                                               double rstd) {
  return bf16_bits_fp64(((double)x0 - mean) * rstd * (double)g0 + (double)b0) |
         (bf16_bits_fp64(((double)x1 - mean) * rstd * (double)g1 + (double)b1) << 16);
}

// Makes the compiler unpack the chunks again where they are used next, instead of
// keeping their 8 NC values in registers.
template <int NC>
__device__ __forceinline__ void unpack_again(uint4 (&u)[NC]) {
#pragma unroll
  for (int c = 0; c < NC; ++c) asm volatile("" : "+r"(u[c].x), "+r"(u[c].y), "+r"(u[c].z), "+r"(u[c].w));
}

template <int TPR, int NC>
__global__ void __launch_bounds__(128, NC == 5 ? 5 : 3)
    ln_rows_int8_kernel(const __nv_bfloat16* __restrict__ x, int ldx, int M, int K,
                        const __nv_bfloat16* __restrict__ gamma, const __nv_bfloat16* __restrict__ beta, double eps,
                        int8_t* __restrict__ q, int ldq, float* __restrict__ s) {
  using E = Elem<__nv_bfloat16>;
  constexpr int ROWS = 128 / TPR;          // rows a CTA works on at a time
  extern __shared__ float4 ln8_smem[];     // gamma, then beta: chunk c of thread t at (2c + half) * TPR + t
  __shared__ double sh_sum[2][4];
  __shared__ uint32_t sh_max[4];
  const int t = threadIdx.x % TPR, warp = threadIdx.x >> 5;
  float4* sg = ln8_smem;
  float4* sb = ln8_smem + 2 * NC * TPR;
  pdl_trigger();
  pdl_wait();
  int row = blockIdx.x * ROWS + threadIdx.x / TPR;
  const int stride = gridDim.x * ROWS;
  auto load_row = [&](int r, uint4 (&u)[NC]) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * TPR + t) * 8;
      u[c] = r < M && col < K ? load_chunk16(x + (size_t)r * ldx, col, K) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  uint4 nxt[NC];
  load_row(row, nxt);
  for (int i = threadIdx.x; i < NC * TPR * 2; i += 128) {   // float4 of 4 columns
    const int half = i / TPR & 1, c = i / (2 * TPR), col = (c * TPR + i % TPR) * 8 + half * 4;
    float g[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      g[k] = col + k < K ? __bfloat162float(gamma[col + k]) : 0.f;
      b[k] = col + k < K ? __bfloat162float(beta[col + k]) : 0.f;
    }
    sg[i] = make_float4(g[0], g[1], g[2], g[3]);
    sb[i] = make_float4(b[0], b[1], b[2], b[3]);
  }
  __syncthreads();
  const double rK = 1.0 / (double)K;
  for (; row < M; row += stride) {   // uniform over the threads of a row
    uint4 u[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) u[c] = nxt[c];
    load_row(row + stride, nxt);
    auto sum2 = [&](double& a, double& b) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
      }
      if (TPR > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
          sh_sum[0][warp] = a;
          sh_sum[1][warp] = b;
        }
        __syncthreads();
        a = (sh_sum[0][0] + sh_sum[0][1]) + (sh_sum[0][2] + sh_sum[0][3]);
        b = (sh_sum[1][0] + sh_sum[1][1]) + (sh_sum[1][2] + sh_sum[1][3]);
      }
    };
    double s1 = 0.0, s2 = 0.0, t1 = 0.0, t2 = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const double a = (double)E::at(u[c], i), b = (double)E::at(u[c], i + 1);
        s1 += a;
        t1 += b;
        s2 = fma(a, a, s2);
        t2 = fma(b, b, t2);
      }
    s1 += t1;
    s2 += t2;
    sum2(s1, s2);
    unpack_again(u);
    const double mean = s1 * rK;
    double var = fma(-mean, mean, s2 * rK);
    if (!(s2 * rK <= 64.0 * var)) {   // also for a NaN
      double d2 = 0.0, none = 0.0;   // reads the row again: rare, and it keeps no registers for it
#pragma unroll 1
      for (int k = t; k < K; k += TPR) {
        const double d = (double)__bfloat162float(x[(size_t)row * ldx + k]) - mean;
        d2 = fma(d, d, d2);
      }
      sum2(d2, none);
      var = d2 * rK;
    }
    const double rstd = rsqrt(var + eps);
    const float mh = (float)mean, ml = (float)(mean - (double)mh), r32 = (float)rstd;
    const bool plain = r32 >= 0x1p-100f && r32 <= 0x1p100f && fabsf(mh) <= 0x1p100f;
    const uint64_t nmh = f2pack(-mh, -mh), rr = f2pack(r32, r32), nmr = f2pack(-ml * r32, -ml * r32);
    const uint64_t up = f2pack(0x1p-21f, 0x1p-21f), dn = f2pack(-0x1p-21f, -0x1p-21f);
    uint32_t m = 0u;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = 2 * c * TPR + t;
      const float4 g0 = sg[at], g1 = sg[at + TPR], b0 = sb[at], b1 = sb[at + TPR];
      const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
      const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
      uint32_t slow = 0u, h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t xc = fadd2(f2pack(E::at(u[c], 2 * i), E::at(u[c], 2 * i + 1)), nmh);
        const uint64_t y = ffma2(ffma2(xc, rr, nmr), f2pack(g[2 * i], g[2 * i + 1]), f2pack(b[2 * i], b[2 * i + 1]));
        const float2 yf = f2unpack(y);
        const uint64_t e = f2pack(fabsf(yf.x) + fabsf(b[2 * i]), fabsf(yf.y) + fabsf(b[2 * i + 1]));
        h[i] = bf16x2_of(ffma2(e, dn, y));
        slow |= (uint32_t)(h[i] != bf16x2_of(ffma2(e, up, y))) << i;
      }
      if (!plain) slow = 15u;
      if (slow) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((slow >> i) & 1u)
            h[i] = ln_pair_exact(E::at(u[c], 2 * i), E::at(u[c], 2 * i + 1), g[2 * i], g[2 * i + 1], b[2 * i],
                                 b[2 * i + 1], mean, rstd);
      }
      u[c] = make_uint4(h[0], h[1], h[2], h[3]);
      // columns past K have gamma = beta = 0, so y = 0 (or NaN, in a row that has one anyway)
      m = max(m, chunk_mag<__nv_bfloat16>(u[c]));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (TPR > 32) {
      if ((threadIdx.x & 31) == 0) sh_max[warp] = m;
      __syncthreads();
      m = max(max(sh_max[0], sh_max[1]), max(sh_max[2], sh_max[3]));
    }
    const RowScale sc = row_scale<__nv_bfloat16>(m);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * TPR + t) * 8;
      if (col < K) store_codes<__nv_bfloat16>(u[c], sc, q + (size_t)row * ldq, col, K);
    }
    if (t == 0) s[row] = sc.s;
  }
}

// ---------------------------------------------------------------- any layout
// Rows of any alignment and width: one CTA per row, single elements, the row read
// again in each pass.
constexpr int kAnyThreads = 256;

template <class T>
__device__ __forceinline__ uint32_t elem_bits(const T* xr, int col) {
  return sizeof(T) == 2 ? (uint32_t)reinterpret_cast<const uint16_t*>(xr)[col]
                        : reinterpret_cast<const uint32_t*>(xr)[col];
}
template <class T>
__device__ __forceinline__ float value_of_bits(uint32_t b) {
  return Elem<T>::at(make_uint4(b, 0u, 0u, 0u), 0);
}

template <int OP, class T>
__global__ void __launch_bounds__(kAnyThreads)
    rows_int8_any_kernel(const T* __restrict__ x, int ldx, int M, int K, const __nv_bfloat16* __restrict__ gamma,
                         const __nv_bfloat16* __restrict__ beta, double eps, int8_t* __restrict__ q, int ldq,
                         float* __restrict__ s) {
  __shared__ double sh_sum[32];
  __shared__ uint32_t sh_max[32];
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x;
  const T* xr = x + (size_t)row * ldx;
  double mean = 0.0, rstd = 0.0;
  if (OP == kI8Ln) {
    double s1 = 0.0, s2 = 0.0;
    for (int k = threadIdx.x; k < K; k += kAnyThreads) s1 += (double)value_of_bits<T>(elem_bits(xr, k));
    mean = row_sum<kAnyThreads>(s1, sh_sum) / (double)K;
    for (int k = threadIdx.x; k < K; k += kAnyThreads) {
      const double d = (double)value_of_bits<T>(elem_bits(xr, k)) - mean;
      s2 = fma(d, d, s2);
    }
    rstd = 1.0 / sqrt(row_sum<kAnyThreads>(s2, sh_sum) / (double)K + eps);
  }
  auto bits = [&](int k) {
    const uint32_t b = elem_bits(xr, k);
    if (OP == kI8Ln)
      return ln_fp64(value_of_bits<T>(b), __bfloat162float(gamma[k]), __bfloat162float(beta[k]), mean, rstd);
    return OP == kI8Gelu ? gelu_bits(b) : b;
  };
  uint32_t m = 0u;
  for (int k = threadIdx.x; k < K; k += kAnyThreads) m = max(m, bits(k) & (sizeof(T) == 2 ? 0x7FFFu : 0x7FFFFFFFu));
  const RowScale sc = row_scale<T>(row_max<kAnyThreads>(m, sh_max));
  for (int k = threadIdx.x; k < K; k += kAnyThreads)
    q[(size_t)row * ldq + k] = (int8_t)code_of<T>(value_of_bits<T>(bits(k)), sc);
  if (threadIdx.x == 0) s[row] = sc.s;
}

// ---------------------------------------------------------------- launch
template <int OP, class T, int TPR, int NC>
cudaError_t rows_launch(const RowsInt8& a, cudaStream_t st) {
  const unsigned grid = TPR == 32 ? (unsigned)((a.M + 7) / 8) : (unsigned)a.M;
  return launch_pdl(rows_int8_kernel<OP, T, TPR, NC>, dim3(grid), dim3(TPR == 32 ? 256 : TPR), 0, st, (const T*)a.x,
                    a.ldx, a.M, a.K, a.q, a.ldq, a.s);
}

template <class T>
bool rows_aligned(const RowsInt8& a) {
  return (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && ((size_t)a.ldx * sizeof(T)) % 16 == 0;
}

template <int OP, class T>
cudaError_t rows_any_launch(const RowsInt8& a, cudaStream_t st) {
  return launch_pdl(rows_int8_any_kernel<OP, T>, dim3((unsigned)a.M), dim3(kAnyThreads), 0, st, (const T*)a.x, a.ldx,
                    a.M, a.K, a.gamma, a.beta, a.eps, a.q, a.ldq, a.s);
}

template <int TPR, int NC>
cudaError_t ln_rows_launch(const RowsInt8& a, int num_sms, cudaStream_t st) {
  constexpr int ROWS = 128 / TPR;
  constexpr size_t smem = (size_t)4 * NC * TPR * sizeof(float4);
  constexpr int per_sm = NC == 5 ? 5 : 3;   // CTAs that fit an SM
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(ln_rows_int8_kernel<TPR, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem);
    if (e != cudaSuccess) return e;
  }
  const long long ctas = ((long long)a.M + ROWS - 1) / ROWS, most = (long long)num_sms * per_sm;
  return launch_pdl(ln_rows_int8_kernel<TPR, NC>, dim3((unsigned)(ctas < most ? ctas : most)), dim3(128), smem, st,
                    (const __nv_bfloat16*)a.x, a.ldx, a.M, a.K, a.gamma, a.beta, a.eps, a.q, a.ldq, a.s);
}

template <int OP, class T>
cudaError_t rows_dispatch(const RowsInt8& a, cudaStream_t st) {
  const int chunks = (a.K + Elem<T>::PER - 1) / Elem<T>::PER;
  if (rows_aligned<T>(a) && chunks <= 8192) {
    if (chunks <= 160) return rows_launch<OP, T, 32, 5>(a, st);
    if (chunks <= 256) return rows_launch<OP, T, 32, 8>(a, st);
    if (chunks <= 640) return rows_launch<OP, T, 128, 5>(a, st);
    if (chunks <= 1024) return rows_launch<OP, T, 128, 8>(a, st);
    if (chunks <= 2048) return rows_launch<OP, T, 256, 8>(a, st);
    return rows_launch<OP, T, 1024, 8>(a, st);
  }
  return rows_any_launch<OP, T>(a, st);
}

}  // namespace

cudaError_t launch_quant_int8(const RowsInt8& a, int dtype, cudaStream_t st) {
  if (a.M == 0) return cudaSuccess;
  if (dtype == 0) return rows_dispatch<kI8Plain, __nv_bfloat16>(a, st);
  if (dtype == 1) return rows_dispatch<kI8Plain, __half>(a, st);
  return rows_dispatch<kI8Plain, float>(a, st);
}
cudaError_t launch_ln_quant_int8(const RowsInt8& a, int num_sms, cudaStream_t st) {
  if (a.M == 0) return cudaSuccess;
  const int chunks = (a.K + 7) / 8;
  if (rows_aligned<__nv_bfloat16>(a)) {
    if (chunks <= 160) return ln_rows_launch<32, 5>(a, num_sms, st);
    if (chunks <= 256) return ln_rows_launch<32, 8>(a, num_sms, st);
    if (chunks <= 640) return ln_rows_launch<128, 5>(a, num_sms, st);
    if (chunks <= 1024) return ln_rows_launch<128, 8>(a, num_sms, st);
  }
  return rows_any_launch<kI8Ln, __nv_bfloat16>(a, st);
}
cudaError_t launch_gelu_quant_int8(const RowsInt8& a, cudaStream_t st) {
  return a.M == 0 ? cudaSuccess : rows_dispatch<kI8Gelu, __nv_bfloat16>(a, st);
}

}  // namespace vitq
