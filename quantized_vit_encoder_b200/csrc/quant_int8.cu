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
#pragma unroll
  for (int g = 0; g < PER / 4; ++g)
    w[g] = pack4(code_of<T>(Elem<T>::at(u, 4 * g), c), code_of<T>(Elem<T>::at(u, 4 * g + 1), c),
                 code_of<T>(Elem<T>::at(u, 4 * g + 2), c), code_of<T>(Elem<T>::at(u, 4 * g + 3), c));
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
    rows_int8_kernel(const T* __restrict__ x, int ldx, int M, int K, const __nv_bfloat16* __restrict__ gamma,
                     const __nv_bfloat16* __restrict__ beta, double eps, int8_t* __restrict__ q, int ldq,
                     float* __restrict__ s) {
  constexpr int PER = Elem<T>::PER;
  __shared__ double sh_sum[32];
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
  if (OP == kI8Ln) {
    double s1 = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < PER; ++i) s1 += (double)Elem<T>::at(u[c], i);
    const double mean = row_sum<TPR>(s1, sh_sum) / (double)K;
    double s2 = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * TPR + t) * PER;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const double d = (double)Elem<T>::at(u[c], i) - mean;
        if (col + i < K) s2 = fma(d, d, s2);
      }
    }
    const double rstd = 1.0 / sqrt(row_sum<TPR>(s2, sh_sum) / (double)K + eps);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * TPR + t) * PER;
      if (col < K) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          uint32_t h = 0u;
          if (col + i < K)
            h = ln_fp64(Elem<T>::at(u[c], i), __bfloat162float(gamma[col + i]), __bfloat162float(beta[col + i]), mean, rstd);
          uint32_t& w = (&u[c].x)[i >> 1];
          w = (i & 1) ? (w & 0xFFFFu) | (h << 16) : (w & 0xFFFF0000u) | h;
        }
      }
    }
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
                    a.ldx, a.M, a.K, a.gamma, a.beta, a.eps, a.q, a.ldq, a.s);
}

template <int OP, class T>
cudaError_t rows_dispatch(const RowsInt8& a, cudaStream_t st) {
  const bool aligned = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && ((size_t)a.ldx * sizeof(T)) % 16 == 0;
  const int chunks = (a.K + Elem<T>::PER - 1) / Elem<T>::PER;
  if (aligned && chunks <= 8192) {
    if (chunks <= 160) return rows_launch<OP, T, 32, 5>(a, st);
    if (chunks <= 256) return rows_launch<OP, T, 32, 8>(a, st);
    if (chunks <= 640) return rows_launch<OP, T, 128, 5>(a, st);
    if (chunks <= 1024) return rows_launch<OP, T, 128, 8>(a, st);
    if (chunks <= 2048) return rows_launch<OP, T, 256, 8>(a, st);
    return rows_launch<OP, T, 1024, 8>(a, st);
  }
  return launch_pdl(rows_int8_any_kernel<OP, T>, dim3((unsigned)a.M), dim3(kAnyThreads), 0, st, (const T*)a.x, a.ldx,
                    a.M, a.K, a.gamma, a.beta, a.eps, a.q, a.ldq, a.s);
}

}  // namespace

cudaError_t launch_quant_int8(const RowsInt8& a, int dtype, cudaStream_t st) {
  if (a.M == 0) return cudaSuccess;
  if (dtype == 0) return rows_dispatch<kI8Plain, __nv_bfloat16>(a, st);
  if (dtype == 1) return rows_dispatch<kI8Plain, __half>(a, st);
  return rows_dispatch<kI8Plain, float>(a, st);
}
cudaError_t launch_ln_quant_int8(const RowsInt8& a, cudaStream_t st) {
  return a.M == 0 ? cudaSuccess : rows_dispatch<kI8Ln, __nv_bfloat16>(a, st);
}
cudaError_t launch_gelu_quant_int8(const RowsInt8& a, cudaStream_t st) {
  return a.M == 0 ? cudaSuccess : rows_dispatch<kI8Gelu, __nv_bfloat16>(a, st);
}

}  // namespace vitq
