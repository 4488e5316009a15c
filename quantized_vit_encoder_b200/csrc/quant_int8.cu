// Row kernels of the INT8 path: one scale per row (token, or output channel of a
// weight), symmetric codes in [-127, 127]; plain, after LayerNorm, after GELU.
//
//   s = fl32(amax / 127),  amax = max_k |y[k]|,   q[k] = round_half_even(y[k] / s)
//
// with the exact quotient by the fp32 number s.  A zero s (amax 0, or below
// 127 * 2^-150) gives zero codes; a row holding an infinity or a NaN gets
// s = NaN and zero codes, so that its row of a product comes out NaN.
//
// (No __restrict__ and no __ldg on what an earlier kernel may have written: such loads could
// be moved before the wait for that kernel.)
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
// (not rounded itself: one FMA adds it to 1.5 2^23, whose spacing is 1) rounds like y / s
// once r is moved by 2^-21 in the right direction: with the 8-bit significands Y of y and A
// of amax, amax / 127 against y / (k + 1/2) is a comparison of 254 Y 2^i with
// (2k + 1) A 2^j, integers below 2^16 times one power of two.  Either they differ by 2^-16
// of their size, which the move and the roundings cannot cross, or they are equal.
// Equality needs 127 | A, and then s is a power of two, r and p are exact and p rounds ties
// to even itself; or 127 | 2k + 1, so |y| = amax / 2, and the sign of amax/2 - 63.5 s (one
// FMA, exact sign) says to which side of 63.5 the quotient falls and r moves.
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
    if (Elem<T>::kMove) return __float_as_uint(__fmaf_rn(y, c.r, 12582912.0f)) & 0xFFu;
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

__device__ __noinline__ void store_codes_edge(int8_t* qc, uint2 w, int n) {
  for (int i = 0; i < n; ++i) qc[i] = (int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
}

// Codes of one chunk at column col of a row with K columns, to qc.  TAIL: the chunk may
// reach past K.
template <class T, bool TAIL>
__device__ __forceinline__ void store_codes(const uint4& u, const RowScale& c, int8_t* qc, int col, int K) {
  constexpr int PER = Elem<T>::PER;
  uint32_t w[PER / 4];
  if (Elem<T>::kMove && c.mode == 0) {   // two values an FMA
    const uint64_t r = f2pack(c.r, c.r), magic = f2pack(12582912.0f, 12582912.0f);
#pragma unroll
    for (int g = 0; g < PER / 4; ++g) {
      const float2 a = f2unpack(ffma2(f2pack(Elem<T>::at(u, 4 * g), Elem<T>::at(u, 4 * g + 1)), r, magic));
      const float2 b = f2unpack(ffma2(f2pack(Elem<T>::at(u, 4 * g + 2), Elem<T>::at(u, 4 * g + 3)), r, magic));
      w[g] = pack4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    }
  } else {
#pragma unroll
    for (int g = 0; g < PER / 4; ++g)
      w[g] = pack4(code_of<T>(Elem<T>::at(u, 4 * g), c), code_of<T>(Elem<T>::at(u, 4 * g + 1), c),
                   code_of<T>(Elem<T>::at(u, 4 * g + 2), c), code_of<T>(Elem<T>::at(u, 4 * g + 3), c));
  }
  if (!TAIL || col + PER <= K) {
    if (PER == 8) *reinterpret_cast<uint2*>(qc) = make_uint2(w[0], w[PER / 4 - 1]);
    else *reinterpret_cast<uint32_t*>(qc) = w[0];
  } else {
    store_codes_edge(qc, make_uint2(w[0], w[PER / 4 - 1]), K - col);
  }
}

// ---------------------------------------------------------------- loads
// The chunk at column col of a row of K columns (zeros past K), element by element.
template <class T>
__device__ __noinline__ uint4 load_chunk_edge(const T* xr, int col, int K) {
  uint4 u = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < Elem<T>::PER; ++i) {
    if (col + i < K) {
      if (sizeof(T) == 2) (&u.x)[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(xr)[col + i] << (16 * (i & 1));
      else (&u.x)[i & 3] = reinterpret_cast<const uint32_t*>(xr)[col + i];
    }
  }
  return u;
}

// Rows of any alignment: the aligned 16-byte units that a row lies in come to shared memory
// by asynchronous copies, and a chunk is put together from two of them.  Other bytes of the
// first and last unit belong to neighbouring rows or the gap between them; of a unit that
// reaches past the matrix (x .. end) only the bytes within it are read.
__device__ __forceinline__ uint32_t row_off(const void* xr) { return (uint32_t)reinterpret_cast<uintptr_t>(xr) & 15u; }

// Unit i of a row to dst.  off: bytes of unit 0 before the row.
template <class T>
__device__ __forceinline__ void fetch_unit(const T* xr, uint32_t off, int i, int K, const T* x, const T* end,
                                           uint4* dst) {
  constexpr int PER = Elem<T>::PER;
  const char* from = reinterpret_cast<const char*>(xr) - off + (size_t)i * 16;
  const long long left = reinterpret_cast<const char*>(end) - from;
  if (from < reinterpret_cast<const char*>(x)) {
    const int lead = (int)(off / sizeof(T));
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int k = 1; k < PER; ++k) {
      if (k >= lead && k - lead < K) {
        if (sizeof(T) == 2) (&u.x)[k >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(xr)[k - lead] << (16 * (k & 1));
        else (&u.x)[k & 3] = reinterpret_cast<const uint32_t*>(xr)[k - lead];
      }
    }
    *dst = u;
  } else {
    cp_async16(smem_u32(dst), from, left < 16 ? (uint32_t)left : 16u);
  }
}
// The chunk at column col from its units a and b (off as above), zeros past K.
template <class T>
__device__ __forceinline__ uint4 chunk_of_units(const uint4& a, const uint4& b, uint32_t off, int col, int K) {
  uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) v[i] = off & 8u ? v[i + 2] : v[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = off & 4u ? v[i + 1] : v[i];
  if (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = off & 2u ? __byte_perm(v[i], v[i + 1], 0x5432) : v[i];
  }
  if (K - col < Elem<T>::PER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int left = (K - col) * (int)sizeof(T) - 4 * i;   // bytes of this word inside the row
      v[i] = left >= 4 ? v[i] : left <= 0 ? 0u : v[i] & 0xFFFFu;
    }
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
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

// ---------------------------------------------------------------- GELU by table
// The magnitudes 2^-14 .. 16 of the GELU table as shared-memory words: GELU(x) and
// GELU(-x) in the low and high half of word bits(x) - kGeluLo (9 KB; lanes that differ
// only in sign read one word).  Chunks with another value (zeros, infinities, about 1 in
// 800 of a unit normal's) take the whole table from global memory.  25024 x 4304: 70.8 us,
// the HBM floor being 49.4; the table reads bound it (3.4 words of one bank among 32 random
// ones: before rows were loaded ahead, shared memory was busy 83 % of 74 us, issue slots 61 %).
constexpr uint32_t kGeluLo = 0x3880u, kGeluN = 0x900u;

__device__ __forceinline__ void gelu_stage(uint32_t* lut) {
  for (int i = threadIdx.x; i < (int)kGeluN / 8; i += blockDim.x) {
    const uint4 a = *reinterpret_cast<const uint4*>(g_gelu_table + kGeluLo + 8 * i);
    const uint4 b = *reinterpret_cast<const uint4*>(g_gelu_table + 0x8000u + kGeluLo + 8 * i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      lut[8 * i + 2 * k] = __byte_perm((&a.x)[k], (&b.x)[k], 0x5410);
      lut[8 * i + 2 * k + 1] = __byte_perm((&a.x)[k], (&b.x)[k], 0x7632);
    }
  }
}

__device__ __noinline__ uint4 gelu_chunk_global(uint4 u) {
#pragma unroll
  for (int j = 0; j < 4; ++j) (&u.x)[j] = gelu_bits((&u.x)[j]) | (gelu_bits((&u.x)[j] >> 16) << 16);
  return u;
}

__device__ __forceinline__ uint4 gelu_chunk(const uint4& u, const uint32_t* lut) {
  const char* base = reinterpret_cast<const char*>(lut);
  uint4 y;
  uint32_t far = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = (&u.x)[j];
    // (magnitude - kGeluLo) of both halves, wrapping around below kGeluLo
    uint32_t t, ok;
    asm("add.u16x2 %0, %1, %2;" : "=r"(t) : "r"(w & 0x7FFF7FFFu), "r"(0x00010001u * (0x10000u - kGeluLo)));
    asm("min.u16x2 %0, %1, %2;" : "=r"(ok) : "r"(t), "r"(0x00010001u * (kGeluN - 1u)));
    far |= t ^ ok;
    const uint32_t at = ok * 4u + ((w >> 14) & 0x00020002u);   // byte offsets; each half stays below 2^16
    const uint32_t lo = *reinterpret_cast<const uint16_t*>(base + (at & 0xFFFFu));
    const uint32_t hi = *reinterpret_cast<const uint16_t*>(base + (at >> 16));
    (&y.x)[j] = __byte_perm(lo, hi, 0x5410);
  }
  return far ? gelu_chunk_global(u) : y;
}

// ---------------------------------------------------------------- the row kernel
// TPR threads per row, the row held in registers as at most NC chunks per thread, read
// once.  ANY: rows of any alignment and K, by way of shared memory (`units` 16-byte units a
// row; the next row's are on their way while this one's codes are stored); otherwise whole
// 16-byte chunks.  Plain rows: one CTA for each (or 8 rows, a warp each); GELU: persistent
// over the rows, since every CTA stages the table.  Bound by memory: 9164 x 1152 bf16
// 4.9 us (floor 4.8; 32 MB, which stay in L2 between calls), 4608 x 4608 fp32 19.5 (16.2).
// Rows of any alignment: 9164 x 1151 bf16 11.0 us (4.8), 25024 x 4303 GELU 127 (49.4): putting
// chunks together from units is 9 instructions an element on top of 15, at few warps (GELU: 23 %
// of the SM's, issue slots 57 % busy).  In fp32 28 warps an SM (4608 x 4607: 31.6 us, floor 16.2,
// by the 20 that the compiler's registers leave 36.6); in 2 bytes that many spill.
// Whole GELU chunks (kAhead): the next row is on its way, in registers, while this one is
// worked on, at 16 warps an SM (25024 x 4304: 70.8 us, 972 x 4304: 5.0; without it 28 warps
// 73.8 and 7.6, 20 warps 73.2 and 5.9; with it by way of shared memory 20 warps 69.4 and 6.1; 256 threads a
// row, 3128 x 18000: 42.1 with it, 40.1 without).
template <int OP, int TPR, bool ANY> constexpr bool kAhead = OP == kI8Gelu && !ANY && TPR <= 128;
// CTAs an SM that the registers leave room for; 0: as the compiler sees fit.
template <int OP, class T, int TPR, bool ANY>
constexpr int kRowCtas = kAhead<OP, TPR, ANY> ? (TPR == 32 ? 2 : 512 / TPR)
                         : ANY && sizeof(T) == 4 && TPR < 1024 ? (TPR == 32 ? 3 : 896 / TPR) : 0;

template <int OP, class T, int TPR, int NC, bool ANY>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR, kRowCtas<OP, T, TPR, ANY>)
    rows_int8_kernel(const T* x, int ldx, int M, int K, int units, int8_t* q, int ldq,
                     float* s) {
  constexpr int PER = Elem<T>::PER;
  constexpr int ROWS = TPR == 32 ? 8 : 1;
  __shared__ uint32_t sh_max[32];
  __shared__ __align__(16) uint32_t lut[OP == kI8Gelu ? kGeluN : 1];
  extern __shared__ uint4 row_units[];   // ANY
  pdl_trigger();
  if (OP == kI8Gelu) {   // the table is this library's own, written before its first launch
    gelu_stage(lut);
    __syncthreads();
  }
  pdl_wait();
  const int t = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
  uint4* mine = row_units + (TPR == 32 ? (threadIdx.x >> 5) * units : 0);
  auto fetch = [&](int row) {
    const T* xr = x + (size_t)row * ldx;
    const uint32_t off = row_off(xr);
    const int n = (K * (int)sizeof(T) + (int)off + 15) / 16;
    for (int i = t; i < n; i += TPR) fetch_unit(xr, off, i, K, x, x + (size_t)(M - 1) * ldx + K, mine + i);
    cp_async_commit();
  };
  // whole warps (TPR = 32) or whole CTAs share a row
  int row = blockIdx.x * ROWS + (TPR == 32 ? threadIdx.x >> 5 : 0);
  if (ANY && row < M) fetch(row);
  uint4 u[NC], next[kAhead<OP, TPR, ANY> ? NC : 1];   // chunks of this row, and of the next
  auto load = [&](int r, uint4* to) {
    const T* xt = x + (size_t)r * ldx + t * PER;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      to[c] = make_uint4(0u, 0u, 0u, 0u);
      if ((c * TPR + t) * PER < K) to[c] = *reinterpret_cast<const uint4*>(xt + c * TPR * PER);
    }
  };
  if (kAhead<OP, TPR, ANY> && row < M) load(row, next);
  for (; row < M; row += gridDim.x * ROWS) {
    if (ANY) {
      cp_async_wait<0>();
      if (TPR == 32) __syncwarp();
      else __syncthreads();
      const uint32_t off = row_off(x + (size_t)row * ldx);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = c * TPR + t, col = i * PER;
        u[c] = col < K ? chunk_of_units<T>(mine[i], mine[i + 1], off, col, K) : make_uint4(0u, 0u, 0u, 0u);
      }
    } else if (kAhead<OP, TPR, ANY>) {
#pragma unroll
      for (int c = 0; c < NC; ++c) u[c] = next[c % (int)(sizeof(next) / sizeof(uint4))];
      if (row + (int)gridDim.x * ROWS < M) load(row + gridDim.x * ROWS, next);
    } else {
      load(row, u);
    }
    uint32_t m = 0u;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (OP == kI8Gelu && (c * TPR + t) * PER < K) u[c] = gelu_chunk(u[c], lut);
      m = max(m, chunk_mag<T>(u[c]));
    }
    const RowScale sc = row_scale<T>(row_max<TPR>(m, sh_max));   // every thread has its chunks in registers now
    if (ANY && row + (int)gridDim.x * ROWS < M) fetch(row + gridDim.x * ROWS);
    int8_t* qt = q + (size_t)row * ldq + t * PER;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * TPR + t) * PER;
      if (col < K) store_codes<T, ANY>(u[c], sc, qt + c * TPR * PER, col, K);
    }
    if (t == 0) s[row] = sc.s;
  }
}

// ---------------------------------------------------------------- LayerNorm
// TPR threads per row: half a warp, a warp, or a CTA of 128.  A thread's chunks (8 columns
// each) go to shared memory by 16-byte asynchronous copies and stay there, private to the
// thread, through the three passes over them (statistics, normalised bf16 values in place,
// codes): the loops stay rolled and the registers few, so that 32 warps share an SM and hide
// each other's latencies, and one kernel takes any width and alignment.  (25024 x 1152:
// 34.9 us, 6256 x 4608: 48.0.  With the row held in registers, 36 a thread and 20 warps an SM,
// 1152 columns took 33.6 when this kernel took 34.3, but that kernel held no wider or unaligned
// row.)  gamma and beta are staged once per CTA as fp32; persistent over the rows.
// Bound by issue slots (70 % busy), not by HBM (floor 13.2 us): about 26 instructions an
// element, of which the bracket below costs 4 us, the codes 5 and the fp64 statistics 1.5; gamma
// and beta are read from shared memory again for every row (four 16-byte loads for 16 bytes of x).
// Rows of any alignment: 25024 x 1151 47.9 us, 25024 x 1153 51.2; units to chunks doubles the
// instructions (47 an element at 1153, issue slots 74 % busy).
//
// Statistics: exact fp64 sums of x and x^2 (bf16 -> fp64 is exact), divided by K: with the sum
// times 1 / K instead, the mean of a constant row is one unit off that constant at one width in
// four or so (0.2 us of 25024 x 1152).  Where the mean is far above the spread (E[x^2] > 2^10
// var), which would cost the difference its bits, the squares are summed again around the mean.
// y = (x - mean) rstd gamma + beta in fp32, mean as a sum of two fp32 numbers: x - mh,
// (x - mh) r - ml r, and the last FMA round once each and r = fl32(rstd) once, so
// |error| <= 3 2^-24 (|y| + |beta|) + 2^-24 |y| < (|y| + |beta|) 2^-21.  Where y minus and
// plus that bound round to the same bf16 value, that value is the rounding of the exact
// y; the other values (about 1 in 2^12) are evaluated in fp64.  Rows whose statistics are
// not finite, whose rstd leaves 2^-100 .. 2^100, or whose mean, or mean times rstd (a constant
// row and a tiny eps; the columns past K hold zeros and meet it), is above 2^100 are evaluated in
// fp64 as a whole.  Below the normal range a rounding is off by up to 2^-150 whatever the value:
// at most 2^-85 of y with |gamma| < 2^64 (other gammas: fp64), which the bound covers from
// |y| = 2^-64 on.  Chunks of 8 columns below 2^-50 take fp64; a smaller value in another chunk
// has code 0 however it is rounded.

// The bf16 results of one chunk (v: its 8 values; g, b: two float4 of gamma and of beta, the
// second `step` behind the first): fp32 where the bracket decides, else (or where !plain) fp64.
__device__ __noinline__ uint4 ln_chunk_exact(const uint4 v, const float4* g, const float4* b, int step, double mean,
                                             double rstd, bool plain) {
  using E = Elem<__nv_bfloat16>;
  const float mh = (float)mean, ml = (float)(mean - (double)mh), r32 = (float)rstd;
  uint4 out;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 gv = reinterpret_cast<const float2*>(g + (i >> 1) * step)[i & 1];
    const float2 bv = reinterpret_cast<const float2*>(b + (i >> 1) * step)[i & 1];
    const float x0 = E::at(v, 2 * i), x1 = E::at(v, 2 * i + 1);
    const float y0 = fmaf(fmaf(x0 - mh, r32, -ml * r32), gv.x, bv.x), y1 = fmaf(fmaf(x1 - mh, r32, -ml * r32), gv.y, bv.y);
    const float e0 = fabsf(y0) + fabsf(bv.x), e1 = fabsf(y1) + fabsf(bv.y);
    uint32_t h = pack_bf16x2(fmaf(e0, -0x1p-21f, y0), fmaf(e1, -0x1p-21f, y1));
    if (!plain || h != pack_bf16x2(fmaf(e0, 0x1p-21f, y0), fmaf(e1, 0x1p-21f, y1)))
      h = bf16_bits_fp64(((double)x0 - mean) * rstd * (double)gv.x + (double)bv.x) |
          (bf16_bits_fp64(((double)x1 - mean) * rstd * (double)gv.y + (double)bv.y) << 16);
    (&out.x)[i] = h;
  }
  return out;
}

constexpr int kLn8Threads = 256;

// nc chunks a thread (nc * TPR * 8 >= K).  TPR = 128: 128 threads a CTA.
// ANY: rows of any alignment and K.
template <int TPR, bool ANY>
__global__ void __launch_bounds__(TPR == 128 ? 128 : kLn8Threads, TPR == 128 ? 8 : 4)
    ln_rows_int8_kernel(const __nv_bfloat16* x, int ldx, int M, int K, int nc,
                        const __nv_bfloat16* gamma, const __nv_bfloat16* beta, double eps,
                        int8_t* q, int ldq, float* s) {
  using E = Elem<__nv_bfloat16>;
  constexpr int LANES = TPR < 32 ? TPR : 32;
  extern __shared__ float4 ln8_smem[];     // gamma, beta: chunk c of thread t at (2c + half) * TPR + t; then the chunks
  __shared__ double sh_sum[2][4];
  __shared__ uint32_t sh_max[4];
  const int t = threadIdx.x % TPR, warp = threadIdx.x >> 5, rows = blockDim.x / TPR;
  float4* sg = ln8_smem;
  float4* sb = ln8_smem + 2 * nc * TPR;
  uint4* mine = reinterpret_cast<uint4*>(ln8_smem + 4 * nc * TPR) + threadIdx.x;   // chunk c at c * blockDim.x
  const int pitch = blockDim.x;
  pdl_trigger();
  pdl_wait();
  // rows in groups, so that the warps that share rows (or a CTA) stay together to the end
  int row0 = blockIdx.x * rows + (TPR < 32 ? warp * (32 / TPR) : TPR == 32 ? warp : 0);
  const int sub = TPR < 32 ? (threadIdx.x & 31) / TPR : 0;
  const int stride = gridDim.x * rows;
  const uint32_t mine_s = smem_u32(mine);
  auto fetch = [&](int r0) {   // a spare half warp repeats its neighbour's row
    const int r = r0 + sub < M ? r0 + sub : r0;
    const __nv_bfloat16* xt = x + (size_t)r * ldx + t * 8;
    if constexpr (ANY) {   // the row's units; unit i has the place of chunk i
      const uint32_t off = row_off(xt - t * 8);
      const int n = (K * 2 + (int)off + 15) / 16;
      const __nv_bfloat16* end = x + (size_t)(M - 1) * ldx + K;
      for (int c = 0, i = t; i < n; ++c, i += TPR) fetch_unit(xt - t * 8, off, i, K, x, end, mine + c * pitch);
    } else {
      uint32_t dst = mine_s;
#pragma unroll 3
      for (int c = 0, col = t * 8; c < nc; ++c, col += 8 * TPR, dst += 16 * pitch)
        cp_async16(dst, col < K ? xt + c * (8 * TPR) : x, col < K ? 16u : 0u);
    }
    cp_async_commit();
  };
  if (row0 < M) fetch(row0);
  const bool wide = !ANY && ((reinterpret_cast<uintptr_t>(gamma) | reinterpret_cast<uintptr_t>(beta)) & 15u) == 0;
  bool huge = false;   // a gamma of 2^64 or more
  for (int i = threadIdx.x; i < nc * TPR; i += blockDim.x) {   // 8 columns
    const int col = i * 8;
    uint4 gu = make_uint4(0u, 0u, 0u, 0u), bu = gu;
    if (col < K) {
      gu = wide ? *reinterpret_cast<const uint4*>(gamma + col) : load_chunk_edge(gamma, col, K);
      bu = wide ? *reinterpret_cast<const uint4*>(beta + col) : load_chunk_edge(beta, col, K);
    }
    huge |= chunk_mag<__nv_bfloat16>(gu) >= 0x5F80u;
    const int at = (2 * (i / TPR)) * TPR + i % TPR;
    sg[at] = make_float4(E::at(gu, 0), E::at(gu, 1), E::at(gu, 2), E::at(gu, 3));
    sg[at + TPR] = make_float4(E::at(gu, 4), E::at(gu, 5), E::at(gu, 6), E::at(gu, 7));
    sb[at] = make_float4(E::at(bu, 0), E::at(bu, 1), E::at(bu, 2), E::at(bu, 3));
    sb[at + TPR] = make_float4(E::at(bu, 4), E::at(bu, 5), E::at(bu, 6), E::at(bu, 7));
  }
  huge = __syncthreads_or(huge);
  auto sum2 = [&](double& a, double& b) {   // over the threads of a row
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
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
  for (; row0 < M; row0 += stride) {
    const int row = row0 + sub;
    cp_async_wait<0>();
    if (ANY) {   // units to chunks, in place: a chunk's second unit is the next thread's, or the next chunk's first
      const uint32_t off = row_off(x + (size_t)(row < M ? row : row0) * ldx);
      const int n = (K * 2 + (int)off + 15) / 16;
      const uint4* next = t + 1 < TPR ? mine + 1 : mine + 1 - TPR + pitch;
#pragma unroll 1
      for (int c = 0; c < nc; ++c) {
        const int i = c * TPR + t;
        if (TPR > 32) __syncthreads();
        else __syncwarp();
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (i * 8 < K) u = chunk_of_units<__nv_bfloat16>(mine[c * pitch], i + 1 < n ? next[c * pitch] : u, off, i * 8, K);
        if (TPR > 32) __syncthreads();
        else __syncwarp();
        mine[c * pitch] = u;
      }
    }
    double s1 = 0.0, s2 = 0.0, t1 = 0.0, t2 = 0.0;
#pragma unroll 3
    for (int c = 0; c < nc; ++c) {
      const uint4 u = mine[c * pitch];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const double a = (double)E::at(u, i), b = (double)E::at(u, i + 1);
        s1 += a;
        t1 += b;
        s2 = fma(a, a, s2);
        t2 = fma(b, b, t2);
      }
    }
    s1 += t1;
    s2 += t2;
    sum2(s1, s2);
    // one division for both: even threads have the mean, odd ones the mean square
    const double of_k = ((t & 1) ? s2 : s1) / (double)K;
    const double mean = __shfl_sync(0xffffffffu, of_k, 0, LANES), square = __shfl_sync(0xffffffffu, of_k, 1, LANES);
    double var = fma(-mean, mean, square);
    const bool again = !(square <= 1024.0 * var);   // also for a NaN
    if (TPR <= 32 ? __any_sync(0xffffffffu, again) : again) {   // the sums are the same in all threads of a row
      double d2 = 0.0, none = 0.0;
#pragma unroll 1
      for (int c = 0; c < nc; ++c) {
        const uint4 u = mine[c * pitch];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double d = (double)E::at(u, i) - mean;
          if ((c * TPR + t) * 8 + i < K) d2 = fma(d, d, d2);
        }
      }
      sum2(d2, none);
      var = d2 / (double)K;
    }
    const double rstd = 1.0 / sqrt(var + eps);
    const float mh = (float)mean, ml = (float)(mean - (double)mh), r32 = (float)rstd;
    const bool plain =
        !huge && r32 >= 0x1p-100f && r32 <= 0x1p100f && fabsf(mh) <= 0x1p100f && fabsf(mh) * r32 <= 0x1p100f;
    const uint64_t nmh = f2pack(-mh, -mh), rr = f2pack(r32, r32), nmr = f2pack(-ml * r32, -ml * r32);
    const uint64_t up = f2pack(0x1p-21f, 0x1p-21f), dn = f2pack(-0x1p-21f, -0x1p-21f);
    uint32_t m = 0u;   // bits of the largest |y|, whose bf16 rounding is the largest |bf16(y)|; a NaN is above all
    const float4 *gp = sg + t, *bp = sb + t;
    uint4* at = mine;
#pragma unroll 1
    for (int c = 0; c < nc; ++c, gp += 2 * TPR, bp += 2 * TPR, at += pitch) {
      const uint4 u = *at;
      const float4 g0 = gp[0], g1 = gp[TPR], b0 = bp[0], b1 = bp[TPR];
      const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
      const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
      uint32_t h[4], differ = plain ? 0u : 1u;
      float cm = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t xc = fadd2(f2pack(E::at(u, 2 * i), E::at(u, 2 * i + 1)), nmh);
        const uint64_t y = ffma2(ffma2(xc, rr, nmr), f2pack(g[2 * i], g[2 * i + 1]), f2pack(b[2 * i], b[2 * i + 1]));
        const float2 yf = f2unpack(y);
        const uint64_t e = f2pack(fabsf(yf.x) + fabsf(b[2 * i]), fabsf(yf.y) + fabsf(b[2 * i + 1]));
        h[i] = bf16x2_of(ffma2(e, dn, y));
        differ |= h[i] ^ bf16x2_of(ffma2(e, up, y));
        cm = fmax3_nan(cm, fabsf(yf.x), fabsf(yf.y));   // gamma or beta may bring a NaN
      }
      uint4 w = make_uint4(h[0], h[1], h[2], h[3]);
      const bool tiny = __float_as_uint(cm) - 1u < __float_as_uint(0x1p-50f) - 1u;   // 0 < cm < 2^-50
      if (differ || tiny) {
        w = ln_chunk_exact(u, gp, bp, TPR, mean, rstd, plain && !tiny);
        cm = E::of_mag(chunk_mag<__nv_bfloat16>(w));
      }
      // columns past K have gamma = beta = 0, so y = 0 (or NaN, in a row that has one anyway)
      m = max(m, __float_as_uint(cm));
      *at = w;
    }
    if (TPR < 32) {
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    } else {
      m = __reduce_max_sync(0xffffffffu, m);
    }
    if (TPR > 32) {
      if ((threadIdx.x & 31) == 0) sh_max[warp] = m;
      __syncthreads();
      m = max(max(sh_max[0], sh_max[1]), max(sh_max[2], sh_max[3]));
    }
    const RowScale sc =
        row_scale<__nv_bfloat16>((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(m))) & 0x7FFFu);
    if (row < M) {
      int8_t* qt = q + (size_t)row * ldq + t * 8;
#pragma unroll 3
      for (int c = 0, col = t * 8; c < nc; ++c, col += 8 * TPR)
        if (col < K) store_codes<__nv_bfloat16, ANY>(mine[c * pitch], sc, qt + c * (8 * TPR), col, K);
    }
    if (row < M && t == 0) s[row] = sc.s;
    if (row0 + stride < M) fetch(row0 + stride);
  }
}

// ---------------------------------------------------------------- any width
// Rows too wide for the kernels above (K > 32768 in fp32; LayerNorm, K > 16384): one CTA
// per row, single elements, the row read again in each pass.
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
    rows_int8_any_kernel(const T* x, int ldx, int M, int K, const __nv_bfloat16* gamma,
                         const __nv_bfloat16* beta, double eps, int8_t* q, int ldq,
                         float* s) {
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
    return b;
  };
  uint32_t m = 0u;
  for (int k = threadIdx.x; k < K; k += kAnyThreads) m = max(m, bits(k) & (sizeof(T) == 2 ? 0x7FFFu : 0x7FFFFFFFu));
  const RowScale sc = row_scale<T>(row_max<kAnyThreads>(m, sh_max));
  for (int k = threadIdx.x; k < K; k += kAnyThreads)
    q[(size_t)row * ldq + k] = (int8_t)code_of<T>(value_of_bits<T>(bits(k)), sc);
  if (threadIdx.x == 0) s[row] = sc.s;
}

// ---------------------------------------------------------------- launch
// Rows that start on 16 bytes and hold whole chunks.
template <class T>
bool rows_whole(const RowsInt8& a) {
  return (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && ((size_t)a.ldx * sizeof(T)) % 16 == 0 &&
         a.K % Elem<T>::PER == 0;
}

template <int OP, class T, int TPR, int NC>
cudaError_t rows_launch(const RowsInt8& a, int num_sms, cudaStream_t st) {
  long long grid = TPR == 32 ? ((long long)a.M + 7) / 8 : a.M;
  const bool whole = rows_whole<T>(a);
  if (OP == kI8Gelu) {   // as many CTAs as fit the GPU: 16 warps an SM, 256 threads a whole row 24
    const long long most = (long long)num_sms * (TPR == 32 ? 2 : TPR >= 1024 ? 1 : TPR == 256 && whole ? 3 : 512 / TPR);
    if (grid > most) grid = most;
  }
  auto kern = whole ? rows_int8_kernel<OP, T, TPR, NC, false> : rows_int8_kernel<OP, T, TPR, NC, true>;
  const int units = (a.K * (int)sizeof(T) + 15) / 16 + 2;   // a row in units it may not start on, and one behind
  const size_t smem = whole ? 0 : (size_t)units * 16 * (TPR == 32 ? 8 : 1);
  if (smem > 32 * 1024) {
    // The limit is the kernel's, not the launch's: always the most that any row takes, so that a call in another
    // thread does not lower it between this and the launch.
    constexpr int kMost = (NC * TPR + 2) * 16 * (TPR == 32 ? 8 : 1);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3((unsigned)grid), dim3(TPR == 32 ? 256 : TPR), smem, st, (const T*)a.x, a.ldx, a.M, a.K,
                    units, a.q, a.ldq, a.s);
}

template <int OP, class T>
cudaError_t rows_any_launch(const RowsInt8& a, cudaStream_t st) {
  return launch_pdl(rows_int8_any_kernel<OP, T>, dim3((unsigned)a.M), dim3(kAnyThreads), 0, st, (const T*)a.x, a.ldx,
                    a.M, a.K, a.gamma, a.beta, a.eps, a.q, a.ldq, a.s);
}

// Chunks a thread at most (launch_ln_quant_int8 goes by it).
template <int TPR> constexpr int kLn8Chunks = TPR == 16 ? 9 : TPR == 32 ? 8 : 16;

template <int TPR>
cudaError_t ln_rows_launch(const RowsInt8& a, int num_sms, cudaStream_t st) {
  const int nc = (a.K + 8 * TPR - 1) / (8 * TPR);
  constexpr int kMostThreads = TPR == 128 ? 128 : kLn8Threads;
  // as many threads a CTA as leave every SM one (gamma and beta are staged once a CTA)
  int threads = kMostThreads;
  while (threads > 32 && TPR < 128 && (long long)num_sms * threads / TPR > a.M) threads /= 2;
  // (one more row of chunks for the unit behind the last in rows that start inside one)
  const size_t smem = (size_t)nc * 16 * (4 * TPR + threads) + (rows_whole<__nv_bfloat16>(a) ? 0 : 16 * threads);
  auto kern = rows_whole<__nv_bfloat16>(a) ? ln_rows_int8_kernel<TPR, false> : ln_rows_int8_kernel<TPR, true>;
  // the kernel's limit, as in rows_launch: the most that any row and number of rows takes
  constexpr int kMost = kLn8Chunks<TPR> * 16 * (4 * TPR + kMostThreads) + 16 * kMostThreads;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  if (e != cudaSuccess) return e;
  const int per_sm = (int)(220 * 1024 / (smem + 1024));
  const int rows = threads / TPR;
  const long long ctas = ((long long)a.M + rows - 1) / rows;
  const long long most = (long long)num_sms * (per_sm < 1024 / threads ? per_sm : 1024 / threads);
  return launch_pdl(kern, dim3((unsigned)(ctas < most ? ctas : most)), dim3(threads), smem, st,
                    (const __nv_bfloat16*)a.x, a.ldx, a.M, a.K, nc, a.gamma, a.beta, a.eps, a.q, a.ldq, a.s);
}

// Threads a row: as few as hold it in 9 chunks each (5 for rows of up to 160).
template <int OP, class T>
cudaError_t rows_dispatch(const RowsInt8& a, int num_sms, cudaStream_t st) {
  const int chunks = (a.K + Elem<T>::PER - 1) / Elem<T>::PER;
  if (chunks <= 160) return rows_launch<OP, T, 32, 5>(a, num_sms, st);
  if (chunks <= 288) return rows_launch<OP, T, 32, 9>(a, num_sms, st);
  if (chunks <= 576) return rows_launch<OP, T, 64, 9>(a, num_sms, st);
  if (chunks <= 1152) return rows_launch<OP, T, 128, 9>(a, num_sms, st);
  if (chunks <= 2304) return rows_launch<OP, T, 256, 9>(a, num_sms, st);
  if (sizeof(T) == 2 || chunks <= 8192) return rows_launch<OP, T, 1024, 8>(a, num_sms, st);   // 2 bytes: K <= 65536
  if constexpr (sizeof(T) == 4) return rows_any_launch<OP, T>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_quant_int8(const RowsInt8& a, int dtype, int num_sms, cudaStream_t st) {
  if (a.M == 0) return cudaSuccess;
  if (dtype == 0) return rows_dispatch<kI8Plain, __nv_bfloat16>(a, num_sms, st);
  if (dtype == 1) return rows_dispatch<kI8Plain, __half>(a, num_sms, st);
  return rows_dispatch<kI8Plain, float>(a, num_sms, st);
}
cudaError_t launch_ln_quant_int8(const RowsInt8& a, int num_sms, cudaStream_t st) {
  if (a.M == 0) return cudaSuccess;
  const int chunks = (a.K + 7) / 8;
  if (chunks <= 16 * kLn8Chunks<16>) return ln_rows_launch<16>(a, num_sms, st);
  if (chunks <= 32 * kLn8Chunks<32>) return ln_rows_launch<32>(a, num_sms, st);
  if (chunks <= 128 * kLn8Chunks<128>) return ln_rows_launch<128>(a, num_sms, st);
  return rows_any_launch<kI8Ln, __nv_bfloat16>(a, st);
}
cudaError_t launch_gelu_quant_int8(const RowsInt8& a, int num_sms, cudaStream_t st) {
  return a.M == 0 ? cudaSuccess : rows_dispatch<kI8Gelu, __nv_bfloat16>(a, num_sms, st);
}

}  // namespace vitq
