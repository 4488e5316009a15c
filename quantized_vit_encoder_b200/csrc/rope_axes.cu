// Rotary positions with several axes (time, row, column) on q and k of any layout.
//
//   angle_j = pos[axis(j)] f_j,   x'_a = x_a cos - x_b sin,   x'_b = x_b cos + x_a sin
//
// for pair j = (a, b) of a head; the inverse (the gradient) turns by -angle_j.
#include "internal.h"
#include "ptx.cuh"

#include <cuda_fp16.h>

namespace vitq {
namespace {

constexpr int kRopeAxThreads = 256;
constexpr int kRopeAxTok = 4;   // tokens per CTA

template <class T, int VEC> struct alignas(sizeof(T) * VEC) RopeVec { T v[VEC]; };

// VEC elements at a time; half style pairs (j, j + pairs), adjacent style (2j, 2j + 1).
template <class T, int VEC, bool ADJ>
__global__ void __launch_bounds__(kRopeAxThreads) rope_axes_kernel(const __grid_constant__ RopeAxes p) {
  using V = RopeVec<T, VEC>;
  extern __shared__ float2 cs[];   // [kRopeAxTok][pairs]: (cos, sin)
  pdl_trigger();
  pdl_wait();
  const int tok0 = blockIdx.x * kRopeAxTok;
  const int ntok = min(kRopeAxTok, p.n - tok0);
  // The angle in turns, in fp64 (a far position times a frequency needs more bits than
  // fp32 has), reduced to half a turn exactly; what is left fits fp32.
  for (int i = threadIdx.x; i < ntok * p.pairs; i += kRopeAxThreads) {
    const int t = i / p.pairs, j = i - t * p.pairs;
    const double turn = (double)p.pos[(tok0 + t) * p.pos_t + p.axis[j] * p.pos_a] * p.turns[j];
    float sn, cn;
    sincospif((float)(2.0 * (turn - rint(turn))), &sn, &cn);
    cs[i] = make_float2(cn, p.inverse ? -sn : sn);
  }
  __syncthreads();
  const int rot = p.pairs / VEC;                       // rotating items per head
  const int heads = p.side[0].heads + p.side[1].heads;
  const int items = heads * (rot + (p.d - 2 * p.pairs) / VEC);
  const int per_head = items / heads;
  for (int i = threadIdx.x; i < ntok * items; i += kRopeAxThreads) {
    const int t = i / items, w = i - t * items;
    int h = w / per_head;
    const int c = w - h * per_head;
    const RopeSide& sd = p.side[h >= p.side[0].heads];
    if (h >= p.side[0].heads) h -= p.side[0].heads;
    const T* x = reinterpret_cast<const T*>(sd.x) + (tok0 + t) * sd.xt + h * sd.xh;
    T* y = reinterpret_cast<T*>(sd.y) + (tok0 + t) * sd.yt + h * sd.yh;
    if (c < rot) {
      const int lo = ADJ ? 2 * c * VEC : c * VEC, hi = ADJ ? lo + VEC : lo + p.pairs;
      V a = *reinterpret_cast<const V*>(x + lo), b = *reinterpret_cast<const V*>(x + hi);
      const float2* f = cs + t * p.pairs + c * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        // element pair k of this item: (a[k], b[k]), or neighbours in the 2 VEC elements
        T& ea = ADJ ? (2 * k < VEC ? a.v[(2 * k) % VEC] : b.v[(2 * k) % VEC]) : a.v[k];
        T& eb = ADJ ? (2 * k + 1 < VEC ? a.v[(2 * k + 1) % VEC] : b.v[(2 * k + 1) % VEC]) : b.v[k];
        const float u = to_f32<T>(ea), v = to_f32<T>(eb);
        const float2 r = f[k];
        ea = of_f32<T>(__fmaf_rn(u, r.x, -__fmul_rn(v, r.y)));
        eb = of_f32<T>(__fmaf_rn(v, r.x, __fmul_rn(u, r.y)));
      }
      *reinterpret_cast<V*>(y + lo) = a;
      *reinterpret_cast<V*>(y + hi) = b;
    } else if (y != x) {   // past the rotary part: copied
      const int at = 2 * p.pairs + (c - rot) * VEC;
      *reinterpret_cast<V*>(y + at) = *reinterpret_cast<const V*>(x + at);
    }
  }
}

template <class T, int VEC>
cudaError_t rope_axes_vec(const RopeAxes& p, cudaStream_t st) {
  auto kern = p.adjacent ? rope_axes_kernel<T, VEC, true> : rope_axes_kernel<T, VEC, false>;
  const unsigned grid = (unsigned)((p.n + kRopeAxTok - 1) / kRopeAxTok);
  return launch_pdl(kern, dim3(grid), dim3(kRopeAxThreads), (size_t)kRopeAxTok * p.pairs * sizeof(float2), st, p);
}

// The widest access that every pointer, stride and split of a head allows.
template <class T>
cudaError_t rope_axes_type(const RopeAxes& p, cudaStream_t st) {
  unsigned long long m = (unsigned long long)p.pairs | (unsigned long long)(p.d - 2 * p.pairs);
  for (const RopeSide& s : p.side) {
    if (!s.heads) continue;
    m |= (unsigned long long)(s.xt | s.xh | s.yt | s.yh);
    m |= (reinterpret_cast<uintptr_t>(s.x) | reinterpret_cast<uintptr_t>(s.y)) / sizeof(T);
  }
  if (sizeof(T) == 2 && m % 8 == 0) return rope_axes_vec<T, 16 / sizeof(T)>(p, st);
  if (m % 4 == 0) return rope_axes_vec<T, 4>(p, st);
  if (m % 2 == 0) return rope_axes_vec<T, 2>(p, st);
  return rope_axes_vec<T, 1>(p, st);
}

}  // namespace

cudaError_t launch_rope_axes(const RopeAxes& p, int dtype, cudaStream_t st) {
  if (p.n == 0 || p.side[0].heads + p.side[1].heads == 0) return cudaSuccess;
  if (dtype == 0) return rope_axes_type<__nv_bfloat16>(p, st);
  if (dtype == 1) return rope_axes_type<__half>(p, st);
  return rope_axes_type<float>(p, st);
}

}  // namespace vitq
