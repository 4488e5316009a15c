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

constexpr int kRopeAxThreads = 256;   // wanted; one head has up to 511 items (head_dim 512, one pair)

template <class T, int VEC> struct alignas(sizeof(T) * VEC) RopeVec { T v[VEC]; };

// (cos, sin) of pair j of a token at pos: the angle in turns, in fp64 (a far position times a
// frequency needs more bits than fp32 has), reduced to half a turn exactly.  For bf16 and fp16
// tensors what is left is rounded to fp32 (2^-23 rad at most, against a last rounding of 2^-9 or
// 2^-12); for fp32 tensors sine and cosine are taken in fp64 and rounded once (4096 tokens of 20
// heads of 128: 19.0 us against 18.8, rms error 3.7e-8 against 5.4e-8 at positions about 10^5).
template <class T>
__device__ __forceinline__ float2 rope_cos_sin(const RopeAxes& p, int token, int j) {
  const double turn = (double)p.pos[token * p.pos_t + p.axis[j] * p.pos_a] * p.turns[j];
  float sn, cn;
  if constexpr (sizeof(T) == 4) {
    double s64, c64;
    sincospi(2.0 * (turn - rint(turn)), &s64, &c64);
    sn = (float)s64;
    cn = (float)c64;
  } else {
    sincospif((float)(2.0 * (turn - rint(turn))), &sn, &cn);
  }
  return make_float2(cn, p.inverse ? -sn : sn);
}

// fp32 -> T, two at a time where T has 2 bytes.
template <class T, int VEC>
__device__ __forceinline__ RopeVec<T, VEC> rope_round(const float (&x)[VEC]) {
  RopeVec<T, VEC> r;
  if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) reinterpret_cast<uint32_t*>(&r)[i / 2] = round2<T>(x[i], x[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.v[i] = of_f32<T>(x[i]);
  }
  return r;
}

// A CTA has `toks` tokens and walks their heads (a token's q, then its k) in memory order,
// `step` heads at a time: a thread keeps its item of a head (VEC pairs, or, behind the rotary
// part, VEC elements to copy), and its head and token advance without a division.  The
// order counts: with several heads of a thread in flight, so that the CTA's accesses spread
// over as many places, 16384 tokens of 40 heads of 128 took 94 us instead of 54, and with
// all tokens' q before their k 58.  Whole 16-byte units of 72-wide heads with the partners
// exchanged by shuffles were slower as well (8192 tokens of 32 heads: 26 us against 20).
// Half style pairs (j, j + pairs), adjacent style (2j, 2j + 1).  Bound by HBM; 8 CTAs an SM
// (32 registers) 55.1 us, 5 with the 40 that the compiler takes by itself 62.5.
template <class T, int VEC, bool ADJ>
__global__ void __launch_bounds__(VEC == 1 ? 2 * kRopeAxThreads : kRopeAxThreads, VEC == 1 ? 1 : 8)
    rope_axes_kernel(const __grid_constant__ RopeAxes p, int toks, int per_head, int step, int step_t, int step_h) {
  using V = RopeVec<T, VEC>;
  extern __shared__ float2 cs[];   // (cos, sin): two pairs in 16 bytes, see cs_at
  pdl_trigger();
  pdl_wait();
  const int rot = p.pairs / VEC, hq = p.side[0].heads, heads = hq + p.side[1].heads;
  const int tok0 = blockIdx.x * toks, ntok = min(toks, p.n - tok0);
  // pair VEC c + k of token t: neighbouring items' 16-byte units side by side
  auto cs_at = [&](int t, int c, int k) {
    return VEC == 1 ? t * p.pairs + c : t * p.pairs + (k / 2 * rot + c) * 2 + k % 2;
  };
  for (int i = threadIdx.x; i < ntok * p.pairs; i += blockDim.x) {
    const int t = i / p.pairs, j = i - t * p.pairs;
    cs[cs_at(t, j / VEC, j % VEC)] = rope_cos_sin<T>(p, tok0 + t, j);
  }
  __syncthreads();
  const int at = threadIdx.x / per_head, c = threadIdx.x - at * per_head;
  if (at >= step) return;   // the last threads of an uneven CTA
  const bool turns = c < rot;
  // where the item's first vector lies in a head, and its second one from there
  const int lo = turns ? (ADJ ? 2 * c * VEC : c * VEC) : 2 * p.pairs + (c - rot) * VEC, ahead = ADJ ? VEC : p.pairs;
  // of head 0 of q, and of the head that would be head 0 if k's heads followed q's
  const T* xq = reinterpret_cast<const T*>(p.side[0].x) + (long long)tok0 * p.side[0].xt + lo;
  const T* xk = reinterpret_cast<const T*>(p.side[1].x) + (long long)tok0 * p.side[1].xt - (long long)hq * p.side[1].xh + lo;
  T* yq = reinterpret_cast<T*>(p.side[0].y) + (long long)tok0 * p.side[0].yt + lo;
  T* yk = reinterpret_cast<T*>(p.side[1].y) + (long long)tok0 * p.side[1].yt - (long long)hq * p.side[1].yh + lo;
  int t = at / heads, h = at - t * heads;
  while (t < ntok) {
    const bool q = h < hq;
    const T* x = (q ? xq : xk) + (long long)t * (q ? p.side[0].xt : p.side[1].xt) + (long long)h * (q ? p.side[0].xh : p.side[1].xh);
    T* y = (q ? yq : yk) + (long long)t * (q ? p.side[0].yt : p.side[1].yt) + (long long)h * (q ? p.side[0].yh : p.side[1].yh);
    const V a = *reinterpret_cast<const V*>(x);
    if (turns) {
      const V b = *reinterpret_cast<const V*>(x + ahead);
      float xa[VEC], xb[VEC];   // as loaded, then turned
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        xa[k] = to_f32<T>(a.v[k]);
        xb[k] = to_f32<T>(b.v[k]);
      }
      float2 f[VEC];
      if constexpr (VEC == 1) {
        f[0] = cs[cs_at(t, c, 0)];
      } else {
#pragma unroll
        for (int k = 0; k < VEC; k += 2)
          *reinterpret_cast<float4*>(f + k) = *reinterpret_cast<const float4*>(cs + cs_at(t, c, k));
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        // pair k of this item: (xa[k], xb[k]), or neighbours in the 2 VEC elements
        float& ea = ADJ ? (2 * k < VEC ? xa[(2 * k) % VEC] : xb[(2 * k) % VEC]) : xa[k];
        float& eb = ADJ ? (2 * k + 1 < VEC ? xa[(2 * k + 1) % VEC] : xb[(2 * k + 1) % VEC]) : xb[k];
        const float va = ea, vb = eb;
        ea = __fmaf_rn(va, f[k].x, -__fmul_rn(vb, f[k].y));
        eb = __fmaf_rn(vb, f[k].x, __fmul_rn(va, f[k].y));
      }
      *reinterpret_cast<V*>(y) = rope_round<T, VEC>(xa);
      *reinterpret_cast<V*>(y + ahead) = rope_round<T, VEC>(xb);
    } else if (y != x) {   // past the rotary part: copied
      *reinterpret_cast<V*>(y) = a;
    }
    t += step_t;
    h += step_h;
    if (h >= heads) {
      h -= heads;
      ++t;
    }
  }
}

// Tokens of a CTA: about as many angles as make it worth the wait, as few as keep its
// accesses together (16384 tokens of 40 heads of 128: 2 tokens 55.2 us, 3 56.8, 5 61.6, 8 64.8;
// 8192 of 32 heads of 72: 3 19.9, 4 19.7, 5 20.6, 8 20.5), and fewer where that leaves SMs
// idle.
int rope_tokens(const RopeAxes& p, int num_sms) {
  int toks = 144 / p.pairs;
  if (toks > p.n / (4 * num_sms)) toks = p.n / (4 * num_sms);
  return toks < 1 ? 1 : toks > 16 ? 16 : toks;
}

template <class T, int VEC>
cudaError_t rope_axes_vec(const RopeAxes& p, int num_sms, cudaStream_t st) {
  const int heads = p.side[0].heads + p.side[1].heads;
  const int per_head = p.pairs / VEC + (p.d - 2 * p.pairs) / VEC;
  auto kern = p.adjacent ? rope_axes_kernel<T, VEC, true> : rope_axes_kernel<T, VEC, false>;
  const int toks = rope_tokens(p, num_sms);
  int step = kRopeAxThreads / per_head;
  if (step < 1) step = 1;
  if (step > toks * heads) step = toks * heads;
  const int threads = (step * per_head + 31) / 32 * 32;
  return launch_pdl(kern, dim3((unsigned)((p.n + toks - 1) / toks)), dim3(threads),
                    (size_t)toks * p.pairs * sizeof(float2), st, p, toks, per_head, step, step / heads, step % heads);
}

// The widest access that every pointer, stride and split of a head allows.
template <class T>
cudaError_t rope_axes_type(const RopeAxes& p, int num_sms, cudaStream_t st) {
  unsigned long long m = (unsigned long long)p.pairs | (unsigned long long)(p.d - 2 * p.pairs);
  for (const RopeSide& s : p.side) {
    if (!s.heads) continue;
    m |= (unsigned long long)(s.xt | s.xh | s.yt | s.yh);
    m |= (reinterpret_cast<uintptr_t>(s.x) | reinterpret_cast<uintptr_t>(s.y)) / sizeof(T);
  }
  if (sizeof(T) == 2 && m % 8 == 0) return rope_axes_vec<T, 16 / sizeof(T)>(p, num_sms, st);
  if (m % 4 == 0) return rope_axes_vec<T, 4>(p, num_sms, st);
  if (m % 2 == 0) return rope_axes_vec<T, 2>(p, num_sms, st);
  return rope_axes_vec<T, 1>(p, num_sms, st);
}

}  // namespace

cudaError_t launch_rope_axes(const RopeAxes& p, int dtype, int num_sms, cudaStream_t st) {
  if (p.n == 0 || p.side[0].heads + p.side[1].heads == 0) return cudaSuccess;
  if (dtype == 0) return rope_axes_type<__nv_bfloat16>(p, num_sms, st);
  if (dtype == 1) return rope_axes_type<__half>(p, num_sms, st);
  return rope_axes_type<float>(p, num_sms, st);
}

}  // namespace vitq
