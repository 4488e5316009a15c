// INT8 GEMM on the sm_100a tensor cores (tcgen05 kind::i8 + TMEM + TMA).
//
//   C[m, n] = T( sA[m] sW[n] sum_k A[m, k] W[n, k] + bias[n] + R[m, n] )
//
// One scale per token and per output channel: nothing changes along K, so the
// whole sum stays in TMEM as exact 32-bit integers (K <= 2^16 and |code| <= 128
// keep it below 2^31) and the scales are applied once per output, in fp32, before
// the one rounding to T.  The sums being exact, every kernel below gives the same bits:
//   few rows    M <= 1024   mma.sync, weights read once for each group of 8 to 32 tokens; bound by
//                           L2 / HBM bytes, and at one group by the rounds of K (see there)
//   split K     M <= 1024   128 x 64 / 128 tiles, a cluster's CTAs share K; bound by latency
//   tiles       128 x 128, one CTA each, persistent
//   pairs       256 x 256, two CTAs each, persistent; bound by the tensor cores
// (int8_choose.h has the choice.)
// 25024 x 3456 x 1152 (pairs, bf16): 84 .. 87 us in short runs, 98 .. 104 under the power
// limit, against 62 .. 64 at the measured FP8 rate (3125 TFLOP/s); the tensor pipe is busy
// half of the time.  A K block of a pair takes about 780 cycles without loads or epilogue.
// 6256 x 1152 x 4304 with residual: 35.9 us (19.8).  243 x 2048 x 4608: 10.4 (1.9).
// 1 x 4608 x 4608: 6.0 (3.3), 21 MB of weights at 3.5 TB/s.
#include "int8_choose.h"
#include "internal.h"
#include "ptx.cuh"

#include <cuda_fp16.h>

#include <type_traits>

namespace vitq {
namespace {

struct I8Args {
  const float* sA;
  const float* sW;
  const void* bias;
  const void* residual;
  void* C;
  int ldr, ldc, M, N, K;
  // whether rows of C and of the residual lie on 16 bytes (base and pitch): boxes of the residual
  // then arrive by TMA, otherwise in words of r_word bytes (4, or 2).  c_tma: boxes of C leave by
  // TMA.  That also takes rows that end on 16 bytes: a store writes whole 16-byte units and so up
  // to 14 bytes behind a row that ends inside one.
  int c_units, c_tma, r_tma, r_word;
};

// ------------------------------------------------------------------ output types
template <class T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T of_f32(float v);
template <> __device__ __forceinline__ float of_f32(float v) { return v; }
template <> __device__ __forceinline__ __half of_f32(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 of_f32(float v) { return __float2bfloat16_rn(v); }

// 16 bytes of T -> fp32 and back.
template <class T>
__device__ __forceinline__ void unpack16(const uint4& u, float* v) {
  const T* p = reinterpret_cast<const T*>(&u);
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(T)); ++i) v[i] = to_f32<T>(p[i]);
}
// Two values, the first in the low half.
template <class T> __device__ __forceinline__ uint32_t round2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t round2<__nv_bfloat16>(float lo, float hi) { return pack_bf16x2(lo, hi); }
template <> __device__ __forceinline__ uint32_t round2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <class T>
__device__ __forceinline__ uint4 pack16(const float* v) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  else
    return make_uint4(round2<T>(v[0], v[1]), round2<T>(v[2], v[3]), round2<T>(v[4], v[5]), round2<T>(v[6], v[7]));
}

// ------------------------------------------------------------------ tiles
// kPair: two CTAs (cta_group::2) share one 256 x BN tile: each holds 128 rows of A, half
// of the W rows, and the accumulator of its own 128 rows.
template <int BN, bool kPair, int kCols>
struct I8Cfg {
  static constexpr int BM = 128, BK = 128;   // 128 codes = one 128B swizzle row
  static constexpr int TILE_M = kPair ? 256 : 128;
  static constexpr int B_ROWS = kPair ? BN / 2 : BN;
  static constexpr int STAGES = BN / kCols > 2 ? 4 : 5;
  static constexpr int A_BYTES = BM * BK;
  static constexpr int B_BYTES = B_ROWS * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int NACC = 2;              // TMEM accumulators, alternating between tiles
  static constexpr int COLS = kCols;                   // columns of an epilogue warp (and a row quadrant)
  static constexpr int EPI_WARPS = BN / COLS * 4, EPI_WARP0 = 4;
  static constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
  static constexpr int BOX_BYTES = 4096;      // 32 rows x 128 bytes of C
  static constexpr int OUT_BYTES = EPI_WARPS * BOX_BYTES;
  static constexpr int COL_BYTES = EPI_WARPS * COLS * 8;   // sW, then bias, of the warp's columns
  static constexpr int BAR_BYTES = (2 * STAGES + 2 * NACC + EPI_WARPS) * 8 + 16;
  static constexpr size_t SMEM = (size_t)STAGES * STAGE_BYTES + OUT_BYTES + COL_BYTES + 1024 + BAR_BYTES;
};

template <class Config>
struct I8Smem {
  using Cfg = Config;
  uint8_t* base;
  __device__ uint32_t a(int s) const { return smem_u32(base + (size_t)s * Cfg::STAGE_BYTES); }
  __device__ uint32_t b(int s) const { return a(s) + Cfg::A_BYTES; }
  __device__ uint8_t* out(int w) const {
    return base + (size_t)Cfg::STAGES * Cfg::STAGE_BYTES + (size_t)w * Cfg::BOX_BYTES;
  }
  __device__ float* cols(int w) const {
    return reinterpret_cast<float*>(base + (size_t)Cfg::STAGES * Cfg::STAGE_BYTES + Cfg::OUT_BYTES) + w * 2 * Cfg::COLS;
  }
  __device__ uint64_t* bars() const {
    return reinterpret_cast<uint64_t*>(base + (size_t)Cfg::STAGES * Cfg::STAGE_BYTES + Cfg::OUT_BYTES + Cfg::COL_BYTES);
  }
  __device__ uint32_t full(int s) const { return smem_u32(bars() + s); }
  __device__ uint32_t empty(int s) const { return smem_u32(bars() + Cfg::STAGES + s); }
  __device__ uint32_t tfull(int b) const { return smem_u32(bars() + 2 * Cfg::STAGES + b); }
  __device__ uint32_t tempty(int b) const { return smem_u32(bars() + 2 * Cfg::STAGES + Cfg::NACC + b); }
  __device__ uint32_t res_full(int w) const { return smem_u32(bars() + 2 * Cfg::STAGES + 2 * Cfg::NACC + w); }
  __device__ uint32_t* tmem_holder() const {
    return reinterpret_cast<uint32_t*>(bars() + 2 * Cfg::STAGES + 2 * Cfg::NACC + Cfg::EPI_WARPS);
  }
  __device__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(tmem_holder() + 1); }
};

// Tile order: down 8 row tiles, then to the next column tile, so that CTAs that run
// together share tiles of both operands (25024 x 3456 x 1152: 101.5 us, against 105.1 in
// the diagonal order of the other GEMMs).
__device__ __forceinline__ void i8_tile_coords(int tile, int tiles_m, int tiles_n, int& m, int& n) {
  const int group = tile / (8 * tiles_n), in = tile - group * 8 * tiles_n, rows = min(8, tiles_m - 8 * group);
  n = in / rows;
  m = 8 * group + in - n * rows;
}

// Tiles of this CTA (or pair): t0, t0 + dt, ...
template <int BN, bool kPair, class Cfg>
__device__ void i8_producer(const I8Smem<Cfg>& sm, const CUtensorMap* tmA, const CUtensorMap* tmB, int tiles_m,
                            int tiles_n, int num_tiles, int nkb, int t0, int dt, int rank) {
  int stage = 0;
  uint32_t phase = 0;
  for (int tile = t0; tile < num_tiles; tile += dt) {
    int mt, nt;
    i8_tile_coords(tile, tiles_m, tiles_n, mt, nt);
    const int m0 = mt * Cfg::TILE_M + rank * Cfg::BM, n0 = nt * BN + rank * Cfg::B_ROWS;
    for (int kb = 0; kb < nkb; ++kb) {
      if (!mbar_wait(sm.empty(stage), phase ^ 1u, sm.abort_flag())) return;
      if (kPair) {   // both CTAs' copies count on the leader's barrier, which expects them all
        const uint32_t full0 = mapa_shared(sm.full(stage), 0);
        if (rank == 0) mbar_arrive_expect_tx(sm.full(stage), 2 * Cfg::STAGE_BYTES);
        tma_load_2d_pair(sm.a(stage), tmA, kb * Cfg::BK, m0, full0);
        tma_load_2d_pair(sm.b(stage), tmB, kb * Cfg::BK, n0, full0);
      } else {
        mbar_arrive_expect_tx(sm.full(stage), Cfg::STAGE_BYTES);
        tma_load_2d(sm.a(stage), tmA, kb * Cfg::BK, m0, sm.full(stage));
        tma_load_2d(sm.b(stage), tmB, kb * Cfg::BK, n0, sm.full(stage));
      }
      if (++stage == Cfg::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
}

template <int BN, bool kPair, class Cfg>
__device__ void i8_mma(const I8Smem<Cfg>& sm, uint32_t tmem_base, int num_tiles, int nkb, int K, int t0, int dt) {
  constexpr uint32_t idesc = make_idesc_i8(Cfg::TILE_M, BN);
  int stage = 0;
  uint32_t phase = 0, it = 0;
  for (int tile = t0; tile < num_tiles; tile += dt, ++it) {
    const uint32_t acc = it % Cfg::NACC;
    if (!mbar_wait(sm.tempty(acc), ((it / Cfg::NACC) & 1u) ^ 1u, sm.abort_flag())) return;
    tc_fence_after();
    for (int kb = 0; kb < nkb; ++kb) {
      if (!mbar_wait(sm.full(stage), phase, sm.abort_flag())) return;
      tc_fence_after();
      const uint32_t a0 = sm.a(stage), b0 = sm.b(stage);
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // 32 codes each; steps that lie past K hold zeros and are left out
        if (kb * Cfg::BK + 32 * k >= K) break;
        const uint64_t ad = make_smem_desc(a0 + 32 * k, 16, 1024, kSwizzle128B);
        const uint64_t bd = make_smem_desc(b0 + 32 * k, 16, 1024, kSwizzle128B);
        if (kPair)
          mma_i8_ss_pair(tmem_base + acc * BN, ad, bd, idesc, (kb > 0 || k > 0) ? 1u : 0u);
        else
          mma_i8_ss(tmem_base + acc * BN, ad, bd, idesc, (kb > 0 || k > 0) ? 1u : 0u);
      }
      if (kPair)
        tc_commit_pair(sm.empty(stage), 0x3);
      else
        tc_commit(sm.empty(stage));
      if (++stage == Cfg::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (kPair)
      tc_commit_pair(sm.tfull(acc), 0x3);
    else
      tc_commit(sm.tfull(acc));
  }
}

// Byte b of row r of a box of 32 rows x 128 bytes (TMA's 128-byte swizzle).
__device__ __forceinline__ int box_at(int r, int b) { return r * 128 + (b ^ ((r & 7) << 4)); }

// A box between shared memory and rows of any alignment, word by word: lanes along the
// row, so that each access of the warp is one run of 128 (or 64) bytes.  rows, bytes:
// what of the box lies inside the matrix.
template <class W>
__device__ __noinline__ void box_load(uint8_t* slot, const uint8_t* mat, size_t pitch, int rows, int bytes) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int b = lane * (int)sizeof(W); b < bytes; b += 32 * (int)sizeof(W)) {
    // 16 in flight (6251 x 1153 x 4303 with residual: 40.3 us; all 32 spill, 48.6)
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 16) {
      W v[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] = *reinterpret_cast<const W*>(mat + min(r0 + r, rows - 1) * pitch + b);
#pragma unroll
      for (int r = 0; r < 16; ++r) *reinterpret_cast<W*>(slot + box_at(r0 + r, b)) = v[r];
    }
  }
}
// A box to rows of any alignment: whole 16-byte units of the matrix, put together from two
// units of the box (8 lanes a row, 4 rows at a time), then the elements before the first
// and behind the last unit.  E: element type by size.
template <class E>
__device__ __noinline__ void box_store(const uint8_t* slot, uint8_t* mat, size_t pitch, int rows, int bytes) {
  const int lane = threadIdx.x & 31, k = lane & 7;
#pragma unroll 2
  for (int r = lane >> 3; r < rows; r += 4) {
    uint8_t* row = mat + r * pitch;
    const int lead = (int)(-reinterpret_cast<uintptr_t>(row) & 15u);   // bytes before the first unit
    const int at = lead + 16 * k, whole = bytes > lead ? (bytes - lead) & ~15 : 0;
    if (at < lead + whole) {
      uint32_t v[8];
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(slot + box_at(r, at & ~15));
      // the unit behind the last is not read from (its bytes are shifted out when lead = 0)
      *reinterpret_cast<uint4*>(v + 4) = *reinterpret_cast<const uint4*>(slot + box_at(r, min(at + 15, 127) & ~15));
#pragma unroll
      for (int i = 0; i < 6; ++i) v[i] = lead & 8 ? v[i + 2] : v[i];
#pragma unroll
      for (int i = 0; i < 5; ++i) v[i] = lead & 4 ? v[i + 1] : v[i];
      if (sizeof(E) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lead & 2 ? __byte_perm(v[i], v[i + 1], 0x5432) : v[i];
      }
      *reinterpret_cast<uint4*>(row + at) = make_uint4(v[0], v[1], v[2], v[3]);
    }
    const int head = min(lead, bytes), edge = bytes - whole;   // bytes: [0, head) and [head + whole, bytes)
    for (int e = k * (int)sizeof(E); e < edge; e += 8 * (int)sizeof(E)) {
      const int b = e < head ? e : e + whole;
      *reinterpret_cast<E*>(row + b) = *reinterpret_cast<const E*>(slot + box_at(r, b));
    }
  }
}

// Epilogue warp: 32 rows (thread = row) and Cfg::COLS columns (64, or 128 where pairs have long
// sums), 32 columns at a time; the 16 warps of a 256-wide tile with 64 columns each, four a
// scheduler, hide each other's latencies (8 with 128 columns: i8_pairs).  A 128-byte-wide box of C (one, or
// two in fp32) has a slot in shared memory: the residual is brought there first (for the
// first box while the tile's sum is still running), the finished box leaves from there.
// kWords: C or the residual may need word-by-word rows (a kernel of its own, so that the
// extra paths cost the others no registers: 6 % of a large product's time).
template <int BN, bool kPair, bool kWords, class T, class Cfg>
__device__ void i8_epilogue(const I8Smem<Cfg>& sm, uint32_t tmem_base, const I8Args& g, const CUtensorMap* tmC,
                            const CUtensorMap* tmR, int tiles_m, int tiles_n, int num_tiles, int t0, int dt, int rank) {
  constexpr int PER = 16 / (int)sizeof(T);          // elements per 16 bytes
  constexpr int BOXC = 128 / (int)sizeof(T);        // columns per box
  constexpr int PER_BOX = BOXC / 32, NBOX = Cfg::COLS / BOXC;
  // the leader's tempty barriers count both CTAs' epilogue warps
  const uint32_t tempty0 = kPair ? mapa_shared(sm.tempty(0), 0) : sm.tempty(0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ew = warp - Cfg::EPI_WARP0, quad = warp & 3, part = ew >> 2;
  uint8_t* slot = sm.out(ew);
  float* sw_s = sm.cols(ew);
  float* bias_s = sw_s + Cfg::COLS;
  const T* bias = reinterpret_cast<const T*>(g.bias);
  const bool has_res = g.residual != nullptr;
  uint32_t it = 0, res_phase = 0;
  for (int tile = t0; tile < num_tiles; tile += dt, ++it) {
    int mt, nt;
    i8_tile_coords(tile, tiles_m, tiles_n, mt, nt);
    const int col0 = nt * BN + part * Cfg::COLS;
    const int y0 = mt * Cfg::TILE_M + rank * Cfg::BM + quad * 32, row = y0 + lane;
    const uint32_t acc = it % Cfg::NACC;
    const int nbox = y0 < g.M ? min(NBOX, (g.N - col0 + BOXC - 1) / BOXC) : 0;   // boxes with a column of C (may be < 0)
    const int rows = min(32, g.M - y0);
    // brings the residual of box b of this tile to the slot, once the last store has read it
    auto fetch_res = [&](int b) {
      const int c0 = col0 + b * BOXC;
      if (lane == 0) bulk_wait_read_all();
      if (!kWords || g.r_tma) {
        fence_proxy_async_smem();   // the warp's own accesses to the slot come before the copy
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_expect_tx(sm.res_full(ew), Cfg::BOX_BYTES);
          tma_load_2d(smem_u32(slot), tmR, c0, y0, sm.res_full(ew));
        }
      } else {
        __syncwarp();
        const uint8_t* mat = reinterpret_cast<const uint8_t*>(g.residual) + ((size_t)y0 * g.ldr + c0) * sizeof(T);
        const int bytes = min(128, (g.N - c0) * (int)sizeof(T));
        if (sizeof(T) == 4 || g.r_word == 4) box_load<uint32_t>(slot, mat, (size_t)g.ldr * sizeof(T), rows, bytes);
        else box_load<uint16_t>(slot, mat, (size_t)g.ldr * sizeof(T), rows, bytes);
        __syncwarp();
      }
    };
    if (has_res && nbox > 0) fetch_res(0);
    __syncwarp();
#pragma unroll
    for (int c = lane; c < Cfg::COLS; c += 32) {
      const int n = col0 + c;
      sw_s[c] = n < g.N ? g.sW[n] : 0.f;
      bias_s[c] = bias && n < g.N ? to_f32<T>(bias[n]) : 0.f;
    }
    const float sa = row < g.M ? g.sA[row] : 0.f;
    const uint64_t sa2 = f2pack(sa, sa);
    __syncwarp();
    bool ok = mbar_wait(sm.tfull(acc), (it / Cfg::NACC) & 1u, sm.abort_flag());
    if (!__all_sync(0xffffffffu, ok)) return;
    tc_fence_after();
    const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + acc * BN + part * Cfg::COLS;
#pragma unroll
    for (int b = 0; b < NBOX; ++b) {
      if (b < nbox) {   // uniform
        if (has_res) {
          if (b > 0) fetch_res(b);
          if (!kWords || g.r_tma) {
            ok = mbar_wait(sm.res_full(ew), res_phase, sm.abort_flag());
            if (!__all_sync(0xffffffffu, ok)) return;
            res_phase ^= 1u;
          }
        } else if (!kWords || g.c_tma) {   // the last store has read the slot
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
        }
#pragma unroll
        for (int h = 0; h < PER_BOX; ++h) {
          const int gr = b * PER_BOX + h;   // 32 columns (past N: zero scales)
          uint32_t r[32];
          tmem_ld32(taddr + gr * 32, r);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32 / PER; ++c) {
            float v[PER];
#pragma unroll
            for (int i = 0; i < PER; i += 4) {
              const int at = gr * 32 + c * PER + i;
              const float4 w = *reinterpret_cast<const float4*>(sw_s + at);
              const float4 bi = *reinterpret_cast<const float4*>(bias_s + at);
              const uint32_t* a = r + c * PER + i;
              const float2 lo = f2unpack(ffma2(fmul2(f2pack(__int2float_rn((int)a[0]), __int2float_rn((int)a[1])), sa2),
                                               f2pack(w.x, w.y), f2pack(bi.x, bi.y)));
              const float2 hi = f2unpack(ffma2(fmul2(f2pack(__int2float_rn((int)a[2]), __int2float_rn((int)a[3])), sa2),
                                               f2pack(w.z, w.w), f2pack(bi.z, bi.w)));
              v[i] = lo.x;
              v[i + 1] = lo.y;
              v[i + 2] = hi.x;
              v[i + 3] = hi.y;
            }
            uint4* at = reinterpret_cast<uint4*>(slot + box_at(lane, h * 32 * (int)sizeof(T) + c * 16));
            if (has_res) {
              float rv[PER];
              unpack16<T>(*at, rv);
#pragma unroll
              for (int i = 0; i < PER; ++i) v[i] += rv[i];
            }
            *at = pack16<T>(v);
          }
        }
        const int c0 = col0 + b * BOXC;
        if (!kWords || g.c_tma) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {   // TMA clips rows past M and columns past N
            tma_store_2d(tmC, smem_u32(slot), c0, y0);
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          uint8_t* mat = reinterpret_cast<uint8_t*>(g.C) + ((size_t)y0 * g.ldc + c0) * sizeof(T);
          const int bytes = min(128, (g.N - c0) * (int)sizeof(T));
          box_store<std::conditional_t<sizeof(T) == 2, uint16_t, uint32_t>>(slot, mat, (size_t)g.ldc * sizeof(T), rows, bytes);
        }
        __syncwarp();
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if (kPair)
        mbar_arrive_cluster(tempty0 + acc * 8);
      else
        mbar_arrive(sm.tempty(acc));
    }
  }
  if (lane == 0) bulk_wait_all();
}

template <int BN, bool kPair, int kCols, bool kWords, class T>
__global__ void __launch_bounds__(I8Cfg<BN, kPair, kCols>::THREADS, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmR,
                     const I8Args args) {
  using Cfg = I8Cfg<BN, kPair, kCols>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  pdl_trigger();
  I8Smem<Cfg> sm;
  sm.base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nkb = (args.K + Cfg::BK - 1) / Cfg::BK;
  const int tiles_m = (args.M + Cfg::TILE_M - 1) / Cfg::TILE_M;
  const int tiles_n = (args.N + BN - 1) / BN;
  const int num_tiles = tiles_m * tiles_n;
  const int rank = kPair ? (int)cluster_ctarank() : 0;
  const int t0 = kPair ? (int)blockIdx.x / 2 : (int)blockIdx.x;
  const int dt = kPair ? (int)gridDim.x / 2 : (int)gridDim.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(sm.full(s), 1);
      mbar_init(sm.empty(s), 1);
    }
    for (int b = 0; b < Cfg::NACC; ++b) {
      mbar_init(sm.tfull(b), 1);
      mbar_init(sm.tempty(b), Cfg::EPI_WARPS * (kPair ? 2 : 1));
    }
    for (int w = 0; w < Cfg::EPI_WARPS; ++w) mbar_init(sm.res_full(w), 1);
    *sm.abort_flag() = 0;
    fence_barrier_init();
  }
  if (kPair) cluster_sync_all();   // the peer's barriers exist before anything signals them
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(smem_u32(sm.tmem_holder()), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(sm.tmem_holder()), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();   // inputs may be the previous kernel's outputs
  const uint32_t tmem_base = *sm.tmem_holder();
  if (warp < Cfg::EPI_WARP0) {
    if (warp == 0 && lane == 0) {
      i8_producer<BN, kPair>(sm, &tmA, &tmB, tiles_m, tiles_n, num_tiles, nkb, t0, dt, rank);
    } else if (warp == 1 && lane == 0 && rank == 0) {
      i8_mma<BN, kPair>(sm, tmem_base, num_tiles, nkb, args.K, t0, dt);
    }
  } else {
    i8_epilogue<BN, kPair, kWords, T>(sm, tmem_base, args, &tmC, &tmR, tiles_m, tiles_n, num_tiles, t0, dt, rank);
  }
  tc_fence_before();
  __syncthreads();
  if (*sm.abort_flag()) settle_pause(50000);
  // neither CTA of a pair leaves while the leader's MMAs may still use the peer's memory
  if (kPair) cluster_sync_all();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (kPair)
      tmem_dealloc_pair(tmem_base, 512);
    else
      tmem_dealloc(tmem_base, 512);
  }
}

// How a box of C leaves and one of the residual arrives (I8Args).
void i8_paths(const Int8Gemm& p, int es, I8Args* a) {
  // widest access that a base address, a row pitch and (word by word) the row's length allow
  auto bytes = [&](const void* base, size_t pitch) {
    const uintptr_t v = reinterpret_cast<uintptr_t>(base) | pitch;
    return v % 16 == 0 ? 16 : (v | (size_t)p.N * es) % 4 == 0 ? 4 : 2;
  };
  a->c_units = bytes(p.C, (size_t)p.ldc * es) == 16;
  a->c_tma = a->c_units && (size_t)p.N * es % 16 == 0;
  a->r_word = p.residual ? bytes(p.residual, (size_t)p.ldr * es) : 0;
  a->r_tma = a->r_word == 16;
}

template <int BN, bool kPair, int kCols, class T>
cudaError_t i8_launch(const Int8Gemm& p, bool words, int num_sms, cudaStream_t st) {
  using Cfg = I8Cfg<BN, kPair, kCols>;
  constexpr int es = (int)sizeof(T);
  I8Args a{p.sA, p.sW, p.bias, p.residual, p.C, p.ldr, p.ldc, p.M, p.N, p.K, 0, 0, 0, 0};
  i8_paths(p, es, &a);
  const size_t pc = (size_t)p.ldc * es, pr = (size_t)p.ldr * es;
  CUtensorMap tmA, tmB, tmC, tmR;
  cudaError_t e = encode_tma_2d_ld(&tmA, 1, p.A, p.K, p.M, (size_t)p.lda, 128, 128);
  if (e != cudaSuccess) return e;
  e = encode_tma_2d_ld(&tmB, 1, p.W, p.K, p.N, (size_t)p.ldw, 128, Cfg::B_ROWS);
  if (e != cudaSuccess) return e;
  tmC = tmR = tmA;   // where not used
  if (a.c_tma) e = encode_tma_2d_ld(&tmC, es, p.C, p.N, p.M, pc, 128 / es, 32);
  if (e == cudaSuccess && a.r_tma) e = encode_tma_2d_ld(&tmR, es, p.residual, p.N, p.M, pr, 128 / es, 32);
  if (e != cudaSuccess) return e;
  constexpr bool kMayWords = kCols == 64;   // see i8_pairs
  auto kern = int8_gemm_kernel<BN, kPair, kCols, false, T>;
  if constexpr (kMayWords)
    if (words) kern = int8_gemm_kernel<BN, kPair, kCols, true, T>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::SMEM);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)((p.M + Cfg::TILE_M - 1) / Cfg::TILE_M) * ((p.N + BN - 1) / BN);
  const int units = kPair ? num_sms / 2 : num_sms;
  const int grid = tiles < units ? (int)tiles : units;
  return kPair ? launch_pdl_cluster(kern, 2, dim3(2 * grid), dim3(Cfg::THREADS), Cfg::SMEM, st, tmA, tmB, tmC, tmR, a)
               : launch_pdl(kern, dim3(grid), dim3(Cfg::THREADS), Cfg::SMEM, st, tmA, tmB, tmC, tmR, a);
}

// ------------------------------------------------------------------ few rows
// A CTA has 8 NT tokens and 16 CT output channels: every weight is read once for 8 NT tokens and
// used a few times, so what counts is bytes in flight.  Its 8 warps take 64-byte pieces of K in
// turn, U at a time, and add up in shared memory at the end.  (A round of pieces waits for the one
// before: at K = 4608 a warp has 9 pieces and takes them 4 + 4 + 1.  1 x 4608 x 4608 takes 6.0 us,
// the floor being 3.3.)  m16n8k32 products with the channels as
// rows; a lane's 16 bytes of a row serve two of them (the sum over K may be taken in any
// order as long as weights and tokens agree), so nothing passes through shared memory
// on the way in.
constexpr int kRowsWarps = 8;

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 codes of a weight row (used once: not kept in L1).
__device__ __forceinline__ uint4 ld_once(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
// The last n < 16 codes of a row, zeros behind them.
__device__ __noinline__ uint4 ld_last(const int8_t* p, int n) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < 15; ++i)
    if (i < n) (&v.x)[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
  return v;
}

// NT: groups of 8 tokens, CT: groups of 16 channels of a CTA; gridDim.y covers more tokens.
template <int NT, int CT, class T>
__global__ void __launch_bounds__(32 * kRowsWarps)
    int8_gemm_rows_kernel(const int8_t* A, int lda, const int8_t* W, int ldw, const I8Args g) {
  constexpr int U = NT + 2 * CT <= 4 ? 4 : NT + 2 * CT <= 6 ? 3 : 2;   // pieces of K in flight
  constexpr int CH = 16 * CT;
  __shared__ int part[kRowsWarps][NT * 8][CH + 1];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * CH, m0 = blockIdx.y * NT * 8;
  // rows past the end repeat the last one; their sums are not used
  const int8_t* w[2 * CT];
  const int8_t* a[NT];
#pragma unroll
  for (int c = 0; c < 2 * CT; ++c) w[c] = W + (size_t)min(n0 + q + 8 * c, g.N - 1) * ldw + t * 16;
#pragma unroll
  for (int j = 0; j < NT; ++j) a[j] = A + (size_t)min(m0 + j * 8 + q, g.M - 1) * lda + t * 16;
  int acc[CT][NT][4] = {};
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int k = warp * 64; k < g.K; k += U * 64 * kRowsWarps) {
    uint4 u[U][2 * CT], b[U][NT];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int kk = k + i * 64 * kRowsWarps;
      const bool in = kk + t * 16 + 16 <= g.K;
#pragma unroll
      for (int c = 0; c < 2 * CT; ++c) u[i][c] = in ? ld_once(w[c] + kk) : zero;
#pragma unroll
      for (int j = 0; j < NT; ++j) b[i][j] = in ? *reinterpret_cast<const uint4*>(a[j] + kk) : zero;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int kk = k + i * 64 * kRowsWarps, left = g.K - (kk + t * 16);   // codes of this piece inside K
      if (left > 0 && left < 16) {
#pragma unroll
        for (int c = 0; c < 2 * CT; ++c) u[i][c] = ld_last(w[c] + kk, left);
#pragma unroll
        for (int j = 0; j < NT; ++j) b[i][j] = ld_last(a[j] + kk, left);
      }
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 &x = u[i][2 * c], &y = u[i][2 * c + 1];
          mma_s8(acc[c][j], x.x, y.x, x.y, y.y, b[i][j].x, b[i][j].y);
          mma_s8(acc[c][j], x.z, y.z, x.w, y.w, b[i][j].z, b[i][j].w);
        }
    }
  }
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 4; ++h) part[warp][j * 8 + 2 * t + (h & 1)][c * 16 + q + 8 * (h >> 1)] = acc[c][j][h];
  __syncthreads();
  for (int e = threadIdx.x; e < NT * 8 * CH; e += 32 * kRowsWarps) {
    const int m = m0 + e / CH, c = e % CH, n = n0 + c;
    if (m >= g.M || n >= g.N) continue;
    int sum = 0;
#pragma unroll
    for (int x = 0; x < kRowsWarps; ++x) sum += part[x][e / CH][c];
    float v = __fmaf_rn(__fmul_rn(__int2float_rn(sum), g.sA[m]), g.sW[n],
                        g.bias ? to_f32<T>(reinterpret_cast<const T*>(g.bias)[n]) : 0.f);
    if (g.residual) v += to_f32<T>(reinterpret_cast<const T*>(g.residual)[(size_t)m * g.ldr + n]);
    reinterpret_cast<T*>(g.C)[(size_t)m * g.ldc + n] = of_f32<T>(v);
  }
}

// ------------------------------------------------------------------ split K
// Few tiles: a cluster of S CTAs (2, 4 or 8) shares one 128 x BN tile, each with its part of
// K.  CTA p finishes the BN / S columns p * BN / S ..; every CTA sorts its integer sums by
// their owner in its own shared memory and sends each owner its block in one bulk copy, the
// owner adds the S blocks (exact, so the order does not matter).  Read by the owner with
// plain loads from the other CTAs' shared memory instead, the same sums took 4 to 6 us.
// One tile per CTA, no persistence.  The ring is as deep as the part of K or shared memory
// allows, so that narrow tiles keep as many bytes in flight as wide ones; A takes the rows
// it has (M < 128), the MMA reads on into what follows, which only reaches sums of rows past
// M.
struct SplitCfg {
  static constexpr int BM = 128, BK = 128, MAX_STAGES = 32;
  static constexpr int THREADS = 384;                   // warps 0: TMA, 1: MMA, 4 .. 11: epilogue
  static constexpr int BAR_BYTES = (2 * MAX_STAGES + 2) * 8 + 16;
  static constexpr int COL_BYTES = 2 * 64 * 4;          // sW and bias of the CTA's columns
  static constexpr int RING_BYTES = 144 * 1024;
  static constexpr int IN_BYTES = 56 * 1024;            // blocks from the other CTAs: BN * 512 * (S - 1) / S
  static constexpr size_t SMEM = (size_t)RING_BYTES + IN_BYTES + COL_BYTES + 1024 + BAR_BYTES;
};
static_assert(128 * 512 * 7 / 8 <= SplitCfg::IN_BYTES && 128 * 512 <= SplitCfg::RING_BYTES, "blocks");

// The 8 epilogue warps of a split-K CTA.
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// 16-byte unit u of row r of a block of rows of `units` units (a power of two), placed so
// that 8 rows' accesses to one unit meet all banks.
__device__ __forceinline__ uint32_t block_at(int r, int u, int units) {
  const int k = units < 8 ? units : 8;
  return (uint32_t)(r * units + (u ^ ((r * k / 8) & (k - 1)))) * 16u;
}

template <int BN, class T>
__global__ void __launch_bounds__(SplitCfg::THREADS, 1)
    int8_gemm_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                           const I8Args g, int a_rows, int parts, int stages) {
  using Cfg = SplitCfg;
  constexpr int PER = 16 / (int)sizeof(T);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  pdl_trigger();
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + Cfg::RING_BYTES + Cfg::IN_BYTES + Cfg::COL_BYTES);
  uint8_t* in_s = base + Cfg::RING_BYTES;   // block of the k-th other CTA at k * block bytes
  float* sw_s = reinterpret_cast<float*>(in_s + Cfg::IN_BYTES);
  float* bias_s = sw_s + 64;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * Cfg::MAX_STAGES + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + Cfg::MAX_STAGES + s); };
  const uint32_t done = smem_u32(bars + 2 * Cfg::MAX_STAGES), arrived = smem_u32(bars + 2 * Cfg::MAX_STAGES + 1);
  const uint32_t stage_bytes = BN * Cfg::BK + (uint32_t)a_rows * Cfg::BK;   // A (whole 8-row units of 1 KB), then W
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)blockIdx.x % parts, tile = (int)blockIdx.x / parts;   // clusters are runs of `parts` blocks
  const int tiles_m = (g.M + Cfg::BM - 1) / Cfg::BM;
  const int m0 = tile % tiles_m * Cfg::BM, n0 = tile / tiles_m * BN;
  const int nkb = (g.K + Cfg::BK - 1) / Cfg::BK;
  const int kb0 = (int)((long long)nkb * rank / parts), kb1 = (int)((long long)nkb * (rank + 1) / parts);
  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    mbar_init(arrived, 1);
    *abort_flag = 0;
    fence_barrier_init();
    mbar_arrive_expect_tx(arrived, (uint32_t)(Cfg::BM * BN * 4 / parts) * (parts - 1));
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 128);
    tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync_all();   // the other CTAs' barriers exist before anything signals them
  tc_fence_after();
  pdl_wait();   // inputs may be the previous kernel's outputs
  const uint32_t tmem_base = *tmem_holder;
  // this CTA's columns of the tile; an epilogue thread has one row of them and units of 8
  // columns (half, half + 2, ...)
  constexpr int UNITS = BN / 32;   // parts >= 2
  const int cols = BN / parts, c_first = rank * cols;
  const int quad = warp & 3, half = (warp >> 2) - 1, r = quad * 32 + lane, row = m0 + r;
  const bool row_in = warp >= 4 && row < g.M;
  const uint32_t block = Cfg::BM * BN * 4 / parts;   // bytes that go to one owner
  bool sums_ok = false;
  float sa = 0.f;
  uint4 ru[UNITS][8 / PER];   // residual
  if (warp == 0 && lane == 0) {
    const uint32_t bytes = (uint32_t)(a_rows + BN) * Cfg::BK;
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(empty(stage), phase ^ 1u, abort_flag)) break;
      const uint32_t a = smem_u32(base) + stage * stage_bytes;
      mbar_arrive_expect_tx(full(stage), bytes);
      tma_load_2d(a + a_rows * Cfg::BK, &tmB, kb * Cfg::BK, n0, full(stage));
      tma_load_2d(a, &tmA, kb * Cfg::BK, m0, full(stage));
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = make_idesc_i8(128, BN);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!(ok = mbar_wait(full(stage), phase, abort_flag))) break;
      tc_fence_after();
      const uint32_t a = smem_u32(base) + stage * stage_bytes, b = a + a_rows * Cfg::BK;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (kb * Cfg::BK + 32 * k >= g.K) break;
        mma_i8_ss(tmem_base, make_smem_desc(a + 32 * k, 16, 1024, kSwizzle128B),
                  make_smem_desc(b + 32 * k, 16, 1024, kSwizzle128B), idesc, (kb > kb0 || k > 0) ? 1u : 0u);
      }
      tc_commit(empty(stage));
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (ok) tc_commit(done);
  } else if (warp >= 4) {   // this CTA's part, to its own shared memory (every load has been used)
    // what the epilogue will need, on its way while the products run
    if (threadIdx.x - 128 < cols) {
      const int c = threadIdx.x - 128, n = n0 + c_first + c;
      sw_s[c] = n < g.N ? g.sW[n] : 0.f;
      bias_s[c] = g.bias && n < g.N ? to_f32<T>(reinterpret_cast<const T*>(g.bias)[n]) : 0.f;
    }
    if (row_in) sa = g.sA[row];
    // no residual: -0, which leaves any sum as it is (a product that underflows to -0 too)
    constexpr uint32_t none = sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      const int u = half + 2 * k, n = n0 + c_first + u * 8;
#pragma unroll
      for (int h = 0; h < 8 / PER; ++h) ru[k][h] = make_uint4(none, none, none, none);
      if (g.residual && row_in && u < cols / 8 && n < g.N) {
        const T* res = reinterpret_cast<const T*>(g.residual) + (size_t)row * g.ldr + n;
        if (n + 8 <= g.N && g.r_tma) {
#pragma unroll
          for (int h = 0; h < 8 / PER; ++h) ru[k][h] = reinterpret_cast<const uint4*>(res)[h];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n + i < g.N) reinterpret_cast<T*>(&ru[k][0])[i] = res[i];
        }
      }
    }
    const bool ok = mbar_wait(done, 0, abort_flag);
    if (__all_sync(0xffffffffu, ok) && m0 + quad * 32 < g.M) {
      tc_fence_after();
#pragma unroll
      for (int gr = 0; gr < (BN + 63) / 64; ++gr) {
        const int c = half * (BN / 2) + gr * 32;
        uint32_t v[32];
        tmem_ld32(tmem_base + ((uint32_t)(quad * 32) << 16) + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int owner = (c + 4 * i) / cols, u = (c + 4 * i - owner * cols) / 4;
          *reinterpret_cast<uint4*>(base + owner * block + block_at(r, u, cols / 4)) =
              make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
      tc_fence_before();
    }
    fence_proxy_async_smem();
    epilogue_sync();   // reached by all 8 warps, after a timed-out wait too
    if (threadIdx.x == 128) {   // rows past M are sent as they are: nobody reads them
      for (int k = 1; k < parts; ++k) {
        const int to = (rank + k) % parts, slot = parts - 1 - k;   // this CTA is `to`'s (parts - k)-th neighbour
        bulk_copy_cluster(mapa_shared(smem_u32(in_s) + slot * block, to), smem_u32(base) + to * block, block,
                          mapa_shared(arrived, to));
      }
    }
    sums_ok = mbar_wait(arrived, 0, abort_flag) && ok;
    sums_ok = __all_sync(0xffffffffu, sums_ok);
  }
  if (row_in && sums_ok) {
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      const int u = half + 2 * k, c = c_first + u * 8, n = n0 + c;
      if (u < cols / 8 && n < g.N) {
        int4 lo = make_int4(0, 0, 0, 0), hi = lo;
#pragma unroll 4
        for (int p = 0; p < parts; ++p) {
          const uint8_t* src = p == 0 ? base + rank * block : in_s + (p - 1) * block;
          const int4 a = *reinterpret_cast<const int4*>(src + block_at(r, 2 * u, cols / 4));
          const int4 b = *reinterpret_cast<const int4*>(src + block_at(r, 2 * u + 1, cols / 4));
          lo = make_int4(lo.x + a.x, lo.y + a.y, lo.z + a.z, lo.w + a.w);
          hi = make_int4(hi.x + b.x, hi.y + b.y, hi.z + b.z, hi.w + b.w);
        }
        const int acc[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        float v[8];
#pragma unroll
        for (int h = 0; h < 8 / PER; ++h) unpack16<T>(ru[k][h], v + h * PER);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] += __fmaf_rn(__fmul_rn(__int2float_rn(acc[i]), sa), sw_s[u * 8 + i], bias_s[u * 8 + i]);
        T* out = reinterpret_cast<T*>(g.C) + (size_t)row * g.ldc + n;
        if (n + 8 <= g.N && g.c_units) {
#pragma unroll
          for (int h = 0; h < 8 / PER; ++h) reinterpret_cast<uint4*>(out)[h] = pack16<T>(v + h * PER);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n + i < g.N) out[i] = of_f32<T>(v[i]);
        }
      }
    }
  }
  __syncthreads();
  if (*abort_flag) settle_pause(50000);
  cluster_sync_all();   // no CTA leaves before every copy between them has arrived
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 128);
  }
}

template <int BN, class T>
cudaError_t i8_launch_split(const Int8Gemm& p, int parts, cudaStream_t st) {
  using Cfg = SplitCfg;
  I8Args a{p.sA, p.sW, p.bias, p.residual, p.C, p.ldr, p.ldc, p.M, p.N, p.K, 0, 0, 0, 0};
  i8_paths(p, (int)sizeof(T), &a);
  const int a_rows = p.M < Cfg::BM ? (p.M + 7) / 8 * 8 : Cfg::BM;
  const int stage_bytes = (BN + a_rows) * Cfg::BK;
  const int nkb = ((p.K + 127) / 128 + parts - 1) / parts;
  // the MMA of the last stage reads 16 KB from the start of its A tile on
  const int behind = stage_bytes < Cfg::BM * Cfg::BK ? Cfg::BM * Cfg::BK - stage_bytes : 0;
  int stages = (Cfg::RING_BYTES - behind) / stage_bytes;
  if (stages > Cfg::MAX_STAGES) stages = Cfg::MAX_STAGES;
  if (stages > nkb) stages = nkb;
  CUtensorMap tmA, tmB;
  cudaError_t e = encode_tma_2d_ld(&tmA, 1, p.A, p.K, p.M, (size_t)p.lda, 128, a_rows);
  if (e != cudaSuccess) return e;
  e = encode_tma_2d_ld(&tmB, 1, p.W, p.K, p.N, (size_t)p.ldw, 128, BN);
  if (e != cudaSuccess) return e;
  auto kern = int8_gemm_split_kernel<BN, T>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::SMEM);
  if (e != cudaSuccess) return e;
  const int tiles = ((p.M + Cfg::BM - 1) / Cfg::BM) * ((p.N + BN - 1) / BN);
  return launch_pdl_cluster(kern, parts, dim3(tiles * parts), dim3(Cfg::THREADS), Cfg::SMEM, st, tmA, tmB, a, a_rows,
                            parts, stages);
}

template <int NT, int CT, class T>
cudaError_t i8_launch_rows(const Int8Gemm& p, cudaStream_t st) {
  const I8Args a{p.sA, p.sW, p.bias, p.residual, p.C, p.ldr, p.ldc, p.M, p.N, p.K, 0, 0, 0, 0};
  return launch_pdl(int8_gemm_rows_kernel<NT, CT, T>, dim3((p.N + 16 * CT - 1) / (16 * CT), (p.M + 8 * NT - 1) / (8 * NT)),
                    dim3(32 * kRowsWarps), 0, st, p.A, p.lda, p.W, p.ldw, a);
}

// Pairs' epilogue: 8 warps (128 columns each) and 5 stages while the sums take longer than
// it, else 16 warps (64 columns) and 4. 25024 x 3456 x 1152: 101.5 against 109.4 us;
// 20000 x 2688 x 221: 38.1 against 32.9 us. Rows moved word by word: always 16 warps.
template <class T>
cudaError_t i8_pairs(const Int8Gemm& p, bool words, int num_sms, cudaStream_t st) {
  return words || p.K <= 512 ? i8_launch<256, true, 64, T>(p, words, num_sms, st)
                             : i8_launch<256, true, 128, T>(p, false, num_sms, st);
}

// Whether C or the residual has rows that TMA cannot move.
bool i8_words(const Int8Gemm& p) {
  I8Args a{};
  i8_paths(p, p.dtype == 2 ? 4 : 2, &a);
  return !a.c_tma || (p.residual && !a.r_tma);
}

template <class T>
cudaError_t i8_run(const Int8Gemm& p, int num_sms, cudaStream_t st) {
  switch (i8_choose(p.M, p.N, p.K, num_sms)) {
    case kRows11: return i8_launch_rows<1, 1, T>(p, st);
    case kRows21: return i8_launch_rows<2, 1, T>(p, st);
    case kRows22: return i8_launch_rows<2, 2, T>(p, st);
    case kRows41: return i8_launch_rows<4, 1, T>(p, st);
    case kTile: return i8_launch<128, false, 64, T>(p, i8_words(p), num_sms, st);
    case kPairs: return i8_pairs<T>(p, i8_words(p), num_sms, st);
    case kSplit64x2: return i8_launch_split<64, T>(p, 2, st);
    case kSplit64x4: return i8_launch_split<64, T>(p, 4, st);
    case kSplit128x2: return i8_launch_split<128, T>(p, 2, st);
    case kSplit128x4: return i8_launch_split<128, T>(p, 4, st);
    case kSplit128x8: return i8_launch_split<128, T>(p, 8, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_int8_gemm(const Int8Gemm& p, int num_sms, cudaStream_t st) {
  if (p.M == 0) return cudaSuccess;
  if (p.dtype == 0) return i8_run<__nv_bfloat16>(p, num_sms, st);
  if (p.dtype == 1) return i8_run<__half>(p, num_sms, st);
  return i8_run<float>(p, num_sms, st);
}

}  // namespace vitq
