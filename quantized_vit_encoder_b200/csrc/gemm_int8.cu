// INT8 GEMM on the sm_100a tensor cores (tcgen05 kind::i8 + TMEM + TMA).
//
//   C[m, n] = T( sA[m] sW[n] sum_k A[m, k] W[n, k] + bias[n] + R[m, n] )
//
// One scale per token and per output channel: nothing changes along K, so the
// whole sum stays in TMEM as exact 32-bit integers (K <= 2^16 and |code| <= 128
// keep it below 2^31) and the scales are applied once per output, in fp32, before
// the one rounding to T.
#include "internal.h"
#include "ptx.cuh"

#include <cuda_fp16.h>

namespace vitq {
namespace {

struct I8Args {
  const float* sA;
  const float* sW;
  const void* bias;
  const void* residual;
  void* C;
  int ldr, ldc, M, N, K;
  // how a 32-row box of C leaves and one of the residual arrives: by TMA (16-byte aligned
  // base and row pitch), or by the warp in words of this many bytes (4, or 2)
  int c_tma, r_tma, c_word, r_word;
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
template <class T>
__device__ __forceinline__ uint4 pack16(const float* v) {
  uint4 u;
  T* p = reinterpret_cast<T*>(&u);
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(T)); ++i) p[i] = of_f32<T>(v[i]);
  return u;
}

// ------------------------------------------------------------------ tiles
// kPair: two CTAs (cta_group::2) share one 256 x BN tile: each holds 128 rows of A, half
// of the W rows, and the accumulator of its own 128 rows.
template <int BN, bool kPair>
struct I8Cfg {
  static constexpr int BM = 128, BK = 128;   // 128 codes = one 128B swizzle row
  static constexpr int TILE_M = kPair ? 256 : 128;
  static constexpr int B_ROWS = kPair ? BN / 2 : BN;
  static constexpr int STAGES = BN == 256 && !kPair ? 3 : 4;
  static constexpr int A_BYTES = BM * BK;
  static constexpr int B_BYTES = B_ROWS * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int NACC = 2;              // TMEM accumulators, alternating between tiles
  static constexpr int EPI_WARPS = 8, EPI_WARP0 = 4;   // a row quadrant and half of the columns each
  static constexpr int COLS = BN / 2;                  // columns of an epilogue warp
  static constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
  static constexpr int BOX_BYTES = 4096;      // 32 rows x 128 bytes of C
  static constexpr int BOXES = 2;             // per epilogue warp
  static constexpr int OUT_BYTES = EPI_WARPS * BOXES * BOX_BYTES;
  static constexpr int COL_BYTES = EPI_WARPS * COLS * 8;   // sW, then bias, of the warp's columns
  static constexpr int BAR_BYTES = (2 * STAGES + 2 * NACC + EPI_WARPS * BOXES) * 8 + 16;
  static constexpr size_t SMEM = (size_t)STAGES * STAGE_BYTES + OUT_BYTES + COL_BYTES + 1024 + BAR_BYTES;
};

template <int BN, bool kPair>
struct I8Smem {
  using Cfg = I8Cfg<BN, kPair>;
  uint8_t* base;
  __device__ uint32_t a(int s) const { return smem_u32(base + (size_t)s * Cfg::STAGE_BYTES); }
  __device__ uint32_t b(int s) const { return a(s) + Cfg::A_BYTES; }
  __device__ uint8_t* out(int w) const {
    return base + (size_t)Cfg::STAGES * Cfg::STAGE_BYTES + (size_t)w * Cfg::BOXES * Cfg::BOX_BYTES;
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
  __device__ uint32_t res_full(int w, int slot) const {
    return smem_u32(bars() + 2 * Cfg::STAGES + 2 * Cfg::NACC + w * Cfg::BOXES + slot);
  }
  __device__ uint32_t* tmem_holder() const {
    return reinterpret_cast<uint32_t*>(bars() + 2 * Cfg::STAGES + 2 * Cfg::NACC + Cfg::EPI_WARPS * Cfg::BOXES);
  }
  __device__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(tmem_holder() + 1); }
};

// Tile order of the other GEMMs: CTAs that run together read different W tiles.
__device__ __forceinline__ void i8_tile_coords(int tile, int tiles_m, int tiles_n, int& m, int& n) {
  m = tile % tiles_m;
  n = (tile / tiles_m + m) % tiles_n;
}

// Tiles of this CTA (or pair): t0, t0 + dt, ...
template <int BN, bool kPair>
__device__ void i8_producer(const I8Smem<BN, kPair>& sm, const CUtensorMap* tmA, const CUtensorMap* tmB, int tiles_m,
                            int tiles_n, int num_tiles, int nkb, int t0, int dt, int rank) {
  using Cfg = I8Cfg<BN, kPair>;
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

template <int BN, bool kPair>
__device__ void i8_mma(const I8Smem<BN, kPair>& sm, uint32_t tmem_base, int num_tiles, int nkb, int K, int t0, int dt) {
  using Cfg = I8Cfg<BN, kPair>;
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
template <class W, bool kStore>
__device__ __forceinline__ void box_words(uint8_t* slot, uint8_t* mat, size_t pitch, int rows, int bytes) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = lane * (int)sizeof(W); b < 128; b += 32 * (int)sizeof(W)) {
    if (b < bytes) {
      W v[32];   // all in flight at once
#pragma unroll
      for (int r = 0; r < 32; ++r)
        if (r < rows) v[r] = kStore ? *reinterpret_cast<W*>(slot + box_at(r, b)) : *reinterpret_cast<W*>(mat + r * pitch + b);
#pragma unroll
      for (int r = 0; r < 32; ++r)
        if (r < rows) *reinterpret_cast<W*>(kStore ? mat + r * pitch + b : slot + box_at(r, b)) = v[r];
    }
  }
}

// Epilogue warp: 32 rows (thread = row) and COLS columns, 32 columns at a time; the next
// 32 columns' accumulators are on their way while the present ones are scaled.  Each
// 128-byte-wide box of C has one of two slots in shared memory: the residual is brought
// there first (for the first two boxes of a tile while its sum is still running), the
// finished box leaves from there.
template <int BN, bool kPair, class T>
__device__ void i8_epilogue(const I8Smem<BN, kPair>& sm, uint32_t tmem_base, const I8Args& g, const CUtensorMap* tmC,
                            const CUtensorMap* tmR, int tiles_m, int tiles_n, int num_tiles, int t0, int dt, int rank) {
  using Cfg = I8Cfg<BN, kPair>;
  constexpr int PER = 16 / (int)sizeof(T);          // elements per 16 bytes
  constexpr int BOXC = 128 / (int)sizeof(T);        // columns per box
  constexpr int GROUPS = Cfg::COLS / 32, PER_BOX = BOXC / 32, NBOX = Cfg::COLS / BOXC;
  // the leader's tempty barriers count both CTAs' epilogue warps
  const uint32_t tempty0 = kPair ? mapa_shared(sm.tempty(0), 0) : sm.tempty(0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ew = warp - Cfg::EPI_WARP0, quad = warp & 3, half = ew >> 2;
  uint8_t* stg = sm.out(ew);
  float* sw_s = sm.cols(ew);
  float* bias_s = sw_s + Cfg::COLS;
  const T* bias = reinterpret_cast<const T*>(g.bias);
  const bool has_res = g.residual != nullptr;
  uint32_t it = 0, slot_it = 0, res_phase = 0;   // boxes so far; phase of each slot's residual barrier
  for (int tile = t0; tile < num_tiles; tile += dt, ++it) {
    int mt, nt;
    i8_tile_coords(tile, tiles_m, tiles_n, mt, nt);
    const int col0 = nt * BN + half * Cfg::COLS;
    const int y0 = mt * Cfg::TILE_M + rank * Cfg::BM + quad * 32, row = y0 + lane;
    const uint32_t acc = it % Cfg::NACC;
    const int groups = y0 < g.M ? min(GROUPS, (g.N - col0 + 31) >> 5) : 0;   // groups inside C (may be < 0)
    const int nbox = (groups + PER_BOX - 1) / PER_BOX;
    const int rows = min(32, g.M - y0);
    // brings the residual of box b of this tile to its slot, once the slot's last store has read it
    auto fetch_res = [&](int b) {
      uint8_t* slot = stg + ((slot_it + b) & 1u) * Cfg::BOX_BYTES;
      const int c0 = col0 + b * BOXC;
      if (g.r_tma) {
        fence_proxy_async_smem();   // the warp's own accesses to the slot come before the copy
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = sm.res_full(ew, (slot_it + b) & 1u);
          mbar_arrive_expect_tx(bar, Cfg::BOX_BYTES);
          tma_load_2d(smem_u32(slot), tmR, c0, y0, bar);
        }
      } else {
        uint8_t* mat = const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(g.residual)) +
                       ((size_t)y0 * g.ldr + c0) * sizeof(T);
        const int bytes = min(128, (g.N - c0) * (int)sizeof(T));
        if (g.r_word == 4) box_words<uint32_t, false>(slot, mat, (size_t)g.ldr * sizeof(T), rows, bytes);
        else box_words<uint16_t, false>(slot, mat, (size_t)g.ldr * sizeof(T), rows, bytes);
        __syncwarp();
      }
    };
    if (has_res && nbox > 0) {
      if (lane == 0) bulk_wait_read_all();
      __syncwarp();
      fetch_res(0);
      if (nbox > 1) fetch_res(1);
    }
    __syncwarp();
#pragma unroll
    for (int c = lane; c < Cfg::COLS; c += 32) {
      const int n = col0 + c;
      sw_s[c] = n < g.N ? __ldg(g.sW + n) : 0.f;
      bias_s[c] = bias && n < g.N ? to_f32<T>(bias[n]) : 0.f;
    }
    const float sa = row < g.M ? __ldg(g.sA + row) : 0.f;
    const uint64_t sa2 = f2pack(sa, sa);
    __syncwarp();
    bool ok = mbar_wait(sm.tfull(acc), (it / Cfg::NACC) & 1u, sm.abort_flag());
    if (!__all_sync(0xffffffffu, ok)) return;
    tc_fence_after();
    const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + acc * BN + half * Cfg::COLS;
    uint32_t r[2][32];
    if (groups > 0) tmem_ld32(taddr, r[0]);
#pragma unroll
    for (int b = 0; b < NBOX; ++b) {
      if (b < nbox) {   // uniform
        const uint32_t s = (slot_it + b) & 1u;
        uint8_t* slot = stg + s * Cfg::BOX_BYTES;
        if (has_res) {
          if (g.r_tma) {
            ok = mbar_wait(sm.res_full(ew, s), (res_phase >> s) & 1u, sm.abort_flag());
            if (!__all_sync(0xffffffffu, ok)) return;
            res_phase ^= 1u << s;
          }
        } else if (g.c_tma) {   // the store before last has read its box
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
        }
#pragma unroll
        for (int h = 0; h < PER_BOX; ++h) {
          const int gr = b * PER_BOX + h;
          if (gr < groups) {
            tmem_wait_ld();
            if (gr + 1 < groups) tmem_ld32(taddr + (gr + 1) * 32, r[(gr + 1) & 1]);
#pragma unroll
            for (int c = 0; c < 32 / PER; ++c) {
              float v[PER];
#pragma unroll
              for (int i = 0; i < PER; i += 4) {
                const int at = gr * 32 + c * PER + i;
                const float4 w = *reinterpret_cast<const float4*>(sw_s + at);
                const float4 bi = *reinterpret_cast<const float4*>(bias_s + at);
                const uint32_t* a = r[gr & 1] + c * PER + i;
                const float2 lo =
                    f2unpack(ffma2(fmul2(f2pack(__int2float_rn((int)a[0]), __int2float_rn((int)a[1])), sa2),
                                   f2pack(w.x, w.y), f2pack(bi.x, bi.y)));
                const float2 hi =
                    f2unpack(ffma2(fmul2(f2pack(__int2float_rn((int)a[2]), __int2float_rn((int)a[3])), sa2),
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
        }
        const int c0 = col0 + b * BOXC;
        if (g.c_tma) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {   // TMA clips rows past M and columns past N
            tma_store_2d(tmC, smem_u32(slot), c0, y0);
            bulk_commit_group();
            if (has_res && b + 2 < nbox) bulk_wait_read<0>();
          }
        } else {
          __syncwarp();
          uint8_t* mat = reinterpret_cast<uint8_t*>(g.C) + ((size_t)y0 * g.ldc + c0) * sizeof(T);
          const int bytes = min(128, (g.N - c0) * (int)sizeof(T));
          if (g.c_word == 4) box_words<uint32_t, true>(slot, mat, (size_t)g.ldc * sizeof(T), rows, bytes);
          else box_words<uint16_t, true>(slot, mat, (size_t)g.ldc * sizeof(T), rows, bytes);
        }
        __syncwarp();
        if (has_res && b + 2 < nbox) fetch_res(b + 2);
      }
    }
    if (nbox > 0) slot_it += nbox;
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

template <int BN, bool kPair, class T>
__global__ void __launch_bounds__(I8Cfg<BN, kPair>::THREADS, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmR,
                     const I8Args args) {
  using Cfg = I8Cfg<BN, kPair>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  pdl_trigger();
  I8Smem<BN, kPair> sm;
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
    for (int w = 0; w < Cfg::EPI_WARPS; ++w)
      for (int b = 0; b < Cfg::BOXES; ++b) mbar_init(sm.res_full(w, b), 1);
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
    i8_epilogue<BN, kPair, T>(sm, tmem_base, args, &tmC, &tmR, tiles_m, tiles_n, num_tiles, t0, dt, rank);
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

template <int BN, bool kPair, class T>
cudaError_t i8_launch(const Int8Gemm& p, int num_sms, cudaStream_t st) {
  using Cfg = I8Cfg<BN, kPair>;
  constexpr int es = (int)sizeof(T);
  I8Args a{p.sA, p.sW, p.bias, p.residual, p.C, p.ldr, p.ldc, p.M, p.N, p.K, 0, 0, 0, 0};
  // widest access that a base address, a row pitch and (word by word) the row's length allow
  auto bytes = [&](const void* base, size_t pitch) {
    const uintptr_t v = reinterpret_cast<uintptr_t>(base) | pitch;
    return v % 16 == 0 ? 16 : (v | (size_t)p.N * es) % 4 == 0 ? 4 : 2;
  };
  const size_t pc = (size_t)p.ldc * es, pr = (size_t)p.ldr * es;
  a.c_word = bytes(p.C, pc);
  a.r_word = p.residual ? bytes(p.residual, pr) : 0;
  a.c_tma = a.c_word == 16;
  a.r_tma = a.r_word == 16;
  CUtensorMap tmA, tmB, tmC, tmR;
  cudaError_t e = encode_tma_2d_ld(&tmA, 1, p.A, p.K, p.M, (size_t)p.lda, 128, 128);
  if (e != cudaSuccess) return e;
  e = encode_tma_2d_ld(&tmB, 1, p.W, p.K, p.N, (size_t)p.ldw, 128, Cfg::B_ROWS);
  if (e != cudaSuccess) return e;
  tmC = tmR = tmA;   // where not used
  if (a.c_tma) e = encode_tma_2d_ld(&tmC, es, p.C, p.N, p.M, pc, 128 / es, 32);
  if (e == cudaSuccess && a.r_tma) e = encode_tma_2d_ld(&tmR, es, p.residual, p.N, p.M, pr, 128 / es, 32);
  if (e != cudaSuccess) return e;
  auto kern = int8_gemm_kernel<BN, kPair, T>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::SMEM);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)((p.M + Cfg::TILE_M - 1) / Cfg::TILE_M) * ((p.N + BN - 1) / BN);
  const int units = kPair ? num_sms / 2 : num_sms;
  const int grid = tiles < units ? (int)tiles : units;
  return kPair ? launch_pdl_pair(kern, dim3(2 * grid), dim3(Cfg::THREADS), Cfg::SMEM, st, tmA, tmB, tmC, tmR, a)
               : launch_pdl(kern, dim3(grid), dim3(Cfg::THREADS), Cfg::SMEM, st, tmA, tmB, tmC, tmR, a);
}

template <class T>
cudaError_t i8_pick(const Int8Gemm& p, int num_sms, cudaStream_t st) {
  if (p.M > 1024 && p.N > 128) return i8_launch<256, true, T>(p, num_sms, st);
  return p.N > 128 ? i8_launch<256, false, T>(p, num_sms, st) : i8_launch<128, false, T>(p, num_sms, st);
}

}  // namespace

cudaError_t launch_int8_gemm(const Int8Gemm& p, int num_sms, cudaStream_t st) {
  if (p.M == 0) return cudaSuccess;
  if (p.dtype == 0) return i8_pick<__nv_bfloat16>(p, num_sms, st);
  if (p.dtype == 1) return i8_pick<__half>(p, num_sms, st);
  return i8_pick<float>(p, num_sms, st);
}

}  // namespace vitq
