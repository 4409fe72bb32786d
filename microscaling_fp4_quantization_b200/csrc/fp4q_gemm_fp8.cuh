// 8-bit GEMM with a scale per block of 128, on the 5th-generation tensor cores (tcgen05
// kind::f8f6f4):
//   D[m][n] = sum over K-blocks j of  sa[m][j] sb[n / 128][j] * (sum over k in block j of qa[m][k] qb[n][k]),
// with A's codes [M][K] and scales [M][ceil(K/128)] as fp4q_quantize_fp8 or fp4q_add_rmsnorm_fp8
// write them, and B's codes [N][K] and scales [ceil(N/128)][ceil(K/128)] from fp4q_quantize_fp8 with
// tiles.  The sum inside a block is the tensor core's (fp32, in tensor memory); the sum over the
// blocks is taken in fp32 registers, each block's sum times its two scales by one fused
// multiply-add, and rounded once, to D's type.
//
// Two kernels, both with one TMA producer warp, one MMA warp and warps that add up the blocks; the
// codes travel through a ring of 128-byte-swizzled stages of one K-block, and two accumulators in
// tensor memory let a block's MMAs run while the block before it is added.  Every wait is bounded.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "fp4q_device.cuh"
#include "fp4q_fp8.cuh"
#include "fp4q_mma.cuh"

namespace fp4q {

struct GemmFp8Args {
  const void* a_scales;   // [M][kb]
  const void* b_scales;   // [ceil(N / 128)][kb]
  void* d;                // [M][N]
  int64_t M, N;
  int kb;                 // K-blocks
  int tiles_m, tiles_n;
  int vec;                // D's rows keep a 32-byte (2), 16-byte (1) or no (0) alignment
};

__device__ __forceinline__ void umma_e4m3(uint32_t tmem_d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(tmem_d),
      "l"(da), "l"(db), "r"(idesc), "r"(acc)
      : "memory");
}

// E4M3 x E4M3 (format 0), K-major, fp32 accumulator, N >> 3, M >> 4.
constexpr uint32_t gemm_fp8_idesc(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// 32 / 16 TMEM columns of this thread's lane as packed pairs; the values are there after tmem_wait_*.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16_bits(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// The wait ties the registers to it, so that nothing reads them before.
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

template <int SF>
__device__ __forceinline__ float load_scale(const void* scales, int64_t i) {
  if constexpr (SF == kSfF32) return __ldg(static_cast<const float*>(scales) + i);
  const uint32_t b = __ldg(static_cast<const uint8_t*>(scales) + i);
  // byte 0 is 2^-127 (a subnormal), 255 NaN
  return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7FFFFFFFu : b << 23);
}

template <int OT>
__device__ __forceinline__ void store_one(void* d, int64_t i, float v) {
  if constexpr (OT == kDtF32)
    static_cast<float*>(d)[i] = v;
  else if constexpr (OT == kDtBf16)
    static_cast<uint16_t*>(d)[i] = static_cast<uint16_t>(pair_from_f32<kDtBf16>(v, 0.0f) & 0xFFFFu);
  else
    static_cast<uint16_t*>(d)[i] = static_cast<uint16_t>(pair_from_f32<kDtFp16>(v, 0.0f) & 0xFFFFu);
}

// Sixteen neighbouring columns of one row of D, as far as they exist.
template <int OT>
__device__ __forceinline__ void store_row16(const GemmFp8Args& g, int64_t row, int64_t col, const f32x2* acc) {
  const int64_t at = row * g.N + col;
  if (g.vec == 0 || col + 16 > g.N) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float lo, hi;
      f2_unpack(acc[i], lo, hi);
      if (col + 2 * i < g.N) store_one<OT>(g.d, at + 2 * i, lo);
      if (col + 2 * i + 1 < g.N) store_one<OT>(g.d, at + 2 * i + 1, hi);
    }
    return;
  }
  if constexpr (OT == kDtF32) {
    float* p = static_cast<float*>(g.d) + at;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float lo, hi;
      f2_unpack(acc[i], lo, hi);
      w[2 * i] = __float_as_uint(lo), w[2 * i + 1] = __float_as_uint(hi);
    }
#pragma unroll
    for (int i = 0; i < 16; i += 4) stg128(p + i, w[i], w[i + 1], w[i + 2], w[i + 3]);
  } else {
    uint16_t* p = static_cast<uint16_t*>(g.d) + at;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pair_from_f32<OT>(acc[i]);
    if (g.vec == 2) {
      stg256(p, w);   // whole 32-byte sectors
    } else {
      stg128(p, w[0], w[1], w[2], w[3]);
      stg128(p + 8, w[4], w[5], w[6], w[7]);
    }
  }
}

// ---------------------------------------------------------------- many rows: tiles of 128 x BN
//
// A is the MMA's row operand, so a thread of the adding warps holds one row of D and half the tile's
// columns: its multiplier is one number a block, sa[row][j] * sb[n / 128][j], and a block costs it
// one fused multiply-add per element.  Persistent CTAs, one per SM, round-robin over the tiles.
template <int BN_, int OT, int SF>
struct GemmFp8Config {
  static constexpr int kBM = 128, kBN = BN_, kBK = kFp8Block;
  static constexpr int kOut = OT, kSf = SF;
  static constexpr int kABytes = kBM * kBK, kBBytes = kBN * kBK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = kBN == 256 ? 4 : 6;
  static constexpr int kBarOffset = kStages * kStageBytes;
  static constexpr int kSmemBytes = 1024 + kBarOffset + 256;
  static constexpr int kTmemCols = 2 * kBN;                 // two accumulators
  static constexpr int kAddWarps = 8, kAddWarp0 = 2;        // two per TMEM lane quarter
  static constexpr int kCols = kBN / 2;                     // columns per adding warp
  static constexpr int kThreads = 32 * (kAddWarp0 + kAddWarps);
  static constexpr uint32_t kIdesc = gemm_fp8_idesc(kBM, kBN);
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, GemmFp8Args g) {
  constexpr int S = Cfg::kStages, BN = Cfg::kBN;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t s_tmem_base;
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t stage0 = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = stage0 + Cfg::kBarOffset;
  auto a_tile = [&](int s) { return stage0 + s * Cfg::kStageBytes; };
  auto b_tile = [&](int s) { return stage0 + s * Cfg::kStageBytes + Cfg::kABytes; };
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
  auto acc_full = [&](int d) { return bars + 8u * (2 * S + d); };
  auto acc_empty = [&](int d) { return bars + 8u * (2 * S + 2 + d); };

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int d = 0; d < 2; ++d) {
      mbar_init(acc_full(d), 1);
      mbar_init(acc_empty(d), Cfg::kAddWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem_base)),
                 "r"(Cfg::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  const int n_tiles = g.tiles_m * g.tiles_n;

  if (warp == 0) {
    // ---------------- producer
    if (lane == 0) {
      pdl_wait();
      int64_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < n_tiles; t += gridDim.x) {
        const int tm = t % g.tiles_m, tn = t / g.tiles_m;
        for (int j = 0; j < g.kb; ++j, ++it) {
          const int s = static_cast<int>(it % S);
          if (!mbar_wait_bounded(empty_bar(s), static_cast<uint32_t>((it / S) & 1) ^ 1u)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full_bar(s), Cfg::kStageBytes);
          tma_load_2d(a_tile(s), &amap, j * Cfg::kBK, tm * Cfg::kBM, full_bar(s));
          tma_load_2d(b_tile(s), &bmap, j * Cfg::kBK, tn * BN, full_bar(s));
        }
      }
      // let every issued copy land before the CTA can leave
      for (int64_t j = (it > S ? it - S : 0); j < it; ++j)
        mbar_wait_bounded(full_bar(static_cast<int>(j % S)), static_cast<uint32_t>((j / S) & 1));
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer: one K-block into one accumulator
    if (lane == 0) {
      int64_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < n_tiles; t += gridDim.x) {
        for (int j = 0; j < g.kb; ++j, ++it) {
          const int s = static_cast<int>(it % S), d = static_cast<int>(it & 1);
          if (!mbar_wait_bounded(acc_empty(d), static_cast<uint32_t>((it >> 1) & 1) ^ 1u) ||
              !mbar_wait_bounded(full_bar(s), static_cast<uint32_t>((it / S) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < Cfg::kBK / 32; ++kk)
            umma_e4m3(tmem_base + d * BN, umma_smem_desc(a_tile(s) + kk * 32, 1024, 2),
                      umma_smem_desc(b_tile(s) + kk * 32, 1024, 2), Cfg::kIdesc, kk != 0 ? 1u : 0u);
          umma_commit(empty_bar(s));
          umma_commit(acc_full(d));
        }
      }
      // the last commits must have landed before TMEM is freed
      if (it > 0) mbar_wait_bounded(acc_full(static_cast<int>((it - 1) & 1)), static_cast<uint32_t>(((it - 1) >> 1) & 1));
    }
  } else {
    // ---------------- adding warps: TMEM lane quarter warp % 4, column half (warp - 2) / 4
    const int q = warp & 3, half = (warp - Cfg::kAddWarp0) >> 2;
    constexpr int NC = Cfg::kCols, CH = 16;
    pdl_wait();
    int64_t it = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < n_tiles; t += gridDim.x) {
      const int tm = t % g.tiles_m, tn = t / g.tiles_m;
      const int64_t row = static_cast<int64_t>(tm) * Cfg::kBM + 32 * q + lane;
      const int64_t col0 = static_cast<int64_t>(tn) * BN + half * NC;
      // rows and columns past the end use the last ones' scales; they are not stored
      const int64_t sa0 = (row < g.M ? row : g.M - 1) * g.kb;
      const int64_t sb0 = (col0 < g.N ? col0 : g.N - 1) / kFp8Block * g.kb;
      // the scales of a block are loaded two blocks ahead
      float s0 = load_scale<Cfg::kSf>(g.a_scales, sa0) * load_scale<Cfg::kSf>(g.b_scales, sb0);
      const int j1 = g.kb > 1 ? 1 : 0;
      float sa1 = load_scale<Cfg::kSf>(g.a_scales, sa0 + j1), sb1 = load_scale<Cfg::kSf>(g.b_scales, sb0 + j1);
      f32x2 acc[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) acc[i] = 0ull;
#pragma unroll 1
      for (int j = 0; j < g.kb; ++j, ++it) {
        const int d = static_cast<int>(it & 1);
        const int j2 = j + 2 < g.kb ? j + 2 : g.kb - 1;
        const float sa2 = load_scale<Cfg::kSf>(g.a_scales, sa0 + j2), sb2 = load_scale<Cfg::kSf>(g.b_scales, sb0 + j2);
        const bool mine = mbar_wait_bounded(acc_full(d), static_cast<uint32_t>((it >> 1) & 1));
        if (!__all_sync(0xFFFFFFFFu, mine)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const f32x2 s2 = f2_pack(s0, s0);
        const uint32_t src = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + d * BN + half * NC;
#pragma unroll
        for (int c = 0; c < NC / CH; ++c) {
          uint32_t p[CH];
          tmem_ld16_bits(src + c * CH, p);
          tmem_wait(p);
          if (c == NC / CH - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty(d));
          }
#pragma unroll
          for (int i = 0; i < CH / 2; ++i) {
            f32x2& x = acc[c * (CH / 2) + i];
            x = f2_fma(f2_pack(__uint_as_float(p[2 * i]), __uint_as_float(p[2 * i + 1])), s2, x);
          }
        }
        s0 = sa1 * sb1;
        sa1 = sa2, sb1 = sb2;
      }
      if (ok && row < g.M) {
#pragma unroll
        for (int c = 0; c < NC / 16; ++c)
          if (col0 + 16 * c < g.N) store_row16<Cfg::kOut>(g, row, col0 + 16 * c, acc + 8 * c);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(Cfg::kTmemCols)
                 : "memory");
  }
}

// ---------------------------------------------------------------- few rows: 128 of B's rows by BT tokens
//
// For decode batches the product is a stream of B: here B is the MMA's row operand (tiles of 128 of
// its rows, one scale per tile and block) and BT rows of A are its columns, so no MMA row is idle.
// The blocks of K are split over a cluster of `split` CTAs, so that enough loads are in flight on
// all SMs; each CTA leaves its sums in shared memory and takes its share of the tokens from all of
// them, in the order of their ranks (no atomics, no workspace).
template <int BT_, int OT, int SF>
struct GemmFp8FewConfig {
  static constexpr int kBT = BT_, kBK = kFp8Block;
  static constexpr int kOut = OT, kSf = SF;
  static constexpr int kWBytes = 128 * kBK, kXBytes = kBT * kBK;
  static constexpr int kStageBytes = kWBytes + kXBytes;
  // two CTAs on an SM: 228 KB less 1 KB of system use each
  static constexpr int kStages = (110 * 1024) / kStageBytes;
  static constexpr int kBarOffset = kStages * kStageBytes;
  static constexpr int kSmemBytes = 1024 + kBarOffset + 256;
  static constexpr int kTmemCols = 2 * kBT < 32 ? 32 : 2 * kBT;
  static constexpr int kAddWarp0 = 2, kAddWarps = 4;
  static constexpr int kThreads = 32 * (kAddWarp0 + kAddWarps);
  static constexpr uint32_t kIdesc = gemm_fp8_idesc(128, kBT);
  static_assert(kStageBytes % 1024 == 0, "stages stay 1024-byte aligned (128-byte swizzle atoms)");
  static_assert(kBT * 128 * 4 <= kBarOffset, "a CTA's sums fit in the ring");
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 2)
    gemm_fp8_few_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                        GemmFp8Args g, int split) {
  constexpr int S = Cfg::kStages, BT = Cfg::kBT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t s_tmem_base;
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t stage0 = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = stage0 + Cfg::kBarOffset;
  auto w_tile = [&](int s) { return stage0 + s * Cfg::kStageBytes; };
  auto x_tile = [&](int s) { return stage0 + s * Cfg::kStageBytes + Cfg::kWBytes; };
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
  auto acc_full = [&](int d) { return bars + 8u * (2 * S + d); };
  auto acc_empty = [&](int d) { return bars + 8u * (2 * S + 2 + d); };
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int d = 0; d < 2; ++d) {
      mbar_init(acc_full(d), 1);
      mbar_init(acc_empty(d), Cfg::kAddWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem_base)),
                 "r"(Cfg::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int t = blockIdx.x / split;
  const int tn = t % g.tiles_n, tm = t / g.tiles_n;
  const int j0 = static_cast<int>(static_cast<int64_t>(g.kb) * rank / split);
  const int j1 = static_cast<int>(static_cast<int64_t>(g.kb) * (rank + 1) / split);
  const int nj = j1 - j0;

  if (warp == 0) {
    if (lane == 0) {
      pdl_wait();
      int it = 0;
      for (; it < nj; ++it) {
        const int s = it % S;
        if (!mbar_wait_bounded(empty_bar(s), static_cast<uint32_t>((it / S) & 1) ^ 1u)) break;
        mbar_arrive_expect_tx(full_bar(s), Cfg::kStageBytes);
        tma_load_2d(w_tile(s), &wmap, (j0 + it) * Cfg::kBK, tn * 128, full_bar(s));
        tma_load_2d(x_tile(s), &xmap, (j0 + it) * Cfg::kBK, tm * BT, full_bar(s));
      }
      for (int j = (it > S ? it - S : 0); j < it; ++j) mbar_wait_bounded(full_bar(j % S), static_cast<uint32_t>((j / S) & 1));
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int it = 0;
      for (; it < nj; ++it) {
        const int s = it % S, d = it & 1;
        if (!mbar_wait_bounded(acc_empty(d), static_cast<uint32_t>((it >> 1) & 1) ^ 1u) ||
            !mbar_wait_bounded(full_bar(s), static_cast<uint32_t>((it / S) & 1)))
          break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < Cfg::kBK / 32; ++kk)
          umma_e4m3(tmem_base + d * BT, umma_smem_desc(w_tile(s) + kk * 32, 1024, 2),
                    umma_smem_desc(x_tile(s) + kk * 32, 1024, 2), Cfg::kIdesc, kk != 0 ? 1u : 0u);
        umma_commit(empty_bar(s));
        umma_commit(acc_full(d));
      }
      if (it > 0) mbar_wait_bounded(acc_full((it - 1) & 1), static_cast<uint32_t>(((it - 1) >> 1) & 1));
    }
  } else {
    // lane quarter warp % 4: this thread holds B's row n and the tile's BT tokens
    const int q = warp & 3;
    const int nl = 32 * q + lane;
    const int64_t n = static_cast<int64_t>(tn) * 128 + nl;
    const int64_t m0 = static_cast<int64_t>(tm) * BT;
    constexpr int TL = (BT + 31) / 32;   // tokens whose scales a lane loads
    pdl_wait();
    const int64_t sb0 = static_cast<int64_t>(tn) * g.kb;
    int64_t sa0[TL];
#pragma unroll
    for (int i = 0; i < TL; ++i) {
      const int64_t m = m0 + i * 32 + lane;
      sa0[i] = (m < g.M ? m : g.M - 1) * g.kb;
    }
    // lane l loads the product of the scales of token 32 i + l, two blocks ahead
    auto scales = [&](int j, float (&v)[TL]) {
      const int jj = j < j1 ? j : (j1 > 0 ? j1 - 1 : 0);
      const float sb = load_scale<Cfg::kSf>(g.b_scales, sb0 + jj);
#pragma unroll
      for (int i = 0; i < TL; ++i) v[i] = load_scale<Cfg::kSf>(g.a_scales, sa0[i] + jj) * sb;
    };
    float s0[TL], s1[TL], s2[TL];
    scales(j0, s0);
    scales(j0 + 1, s1);
    float acc[BT];
#pragma unroll
    for (int i = 0; i < BT; ++i) acc[i] = 0.0f;
#pragma unroll 1
    for (int it = 0; it < nj; ++it) {
      const int d = it & 1;
      scales(j0 + it + 2, s2);
      const bool mine = mbar_wait_bounded(acc_full(d), static_cast<uint32_t>((it >> 1) & 1));
      if (!__all_sync(0xFFFFFFFFu, mine)) break;
      tc_fence_after();
      const uint32_t src = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + d * BT;
#pragma unroll
      for (int c = 0; c < BT / 16; ++c) {
        uint32_t p[16];
        tmem_ld16_bits(src + c * 16, p);
        tmem_wait(p);
        if (c == BT / 16 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty(d));
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int tok = c * 16 + i;
          acc[tok] = fmaf(__uint_as_float(p[i]), __shfl_sync(0xFFFFFFFFu, s0[tok / 32], tok % 32), acc[tok]);
        }
      }
#pragma unroll
      for (int i = 0; i < TL; ++i) s0[i] = s1[i], s1[i] = s2[i];
    }
    if (split == 1) {
      if (n < g.N) {
#pragma unroll
        for (int i = 0; i < BT; ++i)
          if (m0 + i < g.M) store_one<Cfg::kOut>(g.d, (m0 + i) * g.N + n, acc[i]);
      }
    } else {
      // every copy of the ring has landed and been read (the last block's MMAs are complete)
#pragma unroll
      for (int i = 0; i < BT; ++i) sts32(stage0 + 4u * (i * 128 + nl), __float_as_uint(acc[i]));
    }
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync_all();
    if (warp >= Cfg::kAddWarp0) {
      const int nl = 32 * (warp & 3) + lane;
      const int64_t n = static_cast<int64_t>(tn) * 128 + nl;
      for (int i = rank; i < BT; i += split) {
        const int64_t m = static_cast<int64_t>(tm) * BT + i;
        if (m >= g.M) break;
        float v = 0.0f;
        for (int r = 0; r < split; ++r) v += ld_cluster_f32(cluster_map(stage0 + 4u * (i * 128 + nl), r));
        if (n < g.N) store_one<Cfg::kOut>(g.d, m * g.N + n, v);
      }
    }
    __syncwarp();
    cluster_sync_all();   // no CTA leaves while another reads its sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(Cfg::kTmemCols)
                 : "memory");
  }
}

}  // namespace fp4q
