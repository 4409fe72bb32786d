// 8-bit GEMM with a scale per block of 128, on the 5th-generation tensor cores (tcgen05):
//   D[m][n] = sum over K-blocks j of  sa[m][j] sb[n / 128][j] * (sum over k in block j of qa[m][k] qb[n][k]),
// with A's codes [M][K] and scales [M][ceil(K/128)] as fp4q_quantize_fp8 or fp4q_add_rmsnorm_fp8
// write them, and B's codes [N][K] and scales [ceil(N/128)][ceil(K/128)] from fp4q_quantize_fp8 with
// tiles.
//
// Three kernels:
//   gemm_fp8_kernel      many rows, any scales.  The tensor core sums inside a block (kind::f8f6f4, fp32
//                        in tensor memory); the sum over the blocks is taken in fp32 registers, each
//                        block's sum times its two scales by one fused multiply-add;
//   gemm_fp8_mx_kernel   many rows, scales in powers of two.  The tensor core applies the scales
//                        (kind::mxf8f6f4) and sums over all of K;
//   gemm_fp8_few_kernel  few rows: B is the row operand, and K is split over a cluster.
// D is rounded once, to its type.  All three have a TMA producer warp and an MMA warp; the codes travel
// through a ring of 128-byte-swizzled stages of one K-block, and several accumulators in tensor memory
// let MMAs run while what they left before is read.  Every wait is bounded.
//
// Times in this file are of two kinds.  Those of a kernel as it stands are launches of fp4q_gemm_fp8 back to back
// in a graph, on operands that the quantizers made of activations and weights and that pass L2 in turn; GPUs
// differ by 5 to 10 %, most where the power cap holds the clock.  Those that compare variants (marked "variants")
// are of single kernels on codes of random bytes, which draw less power, so that large products run faster:
// they compare with one another alone.
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
  int sf_vec;             // E8M0 scales: rows start on whole words
  int vec;                // D's rows keep a 32-byte (2), 16-byte (1) or no (0) alignment
};

__device__ __forceinline__ void umma_e4m3(uint32_t tmem_d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(tmem_d),
      "l"(da), "l"(db), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void umma_e4m3_scaled(uint32_t tmem_d, uint64_t da, uint64_t db, uint32_t idesc,
                                                 uint32_t tsfa, uint32_t tsfb, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n}" ::"r"(tmem_d),
      "l"(da), "l"(db), "r"(idesc), "r"(acc), "r"(tsfa), "r"(tsfb)
      : "memory");
}

// E4M3 x E4M3 (format 0), K-major, fp32 accumulator, N >> 3, M >> 4.
constexpr uint32_t gemm_fp8_idesc(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// 16 / 8 TMEM columns of this thread's lane, waited for, as pairs: a load's registers are neighbours, so
// pairing them in the same statement costs no moves, which pairing them outside it did.
__device__ __forceinline__ void tmem_ld_pairs(uint32_t taddr, f32x2 (&r)[8]) {
  asm volatile(
      "{\n .reg .b32 t<16>;\n"
      " tcgen05.ld.sync.aligned.32x32b.x16.b32 {t0,t1,t2,t3,t4,t5,t6,t7,t8,t9,t10,t11,t12,t13,t14,t15}, [%8];\n"
      " tcgen05.wait::ld.sync.aligned;\n"
      " mov.b64 %0, {t0, t1};\n"
      " mov.b64 %1, {t2, t3};\n"
      " mov.b64 %2, {t4, t5};\n"
      " mov.b64 %3, {t6, t7};\n"
      " mov.b64 %4, {t8, t9};\n"
      " mov.b64 %5, {t10, t11};\n"
      " mov.b64 %6, {t12, t13};\n"
      " mov.b64 %7, {t14, t15};\n"
      "}"
      : "=l"(r[0]), "=l"(r[1]), "=l"(r[2]), "=l"(r[3]), "=l"(r[4]), "=l"(r[5]), "=l"(r[6]), "=l"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_pairs(uint32_t taddr, f32x2 (&r)[4]) {
  asm volatile(
      "{\n .reg .b32 t<8>;\n"
      " tcgen05.ld.sync.aligned.32x32b.x8.b32 {t0,t1,t2,t3,t4,t5,t6,t7}, [%4];\n"
      " tcgen05.wait::ld.sync.aligned;\n"
      " mov.b64 %0, {t0, t1};\n"
      " mov.b64 %1, {t2, t3};\n"
      " mov.b64 %2, {t4, t5};\n"
      " mov.b64 %3, {t6, t7};\n"
      "}"
      : "=l"(r[0]), "=l"(r[1]), "=l"(r[2]), "=l"(r[3])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// Fetch a tensor map ahead of the first copy that uses it.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// A scale as it lies in memory, and its value.  They are apart so that a loaded scale stays untouched
// until its block is added: converting it where it is loaded would wait for the load.
template <int SF>
__device__ __forceinline__ uint32_t load_scale(const void* scales, int64_t i) {
  if constexpr (SF == kSfF32) return ld_u32(static_cast<const uint32_t*>(scales) + i);
  return ld_u8(static_cast<const uint8_t*>(scales) + i);
}
template <int SF>
__device__ __forceinline__ float scale_value(uint32_t w) {
  if constexpr (SF == kSfF32) return __uint_as_float(w);
  // E8M0: byte 0 is 2^-127 (a subnormal), 255 NaN
  return __uint_as_float(w == 0u ? 0x00400000u : w == 255u ? 0x7FFFFFFFu : w << 23);
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

// Eight neighbouring columns of one row of D, as far as they exist.
template <int OT, int N>
__device__ __forceinline__ void store_row_tail(const GemmFp8Args& g, int64_t row, int64_t col, const f32x2* acc) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float lo, hi;
    f2_unpack(acc[i], lo, hi);
    if (col + 2 * i < g.N) store_one<OT>(g.d, row * g.N + col + 2 * i, lo);
    if (col + 2 * i + 1 < g.N) store_one<OT>(g.d, row * g.N + col + 2 * i + 1, hi);
  }
}
template <int OT>
__device__ __forceinline__ void store_row8(const GemmFp8Args& g, int64_t row, int64_t col, const f32x2* acc) {
  if (g.vec == 0 || col + 8 > g.N) {
    store_row_tail<OT, 8>(g, row, col, acc);
  } else if constexpr (OT == kDtF32) {
    float* p = static_cast<float*>(g.d) + row * g.N + col;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      float v[4];
      f2_unpack(acc[i], v[0], v[1]);
      f2_unpack(acc[i + 1], v[2], v[3]);
      stg128(p + 2 * i, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
  } else {
    stg128(static_cast<uint16_t*>(g.d) + row * g.N + col, pair_from_f32<OT>(acc[0]), pair_from_f32<OT>(acc[1]),
           pair_from_f32<OT>(acc[2]), pair_from_f32<OT>(acc[3]));
  }
}
// Sixteen columns of one row where rows keep a 16-byte alignment, so that a row ends between stores.
template <int OT>
__device__ __forceinline__ void store_row16(const GemmFp8Args& g, int64_t row, int64_t col, const f32x2* acc) {
  if (OT != kDtF32 && g.vec == 2) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pair_from_f32<OT == kDtF32 ? kDtBf16 : OT>(acc[i]);
    stg256(static_cast<uint16_t*>(g.d) + row * g.N + col, w);   // whole 32-byte sectors
  } else if constexpr (OT == kDtF32) {
    float* p = static_cast<float*>(g.d) + row * g.N + col;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float v[4];
      f2_unpack(acc[i], v[0], v[1]);
      f2_unpack(acc[i + 1], v[2], v[3]);
      if (col + 2 * i < g.N)
        stg128(p + 2 * i, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(g.d) + row * g.N + col;
#pragma unroll
    for (int i = 0; i < 8; i += 4)
      if (col + 2 * i < g.N)
        stg128(p + 2 * i, pair_from_f32<OT>(acc[i]), pair_from_f32<OT>(acc[i + 1]), pair_from_f32<OT>(acc[i + 2]),
               pair_from_f32<OT>(acc[i + 3]));
  }
}
// Sixteen columns of a warp's 32 rows (lane: row) where rows keep no such alignment: by way of shared
// memory (`buf`, kUnalignedBytes of the warp's own), so that neighbouring lanes store neighbouring
// columns.  With a lane to a row, every store of 2 bytes would touch a sector of its own.
// Variants, bf16, a lane to a row and this way: 793 x 11180 x 6784 197 and 96 us (256 x 256 tiles), 175 and
// 81 us (E8M0); N = 11181, stores of single elements, 197 and 107 us, 175 and 86 us; UNROLL 16, where 64 sums
// a thread leave the registers for it, 104 -> 101 us with 128 x 128 tiles, else 4.  As it stands, N = 11180 / 11181 /
// 11184 (rows of 16-byte alignment): 99 to 124 / 111 / 86 us, E8M0 91 to 124 / 91 / 83.  All lanes take part.
constexpr int kUnalignedPitch = 17, kUnalignedBytes = 32 * kUnalignedPitch * 4;
template <int OT, int UNROLL>
__device__ __forceinline__ void store_unaligned16(const GemmFp8Args& g, int64_t row0, int64_t col, const f32x2* acc,
                                                  uint32_t buf, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float lo, hi;
    f2_unpack(acc[i], lo, hi);
    sts32(buf + 4u * (lane * kUnalignedPitch + 2 * i), __float_as_uint(lo));
    sts32(buf + 4u * (lane * kUnalignedPitch + 2 * i + 1), __float_as_uint(hi));
  }
  __syncwarp();
  if (OT != kDtF32 && (g.N & 1) == 0) {
    // pairs of columns (D starts on 16 bytes, so a pair on 4), four rows at a time
    const int c = 2 * (lane & 7);
#pragma unroll UNROLL
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      const uint32_t at = buf + 4u * (r * kUnalignedPitch + c);
      if (row0 + r < g.M && col + c < g.N)
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(g.d) + (row0 + r) * g.N + col + c) =
            pair_from_f32<OT == kDtF32 ? kDtBf16 : OT>(__uint_as_float(lds32(at)), __uint_as_float(lds32(at + 4u)));
    }
  } else {
    const int c = lane & 15;
#pragma unroll UNROLL
    for (int i = 0; i < 16; ++i) {
      const int r = 2 * i + (lane >> 4);
      if (row0 + r < g.M && col + c < g.N)
        store_one<OT>(g.d, (row0 + r) * g.N + col + c, __uint_as_float(lds32(buf + 4u * (r * kUnalignedPitch + c))));
    }
  }
  __syncwarp();
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync_all() {
  cluster_arrive();
  cluster_wait();
}
// The address of `addr` (of this CTA's shared memory) in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Arrive on a barrier of another CTA of the cluster.  What it announces is that tensor memory has been
// read, which tcgen05's own fences order: a release at cluster scope took 500 ns of every block.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// Four floats of shared memory as two pairs.
__device__ __forceinline__ void lds_pairs(uint32_t addr, f32x2& a, f32x2& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}

// ---------------------------------------------------------------- many rows: tiles of 128 C x BN
//
// A is the MMA's row operand, so a thread of the adding warps holds one row of D and half the tile's
// columns: its multiplier is one number a block, sa[row][j] * sb[n / 128][j], and a block costs it
// one fused multiply-add per element.  Persistent, round-robin over the tiles.  C = 2 pairs the CTAs
// of a cluster on one tile (cta_group::2, M = 256): each loads its 128 rows of A and half of B's, and
// the leader issues the MMAs of both; that halves what B costs L2 and shared memory (variants at 8192^3:
// 593 us against 627 us with one CTA to a 128 x 256 tile, when it was taken up).
//
// 8192^3 takes 549 to 589 us, 333 x 4104 x 5008 16.7 to 18.7.  What bounds it, variants at 8192^3: the MMAs
// and copies alone take 440 us (at a clock the power cap holds near 1.3 GHz), with the adding 522 us.  A
// block's turn through one of the two accumulators is MMAs (600 cycles with their start), commit and wake-up
// (290), the adding warps' read (500 - 590, in steps of 8 columns: 16, 32 or 64 at a time take 619, 755 and
// 598 us) and the arrival that frees it (300); more accumulators of narrower tiles cost more in operand
// traffic than they hide (256 x 128: 613 us).

// Tile t's row and column of tiles: down kTileGroup rows, then the next column, so that the tiles worked on
// at one time (74 pairs: 16 rows by 4.6 columns) share their rows of A and of B in L2.  Variants at 8192^3:
// 523 us with fp32 scales and 397 us with E8M0, against 555 and 440 us down all 32 rows; groups of 8 and
// 32 rows lie between, and where A's rows are few there is no difference.
constexpr int kTileGroup = 16;
__device__ __forceinline__ void gemm_fp8_tile(const GemmFp8Args& g, int t, int& tm, int& tn) {
  const int per_group = kTileGroup * g.tiles_n, group = t / per_group, in_group = t - group * per_group;
  const int rows = min(kTileGroup, g.tiles_m - group * kTileGroup);
  tn = in_group / rows;
  tm = group * kTileGroup + in_group - tn * rows;
}

constexpr int kMmaTries = 64;   // times an MMA warp asks for its barriers before it suspends

// ALIGNED: D's rows keep a 16-byte alignment.  A parameter: with both kinds of stores in one
// kernel it took 5 % longer at 8192^3 (variants: 525 -> 553 us).
template <int CTAS, int BN_, int OT, int SF, bool ALIGNED>
struct GemmFp8Config {
  static constexpr int kCtas = CTAS;
  static constexpr int kBM = 128 * CTAS, kBN = BN_, kBK = kFp8Block;
  static constexpr int kOut = OT, kSf = SF;
  static constexpr bool kAligned = ALIGNED;
  static constexpr int kARows = 128, kBRows = kBN / CTAS;   // a CTA's share of a stage
  static constexpr int kABytes = kARows * kBK, kBBytes = kBRows * kBK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = (196 * 1024) / kStageBytes;
  static constexpr int kBarOffset = kStages * kStageBytes;
  static constexpr int kAccs = 512 / kBN;                   // accumulators in tensor memory
  static constexpr int kTmemCols = kAccs * kBN;
  static constexpr int kAddWarp0 = 4, kAddWarps = 8;        // two per TMEM lane quarter
  static constexpr int kBufOffset = kBarOffset + 256;       // rows of no alignment: a piece per adding warp
  static constexpr int kSmemBytes = 1024 + kBufOffset + (ALIGNED ? 0 : kAddWarps * kUnalignedBytes);
  static constexpr int kCols = kBN / 2;                     // columns per adding warp
  static constexpr int kThreads = 32 * (kAddWarp0 + kAddWarps);
  // 128 sums a thread need more registers than 384 threads share out evenly (168): the first four
  // warps hand theirs to the adding warps
  static constexpr bool kRegSplit = kCols == 128;
  static constexpr int kRegsLaunch = 168, kRegsFew = 56, kRegsMany = 224;
  static_assert(kRegsFew * kAddWarp0 + kRegsMany * kAddWarps <= kRegsLaunch * (kAddWarp0 + kAddWarps));
  static constexpr uint32_t kIdesc = gemm_fp8_idesc(kBM, kBN);
};

// A position in a ring of N barriers: the slot, and the parity of the pass over the ring (kept rather
// than worked out from a count: the MMA warp's loop has to stay shorter than the MMAs it issues).
template <int N>
struct RingPos {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      parity ^= 1u;
    }
  }
};

// Whether the phase is complete, asked once.  Asking takes some 90 cycles to a branch on the answer (a
// wait that may suspend, 130), so the MMA warps ask for a block's barriers before they issue the block
// in front of it, and wait only where the answer was no.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Two phases at once.
__device__ __forceinline__ bool mbar_test2(uint32_t bar_a, uint32_t parity_a, uint32_t bar_b, uint32_t parity_b) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n"
      " and.pred p, p, q;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar_a), "r"(parity_a), "r"(bar_b), "r"(parity_b)
      : "memory");
  return ok != 0;
}

// Wait of a whole converged warp: ask up to `tries` times, then wait; false when the wait ran out.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int tries) {
#pragma unroll 1
  for (int i = 0; i < tries; ++i)
    if (__all_sync(0xFFFFFFFFu, mbar_test(bar, parity))) return true;
  return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity));
}
__device__ __forceinline__ bool warp_wait2(uint32_t bar_a, uint32_t parity_a, uint32_t bar_b, uint32_t parity_b, int tries) {
#pragma unroll 1
  for (int i = 0; i < tries; ++i)
    if (__all_sync(0xFFFFFFFFu, mbar_test2(bar_a, parity_a, bar_b, parity_b))) return true;
  return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar_a, parity_a) && mbar_wait_bounded(bar_b, parity_b));
}

// Blocks after which two rings are both back at their first slot.
constexpr int ring_unroll(int a, int b) {
  int u = a;
  while (u % b != 0) u += a;
  return u;
}

template <int CTAS>
__device__ __forceinline__ void gemm_fp8_mma(uint32_t tmem_d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t acc) {
  if constexpr (CTAS == 1) {
    umma_e4m3(tmem_d, da, db, idesc, acc);
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(tmem_d),
        "l"(da), "l"(db), "r"(idesc), "r"(acc)
        : "memory");
  }
}
// Arrive on the barrier at this address, in both CTAs of a pair, when the MMAs issued so far are done.
template <int CTAS>
__device__ __forceinline__ void gemm_fp8_commit(uint32_t bar) {
  if constexpr (CTAS == 1) {
    umma_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  }
}
// A box into this CTA's shared memory; a pair's copies complete on the leader's barrier.
template <int CTAS>
__device__ __forceinline__ void gemm_fp8_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CTAS == 1) {
    tma_load_2d(dst, map, x, y, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  }
}

// Producer warp of the many-row kernels: this CTA's rows of A and of B, stage after stage.  full barriers
// lie at `bars`, empty ones behind them; a pair's copies complete on the leader's.  As in the MMA warp the
// whole warp runs the loop, one lane issues, and a stage's barrier is asked for a stage ahead.
template <class Cfg>
__device__ __forceinline__ void gemm_fp8_produce(const GemmFp8Args& g, const CUtensorMap& amap, const CUtensorMap& bmap,
                                                 int rank, int t0, int dt, uint32_t stage0, uint32_t bars) {
  constexpr int S = Cfg::kStages, C = Cfg::kCtas;
  if (elect_one()) {
    prefetch_map(&amap);
    prefetch_map(&bmap);
  }
  __syncwarp();
  pdl_wait();
  const int n_tiles = g.tiles_m * g.tiles_n;
  const uint32_t full0 = C == 2 ? cluster_map(bars, 0) : bars;
  RingPos<S> r;
  bool ok = true, ready = true;
  int filled = 0;
  for (int t = t0; ok && t < n_tiles; t += dt) {
    int tm, tn;
    gemm_fp8_tile(g, t, tm, tn);
    const int ra = tm * Cfg::kBM + rank * Cfg::kARows, rb = tn * Cfg::kBN + rank * Cfg::kBRows;
    for (int j = 0; j < g.kb; ++j) {
      if (!__all_sync(0xFFFFFFFFu, ready)) ok = warp_wait(bars + 8u * (S + r.i), r.parity ^ 1u, 1);
      if (!ok) break;
      RingPos<S> rn = r;
      rn.next();
      ready = mbar_test(bars + 8u * (S + rn.i), rn.parity ^ 1u);
      if (elect_one()) {
        const uint32_t dst = stage0 + r.i * Cfg::kStageBytes, bar = full0 + 8u * r.i;
        if (rank == 0) mbar_arrive_expect_tx(bars + 8u * r.i, C * Cfg::kStageBytes);
        gemm_fp8_load<C>(dst, &amap, j * Cfg::kBK, ra, bar);
        gemm_fp8_load<C>(dst + Cfg::kABytes, &bmap, j * Cfg::kBK, rb, bar);
      }
      __syncwarp();
      filled = filled < S ? filled + 1 : S;
      r = rn;
    }
  }
  // every issued copy has landed once its stage was read (or, where a wait ran out, long before): the
  // ring's slots, from the oldest on
  if (filled < S) r = RingPos<S>{};
  for (int j = 0; j < filled; ++j, r.next())
    mbar_wait_bounded(bars + 8u * (S + r.i), filled < S ? 0u : r.parity ^ 1u);
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, GemmFp8Args g) {
  constexpr int S = Cfg::kStages, BN = Cfg::kBN, C = Cfg::kCtas, NA = Cfg::kAccs;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t s_tmem_base;
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = C == 2 ? static_cast<int>(cluster_rank()) : 0;
  const uint32_t stage0 = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = stage0 + Cfg::kBarOffset;
  auto a_tile = [&](int s) { return stage0 + s * Cfg::kStageBytes; };
  auto b_tile = [&](int s) { return stage0 + s * Cfg::kStageBytes + Cfg::kABytes; };
  auto full_bar = [&](int s) { return bars + 8u * s; };                  // a pair uses the leader's
  auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
  auto acc_full = [&](int d) { return bars + 8u * (2 * S + d); };
  auto acc_empty = [&](int d) { return bars + 8u * (2 * S + NA + d); };   // a pair uses the leader's

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int d = 0; d < NA; ++d) {
      mbar_init(acc_full(d), 1);
      mbar_init(acc_empty(d), C * Cfg::kAddWarps);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (C == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem_base)),
                   "r"(Cfg::kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem_base)),
                   "r"(Cfg::kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (C == 2) cluster_sync_all();   // the pair's barriers are set up
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  const int n_tiles = g.tiles_m * g.tiles_n;
  const int t0 = static_cast<int>(blockIdx.x) / C, dt = static_cast<int>(gridDim.x) / C;
  if constexpr (Cfg::kRegSplit)
    if (warp < Cfg::kAddWarp0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsFew));

  if (warp == 0) {
    gemm_fp8_produce<Cfg>(g, amap, bmap, rank, t0, dt, stage0, bars);
  } else if (warp == 1) {
    // ---------------- MMA issuer (a pair's leader): one K-block into one accumulator.  The whole warp
    // runs the loop, one lane issues.  The loop knows nothing of tiles and is unrolled over the rings, so
    // that a block costs it little besides its instructions: kept rolled, it took 500 cycles a block and
    // held up MMAs of 256.
    if (rank == 0) {
      constexpr int U = ring_unroll(S, NA);
      const int64_t n = t0 < n_tiles ? static_cast<int64_t>((n_tiles - t0 + dt - 1) / dt) * g.kb : 0;   // blocks
      const uint64_t da0 = umma_smem_desc(a_tile(0), 1024, 2), db0 = umma_smem_desc(b_tile(0), 1024, 2);
      bool ok = true, ready = false;
      uint32_t pass = 0;   // over the unrolled loop, modulo 2
#pragma unroll 1
      for (int64_t it = 0; ok && it < n; it += U, pass ^= 1u) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
          // slots and parities of this block and of the next, fixed but for the pass
          constexpr int PF = U / S, PA = U / NA;   // passes over each ring in one over the loop
          const int s = k % S, d = k % NA, kn = (k + 1) % U, sn = kn % S, dn = kn % NA;
          const uint32_t pn = k + 1 == U ? pass ^ 1u : pass;
          const uint32_t full_par = (pass * (PF & 1) + k / S) & 1u, acc_par = (pass * (PA & 1) + k / NA) & 1u;
          const uint32_t full_par_n = (pn * (PF & 1) + kn / S) & 1u, acc_par_n = (pn * (PA & 1) + kn / NA) & 1u;
          if (it + k >= n) break;
          if (!__all_sync(0xFFFFFFFFu, ready))
            ok = warp_wait2(full_bar(s), full_par, acc_empty(d), acc_par ^ 1u, kMmaTries);
          if (!ok) break;
          tc_fence_after();
          ready = mbar_test2(full_bar(sn), full_par_n, acc_empty(dn), acc_par_n ^ 1u);
          // (opaque, so that the sums below are not all worked out ahead and kept in registers)
          uint64_t da = da0, db = db0;
          asm volatile("" : "+l"(da), "+l"(db));
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < Cfg::kBK / 32; ++kk)   // 32 bytes along K: 2 in the descriptors' units
              gemm_fp8_mma<C>(tmem_base + d * BN, da + s * (Cfg::kStageBytes / 16) + 2 * kk,
                              db + s * (Cfg::kStageBytes / 16) + 2 * kk, Cfg::kIdesc, kk != 0 ? 1u : 0u);
            gemm_fp8_commit<C>(empty_bar(s));
            gemm_fp8_commit<C>(acc_full(d));
          }
          __syncwarp();
        }
      }
      // the last commits must have landed before TMEM is freed (one that never came was waited for)
      if (ok && n > 0) mbar_wait_bounded(acc_full(static_cast<int>((n - 1) % NA)), static_cast<uint32_t>((n - 1) / NA & 1));
    }
  } else if (warp >= Cfg::kAddWarp0) {
    // ---------------- adding warps: TMEM lane quarter warp % 4, column half (warp - 4) / 4
    if constexpr (Cfg::kRegSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsMany));
    const int q = warp & 3, half = (warp - Cfg::kAddWarp0) >> 2;
    constexpr int NC = Cfg::kCols, CH = 8;
    pdl_wait();
    RingPos<NA> u;
    bool ok = true;
    for (int t = t0; ok && t < n_tiles; t += dt) {
      int tm, tn;
      gemm_fp8_tile(g, t, tm, tn);
      const int64_t row = static_cast<int64_t>(tm) * Cfg::kBM + rank * 128 + 32 * q + lane;
      const int64_t col0 = static_cast<int64_t>(tn) * BN + half * NC;
      // rows and columns past the end use the last ones' scales; they are not stored
      const int64_t sa0 = (row < g.M ? row : g.M - 1) * g.kb;
      const int64_t sb0 = (col0 < g.N ? col0 : g.N - 1) / kFp8Block * g.kb;
      // A block's scales are loaded two blocks ahead, into registers of their own by parity: a copy from
      // one register to the next would wait for the load
      uint32_t sa[2], sb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = i < g.kb ? i : 0;
        sa[i] = load_scale<Cfg::kSf>(g.a_scales, sa0 + j);
        sb[i] = load_scale<Cfg::kSf>(g.b_scales, sb0 + j);
      }
      f32x2 acc[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) acc[i] = 0ull;
#pragma unroll 1
      for (int jj = 0; ok && jj < g.kb; jj += 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (jj + i >= g.kb) break;
          ok = warp_wait(acc_full(u.i), u.parity, 1);
          if (!ok) break;
          tc_fence_after();
          const float s = scale_value<Cfg::kSf>(sa[i]) * scale_value<Cfg::kSf>(sb[i]);
          const int j2 = jj + i + 2 < g.kb ? jj + i + 2 : g.kb - 1;
          sa[i] = load_scale<Cfg::kSf>(g.a_scales, sa0 + j2);
          sb[i] = load_scale<Cfg::kSf>(g.b_scales, sb0 + j2);
          const f32x2 s2 = f2_pack(s, s);
          const uint32_t src = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + u.i * BN + half * NC;
#pragma unroll
          for (int c = 0; c < NC / CH; ++c) {
            f32x2 p[CH / 2];
            tmem_ld_pairs(src + c * CH, p);
            if (c == NC / CH - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if constexpr (C == 2)
                  mbar_arrive_cluster(cluster_map(acc_empty(u.i), 0));
                else
                  mbar_arrive(acc_empty(u.i));
              }
            }
#pragma unroll
            for (int k = 0; k < CH / 2; ++k) acc[c * (CH / 2) + k] = f2_fma(p[k], s2, acc[c * (CH / 2) + k]);
          }
          u.next();
        }
      }
      if constexpr (Cfg::kAligned) {
        if (ok && row < g.M) {
#pragma unroll
          for (int c = 0; c < NC / 16; ++c)
            if (col0 + 16 * c < g.N) store_row16<Cfg::kOut>(g, row, col0 + 16 * c, acc + 8 * c);
        }
      } else if (ok) {
        const uint32_t buf = stage0 + Cfg::kBufOffset + (warp - Cfg::kAddWarp0) * kUnalignedBytes;
#pragma unroll
        for (int c = 0; c < NC / 16; ++c)
          if (col0 + 16 * c < g.N)
            store_unaligned16<Cfg::kOut, NC == 64 ? 16 : 4>(g, row - lane, col0 + 16 * c, acc + 8 * c, buf, lane);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (C == 2) cluster_sync_all();   // nothing of the pair's is in flight towards the other CTA
  if (warp == 1) {
    tc_fence_after();
    if constexpr (C == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(Cfg::kTmemCols)
                   : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(Cfg::kTmemCols)
                   : "memory");
  }
}

// ---------------------------------------------------------------- many rows, scales in powers of two
//
// With E8M0 scales the tensor core applies them itself (kind::mxf8f6f4, a scale per row and 32
// channels: a block's four MMAs name the same one), so a tile's whole sum stays in tensor memory and
// nothing is added in registers.  A pair of CTAs takes 256 x 224 of D: two accumulators of 224 columns
// leave room for the scales (12 columns, twice), and the epilogue of one tile runs under the MMAs of
// the next.  The scales reach tensor memory without a copy instruction, which would wait its turn with
// the MMAs: four warps, one per lane quarter, load four blocks' bytes of a row as one word and store it
// (row r of the tile: lane r mod 32 of every quarter, column r / 32, byte j mod 4).
//
// Measured: 8192^3 in 450 to 473 us, 2.4 PFLOP/s, where adding in registers takes 549 to 589 (variants: 397 and
// 523 us); 4096 x 14336 x 4096 in 201 to 215 us.  4096 x 8192 x 8192 keeps the tensor pipe 85 % busy (58 % when
// added in registers).  What bounds it is the power cap, and
// below that the MMAs.
template <int OT, bool ALIGNED>
struct GemmFp8MxConfig {
  static constexpr int kCtas = 2, kBM = 256, kBN = 224, kBK = kFp8Block;
  static constexpr int kOut = OT;
  static constexpr bool kAligned = ALIGNED;                 // as in GemmFp8Config
  static constexpr int kARows = 128, kBRows = kBN / 2;      // a CTA's share of a stage
  static constexpr int kABytes = kARows * kBK, kBBytes = kBRows * kBK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static_assert(kStageBytes % 1024 == 0 && kBBytes % 1024 == 0, "swizzle atoms");
  static constexpr int kStages = (196 * 1024) / kStageBytes;
  static constexpr int kBarOffset = kStages * kStageBytes;
  static constexpr int kBufOffset = kBarOffset + 256;
  static constexpr int kSfCols = 4 + 8;                     // A's 128 rows, B's 224 in 32-row cells
  static constexpr int kSfCol0 = 2 * kBN;
  static constexpr int kTmemCols = 512;
  static_assert(kSfCol0 + 2 * kSfCols <= kTmemCols);
  static constexpr int kSfWarp0 = 4, kEpiWarp0 = 8, kEpiWarps = 8;
  static constexpr int kSmemBytes = 1024 + kBufOffset + (ALIGNED ? 0 : kEpiWarps * kUnalignedBytes);
  static constexpr int kCols = kBN / 2;                     // columns per epilogue warp
  static constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
  // as gemm_fp8_idesc, with E8M0 scales (bit 23)
  static constexpr uint32_t kIdesc =
      (1u << 23) | (static_cast<uint32_t>(kBN >> 3) << 17) | (static_cast<uint32_t>(kBM >> 4) << 24);
};

// The scale bytes of blocks j .. j + 3 of row `row` as one word; past the end of the row or of the rows
// zeros, which meet no code but zeros.  vec: rows start on whole words.
__device__ __forceinline__ uint32_t load_scale_word(const uint8_t* scales, int64_t row, int64_t rows, int j, int kb,
                                                    bool vec) {
  if (row >= rows) return 0u;
  const uint8_t* p = scales + row * kb + j;
  if (vec) return ld_u32(p);
  uint32_t w = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (j + i < kb) w |= ld_u8(p + i) << (8 * i);
  return w;
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    gemm_fp8_mx_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                       GemmFp8Args g) {
  constexpr int S = Cfg::kStages, BN = Cfg::kBN, C = Cfg::kCtas;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t s_tmem_base;
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  const uint32_t stage0 = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = stage0 + Cfg::kBarOffset;
  auto a_tile = [&](int s) { return stage0 + s * Cfg::kStageBytes; };
  auto b_tile = [&](int s) { return stage0 + s * Cfg::kStageBytes + Cfg::kABytes; };
  // what the MMA warp waits for is on the leader's barriers; what it commits arrives on both CTAs'
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
  auto acc_full = [&](int d) { return bars + 8u * (2 * S + d); };
  auto acc_empty = [&](int d) { return bars + 8u * (2 * S + 2 + d); };
  auto sf_full = [&](int d) { return bars + 8u * (2 * S + 4 + d); };
  auto sf_empty = [&](int d) { return bars + 8u * (2 * S + 6 + d); };

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int d = 0; d < 2; ++d) {
      mbar_init(acc_full(d), 1);
      mbar_init(acc_empty(d), C * Cfg::kEpiWarps);
      mbar_init(sf_full(d), C * 4);
      mbar_init(sf_empty(d), 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem_base)),
                 "r"(Cfg::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // the pair's barriers are set up
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  const int n_tiles = g.tiles_m * g.tiles_n;
  const int t0 = static_cast<int>(blockIdx.x) / C, dt = static_cast<int>(gridDim.x) / C;

  if (warp == 0) {
    gemm_fp8_produce<Cfg>(g, amap, bmap, rank, t0, dt, stage0, bars);
  } else if (warp == 1) {
    // ---------------- MMA issuer (the leader)
    if (rank == 0) {
      RingPos<S> r;
      RingPos<2> u, f;
      bool ok = true, ready = false;
      uint32_t last = 0;   // 1 | accumulator << 1 | parity << 8 of the last commit, 0: none
      const uint64_t da0 = umma_smem_desc(a_tile(0), 1024, 2), db0 = umma_smem_desc(b_tile(0), 1024, 2);
      for (int t = t0; ok && t < n_tiles; t += dt) {
        ok = warp_wait(acc_empty(u.i), u.parity ^ 1u, kMmaTries);
        for (int j = 0; ok && j < g.kb; ++j) {
          if ((j & 3) == 0) ok = warp_wait(sf_full(f.i), f.parity, kMmaTries);
          if (!__all_sync(0xFFFFFFFFu, ready)) ok = ok && warp_wait(full_bar(r.i), r.parity, kMmaTries);
          if (!ok) break;
          tc_fence_after();
          const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(r.i) * (Cfg::kStageBytes / 16));
          RingPos<S> rn = r;
          rn.next();
          ready = mbar_test(full_bar(rn.i), rn.parity);
          const uint32_t id = static_cast<uint32_t>(j & 3);   // the block's byte in the scales' cells
          const uint32_t idesc = Cfg::kIdesc | (id << 4) | (id << 29);
          const uint32_t sfa = (tmem_base + Cfg::kSfCol0 + f.i * Cfg::kSfCols) | (id << 30), sfb = sfa + 4;
          const bool group_end = (j & 3) == 3 || j == g.kb - 1;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < Cfg::kBK / 32; ++kk)
              umma_e4m3_scaled(tmem_base + u.i * BN, da0 + off + 2 * kk, db0 + off + 2 * kk, idesc, sfa, sfb,
                               (j | kk) != 0 ? 1u : 0u);
            gemm_fp8_commit<C>(empty_bar(r.i));
            if (group_end) gemm_fp8_commit<C>(sf_empty(f.i));
            if (j == g.kb - 1) gemm_fp8_commit<C>(acc_full(u.i));
          }
          __syncwarp();
          if (group_end) f.next();
          r = rn;
        }
        if (ok) last = 1u | static_cast<uint32_t>(u.i) << 1 | u.parity << 8;
        u.next();
      }
      // the last commits must have landed before TMEM is freed
      if (last) mbar_wait_bounded(acc_full((last >> 1) & 1u), last >> 8);
    }
  } else if (warp >= Cfg::kEpiWarp0) {
    // ---------------- epilogue: lane quarter warp % 4, column half (warp - 8) / 4
    const int q = warp & 3, half = (warp - Cfg::kEpiWarp0) >> 2;
    constexpr int NC = Cfg::kCols;
    pdl_wait();   // D may still be read by an earlier kernel
    RingPos<2> u;
    for (int t = t0; t < n_tiles; t += dt, u.next()) {
      int tm, tn;
      gemm_fp8_tile(g, t, tm, tn);
      const int64_t row = static_cast<int64_t>(tm) * Cfg::kBM + rank * 128 + 32 * q + lane;
      const int64_t col0 = static_cast<int64_t>(tn) * BN + half * NC;
      if (!warp_wait(acc_full(u.i), u.parity, 0)) break;
      tc_fence_after();
      const uint32_t src = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + u.i * BN + half * NC;
#pragma unroll 1
      for (int c = 0; c < NC / 16; ++c) {
        f32x2 p[8];
        tmem_ld_pairs(src + 16 * c, p);
        if constexpr (Cfg::kAligned) {
          if (row < g.M && col0 + 16 * c < g.N) store_row16<Cfg::kOut>(g, row, col0 + 16 * c, p);
        } else if (col0 + 16 * c < g.N) {
          const uint32_t buf = stage0 + Cfg::kBufOffset + (warp - Cfg::kEpiWarp0) * kUnalignedBytes;
          store_unaligned16<Cfg::kOut, 4>(g, row - lane, col0 + 16 * c, p, buf, lane);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_map(acc_empty(u.i), 0));
    }
  } else if (warp >= Cfg::kSfWarp0) {
    // ---------------- scales into tensor memory: lane quarter warp % 4, all quarters alike
    const int q = warp & 3;
    const auto* as = static_cast<const uint8_t*>(g.a_scales);
    const auto* bs = static_cast<const uint8_t*>(g.b_scales);
    const int64_t b_rows = (g.N + kFp8Block - 1) / kFp8Block;
    pdl_wait();
    RingPos<2> f;
    bool ok = true;
    for (int t = t0; ok && t < n_tiles; t += dt) {
      int tm, tn;
      gemm_fp8_tile(g, t, tm, tn);
      const int64_t ra = static_cast<int64_t>(tm) * Cfg::kBM + rank * 128 + lane;
      const int64_t rb = static_cast<int64_t>(tn) * BN + lane;
      for (int j = 0; j < g.kb; j += 4, f.next()) {
        uint32_t wa[4], wb[8];   // the loads run while the buffer is waited for
#pragma unroll
        for (int i = 0; i < 4; ++i) wa[i] = load_scale_word(as, ra + 32 * i, g.M, j, g.kb, g.sf_vec);
#pragma unroll
        for (int i = 0; i < 8; ++i) wb[i] = i < BN / 32 ? load_scale_word(bs, (rb + 32 * i) / kFp8Block, b_rows, j, g.kb, g.sf_vec) : 0u;
        ok = warp_wait(sf_empty(f.i), f.parity ^ 1u, 0);
        if (!ok) break;
        tc_fence_after();
        const uint32_t dst = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + Cfg::kSfCol0 + f.i * Cfg::kSfCols;
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(wa[0]), "r"(wa[1]),
                     "r"(wa[2]), "r"(wa[3])
                     : "memory");
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(dst + 4), "r"(wb[0]),
                     "r"(wb[1]), "r"(wb[2]), "r"(wb[3]), "r"(wb[4]), "r"(wb[5]), "r"(wb[6]), "r"(wb[7])
                     : "memory");
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_map(sf_full(f.i), 0));
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // nothing of the pair's is in flight towards the other CTA
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(Cfg::kTmemCols)
                 : "memory");
  }
}

// ---------------------------------------------------------------- few rows: 128 of B's rows by BT tokens
//
// For decode batches the product is a stream of B: here B is the MMA's row operand (tiles of 128 of
// its rows, one scale per tile and block) and BT rows of A are its columns, so no MMA row is idle.
// One CTA to an SM and one tile to a CTA; where there are fewer tiles than SMs, the blocks of K are
// split over a cluster.  A CTA's sums then go to the CTA of the cluster that owns their token (pushed
// into its shared memory), which adds them in the order of their ranks: no atomics, no workspace.
//
// Measured, with weights that are not in L2 (and, in brackets, ones that are): 1 x 14336 x 4096 12.4 us (10.6),
// 16 x 4096 x 14336 13.1 (10.6), 16 x 8192 x 8192 13.9 (11.3), 64 x 14336 x 4096 14.5 (13.3), 16 x 4096 x 4096 6.9
// (5.7).  Of the first, B's 58.7 MB stream in 8.3 us (7.1 TB/s); the rest is the first load (1.7 us), the sums and
// stores (0.6 us) and the gap to the next launch.  Variants: 16 x 4096 x 14336 with K over 1 / 2 / 3 / 4 CTAs
// 29.4 / 17.1 / 14.1 / 13.7 us; with two smaller CTAs to an SM the early start of the next launch put two CTAs
// of one grid on an SM beside idle ones (64 x 14336 x 4096: 26.6 us against 14.9).
template <int BT_, int OT, int SF>
struct GemmFp8FewConfig {
  static constexpr int kBT = BT_, kBK = kFp8Block;
  static constexpr int kOut = OT, kSf = SF;
  static constexpr int kMaxSplit = 8;                                // portable cluster size
  static constexpr int kWBytes = 128 * kBK, kXBytes = kBT * kBK;
  static constexpr int kStageBytes = kWBytes + kXBytes;
  static constexpr int kHalves = kBT > 32 ? 2 : 1;                   // adding warps per TMEM lane quarter
  static constexpr int kTok = kBT / kHalves;                         // tokens per adding warp
  static constexpr int kAddWarp0 = 4, kAddWarps = 4 * kHalves;
  static constexpr int kThreads = 32 * (kAddWarp0 + kAddWarps);
  static constexpr int kSumBytes = (kBT + kMaxSplit - 1) * 128 * 4;  // split x few_own rows of sums, at most
  static constexpr int kMultBytes = kAddWarps * 2 * kTok * 4;        // per adding warp: two blocks' multipliers
  static constexpr int kStages = (222 * 1024 - kSumBytes - kMultBytes) / kStageBytes;
  static constexpr int kBarOffset = kStages * kStageBytes;
  static constexpr int kMultOffset = kBarOffset + 512;
  static constexpr int kSumOffset = kMultOffset + kMultBytes;
  static constexpr int kSmemBytes = 1024 + kSumOffset + kSumBytes;
  static constexpr int kAccs = 4;
  static constexpr int kTmemCols = kAccs * kBT;
  static constexpr uint32_t kIdesc = gemm_fp8_idesc(128, kBT);
  static_assert(kStageBytes % 1024 == 0, "stages stay 1024-byte aligned (128-byte swizzle atoms)");
  static_assert(8 * (2 * kStages + 2 * kAccs) <= 512 && kSumOffset % 16 == 0 && kSmemBytes <= 227 * 1024);
};

// Tokens whose sums one CTA of a cluster takes.
__host__ __device__ constexpr int few_own(int bt, int split) { return (bt + split - 1) / split; }

// One thread's sums to the CTAs that own their tokens (token i: CTA i / own), as
// sums[rank][token of the owner][row nl].  SPLIT is a constant so that the division is one by a
// constant: with a variable one the 64 stores of a thread took 6.7 us.
template <int SPLIT, int BT, int TOK>
__device__ __forceinline__ void few_push(const f32x2 (&acc)[TOK / 2], uint32_t sums, int rank, int tok0, int nl) {
  constexpr int OWN = few_own(BT, SPLIT);
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    float v[2];
    f2_unpack(acc[i / 2], v[0], v[1]);
    const int tok = tok0 + i, owner = tok / OWN;
    const uint32_t local = sums + 4u * ((rank * OWN + (tok - owner * OWN)) * 128 + nl);
    if constexpr (SPLIT > 1)
      st_cluster_f32(cluster_map(local, owner), v[i & 1]);
    else
      sts32(local, __float_as_uint(v[i & 1]));
  }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    gemm_fp8_few_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                        GemmFp8Args g, int split) {
  constexpr int S = Cfg::kStages, BT = Cfg::kBT, NA = Cfg::kAccs, TOK = Cfg::kTok;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t s_tmem_base;
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t stage0 = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = stage0 + Cfg::kBarOffset, sums = stage0 + Cfg::kSumOffset;
  auto w_tile = [&](int s) { return stage0 + s * Cfg::kStageBytes; };
  auto x_tile = [&](int s) { return stage0 + s * Cfg::kStageBytes + Cfg::kWBytes; };
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
  auto acc_full = [&](int d) { return bars + 8u * (2 * S + d); };
  auto acc_empty = [&](int d) { return bars + 8u * (2 * S + NA + d); };
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int d = 0; d < NA; ++d) {
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
  // the cluster's CTAs are running, so that their shared memory can be written; awaited below
  if (split > 1) cluster_arrive();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int t = blockIdx.x / split;
  const int tn = t % g.tiles_n, tm = t / g.tiles_n;
  const int j0 = static_cast<int>(static_cast<int64_t>(g.kb) * rank / split);
  const int j1 = static_cast<int>(static_cast<int64_t>(g.kb) * (rank + 1) / split);
  const int64_t m0 = static_cast<int64_t>(tm) * BT, n0 = static_cast<int64_t>(tn) * 128;
  const int own = few_own(BT, split);   // this CTA takes the sums of tokens rank * own ...

  if (warp == 0) {
    if (lane == 0) {
      prefetch_map(&wmap);
      prefetch_map(&xmap);
      pdl_wait();
      RingPos<S> r;
      int filled = 0;
      for (int j = j0; j < j1; ++j, r.next()) {
        if (!mbar_test(empty_bar(r.i), r.parity ^ 1u) && !mbar_wait_bounded(empty_bar(r.i), r.parity ^ 1u)) break;
        mbar_arrive_expect_tx(full_bar(r.i), Cfg::kStageBytes);
        tma_load_2d(w_tile(r.i), &wmap, j * Cfg::kBK, tn * 128, full_bar(r.i));
        tma_load_2d(x_tile(r.i), &xmap, j * Cfg::kBK, tm * BT, full_bar(r.i));
        filled = filled < S ? filled + 1 : S;
      }
      // every issued copy lands before the CTA leaves
      if (filled < S) r = RingPos<S>{};
      for (int j = 0; j < filled; ++j, r.next()) mbar_wait_bounded(full_bar(r.i), filled < S ? 0u : r.parity ^ 1u);
    }
  } else if (warp == 1) {
    RingPos<S> r;
    RingPos<NA> u;
    bool ready = false;
    uint32_t last = 0;   // 1 | accumulator << 1 | parity << 8 of the last commit, 0: none
    const uint64_t dw0 = umma_smem_desc(w_tile(0), 1024, 2), dx0 = umma_smem_desc(x_tile(0), 1024, 2);
    for (int j = j0; j < j1; ++j) {
      if (!__all_sync(0xFFFFFFFFu, ready) &&
          !warp_wait2(full_bar(r.i), r.parity, acc_empty(u.i), u.parity ^ 1u, kMmaTries))
        break;
      tc_fence_after();
      const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(r.i) * (Cfg::kStageBytes / 16));
      RingPos<S> rn = r;
      RingPos<NA> un = u;
      rn.next();
      un.next();
      ready = mbar_test2(full_bar(rn.i), rn.parity, acc_empty(un.i), un.parity ^ 1u);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < Cfg::kBK / 32; ++kk)
          umma_e4m3(tmem_base + u.i * BT, dw0 + off + 2 * kk, dx0 + off + 2 * kk, Cfg::kIdesc, kk != 0 ? 1u : 0u);
        umma_commit(empty_bar(r.i));
        umma_commit(acc_full(u.i));
      }
      __syncwarp();
      last = 1u | static_cast<uint32_t>(u.i) << 1 | u.parity << 8;
      r = rn;
      u = un;
    }
    if (last) mbar_wait_bounded(acc_full((last >> 1) & 0x7F), last >> 8);
  } else if (warp == 2) {
    // B's first stages into L2 while the kernel in front still runs (which may even be writing them: L2 is
    // where all copies meet, and the ring's own loads come after the wait)
    if (lane == 0)
      for (int j = j0; j < j1 && j < j0 + S; ++j) tma_prefetch_2d(&wmap, j * Cfg::kBK, tn * 128);
  } else if (warp >= Cfg::kAddWarp0) {
    // lane quarter warp % 4: this thread holds B's row n0 + nl and TOK of the tile's tokens, from `tok0` on
    const int q = warp & 3, nl = 32 * q + lane;
    const int tok0 = ((warp - Cfg::kAddWarp0) >> 2) * TOK;
    constexpr int TL = (TOK + 31) / 32;   // tokens whose multipliers a lane works out
    const uint32_t mult = stage0 + Cfg::kMultOffset + (warp - Cfg::kAddWarp0) * (2 * TOK * 4);
    pdl_wait();
    const int64_t sb0 = static_cast<int64_t>(tn) * g.kb;
    int64_t sa0[TL];
#pragma unroll
    for (int i = 0; i < TL; ++i) {
      const int64_t m = m0 + tok0 + i * 32 + lane;
      sa0[i] = (m < g.M ? m : g.M - 1) * g.kb;
    }
    // lane l takes tokens 32 i + l: their scales of a block and the tile's, loaded two blocks ahead (into
    // registers of their own by parity, as above), multiplied, and passed to the warp's other lanes
    // through shared memory
    auto scales = [&](int j, uint32_t (&v)[TL], uint32_t& sb) {
      const int jj = j < j1 ? j : (j1 > 0 ? j1 - 1 : 0);
      sb = load_scale<Cfg::kSf>(g.b_scales, sb0 + jj);
#pragma unroll
      for (int i = 0; i < TL; ++i) v[i] = load_scale<Cfg::kSf>(g.a_scales, sa0[i] + jj);
    };
    auto put = [&](int slot, const uint32_t (&v)[TL], uint32_t sb) {
#pragma unroll
      for (int i = 0; i < TL; ++i)
        if (32 * i + lane < TOK) sts32(mult + 4u * (slot * TOK + 32 * i + lane), __float_as_uint(scale_value<Cfg::kSf>(v[i]) * scale_value<Cfg::kSf>(sb)));
    };
    uint32_t sa[2][TL], sb[2];
    scales(j0, sa[0], sb[0]);
    scales(j0 + 1, sa[1], sb[1]);
    f32x2 acc[TOK / 2];
#pragma unroll
    for (int i = 0; i < TOK / 2; ++i) acc[i] = 0ull;
    RingPos<NA> u;
    bool ok = true;
#pragma unroll 1
    for (int jj = j0; ok && jj < j1; jj += 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (jj + i >= j1) break;
        put(i, sa[i], sb[i]);
        scales(jj + i + 2, sa[i], sb[i]);
        ok = warp_wait(acc_full(u.i), u.parity, 1);
        if (!ok) break;
        __syncwarp();   // the lanes' multipliers
        tc_fence_after();
        const uint32_t src = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + u.i * BT + tok0;
#pragma unroll
        for (int c = 0; c < TOK / 16; ++c) {
          f32x2 p[8], m[8];
#pragma unroll
          for (int k = 0; k < 8; k += 2) lds_pairs(mult + 4u * (i * TOK + 16 * c + 2 * k), m[k], m[k + 1]);
          tmem_ld_pairs(src + c * 16, p);
          if (c == TOK / 16 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty(u.i));
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[8 * c + k] = f2_fma(p[k], m[k], acc[8 * c + k]);
        }
        u.next();
      }
    }
    if (split > 1) cluster_wait();
    switch (split) {
      case 8: few_push<8, BT, TOK>(acc, sums, rank, tok0, nl); break;
      case 7: few_push<7, BT, TOK>(acc, sums, rank, tok0, nl); break;
      case 6: few_push<6, BT, TOK>(acc, sums, rank, tok0, nl); break;
      case 5: few_push<5, BT, TOK>(acc, sums, rank, tok0, nl); break;
      case 4: few_push<4, BT, TOK>(acc, sums, rank, tok0, nl); break;
      case 3: few_push<3, BT, TOK>(acc, sums, rank, tok0, nl); break;
      case 2: few_push<2, BT, TOK>(acc, sums, rank, tok0, nl); break;
      default: few_push<1, BT, TOK>(acc, sums, rank, tok0, nl); break;
    }
  }
  __syncwarp();
  if (split > 1) {
    if (warp < Cfg::kAddWarp0) cluster_wait();
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  // eight neighbouring columns of one token a thread: 16-byte reads and stores
  for (int c = tid; c < own * 16; c += Cfg::kThreads) {
    const int tok = rank * own + c / 16;
    const int64_t m = m0 + tok, n = n0 + 8 * (c % 16);
    if (tok >= BT || m >= g.M || n >= g.N) continue;
    f32x2 v[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
    for (int r = 0; r < split; ++r) {
      f32x2 a[4];
      const uint32_t at = sums + 4u * ((r * own + c / 16) * 128 + 8 * (c % 16));
      lds_pairs(at, a[0], a[1]);
      lds_pairs(at + 16, a[2], a[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = f2_add(v[i], a[i]);
    }
    store_row8<Cfg::kOut>(g, m, n, v);
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
