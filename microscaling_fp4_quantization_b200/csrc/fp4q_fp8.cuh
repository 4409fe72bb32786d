// 8-bit (E4M3) quantization with a scale per 128 channels: the quantizer (a scale per row and
// 128 channels, or per 128 x 128 tile) and the RMS norm, with the residual's addition, that ends
// in it.  The rules of the scale and of the codes are in fp4q.h (fp4q_quantize_fp8).
//
// Times: us a launch, launches back to back in a graph on bf16 inputs that pass L2 in turn.  The tensor call shows
// its host time where that is longer (6 to 9 us), and a little more where it is not (large norm 146, call 158).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "fp4q_device.cuh"

namespace fp4q {

constexpr int kFp8Block = 128;          // channels (and weight rows) per scale
constexpr int kFp8Chunk = 16;           // channels per thread: 32 bytes in, one 16-byte store of codes
constexpr int kFp8Lanes = kFp8Block / kFp8Chunk;   // lanes that share a block

enum : int { kDtBf16 = 0, kDtFp16 = 1, kDtF32 = 2 };   // fp4q_dtype
enum : int { kSfF32 = 0, kSfE8m0 = 1 };                // fp4q_fp8_scale

// 16-bit pair word (element 2k in the low half) <-> two fp32 values.
template <int DT>
__device__ __forceinline__ f32x2 pair_to_f32(uint32_t w) {
  if constexpr (DT == kDtBf16) {
    return f2_pack(bf16_lo(w), bf16_hi(w));
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return f2_pack(f.x, f.y);
  }
}
template <int DT>
__device__ __forceinline__ uint32_t pair_from_f32(float lo, float hi) {
  uint32_t r;
  if constexpr (DT == kDtBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int DT>
__device__ __forceinline__ uint32_t pair_from_f32(f32x2 p) {
  float lo, hi;
  f2_unpack(p, lo, hi);
  return pair_from_f32<DT>(lo, hi);
}

// Four fp32 values -> four E4M3 bytes (nearest even, saturating at 448; NaN -> 0x7F).
__device__ __forceinline__ uint32_t e4m3x4(f32x2 a, f32x2 b) {
  float a0, a1, b0, b1;
  f2_unpack(a, a0, a1);
  f2_unpack(b, b0, b1);
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n"
      " cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n}"
      : "=r"(r)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
  return r;
}

// The scale of a block whose largest magnitude has the fp32 bit pattern A (sign clear), and what
// the elements are divided by: v = y / s.
//   F32   s = max(RN(A / 448), 2^-126); the quotient is corrected once by its remainder (Markstein's step, as
//         div_rn_markstein), so it is the correctly rounded one while s >= 2^-90 (below, the remainder
//         falls under fp32's range and v may be one ulp off);
//   E8M0  s = 2^e, byte e + 127, e = ceil(log2(A / 448)) >= -126, from A's bits: 448 = 1.75 * 2^8;
//         the product with 2^-e is exact.
// An infinity or a NaN in the block gives the scale NaN (byte 255), and so NaN codes.
// The bit patterns of magnitudes are ordered as the magnitudes are, NaN above infinity: maxima
// are taken on them, which keeps a NaN that fmaxf would drop.
template <int SF>
struct Fp8Scale {
  float s;        // F32: the scale; E8M0: unused
  float r;        // 1 / s
  uint32_t byte;  // E8M0
  __device__ __forceinline__ explicit Fp8Scale(uint32_t A) {
    const bool finite = A < 0x7F800000u;
    if constexpr (SF == kSfF32) {
      // RN(A / 448) by one correction of the product with RN(1 / 448); its remainder is exact
      // wherever the quotient is above the lower bound 2^-126
      constexpr float r448 = 1.0f / 448.0f;
      const float a = __uint_as_float(A), q0 = a * r448;
      const float q = fmaf(fmaf(-q0, 448.0f, a), r448, q0);
      s = finite ? fmaxf(q, __uint_as_float(0x00800000u)) : __uint_as_float(0x7FFFFFFFu);
      r = __frcp_rn(s);
      byte = 0;
    } else {
      const int e = static_cast<int>(A >> 23) - 8 + ((A & 0x7FFFFFu) > 0x600000u ? 1 : 0);
      byte = finite ? static_cast<uint32_t>(e < 1 ? 1 : e) : 255u;
      s = 0.0f;
      r = __uint_as_float(finite ? (254u - byte) << 23 : 0x7FFFFFFFu);
    }
  }
  // v = y / s of a pair
  __device__ __forceinline__ f32x2 quotient(f32x2 y) const {
    const f32x2 r2 = f2_pack(r, r);
    const f32x2 q0 = f2_mul(y, r2);
    if constexpr (SF == kSfE8m0) return q0;
    const f32x2 rem = f2_fma(q0, f2_pack(-s, -s), y);
    return f2_fma(rem, r2, q0);
  }
  __device__ __forceinline__ void store(void* scales, int64_t i) const {
    if constexpr (SF == kSfF32)
      static_cast<float*>(scales)[i] = s;
    else
      static_cast<uint8_t*>(scales)[i] = static_cast<uint8_t>(byte);
  }
};

// Magnitude patterns of a pair word as two packed 16-bit values, and of one of them as fp32 bits.
__device__ __forceinline__ uint32_t pair_abs(uint32_t w) { return w & 0x7FFF7FFFu; }
template <int DT>
__device__ __forceinline__ uint32_t half_bits_to_f32(uint32_t h) {
  if constexpr (DT == kDtBf16) return h << 16;
  return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
}

// Unsigned division by a fixed d of n < 2^31: (n * mul) >> shift, mul = ceil(2^shift / d),
// shift = 31 + ceil(log2 d).
struct FastDiv {
  uint32_t d, mul, shift;
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * mul) >> shift);
  }
};

struct Fp8QuantArgs {
  const uint16_t* x;   // [M] rows, ldx elements apart
  int64_t ldx, M, K;
  FastDiv kb;          // blocks per row, ceil(K / 128)
  uint32_t n_blocks;   // scales: rows of blocks x kb.d
  uint8_t* codes;      // [M][K]
  void* scales;
};

// ---------------------------------------------------------------- a scale per row and 128 channels
//
// One pass: eight lanes hold a block (16 channels each, two 16-byte loads and one 16-byte store),
// its maximum takes three shuffles, and a warp's four blocks are neighbours in memory.  The floor
// is the traffic, 3 bytes an element.  A CTA does 32 blocks and leaves: the next one's loads start
// as soon as there is room, where the CTAs of a persistent grid load and store in step.  32768 x 14336:
// 204 us, 7.0 TB/s (E8M0 196); in one run of variants 198 us, 251 on a persistent grid of one wave and 228
// with two waves of four blocks to a group of lanes.
constexpr int kFp8QuantThreads = 256;

template <int DT>
__device__ __forceinline__ void load_chunk(const uint16_t* p, uint32_t (&w)[8]) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
  const uint4 v0 = q[0], v1 = q[1];
  w[0] = v0.x, w[1] = v0.y, w[2] = v0.z, w[3] = v0.w;
  w[4] = v1.x, w[5] = v1.y, w[6] = v1.z, w[7] = v1.w;
}

template <int DT, int SF>
__global__ void __launch_bounds__(kFp8QuantThreads) quantize_fp8_rows_kernel(Fp8QuantArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t sub = threadIdx.x & (kFp8Lanes - 1);
  const uint32_t block = blockIdx.x * (kFp8QuantThreads / kFp8Lanes) + threadIdx.x / kFp8Lanes;
  uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  int64_t out = -1;   // offset of this lane's codes; none past the end of the row or of the blocks
  if (block < a.n_blocks) {
    const uint32_t row = a.kb.div(block);
    const int64_t col = static_cast<int64_t>(block - row * a.kb.d) * kFp8Block + sub * kFp8Chunk;
    if (col < a.K) {
      load_chunk<DT>(a.x + row * a.ldx + col, w);
      out = row * a.K + col;
    }
  }
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, pair_abs(w[i]));
#pragma unroll
  for (int d = 1; d < kFp8Lanes; d *= 2) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  const Fp8Scale<SF> sc(half_bits_to_f32<DT>(max(m & 0xFFFFu, m >> 16)));
  if (out >= 0) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = e4m3x4(sc.quotient(pair_to_f32<DT>(w[2 * i])), sc.quotient(pair_to_f32<DT>(w[2 * i + 1])));
    stg128(a.codes + out, c[0], c[1], c[2], c[3]);
    if (sub == 0) sc.store(a.scales, block);
  }
}

// ---------------------------------------------------------------- a scale per 128 x 128 tile
//
// One CTA per tile, held in registers (64 elements a thread: four rows 32 apart), so that it is
// read once; the maximum goes over a warp by shuffles and over the CTA's eight warps through
// shared memory.  14336 x 4096: 28.4 us, 6.2 TB/s (E8M0 26.9), bound by the traffic; in one run of variants
// 27.2 us, and 27.7 to 34.6 with 512 threads a tile.
template <int DT, int SF>
__global__ void __launch_bounds__(kFp8QuantThreads) quantize_fp8_tiles_kernel(Fp8QuantArgs a) {
  __shared__ uint32_t s_max[kFp8QuantThreads / 32];
  constexpr int R = kFp8Block / (kFp8QuantThreads / kFp8Lanes);   // rows per thread
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t tile = blockIdx.x;
  const uint32_t rb = a.kb.div(tile);
  const int64_t col = static_cast<int64_t>(tile - rb * a.kb.d) * kFp8Block + (threadIdx.x & (kFp8Lanes - 1)) * kFp8Chunk;
  const int64_t row0 = static_cast<int64_t>(rb) * kFp8Block + threadIdx.x / kFp8Lanes;
  uint32_t w[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = row0 + i * (kFp8QuantThreads / kFp8Lanes);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = 0u;
    if (row < a.M && col < a.K) load_chunk<DT>(a.x + row * a.ldx + col, w[i]);
  }
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = __vmaxu2(m, pair_abs(w[i][j]));
  m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kFp8QuantThreads / 32; ++i) m = max(m, s_max[i]);
  const Fp8Scale<SF> sc(half_bits_to_f32<DT>(m));
  if (threadIdx.x == 0) sc.store(a.scales, tile);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = row0 + i * (kFp8QuantThreads / kFp8Lanes);
    if (row < a.M && col < a.K) {
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c[j] = e4m3x4(sc.quotient(pair_to_f32<DT>(w[i][2 * j])), sc.quotient(pair_to_f32<DT>(w[i][2 * j + 1])));
      stg128(a.codes + row * a.K + col, c[0], c[1], c[2], c[3]);
    }
  }
}

// ---------------------------------------------------------------- RMS norm with the residual's addition
//
//   h = x + r,  stored = RN(h),  y = h * (1 / sqrt(mean(h^2) + eps)) * w,  then codes and scales of y.
//
// A CTA takes whole rows, one after another, and holds a row in registers between its one read and
// its one write: C chunks of 16 channels a thread.  C = 2 where there are many rows (smaller CTAs, more
// of them on an SM in different phases), C = 1 where a row has an SM to itself and its latency counts.
// C = 4 took 182 us at 16384 x 8192.  Measured, us with C = 1 / 2, by channels (down) and rows:
//                1           148         149         333         600         1200        2400        16384
//   with a residual
//     4096   2.0 / 2.6   2.7 / 3.7   3.1 / 3.8   4.2 / 6.1   5.3 / 6.4   8.2 / 8.9  13.7 / 14.1   76 / 73
//     5008   2.2 / 2.8   3.0 / 4.1   3.7 / 4.3   4.5 / 6.3   6.9 / 7.1  10.1 / 10.8 17.1 / 17.4  101 / 97
//     8192   2.6 / 3.0   3.8 / 4.5   4.2 / 5.0   6.8 / 6.8   9.3 / 9.5  15.1 / 14.9 26.3 / 26.3  157 / 146
//    14336   3.6 / 4.0   5.1 / 5.8   7.4 / 6.2  10.9 / 10.7 16.9 / 15.2 28.5 / 26.7 50.5 / 46.2  305 / 276
//   without
//     4096   1.9 / 2.4   2.1 / 2.6   2.5 / 2.8   3.4 / 3.5   3.9 / 5.1   6.3 / 5.8   9.4 / 9.7    52 / 47
//     8192   2.2 / 2.6   2.8 / 3.4   3.1 / 3.7   5.5 / 5.2   7.3 / 7.3  11.9 / 10.6 20.0 / 18.4  116 / 100
//    14336   2.7 / 3.0   3.7 / 4.3   5.5 / 4.7   8.6 / 8.3  13.2 / 11.7 22.6 / 19.6 40.9 / 33.4  247 / 195
// The border at one row to an SM suits long rows; up to 5008 channels C = 1 stays ahead to some 2400 rows, by
// 2 us at most.  h, the square sum and y stay in fp32: y is rounded once, to its code, and the
// norm is of h as it was before it is rounded to be stored.  The square sum goes over a chunk, then over
// groups of 32 chunks, then over the groups: one order for both values of C, so that a row's result does not
// depend on the batch it is in.
struct Fp8NormArgs {
  const uint16_t* x;
  const uint16_t* residual;   // or null
  const uint16_t* weight;
  uint16_t* residual_out;
  uint8_t* codes;
  void* scales;
  int64_t ldx, ldr, ldo, M;
  int K, kb;
  float eps;
};

constexpr int kFp8NormThreads = 1024;   // at most; K / (16 C) rounded up to whole warps

template <int DT, int SF, int C, bool RES>
__global__ void __launch_bounds__(kFp8NormThreads) add_rmsnorm_fp8_kernel(Fp8NormArgs a) {
  constexpr int kGroups = 2 * kFp8NormThreads / 32;   // groups of 32 chunks in the longest row
  __shared__ float s_part[2][kGroups];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x, n_warps = T >> 5;
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, parity ^= 1) {
    f32x2 h[C][8];
    float ss[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (tid + c * T) * kFp8Chunk;
      uint32_t w[8];
      if (col < a.K) {
        load_chunk<DT>(a.x + row * a.ldx + col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] = pair_to_f32<DT>(w[i]);
        if constexpr (RES) {
          load_chunk<DT>(a.residual + row * a.ldr + col, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[c][i] = f2_add(h[c][i], pair_to_f32<DT>(w[i]));
          uint16_t* o = a.residual_out + row * a.ldo + col;
          stg128(o, pair_from_f32<DT>(h[c][0]), pair_from_f32<DT>(h[c][1]), pair_from_f32<DT>(h[c][2]),
                 pair_from_f32<DT>(h[c][3]));
          stg128(o + 8, pair_from_f32<DT>(h[c][4]), pair_from_f32<DT>(h[c][5]), pair_from_f32<DT>(h[c][6]),
                 pair_from_f32<DT>(h[c][7]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] = 0ull;
      }
      f32x2 sq = 0ull;
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = f2_fma(h[c][i], h[c][i], sq);
      float s0, s1;
      f2_unpack(sq, s0, s1);
      ss[c] = s0 + s1;
    }
    // group g holds chunks 32 g ... 32 g + 31, whatever C is
#pragma unroll
    for (int d = 16; d > 0; d /= 2)
#pragma unroll
      for (int c = 0; c < C; ++c) ss[c] += __shfl_xor_sync(0xFFFFFFFFu, ss[c], d);
    if (lane == 0)
#pragma unroll
      for (int c = 0; c < C; ++c) s_part[parity][warp + c * n_warps] = ss[c];
    __syncthreads();   // the other half of s_part is written only after every thread passed this
    const int n_groups = C * n_warps;
    float tot = lane < n_groups ? s_part[parity][lane] : 0.0f;
    tot += lane + 32 < n_groups ? s_part[parity][lane + 32] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) tot += __shfl_xor_sync(0xFFFFFFFFu, tot, d);
    const float rstd = __frsqrt_rn(__fdiv_rn(tot, static_cast<float>(a.K)) + a.eps);
    const f32x2 rstd2 = f2_pack(rstd, rstd);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (tid + c * T) * kFp8Chunk;
      uint32_t m = 0u;
      if (col < a.K) {
        uint32_t w[8];
        load_chunk<DT>(a.weight + col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[c][i] = f2_mul(f2_mul(h[c][i], rstd2), pair_to_f32<DT>(w[i]));
          float y0, y1;
          f2_unpack(h[c][i], y0, y1);
          m = max(m, max(__float_as_uint(y0) & 0x7FFFFFFFu, __float_as_uint(y1) & 0x7FFFFFFFu));
        }
      }
#pragma unroll
      for (int d = 1; d < kFp8Lanes; d *= 2) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
      const Fp8Scale<SF> sc(m);
      if (col < a.K) {
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = e4m3x4(sc.quotient(h[c][2 * i]), sc.quotient(h[c][2 * i + 1]));
        stg128(a.codes + row * a.K + col, q[0], q[1], q[2], q[3]);
        if ((lane & (kFp8Lanes - 1)) == 0) sc.store(a.scales, row * a.kb + col / kFp8Block);
      }
    }
  }
}

}  // namespace fp4q
