// 8-bit GEMM (fp4q_gemm_fp8.cuh): its launcher.  One kernel family per translation unit, so that
// the library's kernels compile in parallel (see fp4q_host.cuh).
#include "fp4q_gemm_fp8.cuh"

#include <atomic>

#include "fp4q_launch.cuh"

namespace fp4q {
namespace host {

namespace {

// Codes [rows][K]: boxes of 128 bytes (one K-block) x box_rows, 128-byte swizzled; past the end of
// a row or of the rows zeros are read.
fp4q_status codes_map(CUtensorMap* map, const void* codes, int64_t rows, int64_t K, int box_rows) {
  EncodeTiledFn enc;
  fp4q_status st = encode_fn(&enc);
  if (st != FP4Q_OK) return st;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t box[2] = {kFp8Block, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    std::snprintf(last_error_buffer(), kLastErrorBytes, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return FP4Q_ERR_CUDA;
  }
  return FP4Q_OK;
}

struct Problem {
  const void *a_codes, *b_codes;
  GemmFp8Args g;
  int64_t K;
  cudaStream_t stream;
};

// The many-row kernels: persistent clusters (pairs) or CTAs, as many as are resident at once.
template <class Cfg, class Kernel>
fp4q_status launch_many(Kernel kernel, Problem p) {
  CUtensorMap amap, bmap;
  fp4q_status st = codes_map(&amap, p.a_codes, p.g.M, p.K, Cfg::kARows);
  if (st == FP4Q_OK) st = codes_map(&bmap, p.b_codes, p.g.N, p.K, Cfg::kBRows);
  if (st != FP4Q_OK) return st;
  p.g.tiles_m = static_cast<int>((p.g.M + Cfg::kBM - 1) / Cfg::kBM);
  p.g.tiles_n = static_cast<int>((p.g.N + Cfg::kBN - 1) / Cfg::kBN);
  KernelInfo ki;
  st = kernel_info(kernel, Cfg::kSmemBytes, Cfg::kThreads, &ki, 0, 100, Cfg::kCtas);
  if (st != FP4Q_OK) return st;
  int64_t n = static_cast<int64_t>(p.g.tiles_m) * p.g.tiles_n;
  const int64_t resident = Cfg::kCtas > 1 ? ki.max_clusters : ki.sm_count;
  if (n > resident) n = resident;
  cudaError_t e = launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(n * Cfg::kCtas)), dim3(Cfg::kThreads),
                                     Cfg::kSmemBytes, Cfg::kCtas, p.stream, amap, bmap, p.g);
  if (e != cudaSuccess) return cuda_fail(e, "gemm_fp8 launch");
  return FP4Q_OK;
}

// The warps that hand their registers over can do so only if the launch holds them.
template <class Cfg, class Kernel>
fp4q_status check_registers(Kernel kernel) {
  if constexpr (Cfg::kRegSplit) {
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_relaxed) == 0) {
      cudaFuncAttributes fa = {};
      cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes");
      regs.store(fa.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) < Cfg::kRegsLaunch) {
      std::snprintf(last_error_buffer(), kLastErrorBytes, "gemm_fp8: built with %d registers a thread, not %d",
                    regs.load(), Cfg::kRegsLaunch);
      return FP4Q_ERR_UNSUPPORTED;
    }
  }
  return FP4Q_OK;
}

template <int CTAS, int BN, int OT, int SF, bool ALIGNED>
fp4q_status launch_add(const Problem& p) {
  using Cfg = GemmFp8Config<CTAS, BN, OT, SF, ALIGNED>;
  fp4q_status st = check_registers<Cfg>(gemm_fp8_kernel<Cfg>);
  return st == FP4Q_OK ? launch_many<Cfg>(gemm_fp8_kernel<Cfg>, p) : st;
}

template <class Cfg>
fp4q_status launch_few(Problem p, int split) {
  CUtensorMap wmap, xmap;
  fp4q_status st = codes_map(&wmap, p.b_codes, p.g.N, p.K, 128);
  if (st == FP4Q_OK) st = codes_map(&xmap, p.a_codes, p.g.M, p.K, Cfg::kBT);
  if (st != FP4Q_OK) return st;
  p.g.tiles_m = static_cast<int>((p.g.M + Cfg::kBT - 1) / Cfg::kBT);
  p.g.tiles_n = static_cast<int>((p.g.N + 127) / 128);
  auto kernel = gemm_fp8_few_kernel<Cfg>;
  const int64_t tiles = static_cast<int64_t>(p.g.tiles_m) * p.g.tiles_n;
  KernelInfo ki;
  st = kernel_info(kernel, Cfg::kSmemBytes, Cfg::kThreads, &ki, 0, 100, split);
  if (st != FP4Q_OK) return st;
  // a cluster takes `split` SMs of one GPC, and GPCs differ: where the clusters do not all fit at once,
  // split less
  while (split > 1 && tiles > ki.max_clusters) {
    --split;
    st = kernel_info(kernel, Cfg::kSmemBytes, Cfg::kThreads, &ki, 0, 100, split);
    if (st != FP4Q_OK) return st;
  }
  cudaError_t e = launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(tiles * split)), dim3(Cfg::kThreads),
                                     Cfg::kSmemBytes, split, p.stream, wmap, xmap, p.g, split);
  if (e != cudaSuccess) return cuda_fail(e, "gemm_fp8 launch");
  return FP4Q_OK;
}

// Which kernel: the one whose time comes out least, as a start, a cost for each round of tiles over the
// SMs, and one for each block of K that a round works off (units of 10 ns).  The costs are fitted to
// measurements of all four kernels at M = 1 ... 4096 and nine pairs of N and K (1024 x 4096 to
// 8192 x 8192, 600 x 784): over those the choice takes 0.7 % longer than the fastest of the four on
// average (1.7 % with one cost per block alone).  Examples, of single kernels on random codes, in us as
// few / 128 x 128 / 256 x 128 / wide: 96 x 8192 x 8192 25.6 / 24.6 / 23.7 / 34.5; 333 x 4104 x 5008 31.3 / 20.4 /
// 17.8 / 24.4; 256 x 4096 x 4096 13.5 / 13.9 / 13.6 / 20.4; 1024 x 4096 x 4096 E8M0 49.4 / 27.3 / 27.9 / 22.7.
struct Variant {
  int tile_m, tile_n;   // of D
  int ctas;             // per tile
  int start, round, block;
};
constexpr Variant kFew16{16, 128, 1, 250, 60, 36}, kFew32{32, 128, 1, 250, 110, 31}, kFew64{64, 128, 1, 170, 250, 31};
// by scale format: with E8M0 the widest tile has its scales applied by the tensor core
constexpr Variant kOne[2] = {{128, 128, 1, 300, 140, 32}, {128, 128, 1, 280, 140, 33}};
constexpr Variant kWide[2] = {{256, 256, 2, 430, 150, 48}, {256, 224, 2, 470, 90, 30}};
// fp32 scales alone: with E8M0 a pair's rounds are as many as those of the 128 x 128 tiles or more, and one
// of its neighbours is never slower
constexpr Variant kPair{256, 128, 2, 320, 130, 30};

struct Estimate {
  int64_t time;
  int split;
};
Estimate estimate(const Variant& v, const GemmFp8Args& g, int sms, bool may_split) {
  const int64_t tiles = ((g.M + v.tile_m - 1) / v.tile_m) * ((g.N + v.tile_n - 1) / v.tile_n);
  const int64_t at_once = sms / v.ctas;
  const int64_t rounds = (tiles + at_once - 1) / at_once;
  // the blocks of K over as many CTAs as there are SMs for, two at least to each
  int64_t split = may_split ? at_once / tiles : 1;
  if (split > g.kb / 2) split = g.kb / 2;
  split = split < 1 ? 1 : split > 8 ? 8 : split;
  return {v.start + (split > 1 ? 40 : 0) + rounds * (v.round + (g.kb + split - 1) / split * v.block),
          static_cast<int>(split)};
}

// The variant for a product, and the CTAs its K is split over.
struct Choice {
  const Variant* v;
  int split;
};
Choice choose(int scale_format, const GemmFp8Args& g, int sms) {
  const Variant* few = g.M <= 16 ? &kFew16 : g.M <= 32 ? &kFew32 : &kFew64;
  const Estimate e = estimate(*few, g, sms, true);
  Choice c{few, e.split};
  int64_t best = e.time;
  auto consider = [&](const Variant* v) {   // a tie goes to the one considered first
    const int64_t t = estimate(*v, g, sms, false).time;
    if (t < best) c = {v, 1}, best = t;
  };
  consider(&kWide[scale_format]);
  consider(&kOne[scale_format]);
  if (scale_format == FP4Q_FP8_SCALE_F32) consider(&kPair);
  return c;
}

template <int OT, int SF, bool ALIGNED>
fp4q_status launch_tiles(const Variant* v, const Problem& p) {
  if (v == &kWide[SF]) {
    if constexpr (SF == kSfE8m0) {
      using Cfg = GemmFp8MxConfig<OT, ALIGNED>;
      return launch_many<Cfg>(gemm_fp8_mx_kernel<Cfg>, p);
    } else {
      return launch_add<2, 256, OT, SF, ALIGNED>(p);
    }
  }
  if constexpr (SF == kSfF32)
    if (v == &kPair) return launch_add<2, 128, OT, SF, ALIGNED>(p);
  return launch_add<1, 128, OT, SF, ALIGNED>(p);
}

fp4q_status current_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? FP4Q_OK : cuda_fail(e, "cudaDeviceGetAttribute");
}

template <int OT, int SF>
fp4q_status dispatch(const Problem& p) {
  int sms = 0;
  fp4q_status st = current_sms(&sms);
  if (st != FP4Q_OK) return st;
  const Choice c = choose(SF, p.g, sms);
  if (c.v == &kFew16) return launch_few<GemmFp8FewConfig<16, OT, SF>>(p, c.split);
  if (c.v == &kFew32) return launch_few<GemmFp8FewConfig<32, OT, SF>>(p, c.split);
  if (c.v == &kFew64) return launch_few<GemmFp8FewConfig<64, OT, SF>>(p, c.split);
  return p.g.vec != 0 ? launch_tiles<OT, SF, true>(c.v, p) : launch_tiles<OT, SF, false>(c.v, p);
}

template <int OT>
fp4q_status dispatch_sf(int scale_format, const Problem& p) {
  return scale_format == FP4Q_FP8_SCALE_F32 ? dispatch<OT, kSfF32>(p) : dispatch<OT, kSfE8m0>(p);
}

}  // namespace

fp4q_status gemm_fp8_choice(int scale_format, int64_t M, int64_t N, int64_t K, int sms, int* tile_m, int* tile_n,
                            int* split) {
  if (sms == 0) {
    fp4q_status st = current_sms(&sms);
    if (st != FP4Q_OK) return st;
  }
  GemmFp8Args g = {};
  g.M = M;
  g.N = N;
  g.kb = static_cast<int>((K + kFp8Block - 1) / kFp8Block);
  const Choice c = choose(scale_format, g, sms);
  *tile_m = c.v->tile_m;
  *tile_n = c.v->tile_n;
  *split = c.split;
  return FP4Q_OK;
}

fp4q_status launch_gemm_fp8(int scale_format, int out_dtype, const void* a_codes, const void* a_scales,
                            const void* b_codes, const void* b_scales, int64_t M, int64_t N, int64_t K, void* d,
                            cudaStream_t stream) {
  GemmFp8Args g = {};
  g.a_scales = a_scales;
  g.b_scales = b_scales;
  g.d = d;
  g.M = M;
  g.N = N;
  g.kb = static_cast<int>((K + kFp8Block - 1) / kFp8Block);
  const int64_t esize = out_dtype == FP4Q_DTYPE_F32 ? 4 : 2;
  const uintptr_t at = reinterpret_cast<uintptr_t>(d);
  g.vec = (at % 32 == 0 && N * esize % 32 == 0) ? 2 : (N * esize % 16 == 0) ? 1 : 0;   // d itself: 16 bytes
  g.sf_vec = g.kb % 4 == 0 && reinterpret_cast<uintptr_t>(a_scales) % 4 == 0 &&
             reinterpret_cast<uintptr_t>(b_scales) % 4 == 0;
  const Problem p{a_codes, b_codes, g, K, stream};
  switch (out_dtype) {
    case FP4Q_DTYPE_BF16: return dispatch_sf<kDtBf16>(scale_format, p);
    case FP4Q_DTYPE_FP16: return dispatch_sf<kDtFp16>(scale_format, p);
    default: return dispatch_sf<kDtF32>(scale_format, p);
  }
}

}  // namespace host
}  // namespace fp4q

FP4Q_DEFINE_STATUS_READER(status_gemm_fp8)
