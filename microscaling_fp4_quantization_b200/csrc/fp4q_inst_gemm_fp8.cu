// 8-bit GEMM (fp4q_gemm_fp8.cuh): its launcher.  One kernel family per translation unit, so that
// the library's kernels compile in parallel (see fp4q_host.cuh).
#include "fp4q_gemm_fp8.cuh"

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

template <class Cfg>
fp4q_status launch_many(const void* a_codes, const void* b_codes, GemmFp8Args g, int64_t K, cudaStream_t stream) {
  CUtensorMap amap, bmap;
  fp4q_status st = codes_map(&amap, a_codes, g.M, K, Cfg::kBM);
  if (st == FP4Q_OK) st = codes_map(&bmap, b_codes, g.N, K, Cfg::kBN);
  if (st != FP4Q_OK) return st;
  g.tiles_m = static_cast<int>((g.M + Cfg::kBM - 1) / Cfg::kBM);
  g.tiles_n = static_cast<int>((g.N + Cfg::kBN - 1) / Cfg::kBN);
  auto kernel = gemm_fp8_kernel<Cfg>;
  KernelInfo ki;
  st = kernel_info(kernel, Cfg::kSmemBytes, Cfg::kThreads, &ki);
  if (st != FP4Q_OK) return st;
  int64_t ctas = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
  if (ctas > ki.sm_count) ctas = ki.sm_count;
  cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(Cfg::kThreads), Cfg::kSmemBytes, stream,
                             amap, bmap, g);
  if (e != cudaSuccess) return cuda_fail(e, "gemm_fp8 launch");
  return FP4Q_OK;
}

template <class Cfg>
fp4q_status launch_few(const void* a_codes, const void* b_codes, GemmFp8Args g, int64_t K, cudaStream_t stream) {
  CUtensorMap wmap, xmap;
  fp4q_status st = codes_map(&wmap, b_codes, g.N, K, 128);
  if (st == FP4Q_OK) st = codes_map(&xmap, a_codes, g.M, K, Cfg::kBT);
  if (st != FP4Q_OK) return st;
  g.tiles_m = static_cast<int>((g.M + Cfg::kBT - 1) / Cfg::kBT);
  g.tiles_n = static_cast<int>((g.N + 127) / 128);
  auto kernel = gemm_fp8_few_kernel<Cfg>;
  KernelInfo ki;
  st = kernel_info(kernel, Cfg::kSmemBytes, Cfg::kThreads, &ki);
  if (st != FP4Q_OK) return st;
  // split K over a cluster as long as all CTAs stay resident together (two on an SM)
  const int64_t tiles = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
  int split = 1;
  while (split < 8 && 2 * split <= g.kb && tiles * 2 * split <= 2 * static_cast<int64_t>(ki.sm_count)) split *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * split));
  cfg.blockDim = dim3(Cfg::kThreads);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, wmap, xmap, g, split);
  if (e != cudaSuccess) return cuda_fail(e, "gemm_fp8 launch");
  return FP4Q_OK;
}

template <int OT, int SF>
fp4q_status dispatch(const void* a_codes, const void* b_codes, const GemmFp8Args& g, int64_t K, cudaStream_t stream) {
  if (g.M <= 16) return launch_few<GemmFp8FewConfig<16, OT, SF>>(a_codes, b_codes, g, K, stream);
  if (g.M <= 32) return launch_few<GemmFp8FewConfig<32, OT, SF>>(a_codes, b_codes, g, K, stream);
  if (g.M <= 64) return launch_few<GemmFp8FewConfig<64, OT, SF>>(a_codes, b_codes, g, K, stream);
  const int64_t tiles256 = (g.M + 127) / 128 * ((g.N + 255) / 256);
  if (tiles256 < 148) return launch_many<GemmFp8Config<128, OT, SF>>(a_codes, b_codes, g, K, stream);
  return launch_many<GemmFp8Config<256, OT, SF>>(a_codes, b_codes, g, K, stream);
}

template <int OT>
fp4q_status dispatch_sf(int scale_format, const void* a_codes, const void* b_codes, const GemmFp8Args& g, int64_t K,
                        cudaStream_t stream) {
  return scale_format == FP4Q_FP8_SCALE_F32 ? dispatch<OT, kSfF32>(a_codes, b_codes, g, K, stream)
                                            : dispatch<OT, kSfE8m0>(a_codes, b_codes, g, K, stream);
}

}  // namespace

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
  switch (out_dtype) {
    case FP4Q_DTYPE_BF16: return dispatch_sf<kDtBf16>(scale_format, a_codes, b_codes, g, K, stream);
    case FP4Q_DTYPE_FP16: return dispatch_sf<kDtFp16>(scale_format, a_codes, b_codes, g, K, stream);
    default: return dispatch_sf<kDtF32>(scale_format, a_codes, b_codes, g, K, stream);
  }
}

}  // namespace host
}  // namespace fp4q

FP4Q_DEFINE_STATUS_READER(status_gemm_fp8)
