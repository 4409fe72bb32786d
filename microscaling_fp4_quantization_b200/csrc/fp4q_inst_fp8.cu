// 8-bit quantizer and RMS norm (fp4q_fp8.cuh): their launchers.  One kernel family per
// translation unit, so that the library's kernels compile in parallel (see fp4q_host.cuh).
#include "fp4q_fp8.cuh"

#include "fp4q_host.cuh"

namespace fp4q {
namespace host {

namespace {

FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((uint64_t(1) << l) < d) ++l;
  const uint64_t p = uint64_t(1) << (31 + l);
  return FastDiv{d, static_cast<uint32_t>((p + d - 1) / d), 31 + l};
}

// f.template operator()<DT, SF>() for an input type and a scale format (validated by the caller).
template <class F>
fp4q_status with_types(int dtype, int scale_format, F&& f) {
  if (dtype == FP4Q_DTYPE_BF16)
    return scale_format == FP4Q_FP8_SCALE_F32 ? f.template operator()<kDtBf16, kSfF32>()
                                              : f.template operator()<kDtBf16, kSfE8m0>();
  return scale_format == FP4Q_FP8_SCALE_F32 ? f.template operator()<kDtFp16, kSfF32>()
                                            : f.template operator()<kDtFp16, kSfE8m0>();
}

}  // namespace

fp4q_status launch_quantize_fp8(int scale_format, int dtype, int block_rows, const void* x, int64_t ldx, int64_t M,
                                int64_t K, void* codes, void* scales, cudaStream_t stream) {
  Fp8QuantArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx, a.M = M, a.K = K;
  a.kb = fast_div(static_cast<uint32_t>((K + kFp8Block - 1) / kFp8Block));
  a.n_blocks = static_cast<uint32_t>((M + block_rows - 1) / block_rows * a.kb.d);
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  return with_types(dtype, scale_format, [&]<int DT, int SF>() -> fp4q_status {
    cudaError_t e;
    if (block_rows == 1) {
      constexpr uint32_t per_cta = kFp8QuantThreads / kFp8Lanes;   // blocks
      e = launch_pdl(quantize_fp8_rows_kernel<DT, SF>, dim3((a.n_blocks + per_cta - 1) / per_cta),
                     dim3(kFp8QuantThreads), 0, stream, a);
    } else {
      e = launch_pdl(quantize_fp8_tiles_kernel<DT, SF>, dim3(a.n_blocks), dim3(kFp8QuantThreads), 0, stream, a);
    }
    if (e != cudaSuccess) return cuda_fail(e, "quantize_fp8 launch");
    return FP4Q_OK;
  });
}

fp4q_status launch_add_rmsnorm_fp8(int scale_format, int dtype, const void* x, int64_t ldx, const void* residual,
                                   int64_t ldr, const void* weight, float eps, int64_t M, int64_t K,
                                   void* residual_out, int64_t ldo, void* codes, void* scales, cudaStream_t stream) {
  Fp8NormArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.weight = static_cast<const uint16_t*>(weight);
  a.residual_out = static_cast<uint16_t*>(residual_out);
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.ldx = ldx, a.ldr = ldr, a.ldo = ldo, a.M = M;
  a.K = static_cast<int>(K);
  a.kb = static_cast<int>((K + kFp8Block - 1) / kFp8Block);
  a.eps = eps;
  const int chunks = static_cast<int>(K / kFp8Chunk);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
  const int per_thread = M <= sms && chunks <= kFp8NormThreads ? 1 : 2;   // both are timed beside the kernel
  auto launch = [&]<int DT, int SF, int C, bool RES>() -> fp4q_status {
    auto kernel = add_rmsnorm_fp8_kernel<DT, SF, C, RES>;
    const int threads = ((chunks + C - 1) / C + 31) / 32 * 32;
    KernelInfo ki;
    fp4q_status st = kernel_info(kernel, 0, threads, &ki, 0, -1);
    if (st != FP4Q_OK) return st;
    int64_t ctas = 2 * static_cast<int64_t>(ki.sm_count) * ki.ctas_per_sm;   // two waves: their ends overlap
    if (ctas > M) ctas = M;
    cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(threads), 0, stream, a);
    if (e != cudaSuccess) return cuda_fail(e, "add_rmsnorm_fp8 launch");
    return FP4Q_OK;
  };
  return with_types(dtype, scale_format, [&]<int DT, int SF>() -> fp4q_status {
    if (residual)
      return per_thread == 1 ? launch.template operator()<DT, SF, 1, true>()
                             : launch.template operator()<DT, SF, 2, true>();
    return per_thread == 1 ? launch.template operator()<DT, SF, 1, false>()
                           : launch.template operator()<DT, SF, 2, false>();
  });
}

}  // namespace host
}  // namespace fp4q
