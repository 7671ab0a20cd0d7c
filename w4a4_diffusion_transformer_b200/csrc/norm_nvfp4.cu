// The normalising kernel (norm_quant.cuh) for NVFP4 codes.
#include "norm_quant.cuh"

namespace svdq {

cudaError_t launch_norm_nvfp4(NormParams& p, int num_sms, cudaStream_t stream) {
  if (p.nmt == 0) return launch_plain<kFmtNvfp4>(p, num_sms, stream);
  if (p.nmt == 2) return launch_project<kFmtNvfp4, 2>(p, num_sms, stream);
  if (p.nmt == 4) return launch_project<kFmtNvfp4, 4>(p, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace svdq
