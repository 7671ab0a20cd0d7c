// The normalising kernel (norm_quant.cuh) for INT8 codes.
#include "norm_quant.cuh"

namespace svdq {

cudaError_t launch_norm_int8(NormParams& p, int num_sms, cudaStream_t stream) {
  if (p.nmt == 0) return launch_plain<kFmtInt8>(p, num_sms, stream);
  if (p.nmt == 1) return launch_project<kFmtInt8, 1>(p, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace svdq
