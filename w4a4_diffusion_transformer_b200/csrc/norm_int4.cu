// The normalising kernel (norm_quant.cuh) for INT4 codes.
#include "norm_quant.cuh"

namespace svdq {

cudaError_t launch_norm_int4(NormParams& p, int num_sms, cudaStream_t stream) {
  if (p.nmt == 0) return launch_plain<kFmtInt4>(p, num_sms, stream);
  if (p.nmt == 2) return launch_project<kFmtInt4, 2>(p, num_sms, stream);
  if (p.nmt == 4) return launch_project<kFmtInt4, 4>(p, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace svdq
