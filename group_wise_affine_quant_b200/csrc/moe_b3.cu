// moe_b3.cu — the mixture-of-experts kernels for 3-bit affine experts.
#include "moe_kernel.cuh"

namespace aq {
namespace moe {
cudaError_t launch_bits3(const Params& p, int sms, int dtype, cudaStream_t st) {
  return launch_affine<3>(p, sms, dtype, st);
}
}  // namespace moe
}  // namespace aq
