// moe_b2.cu — the mixture-of-experts kernels for 2-bit affine experts.
#include "moe_kernel.cuh"

namespace aq {
namespace moe {
cudaError_t launch_bits2(const Params& p, int sms, int dtype, cudaStream_t st) {
  return launch_affine<2>(p, sms, dtype, st);
}
}  // namespace moe
}  // namespace aq
