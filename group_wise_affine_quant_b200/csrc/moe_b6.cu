// moe_b6.cu — the mixture-of-experts kernels for 6-bit affine experts.
#include "moe_kernel.cuh"

namespace aq {
namespace moe {
cudaError_t launch_bits6(const Params& p, int sms, int dtype, cudaStream_t st) {
  return launch_affine<6>(p, sms, dtype, st);
}
}  // namespace moe
}  // namespace aq
