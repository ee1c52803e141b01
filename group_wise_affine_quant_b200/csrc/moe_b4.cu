// moe_b4.cu — the mixture-of-experts kernels for 4-bit affine experts.
#include "moe_kernel.cuh"

namespace aq {
namespace moe {
cudaError_t launch_bits4(const Params& p, int sms, int dtype, cudaStream_t st) {
  return launch_affine<4>(p, sms, dtype, st);
}
}  // namespace moe
}  // namespace aq
