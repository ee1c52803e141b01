// moe_b5.cu — the mixture-of-experts kernels for 5-bit affine experts.
#include "moe_kernel.cuh"

namespace aq {
namespace moe {
cudaError_t launch_bits5(const Params& p, int sms, int dtype, cudaStream_t st) {
  return launch_affine<5>(p, sms, dtype, st);
}
}  // namespace moe
}  // namespace aq
