// moe_b8.cu — the mixture-of-experts kernels for 8-bit affine experts.
#include "moe_kernel.cuh"

namespace aq {
namespace moe {
cudaError_t launch_bits8(const Params& p, int sms, int dtype, cudaStream_t st) {
  return launch_affine<8>(p, sms, dtype, st);
}
}  // namespace moe
}  // namespace aq
