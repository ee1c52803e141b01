// moe_fp4.cu — the mixture-of-experts kernels for FP4 experts.
#include "moe_kernel.cuh"

namespace aq {
namespace moe {
cudaError_t launch_fp4(const Params& p, int sms, int dtype, cudaStream_t st) {
  return p.a.gs == 16 ? launch_gs<4, true, 16>(p, sms, dtype, st)
                      : launch_gs<4, true, 32>(p, sms, dtype, st);
}
}  // namespace moe
}  // namespace aq
