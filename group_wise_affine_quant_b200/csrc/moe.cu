// moe.cu — workspace and launch of the mixture-of-experts layer; the kernel
// and its formats are in moe_kernel.cuh and moe_*.cu.
#include "moe_kernel.cuh"

namespace aq {
namespace {

__device__ unsigned int g_moe_device_error = 0u;

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// Per device: its SMs and the address of its error word.
struct Device {
  std::atomic<int> sms{0};
  std::atomic<unsigned*> error{nullptr};
};
Device g_devices[64];

cudaError_t device_of(int* sms, unsigned** error) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*sms = g_devices[dev].sms.load(std::memory_order_acquire)) > 0) {
    *error = g_devices[dev].error.load(std::memory_order_relaxed);
    return cudaSuccess;
  }
  void* p = nullptr;
  e = cudaGetSymbolAddress(&p, g_moe_device_error);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  *error = static_cast<unsigned*>(p);
  if (dev < 64) {
    g_devices[dev].error.store(*error, std::memory_order_relaxed);
    g_devices[dev].sms.store(*sms, std::memory_order_release);
  }
  return cudaSuccess;
}

}  // namespace

// The counter area that every entry point shares, the logits, h (two bf16
// per element) and the fp32 results of each pair.
size_t moe_workspace(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
  return (size_t)moe::kCounterBytes + up256((size_t)(T * E) * 8) +
         up256((size_t)(T * top_k * I) * 4) + up256((size_t)(T * top_k * H) * 4);
}

cudaError_t launch_moe(const MoeArgs& a, int bits, int mode, int dtype, cudaStream_t st) {
  moe::Params p{};
  int sms = 0;
  cudaError_t e = device_of(&sms, &p.error);
  if (e != cudaSuccess) return e;
  p.wait_ns = testing_wait_ns();
  p.delay_ns = testing_delay_ns();
  const int64_t pairs = (int64_t)a.T * a.top_k;
  p.a = a;
  p.bars = reinterpret_cast<unsigned*>(a.workspace);
  uint8_t* at = a.workspace + moe::kCounterBytes;
  p.logits = reinterpret_cast<double*>(at);
  at += up256((size_t)a.T * a.E * 8);
  p.h = at;
  at += up256((size_t)(pairs * a.I) * 4);
  p.part = reinterpret_cast<float*>(at);
  if (mode == AQ_MODE_FP4) return moe::launch_fp4(p, sms, dtype, st);
  switch (bits) {
    case 2: return moe::launch_bits2(p, sms, dtype, st);
    case 3: return moe::launch_bits3(p, sms, dtype, st);
    case 4: return moe::launch_bits4(p, sms, dtype, st);
    case 5: return moe::launch_bits5(p, sms, dtype, st);
    case 6: return moe::launch_bits6(p, sms, dtype, st);
    case 8: return moe::launch_bits8(p, sms, dtype, st);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t read_device_error_moe(unsigned* out) {
  return cudaMemcpyFromSymbol(out, g_moe_device_error, sizeof(unsigned));
}
cudaError_t testing_clear_device_error_moe() {
  const unsigned z = 0;
  return cudaMemcpyToSymbol(g_moe_device_error, &z, sizeof(z));
}

}  // namespace aq
