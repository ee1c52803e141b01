// int8.cu — W8A8: the symmetric row quantizer and the 8-bit integer matrix
// product with one scale per token and one per channel.
//
// Quantizer: a = max |x| over the row, s = a / 127, q = rint(x / s), both
// divisions and the rounding as fp32 IEEE operations (bit-exact codes).  A
// row with a NaN has s = NaN, one with an infinity s = inf, and codes 0, so
// that the products of such a row show it (NaN).  The row stays in registers
// between the two passes up to K = 16384 (longer rows are read twice, the
// second time from L2): 2 bytes in and 1 out per element.  The maximum is
// taken on the 16-bit patterns without their sign (NaN > inf > finite).  What
// bounds it is HBM: 8192 x 4096 bf16 19.2 us, 5.2 TB/s.
//
// Product: y[m, n] = T(((float)sum_k x_q w_q * s_x[m]) * s_w[n]).  The sum is
// exact in 32-bit integers (K is limited so that it cannot overflow),
// whatever the split; the conversion to fp32 rounds by at most 2^-24.  Tensor
// cores bound large products (8192 x 8192 x 2048 93 us, 3.0 POP/s; 107 us in a
// loop under the power cap), a tile's start and end small ones (1 x 2048 x 2048
// 4.1 us, from HBM 4.5).
#include <atomic>
#include <cooperative_groups.h>

#include "common.cuh"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace aq {
namespace {

using namespace sm100;

__device__ unsigned int g_int8_device_error = 0u;

// ---------------------------------------------------------------- quantizer
// 16 elements (two 16-byte vectors) of a row.
struct Vec16 {
  uint4 a, b;
};

__device__ __forceinline__ uint32_t abs_max2(const Vec16& v) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t p = __vmaxu2(__vmaxu2(v.a.x & m, v.a.y & m), __vmaxu2(v.a.z & m, v.a.w & m));
  const uint32_t q = __vmaxu2(__vmaxu2(v.b.x & m, v.b.y & m), __vmaxu2(v.b.z & m, v.b.w & m));
  return __vmaxu2(p, q);
}
__device__ __forceinline__ uint32_t max_half(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t v);
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <typename T> __device__ __forceinline__ float from_bits(uint32_t b) {
  return unpack2<T>(b).x;
}

// Adding 1.5 * 2^23 rounds to the nearest integer, ties to even, and leaves
// its two's complement in the low bits (|v| < 2^22).
constexpr float kRoundMagic = 12582912.0f;

struct RowScale {
  float s, inv;
  int how;               // 0: codes 0, 1: product with 1/s, 2: division (1/s may overflow)
};
__device__ __forceinline__ RowScale row_scale(float amax) {
  RowScale r;
  if (amax > 1e-28f && amax <= 3.4e38f) {
    // amax / 127, correctly rounded: the rounded reciprocal's quotient corrected
    // by its exact remainder (as for the codes below)
    const float y = 1.0f / 127.0f, q = __fmul_rn(amax, y);
    r.s = __fmaf_rn(__fmaf_rn(q, -127.0f, amax), y, q);
    r.how = 1;
    r.inv = __frcp_rn(r.s);
  } else {
    r.s = __fdiv_rn(amax, 127.0f);
    r.how = r.s > 0.0f && r.s <= 3.4e38f ? 2 : 0;          // 0 for zero, inf and NaN
    r.inv = 0.0f;
  }
  return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  return (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// The codes of two elements in the low bytes of two words: a quotient from the
// rounded reciprocal, corrected by its exact remainder (Markstein 1990: the
// result is the correctly rounded x / s).
__device__ __forceinline__ uint32_t codes2(float2 x, const RowScale& r) {
  uint64_t q;
  if (r.how == 2) {
    q = pack2(__fdiv_rn(x.x, r.s), __fdiv_rn(x.y, r.s));
  } else {
    const uint64_t v = pack2(x.x, x.y), inv = pack2(r.inv, r.inv);
    q = mul2(v, inv);
    q = fma2(fma2(q, pack2(-r.s, -r.s), v), inv, q);
  }
  q = add2(q, pack2(kRoundMagic, kRoundMagic));
  return __byte_perm((uint32_t)q, (uint32_t)(q >> 32), 0x0040);
}
template <typename T>
__device__ __forceinline__ uint32_t codes4(uint32_t lo, uint32_t hi, const RowScale& r) {
  return __byte_perm(codes2(unpack2<T>(lo), r), codes2(unpack2<T>(hi), r), 0x5410);
}
template <typename T>
__device__ __forceinline__ uint4 codes16(const Vec16& v, const RowScale& r) {
  if (r.how == 0) return make_uint4(0u, 0u, 0u, 0u);
  return make_uint4(codes4<T>(v.a.x, v.a.y, r), codes4<T>(v.a.z, v.a.w, r),
                    codes4<T>(v.b.x, v.b.y, r), codes4<T>(v.b.z, v.b.w, r));
}
__device__ __forceinline__ Vec16 load16(const uint4* row, int64_t i) {
  Vec16 v;
  v.a = __ldg(row + 2 * i);
  v.b = __ldg(row + 2 * i + 1);
  return v;
}

// WARPS warps per row (16 elements a thread keep most threads in flight: a warp
// for rows of 2048 took 19.2 us for 8192 of them, four warps 11.4), V vectors
// per thread; V = 0 reads the row twice (K > 16384).
constexpr int kQuantThreads = 256;
template <typename T, int WARPS, int V>
__global__ void __launch_bounds__(kQuantThreads)
quantize_int8_kernel(const uint4* __restrict__ x, uint4* __restrict__ xq, float* __restrict__ scales,
                     int64_t rows, int nvec) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ uint32_t part[kQuantThreads / 32];
  constexpr int kRow = 32 * WARPS;                       // threads of a row
  const int at = threadIdx.x % kRow, team = threadIdx.x / kRow;
  const int64_t row = (int64_t)blockIdx.x * (kQuantThreads / kRow) + team;
  const bool live = row < rows;
  const uint4* src = x + row * nvec * 2;
  Vec16 v[V > 0 ? V : 1];
  uint32_t m = 0u;
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = at + kRow * i;
      if (live && c < nvec) {
        v[i] = load16(src, c);
        m = __vmaxu2(m, abs_max2(v[i]));
      }
    }
  } else {
    for (int c = at; c < nvec; c += kRow) m = __vmaxu2(m, abs_max2(load16(src, c)));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, max_half(m));
  if constexpr (WARPS > 1) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = 0u;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) m = max(m, part[team * WARPS + i]);
  }
  if (!live) return;
  const RowScale r = row_scale(from_bits<T>(m));
  uint4* dst = xq + row * nvec;
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = at + kRow * i;
      if (c < nvec) dst[c] = codes16<T>(v[i], r);
    }
  } else {
    for (int c = at; c < nvec; c += kRow) dst[c] = codes16<T>(load16(src, c), r);
  }
  if (at == 0) scales[row] = r.s;
}

template <typename T>
cudaError_t quantize_rows(const void* x, void* xq, float* scales, int64_t rows, int64_t K,
                          cudaStream_t st) {
  const int nvec = (int)(K / 16);
  const int warps = nvec <= 32 ? 1 : nvec <= 64 ? 2 : nvec <= 128 ? 4 : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows * warps + 7) / 8));
  cfg.blockDim = dim3(kQuantThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = warps == 1   ? quantize_int8_kernel<T, 1, 1>
              : warps == 2 ? quantize_int8_kernel<T, 2, 1>
              : warps == 4 ? quantize_int8_kernel<T, 4, 1>
              : nvec <= kQuantThreads     ? quantize_int8_kernel<T, 8, 1>
              : nvec <= 2 * kQuantThreads ? quantize_int8_kernel<T, 8, 2>
              : nvec <= 4 * kQuantThreads ? quantize_int8_kernel<T, 8, 4>
                                          : quantize_int8_kernel<T, 8, 0>;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const uint4*>(x), static_cast<uint4*>(xq), scales,
                            rows, nvec);
}

// ------------------------------------------------------------------ product
// Both operands are K-major 8-bit tiles of 128 bytes per row (128-byte swizzle)
// that TMA brings into a ring of stages; an elected lane issues tcgen05.mma
// kind::i8 into one of two accumulators in TMEM while the epilogue warps scale and
// store the other.
//   * Few tokens: the weight is the MMA's A operand (128 channels per CTA) and
//     x its B operand (BN tokens), so that a few tokens still fill the MMA.
//     splits > 1 (few tiles): the CTAs of a cluster take slices of K, park their
//     integer tiles in shared memory and add each other's through distributed
//     shared memory, each CTA a share of the columns.
//   * kPair: two CTAs of a cluster share a tile of 256 tokens x BN channels
//     (cta_group::2), tokens as A operand; each loads its 128 tokens and half of
//     the channels.  A 256 x 256 tile then costs each SM 32 KB per 128 of K
//     instead of 48 KB, which is what bounds a single CTA's tile.  A thread
//     holds a token's run of channels, which leaves through shared memory in
//     TMA stores (rows of y of odd length: by the warps).
constexpr int kBK = 128;                 // bytes (elements) of K per stage
constexpr int kBM = 128;                 // rows of the A operand per CTA: channels, kPair: tokens

template <int BN, bool PAIR>
struct MmShape {
  static constexpr int kBRows = PAIR ? BN / 2 : BN;
  static constexpr int kABytes = kBM * kBK;
  static constexpr int kBBytes = kBRows * kBK;
  static constexpr int kStage = kABytes + kBBytes;
  // BN <= 32 streams weights: five stages, so that two CTAs fit on an SM and
  // one's start and end overlap the other's stream.
  static constexpr int kStages = BN <= 32 ? 5 : (192 * 1024) / kStage > 8 ? 8 : PAIR && BN == 256 ? 5 : (192 * 1024) / kStage;
  static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
  static constexpr int kBars = 2 * kStages + 5;
  // A quarter of the accumulator's rows to a warp, kPair: to two warps, half of
  // the columns each (4096 x 4096 x 1024 in tiles of 256 x 128: 21.0 us, with
  // four warps 22.4; in tiles of 256 x 256 18.6 and 18.9).
  static constexpr int kEpilogue = PAIR ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kEpilogue;           // TMA warp, MMA warp, epilogue
  static constexpr int kOut = PAIR ? kEpilogue * 4096 : 0;       // staged rows of y
  static constexpr int kTail = 2 * BN * 4 + kBars * 8 + 16;     // column scales, barriers, slots
  static constexpr int kSmem = 1024 + kStages * kStage + kOut + kTail;
  static_assert(PAIR || kStages * kStage >= BN * kBM * 4, "split-K parking reuses the ring");
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

struct MmArgs {
  const float* xs;
  const float* ws;
  void* y;
  int M, N, K;
  int kblocks;           // ceil(K / 128)
  int splits, kb_split;  // K-slices and 128-blocks per slice
  int m_tiles, n_tiles;
  int prefetch;          // weights may be read before the previous kernel has ended
  int tma_out;           // y's rows suit TMA (N a multiple of 8)
  uint64_t wait_ns;      // bound of every mbarrier wait
  uint64_t delay_ns;     // test hook: TMA warp start delay (0: none)
};

// Sets the flag at this shared-memory offset in another CTA of the cluster.
__device__ __forceinline__ void raise_remote(uint32_t cluster_addr) {
  asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], 1;" ::"r"(cluster_addr) : "memory");
}
constexpr uint64_t kDrainNs = 200000000ull;   // bound of the waits after giving up

__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_i8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Two values rounded to T, a in the low half.
template <typename T> __device__ __forceinline__ uint32_t pack_t(float a, float b);
template <> __device__ __forceinline__ uint32_t pack_t<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <> __device__ __forceinline__ uint32_t pack_t<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Arrive on the barrier at this offset in both CTAs of the pair once the MMAs
// issued so far have completed.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// Tile load whose bytes complete on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t cluster_bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(c0), "r"(c1)
      : "memory");
}
// Tile store from shared memory; its rows outside the map are dropped.
__device__ __forceinline__ void tma_store_2d(uint32_t src, const CUtensorMap* map, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Until the sources of all but this thread's last N store groups are read.
template <int N> __device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// Instruction descriptor, kind::i8: s32 accumulator (bits 4-5 = 2), signed A
// and B (bits 7-9 and 10-12 = 1), both K-major, N >> 3 (17-22), M >> 4 (24-28).
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// Tile t in bands of eight token tiles: the tiles in flight then share both
// operands in L2.
__device__ __forceinline__ void tile_at(int t, int m_tiles, int n_tiles, int& mt, int& nt) {
  const int band = t / (8 * n_tiles);
  const int in = t - band * 8 * n_tiles;
  const int rows = min(8, m_tiles - band * 8);
  nt = in / rows;
  mt = band * 8 + in - nt * rows;
}

template <typename T, int BN, bool PAIR>
__global__ void __launch_bounds__(MmShape<BN, PAIR>::kThreads)
int8_mm_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
               const __grid_constant__ CUtensorMap my, const MmArgs a) {
  using S = MmShape<BN, PAIR>;
  constexpr int ST = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* tail = smem_raw + (base - raw) + ST * S::kStage + S::kOut;
  float* sx = reinterpret_cast<float*>(tail);                         // [2][BN]
  const uint32_t bars = smem_u32(tail + 2 * BN * 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 2 * BN * 4 + S::kBars * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(const_cast<int*>(abort_flag) + 1);
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (ST + s); };
  auto tfull = [&](int b) { return bars + 8u * (2 * ST + b); };
  auto tempty = [&](int b) { return bars + 8u * (2 * ST + 2 + b); };
  const uint32_t drain = bars + 8u * (2 * ST + 4);
  // A role that gives up ends its CTA's waits by the flag, and the other CTA's
  // of a pair by that one's: neither can finish alone.
  auto tell_peer = [&]() {
    if constexpr (PAIR) raise_remote(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), cluster_rank() ^ 1u));
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool clustered = PAIR || a.splits > 1;
  const uint32_t rank = clustered ? cluster_rank() : 0u;
  const bool leader = !PAIR || rank == 0;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < ST; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), PAIR ? 2 * S::kEpilogue : S::kEpilogue);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    prefetch_tensormap(&mw);
    prefetch_tensormap(&mx);
    if (PAIR && a.tma_out) prefetch_tensormap(&my);
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_alloc_pair(smem_u32(tmem_slot), S::kTmemCols);
    else tmem_alloc(smem_u32(tmem_slot), S::kTmemCols);
  }
  tc_fence_before();
  if (PAIR) {
    cluster_arrive();
    cluster_wait();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();

  const int group = PAIR ? 2 : a.splits;                 // CTAs per tile
  const int first = (int)blockIdx.x / group, step = (int)gridDim.x / group;
  const int tiles = a.m_tiles * a.n_tiles;
  const int kb0 = PAIR ? 0 : (int)rank * a.kb_split;
  const int nkb = PAIR ? a.kblocks : min(a.kb_split, a.kblocks - kb0);   // > 0 by the plan
  constexpr int kRowsA = PAIR ? 2 * kBM : kBM;           // rows of the A operand per tile
  uint32_t issued = 0;                                   // stages the TMA warp has asked for

  if (warp == 0) {
    // ------------------------------------------------------------- TMA warp
    uint32_t it = 0;                                     // stages used so far
    bool ok = true;
    int pre = 0;                                         // stages whose weights are under way
    auto load_w = [&](int s, int nt, int kb) {
      const uint32_t dst = base + s * S::kStage;
      if constexpr (PAIR)
        tma_load_2d_pair(dst + S::kABytes, &mw, mapa_shared(full(s), 0), kb * kBK,
                         nt * BN + (int)rank * S::kBRows);
      else tma_load_2d(dst, &mw, full(s), kb * kBK, nt * kBM);
    };
    auto load_x = [&](int s, int mt, int kb) {
      const uint32_t dst = base + s * S::kStage;
      if constexpr (PAIR)
        tma_load_2d_pair(dst, &mx, mapa_shared(full(s), 0), kb * kBK, mt * kRowsA + (int)rank * kBM);
      else tma_load_2d(dst + S::kABytes, &mx, full(s), kb * kBK, mt * BN);
    };
    const uint32_t bytes = (PAIR ? 2u : 1u) * S::kStage;
    if (a.prefetch && first < tiles) {
      int mt, nt;
      tile_at(first, a.m_tiles, a.n_tiles, mt, nt);
      pre = min(ST, nkb);
      if (elect_one()) {
        for (int s = 0; s < pre; ++s) {
          if (leader) mbar_arrive_expect_tx(full(s), bytes);
          load_w(s, nt, kb0 + s);
        }
      }
      __syncwarp();
    }
    pdl_wait();
    if (a.delay_ns) {                                    // test hook
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < a.delay_ns && !*abort_flag) {
      }
      __syncwarp();
    }
    for (int t = first; t < tiles && ok; t += step) {
      int mt, nt;
      tile_at(t, a.m_tiles, a.n_tiles, mt, nt);
      for (int k = 0; k < nkb; ++k, ++it) {
        const int s = (int)(it % ST);
        const bool early = it < (uint32_t)pre;
        if (!mbar_wait(empty(s), ((it / ST) & 1u) ^ 1u, abort_flag, a.wait_ns)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          if (!early) {
            if (leader) mbar_arrive_expect_tx(full(s), bytes);
            load_w(s, nt, kb0 + k);
          }
          load_x(s, mt, kb0 + k);
        }
        __syncwarp();
      }
    }
    issued = it;
    if (!ok) tell_peer();
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA warp
    if (leader) {
      constexpr uint32_t idesc = idesc_i8(kRowsA, BN);
      uint32_t it = 0, tile_i = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step, ++tile_i) {
        const int b = (int)(tile_i & 1u);
        const uint32_t use = tile_i >> 1;
        ok = PAIR ? mbar_wait_cluster(tempty(b), (use & 1u) ^ 1u, abort_flag, a.wait_ns)
                  : mbar_wait(tempty(b), (use & 1u) ^ 1u, abort_flag, a.wait_ns);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(b * BN);
        for (int k = 0; k < nkb; ++k, ++it) {
          const int s = (int)(it % ST);
          if (!mbar_wait(full(s), (it / ST) & 1u, abort_flag, a.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t da = sdesc_sw128(base + s * S::kStage);
            const uint64_t db = sdesc_sw128(base + s * S::kStage + S::kABytes);
            const int left = a.K - (kb0 + k) * kBK;      // K elements of this stage
#pragma unroll
            for (int q = 0; q < kBK / 32; ++q) {
              if (q * 32 < left) {
                const uint32_t acc = (k | q) ? 1u : 0u;
                if constexpr (PAIR) mma_i8_pair(d, da + 2 * q, db + 2 * q, idesc, acc);
                else mma_i8(d, da + 2 * q, db + 2 * q, idesc, acc);
              }
            }
            if constexpr (PAIR) mma_commit_pair(empty(s));
            else mma_commit(empty(s));
            if (k == nkb - 1) {
              if constexpr (PAIR) mma_commit_pair(tfull(b));
              else mma_commit(tfull(b));
            }
          }
          __syncwarp();
        }
      }
      if (!ok) {
        // Gave up: the MMAs issued end before the TMEM is freed.
        tell_peer();
        int ignore = 0;
        if (elect_one()) {
          if constexpr (PAIR) mma_commit_pair(drain);
          else mma_commit(drain);
        }
        __syncwarp();
        mbar_wait(drain, 0, &ignore, kDrainNs);
      }
    }
  } else {
    // ------------------------------------------------------- epilogue warps
    pdl_wait();
    const int q = warp & 3;                              // TMEM lane quarter
    constexpr int kEt = 32 * S::kEpilogue;
    const int et = (int)threadIdx.x - 64;                // 0..kEt - 1
    T* y = static_cast<T*>(a.y);
    uint32_t tile_i = 0;
    bool ok = true;
    // The scales of a tile's columns and of the thread's row are asked for a
    // tile ahead.
    float column = 0.0f, row = 0.0f;
    auto ask = [&](int t) {
      if (t >= tiles) return;
      int mt, nt;
      tile_at(t, a.m_tiles, a.n_tiles, mt, nt);
      if constexpr (PAIR) {
        const int m = mt * kRowsA + (int)rank * kBM + q * 32 + lane;
        column = et < BN && nt * BN + et < a.N ? a.ws[nt * BN + et] : 0.0f;
        row = m < a.M ? a.xs[m] : 0.0f;
      } else {
        const int n = nt * kBM + q * 32 + lane;
        column = et < BN && mt * BN + et < a.M ? a.xs[mt * BN + et] : 0.0f;
        row = n < a.N ? a.ws[n] : 0.0f;
      }
    };
    static_assert(BN <= kEt, "a column to a thread");
    ask(first);
    for (int t = first; t < tiles; t += step, ++tile_i) {
      int mt, nt;
      tile_at(t, a.m_tiles, a.n_tiles, mt, nt);
      const int b = (int)(tile_i & 1u);
      float* sxb = sx + b * BN;                          // scales of the columns
      if (et < BN) sxb[et] = column;
      const float s_row = row;
      named_barrier_sync(1, kEt);
      ask(t + step);
      // after giving up the warps still meet at the barrier above
      if (ok) ok = mbar_wait(tfull(b), (tile_i >> 1) & 1u, abort_flag, a.wait_ns);
      if (!ok) continue;
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * BN);
      if constexpr (PAIR) {
        const int row0 = mt * kRowsA + (int)rank * kBM + q * 32;   // the warp's tokens
        uint8_t* out = smem_raw + (base - raw) + ST * S::kStage + (warp - 2) * 4096;
        const int end = (warp - 2) / 4 * (BN / 2) + BN / 2;
#pragma unroll 1
        for (int c0 = end - BN / 2; c0 < end; c0 += 64) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[32];
            tmem_ld_32(d + c0 + 32 * h, r);
            float4 sc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) sc[i] = *reinterpret_cast<const float4*>(sxb + c0 + 32 * h + 4 * i);
            tmem_ld_wait();
            auto v = [&](int c, float w) { return __fmul_rn(__fmul_rn(__int2float_rn((int)r[c]), s_row), w); };
            uint4 o[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float4 a0 = sc[2 * u], a1 = sc[2 * u + 1];
              o[u] = make_uint4(pack_t<T>(v(8 * u, a0.x), v(8 * u + 1, a0.y)),
                                pack_t<T>(v(8 * u + 2, a0.z), v(8 * u + 3, a0.w)),
                                pack_t<T>(v(8 * u + 4, a1.x), v(8 * u + 5, a1.y)),
                                pack_t<T>(v(8 * u + 6, a1.z), v(8 * u + 7, a1.w)));
            }
            if (h == 0) {
              if (lane == 0) bulk_wait_read<0>();        // the last store has left
              __syncwarp();
            }
            // 128-byte rows, 16-byte units swizzled by the row
#pragma unroll
            for (int u = 0; u < 4; ++u)
              *reinterpret_cast<uint4*>(out + lane * 128 + (((4 * h + u) ^ (lane & 7)) * 16)) = o[u];
          }
          if (c0 + 64 >= end) {                          // the accumulator is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(mapa_shared(tempty(b), 0));
          }
          const int n0 = nt * BN + c0;
          if (a.tma_out) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (row0 < a.M && n0 < a.N) tma_store_2d(smem_u32(out), &my, n0, row0);
              bulk_commit();
            }
          } else {
            __syncwarp();
            const int rows = min(32, a.M - row0), cols = min(64, a.N - n0);
            T* to = y + (int64_t)row0 * a.N + n0;
            // (eight reads before their stores, which the compiler takes for
            // ones that might change what is read)
            if (a.N % 4 == 0) {
              // rows start at a multiple of 8 bytes: two at a time
              const int c = lane & 15;
#pragma unroll
              for (int i = 0; i < 16; i += 8) {
                uint2 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const int r = 2 * (i + k) + (lane >> 4);
                  v[k] = *reinterpret_cast<const uint2*>(out + r * 128 + (((c >> 1) ^ (r & 7)) * 16) + (c & 1) * 8);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const int r = 2 * (i + k) + (lane >> 4);
                  if (r < rows && 4 * c < cols) *reinterpret_cast<uint2*>(to + (int64_t)r * a.N + 4 * c) = v[k];
                }
              }
            } else {
              // pairs from the row's first multiple of 4 bytes on, and what is
              // left at its ends
              auto at = [&](int r, int c) {
                return *reinterpret_cast<const uint16_t*>(out + r * 128 + (((c >> 3) ^ (r & 7)) * 16) + (c & 7) * 2);
              };
              uint16_t* row = reinterpret_cast<uint16_t*>(to);
#pragma unroll 1
              for (int r = 0; r < rows; r += 8) {
                uint32_t v[8], first[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const int odd = (int)(((row0 + k) & a.N) & 1);       // n0 and r are even
                  const int c = 2 * lane + odd;
                  v[k] = at(r + k, c) | (uint32_t)at(r + k, (c + 1) & 63) << 16;
                  first[k] = at(r + k, 0);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const int odd = (int)(((row0 + k) & a.N) & 1), c = 2 * lane + odd;
                  if (r + k < rows) {
                    if (c + 1 < cols) *reinterpret_cast<uint32_t*>(row + c) = v[k];
                    else if (c < cols) row[c] = (uint16_t)v[k];
                    if (odd && lane == 0 && cols > 0) row[0] = (uint16_t)first[k];
                  }
                  row += a.N;
                }
              }
            }
          }
        }
      } else {
        const int m0 = mt * BN;
        const int n = nt * kBM + q * 32 + lane;
        constexpr int kCols = BN < 32 ? BN : 32;
#pragma unroll 1
        for (int c0 = 0; c0 < BN; c0 += kCols) {
          uint32_t r[kCols];
          if constexpr (kCols == 32) tmem_ld_32(d + c0, r);
          else tmem_ld_16(d + c0, r);
          if (a.splits == 1) {
            // all scales before the first store, which the compiler takes for
            // one that might change them
            float4 sc[kCols / 4];
#pragma unroll
            for (int i = 0; i < kCols / 4; ++i) sc[i] = *reinterpret_cast<const float4*>(sxb + c0 + 4 * i);
            tmem_ld_wait();
            if (n < a.N) {
              T* out = y + (int64_t)(m0 + c0) * a.N + n;
              const int cols = min(kCols, a.M - m0 - c0);
#pragma unroll
              for (int c = 0; c < kCols; ++c) {
                const float4 v = sc[c / 4];
                const float s = c % 4 == 0 ? v.x : c % 4 == 1 ? v.y : c % 4 == 2 ? v.z : v.w;
                if (c < cols)
                  out[(int64_t)c * a.N] = TT<T>::from_f(__fmul_rn(__fmul_rn(__int2float_rn((int)r[c]), s), s_row));
              }
            }
          } else {
            tmem_ld_wait();
            int* park = reinterpret_cast<int*>(smem_raw + (base - raw));
#pragma unroll
            for (int c = 0; c < kCols; ++c) park[(c0 + c) * kBM + q * 32 + lane] = (int)r[c];
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty(b));
      }
    }
    if (!ok) tell_peer();
    if (PAIR && lane == 0) bulk_wait_all();              // y is written, the buffers are free
  }

  if (!PAIR && a.splits > 1) {
    // One tile per cluster: the parked integer tiles of all slices, added by
    // each CTA for its share of the columns.
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (warp >= 2 && *abort_flag == 0) {
      int mt, nt;
      tile_at(first, a.m_tiles, a.n_tiles, mt, nt);
      // a warp per column, four channels to a lane: all slices' loads of a
      // column are under way at once
      int* park = reinterpret_cast<int*>(smem_raw + (base - raw));
      T* y = static_cast<T*>(a.y);
      const int n = nt * kBM + lane * 4;
      float sw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sw[i] = n + i < a.N ? a.ws[n + i] : 0.0f;
      const int per = (BN + a.splits - 1) / a.splits;
      const int m0 = mt * BN;
      const int c_end = min(min((int)(rank + 1) * per, BN), a.M - m0);
      for (int c = (int)rank * per + warp - 2; c < c_end; c += 4) {
        int4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          v[r] = r < a.splits ? *reinterpret_cast<const int4*>(cluster.map_shared_rank(park + c * kBM + lane * 4, r))
                              : make_int4(0, 0, 0, 0);
        int sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          sum[0] += v[r].x;
          sum[1] += v[r].y;
          sum[2] += v[r].z;
          sum[3] += v[r].w;
        }
        T o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = TT<T>::from_f(__fmul_rn(__fmul_rn(__int2float_rn(sum[i]), sx[c]), sw[i]));
        T* out = y + (int64_t)(m0 + c) * a.N + n;
        if (a.N % 4 == 0 && n < a.N) {
          *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(o);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < a.N) out[i] = o[i];
        }
      }
    }
    cluster.sync();
  }
  tc_fence_before();
  if (PAIR) {
    cluster_arrive();
    cluster_wait();
  }
  __syncthreads();
  if (*abort_flag) {
    // Gave up (both CTAs of a pair know by now).  The copies in flight land before
    // a CTA exits, also those that the TMA warp asked for without waiting for
    // anything later.
    if (warp == 0 && leader) {
      int ignore = 0;
      const uint32_t n = issued < (uint32_t)ST ? issued : (uint32_t)ST;
      for (uint32_t j = 0; j < n; ++j) {
        const uint32_t i = issued - 1 - j;
        mbar_wait(full((int)(i % ST)), (i / ST) & 1u, &ignore, kDrainNs);
      }
    } else if (warp == 0) {
      // A stage that the leader did not ask for completes on no barrier: 10 ms
      // are a thousand times as long as a copy takes.
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 10000000ull) {
      }
    }
    if (PAIR) {
      cluster_arrive();
      cluster_wait();
    }
    __syncthreads();
    if (threadIdx.x == 0) atomicOr(&g_int8_device_error, 1u);
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, S::kTmemCols);
    else tmem_dealloc(tmem, S::kTmemCols);
  }
}

// -------------------------------------------------------------------- host
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(p);
    return nullptr;
  }();
  return fn;
}

// Rows of `row` elements, boxes of 128 bytes x box_rows, 128-byte swizzle, zero
// fill.
cudaError_t tile_map(CUtensorMap* map, CUtensorMapDataType type, int size, const void* base,
                     int64_t rows, int64_t row, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {(cuuint64_t)row, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(row * size)};
  cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int BN, bool PAIR>
cudaError_t launch_mm(const Int8Plan& p, const void* x_q, const void* w_q, MmArgs a,
                      cudaStream_t st) {
  using S = MmShape<BN, PAIR>;
  auto kern = int8_mm_kernel<T, BN, PAIR>;
  static std::atomic<bool> attr_done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr_done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done[dev].store(true, std::memory_order_release);
  }
  CUtensorMap mw, mx, my{};
  e = tile_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w_q, a.N, a.K, PAIR ? S::kBRows : kBM);
  if (e == cudaSuccess)
    e = tile_map(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, x_q, a.M, a.K, PAIR ? kBM : BN);
  a.tma_out = PAIR && a.N % 8 == 0;
  if (e == cudaSuccess && a.tma_out)
    e = tile_map(&my, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.y, a.M, a.N, 32);
  if (e != cudaSuccess) return e;
  a.splits = p.splits;
  a.kb_split = p.kb_split;
  a.m_tiles = (a.M + (PAIR ? 2 * kBM : BN) - 1) / (PAIR ? 2 * kBM : BN);
  a.n_tiles = (a.N + (PAIR ? BN : kBM) - 1) / (PAIR ? BN : kBM);
  const int group = PAIR ? 2 : p.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.groups * group), 1, 1);
  cfg.blockDim = dim3(S::kThreads, 1, 1);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)group;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = group > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, mw, mx, my, a);
}

template <typename T>
cudaError_t by_plan(const Int8Plan& p, const void* x_q, const void* w_q, const MmArgs& a,
                    cudaStream_t st) {
  if (p.pair)
    return p.bn == 128 ? launch_mm<T, 128, true>(p, x_q, w_q, a, st)
                       : launch_mm<T, 256, true>(p, x_q, w_q, a, st);
  switch (p.bn) {
    case 16: return launch_mm<T, 16, false>(p, x_q, w_q, a, st);
    case 32: return launch_mm<T, 32, false>(p, x_q, w_q, a, st);
    case 64: return launch_mm<T, 64, false>(p, x_q, w_q, a, st);
    default: return launch_mm<T, 128, false>(p, x_q, w_q, a, st);
  }
}

// Plan forced by a test: Int8Plan's bn (0: automatic), pair, K-slices.
std::atomic<int> g_force_bn{0}, g_force_pair{0}, g_force_splits{0};

}  // namespace

// Tile and split with the least estimated time, in clocks of one SM, from a fit
// to 16 shapes (1 x 2048 x 2048 to 8192 x 8192 x 2048) of all plans: a
// 128-element block of K costs what its loads take (a few bytes per clock less
// when every SM loads), a CTA of its own what its start and end take, and the
// stores of a tile hide behind the next one's products if those take longer.
// Clusters do not fill the GPU: `slots` is how many run at once.
Int8Plan plan_int8_mm(int64_t M, int64_t N, int64_t K) {
  struct Tile {
    int bn;                              // as in Int8Plan
    bool pair;
    int block, full, start, column;      // clocks: per block, more at full load, start, per column
  };
  static const Tile kTiles[6] = {{16, false, 458, 135, 4366, 130}, {32, false, 462, 160, 4800, 130},
                                 {64, false, 469, 55, 6200, 75},   {128, false, 502, 134, 8700, 75},
                                 {128, true, 389, 65, 6750, 23},   {256, true, 500, 130, 8500, 20}};
  const int ragged = N % 8 == 0 ? 0 : N % 4 == 0 ? 9 : 29;           // rows of y that TMA cannot store
  static const int kSlotsTwo[9] = {0, 296, 148, 93, 71, 56, 45, 37, 33};   // two CTAs on an SM
  static const int kSlotsOne[9] = {0, 148, 74, 45, 33, 26, 22, 15, 15};
  Int8Plan best{};
  double best_cost = 0;
  const int kblocks = (int)((K + kBK - 1) / kBK);
  const int fbn = g_force_bn.load(std::memory_order_relaxed);
  const int fpair = g_force_pair.load(std::memory_order_relaxed);
  const int fsplit = g_force_splits.load(std::memory_order_relaxed);
  for (const Tile& t : kTiles) {
    if (fbn && (t.bn != fbn || t.pair != (fpair != 0))) continue;
    const int64_t tm = t.pair ? 2 * kBM : t.bn, tn = t.pair ? t.bn : kBM;
    const int64_t tiles = ((M + tm - 1) / tm) * ((N + tn - 1) / tn);
    const double columns = t.pair ? (double)t.bn : (double)(M < t.bn ? M : t.bn);
    for (int s = 1; s <= (t.pair ? 1 : 8) && s <= kblocks; ++s) {
      const int slots = t.pair ? 74 : t.bn <= 32 ? kSlotsTwo[s] : kSlotsOne[s];
      if (s > 1 && (fsplit ? s > fsplit : tiles > slots)) break;
      const int kb = (kblocks + s - 1) / s;
      if ((kblocks + kb - 1) / kb != s) continue;        // an empty slice
      const double waves = (double)((tiles + slots - 1) / slots);
      const double load = tiles < slots ? (double)tiles / slots : 1.0;
      const double products = kb * (t.block + t.full * load), stores = (t.column + (t.pair ? ragged : 0)) * columns * load;
      const double cost = waves * (products > stores ? products : stores) +
                          (s > 1 ? 5400.0 + 10.0 * t.bn + 30.0 * columns + 150.0 * s
                                 : t.start + (t.pair ? 0.0 : 25.0 * columns));
      if (best.bn == 0 || cost < best_cost || fsplit) {
        best_cost = cost;
        best.bn = t.bn;
        best.pair = t.pair;
        best.splits = s;
        best.kb_split = kb;
        best.groups = s > 1 || tiles < slots ? tiles : slots;
      }
    }
  }
  return best;
}

cudaError_t launch_quantize_int8(const void* x, void* xq, float* scales, int64_t rows, int64_t K,
                                 int dtype, cudaStream_t st) {
  return dtype == AQ_F16 ? quantize_rows<__half>(x, xq, scales, rows, K, st)
                         : quantize_rows<__nv_bfloat16>(x, xq, scales, rows, K, st);
}

cudaError_t launch_int8_mm(const void* x_q, const float* x_scales, const void* w_q,
                           const float* w_scales, void* y, int64_t M, int64_t N, int64_t K,
                           int dtype, int prefetch, cudaStream_t st) {
  const Int8Plan p = plan_int8_mm(M, N, K);
  if (p.bn == 0) return cudaErrorInvalidValue;
  MmArgs a{};
  a.xs = x_scales;
  a.ws = w_scales;
  a.y = y;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.kblocks = (int)((K + kBK - 1) / kBK);
  a.prefetch = prefetch;
  a.wait_ns = testing_wait_ns();
  a.delay_ns = testing_delay_ns();
  return dtype == AQ_F16 ? by_plan<__half>(p, x_q, w_q, a, st)
                         : by_plan<__nv_bfloat16>(p, x_q, w_q, a, st);
}

cudaError_t read_device_error_int8(unsigned* out) {
  return cudaMemcpyFromSymbol(out, g_int8_device_error, sizeof(unsigned));
}
cudaError_t testing_clear_device_error_int8() {
  const unsigned z = 0;
  return cudaMemcpyToSymbol(g_int8_device_error, &z, sizeof(z));
}

void testing_set_int8_plan(int bn, int pair, int splits) {
  g_force_bn.store(bn, std::memory_order_relaxed);
  g_force_pair.store(pair, std::memory_order_relaxed);
  g_force_splits.store(splits, std::memory_order_relaxed);
}

}  // namespace aq
