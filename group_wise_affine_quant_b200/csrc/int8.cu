// int8.cu — W8A8: the symmetric row quantizer and the 8-bit integer matrix
// product with one scale per token and one per channel.
//
// Quantizer: a = max |x| over the row, s = a / 127, q = rint(x / s), both
// divisions and the rounding as fp32 IEEE operations (bit-exact codes).  A
// row with a NaN has s = NaN, one with an infinity s = inf, and codes 0, so
// that the products of such a row show it (NaN).  The row stays in registers
// between the two passes up to K = 16384 (longer rows are read twice, the
// second time from L2): 2 bytes in and 1 out per element.  The maximum is
// taken on the 16-bit patterns without their sign (NaN > inf > finite).  The
// division per element is replaced by a product with 1/s: r = x * fl(1/s) is
// within 127 * 2^-22 of x / s, so rint agrees unless r is within 1e-4 of a
// tie, and only then is the IEEE division done.
//
// Product: y[m, n] = T(((float)sum_k x_q w_q * s_x[m]) * s_w[n]).  The sum is
// exact in 32-bit integers (K is limited so that it cannot overflow),
// whatever the split; the conversion to fp32 rounds by at most 2^-24.
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
  r.s = __fdiv_rn(amax, 127.0f);
  const bool finite = r.s <= 3.0e38f;                       // false for inf and NaN
  r.how = !finite || r.s == 0.0f ? 0 : r.s < 1e-30f ? 2 : 1;
  r.inv = r.how == 1 ? __fdiv_rn(1.0f, r.s) : 0.0f;
  return r;
}
__device__ __forceinline__ uint32_t code_of(float x, const RowScale& r) {
  if (r.how == 2) {
    const float v = fminf(fmaxf(__fdiv_rn(x, r.s), -127.0f), 127.0f);
    return __float_as_uint(__fadd_rn(v, kRoundMagic));
  }
  const float v = __fmul_rn(x, r.inv);
  float t = __fadd_rn(v, kRoundMagic);
  if (fabsf(__fsub_rn(v, __fsub_rn(t, kRoundMagic))) > 0.4999f)
    t = __fadd_rn(__fdiv_rn(x, r.s), kRoundMagic);
  return __float_as_uint(t);
}
template <typename T>
__device__ __forceinline__ uint32_t codes4(uint32_t lo, uint32_t hi, const RowScale& r) {
  const float2 a = unpack2<T>(lo), b = unpack2<T>(hi);
  const uint32_t p = __byte_perm(code_of(a.x, r), code_of(a.y, r), 0x0040);
  const uint32_t q = __byte_perm(code_of(b.x, r), code_of(b.y, r), 0x0040);
  return __byte_perm(p, q, 0x5410);
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

// A warp per row (K <= 512 * V): rows too short to keep a block busy.
constexpr int kWarpRows = 8;
template <typename T, int V>
__global__ void __launch_bounds__(kWarpRows * 32)
quantize_int8_warp_kernel(const uint4* __restrict__ x, uint4* __restrict__ xq,
                          float* __restrict__ scales, int64_t rows, int nvec) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5);
  if (row >= rows) return;
  const uint4* src = x + row * nvec * 2;
  Vec16 v[V];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = lane + 32 * i;
    if (c < nvec) {
      v[i] = load16(src, c);
      m = __vmaxu2(m, abs_max2(v[i]));
    }
  }
  const RowScale r = row_scale(from_bits<T>(__reduce_max_sync(0xFFFFFFFFu, max_half(m))));
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = lane + 32 * i;
    if (c < nvec) xq[row * nvec + c] = codes16<T>(v[i], r);
  }
  if (lane == 0) scales[row] = r.s;
}

// A block per row; V = 0 reads the row twice (K > 16384).
constexpr int kRowThreads = 256;
template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads)
quantize_int8_row_kernel(const uint4* __restrict__ x, uint4* __restrict__ xq,
                         float* __restrict__ scales, int nvec) {
  pdl_launch_dependents();
  __shared__ uint32_t part[kRowThreads / 32];
  const int64_t row = blockIdx.x;
  const uint4* src = x + row * nvec * 2;
  uint4* dst = xq + row * nvec;
  constexpr int kHeld = V > 0 ? V : 1;
  Vec16 v[kHeld];
  uint32_t m = 0u;
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + kRowThreads * i;
      if (c < nvec) {
        v[i] = load16(src, c);
        m = __vmaxu2(m, abs_max2(v[i]));
      }
    }
  } else {
    for (int c = threadIdx.x; c < nvec; c += kRowThreads) m = __vmaxu2(m, abs_max2(load16(src, c)));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, max_half(m));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  m = 0u;
#pragma unroll
  for (int i = 0; i < kRowThreads / 32; ++i) m = max(m, part[i]);
  const RowScale r = row_scale(from_bits<T>(m));
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + kRowThreads * i;
      if (c < nvec) dst[c] = codes16<T>(v[i], r);
    }
  } else {
    for (int c = threadIdx.x; c < nvec; c += kRowThreads) dst[c] = codes16<T>(load16(src, c), r);
  }
  if (threadIdx.x == 0) scales[row] = r.s;
}

template <typename T>
cudaError_t quantize_rows(const void* x, void* xq, float* scales, int64_t rows, int64_t K,
                          cudaStream_t st) {
  const uint4* px = static_cast<const uint4*>(x);
  uint4* pq = static_cast<uint4*>(xq);
  const int nvec = (int)(K / 16);
  if (nvec <= 128) {
    const unsigned grid = (unsigned)((rows + kWarpRows - 1) / kWarpRows);
    if (nvec <= 32)
      quantize_int8_warp_kernel<T, 1><<<grid, kWarpRows * 32, 0, st>>>(px, pq, scales, rows, nvec);
    else if (nvec <= 64)
      quantize_int8_warp_kernel<T, 2><<<grid, kWarpRows * 32, 0, st>>>(px, pq, scales, rows, nvec);
    else
      quantize_int8_warp_kernel<T, 4><<<grid, kWarpRows * 32, 0, st>>>(px, pq, scales, rows, nvec);
  } else {
    const unsigned grid = (unsigned)rows;
    if (nvec <= kRowThreads)
      quantize_int8_row_kernel<T, 1><<<grid, kRowThreads, 0, st>>>(px, pq, scales, nvec);
    else if (nvec <= 2 * kRowThreads)
      quantize_int8_row_kernel<T, 2><<<grid, kRowThreads, 0, st>>>(px, pq, scales, nvec);
    else if (nvec <= 4 * kRowThreads)
      quantize_int8_row_kernel<T, 4><<<grid, kRowThreads, 0, st>>>(px, pq, scales, nvec);
    else
      quantize_int8_row_kernel<T, 0><<<grid, kRowThreads, 0, st>>>(px, pq, scales, nvec);
  }
  return cudaGetLastError();
}

// ------------------------------------------------------------------ product
// The weight is the MMA's A operand (128 channels per CTA) and x its B
// operand (BN tokens), so that a few tokens still fill the MMA and a column
// of the accumulator is a run of y.  Both operands are K-major 8-bit tiles of
// 128 bytes per row (128-byte swizzle) that TMA brings into a ring of stages;
// an elected lane issues tcgen05.mma kind::i8 into one of two accumulators in
// TMEM while four epilogue warps scale and store the other.
//   * kPair: two CTAs of a cluster share a tile of 256 channels x BN tokens
//     (cta_group::2); each loads its 128 channels and half of the tokens.  A
//     256 x 256 tile then costs each SM 32 KB per 128 of K instead of 48 KB,
//     which is what bounds a single CTA's tile.
//   * splits > 1 (few tiles): the CTAs of a cluster take slices of K, park
//     their integer tiles in shared memory and add each other's through
//     distributed shared memory, each CTA a share of the columns.
constexpr int kBK = 128;                 // bytes (elements) of K per stage
constexpr int kBM = 128;                 // channels per CTA
constexpr int kMmThreads = 192;          // TMA warp, MMA warp, 4 epilogue warps

template <int BN, bool PAIR>
struct MmShape {
  static constexpr int kBRows = PAIR ? BN / 2 : BN;
  static constexpr int kABytes = kBM * kBK;
  static constexpr int kBBytes = kBRows * kBK;
  static constexpr int kStage = kABytes + kBBytes;
  // BN <= 32 streams weights: five stages, so that two CTAs fit on an SM and
  // one's start and end overlap the other's stream.
  static constexpr int kStages = BN <= 32 ? 5 : (192 * 1024) / kStage > 8 ? 8 : (192 * 1024) / kStage;
  static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
  static constexpr int kBars = 2 * kStages + 5;
  static constexpr int kTail = 2 * BN * 4 + kBars * 8 + 16;     // token scales, barriers, slots
  static constexpr int kSmem = 1024 + kStages * kStage + kTail;
  static_assert(kStages * kStage >= BN * kBM * 4, "split-K parking reuses the ring");
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
};

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
__global__ void __launch_bounds__(kMmThreads)
int8_mm_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
               const MmArgs a) {
  using S = MmShape<BN, PAIR>;
  constexpr int ST = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* tail = smem_raw + (base - raw) + ST * S::kStage;
  float* sx = reinterpret_cast<float*>(tail);                         // [2][BN]
  const uint32_t bars = smem_u32(tail + 2 * BN * 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 2 * BN * 4 + S::kBars * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(const_cast<int*>(abort_flag) + 1);
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (ST + s); };
  auto tfull = [&](int b) { return bars + 8u * (2 * ST + b); };
  auto tempty = [&](int b) { return bars + 8u * (2 * ST + 2 + b); };
  const uint32_t drain = bars + 8u * (2 * ST + 4);

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
      mbar_init(tempty(b), PAIR ? 8 : 4);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    prefetch_tensormap(&mw);
    prefetch_tensormap(&mx);
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
  constexpr int kChannels = PAIR ? 2 * kBM : kBM;        // channels per tile

  if (warp == 0) {
    // ------------------------------------------------------------- TMA warp
    uint32_t it = 0;                                     // stages used so far
    bool ok = true;
    int pre = 0;                                         // stages whose weights are under way
    auto load_w = [&](int s, int nt, int kb) {
      const uint32_t dst = base + s * S::kStage;
      const int row = nt * kChannels + (PAIR ? (int)rank * kBM : 0);
      if constexpr (PAIR) tma_load_2d_pair(dst, &mw, mapa_shared(full(s), 0), kb * kBK, row);
      else tma_load_2d(dst, &mw, full(s), kb * kBK, row);
    };
    auto load_x = [&](int s, int mt, int kb) {
      const uint32_t dst = base + s * S::kStage + S::kABytes;
      const int row = mt * BN + (PAIR ? (int)rank * S::kBRows : 0);
      if constexpr (PAIR) tma_load_2d_pair(dst, &mx, mapa_shared(full(s), 0), kb * kBK, row);
      else tma_load_2d(dst, &mx, full(s), kb * kBK, row);
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
    for (int t = first; t < tiles && ok; t += step) {
      int mt, nt;
      tile_at(t, a.m_tiles, a.n_tiles, mt, nt);
      for (int k = 0; k < nkb; ++k, ++it) {
        const int s = (int)(it % ST);
        const bool early = it < (uint32_t)pre;
        if (!mbar_wait(empty(s), ((it / ST) & 1u) ^ 1u, abort_flag)) {
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
    if (!ok && leader) {
      // Gave up: the copies in flight land before the CTA may exit.
      int ignore = 0;
      const uint32_t n = it < (uint32_t)ST ? it : (uint32_t)ST;
      for (uint32_t j = 0; j < n; ++j) {
        const uint32_t i = it - 1 - j;
        mbar_wait(full((int)(i % ST)), (i / ST) & 1u, &ignore, 200000000ull);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA warp
    if (leader) {
      constexpr uint32_t idesc = idesc_i8(kChannels, BN);
      uint32_t it = 0, tile_i = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step, ++tile_i) {
        const int b = (int)(tile_i & 1u);
        const uint32_t use = tile_i >> 1;
        ok = PAIR ? mbar_wait_cluster(tempty(b), (use & 1u) ^ 1u, abort_flag)
                  : mbar_wait(tempty(b), (use & 1u) ^ 1u, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(b * BN);
        for (int k = 0; k < nkb; ++k, ++it) {
          const int s = (int)(it % ST);
          if (!mbar_wait(full(s), (it / ST) & 1u, abort_flag)) {
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
        int ignore = 0;
        if (elect_one()) mma_commit(drain);
        __syncwarp();
        mbar_wait(drain, 0, &ignore, 200000000ull);
      }
    }
  } else {
    // ------------------------------------------------------- epilogue warps
    pdl_wait();
    const int q = warp & 3;                              // TMEM lane quarter
    const int et = (int)threadIdx.x - 64;                // 0..127
    T* y = static_cast<T*>(a.y);
    uint32_t tile_i = 0;
    bool ok = true;
    for (int t = first; t < tiles; t += step, ++tile_i) {
      int mt, nt;
      tile_at(t, a.m_tiles, a.n_tiles, mt, nt);
      const int b = (int)(tile_i & 1u);
      const int m0 = mt * BN;
      const int n = nt * kChannels + (PAIR ? (int)rank * kBM : 0) + q * 32 + lane;
      float* sxb = sx + b * BN;
      for (int i = et; i < BN; i += 128) sxb[i] = m0 + i < a.M ? a.xs[m0 + i] : 0.0f;
      const float sw = n < a.N ? a.ws[n] : 0.0f;
      named_barrier_sync(1, 128);
      // after giving up the warps still meet at the barrier above
      if (ok) ok = mbar_wait(tfull(b), (tile_i >> 1) & 1u, abort_flag);
      if (!ok) continue;
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * BN);
      constexpr int kCols = BN < 32 ? BN : 32;
#pragma unroll 1
      for (int c0 = 0; c0 < BN; c0 += kCols) {
        uint32_t r[kCols];
        if constexpr (kCols == 32) tmem_ld_32(d + c0, r);
        else tmem_ld_16(d + c0, r);
        tmem_ld_wait();
        if (PAIR || a.splits == 1) {
          if (n < a.N) {
            T* out = y + (int64_t)(m0 + c0) * a.N + n;
            const int cols = min(kCols, a.M - m0 - c0);
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
              if (c < cols)
                out[(int64_t)c * a.N] =
                    TT<T>::from_f(__fmul_rn(__fmul_rn(__int2float_rn((int)r[c]), sxb[c0 + c]), sw));
            }
          }
        } else {
          int* park = reinterpret_cast<int*>(smem_raw + (base - raw));
#pragma unroll
          for (int c = 0; c < kCols; ++c) park[(c0 + c) * kBM + q * 32 + lane] = (int)r[c];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_remote(mapa_shared(tempty(b), 0));
        else mbar_arrive(tempty(b));
      }
    }
  }

  if (!PAIR && a.splits > 1) {
    // One tile per cluster: the parked integer tiles of all slices, added by
    // each CTA for its share of the columns.
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (warp >= 2 && *abort_flag == 0) {
      int mt, nt;
      tile_at(first, a.m_tiles, a.n_tiles, mt, nt);
      const int row = (int)threadIdx.x - 64;
      const int n = nt * kBM + row;
      int* park = reinterpret_cast<int*>(smem_raw + (base - raw));
      const float sw = n < a.N ? a.ws[n] : 0.0f;
      T* y = static_cast<T*>(a.y);
      const int per = (BN + a.splits - 1) / a.splits;
      const int m0 = mt * BN;
      const int c_end = min(min((int)(rank + 1) * per, BN), a.M - m0);
      for (int c = (int)rank * per; c < c_end; ++c) {
        int sum = 0;
        for (int r = 0; r < a.splits; ++r)
          sum += *cluster.map_shared_rank(park + c * kBM + row, r);
        if (n < a.N)
          y[(int64_t)(m0 + c) * a.N + n] =
              TT<T>::from_f(__fmul_rn(__fmul_rn(__int2float_rn(sum), sx[c]), sw));
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
  if (threadIdx.x == 0 && *abort_flag) atomicOr(&g_int8_device_error, 1u);
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

// Rows of K bytes, boxes of 128 bytes x box_rows, 128-byte swizzle, zero fill.
cudaError_t code_map(CUtensorMap* map, const void* base, int64_t rows, int64_t K, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)K};
  cuuint32_t box[2] = {kBK, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
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
  CUtensorMap mw, mx;
  e = code_map(&mw, w_q, a.N, a.K, kBM);
  if (e == cudaSuccess) e = code_map(&mx, x_q, a.M, a.K, S::kBRows);
  if (e != cudaSuccess) return e;
  a.splits = p.splits;
  a.kb_split = p.kb_split;
  a.m_tiles = (a.M + BN - 1) / BN;
  a.n_tiles = (int)((a.N + (PAIR ? 2 * kBM : kBM) - 1) / (PAIR ? 2 * kBM : kBM));
  const int group = PAIR ? 2 : p.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.groups * group), 1, 1);
  cfg.blockDim = dim3(kMmThreads, 1, 1);
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
  return cudaLaunchKernelEx(&cfg, kern, mw, mx, a);
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

// Plan forced by a test: tokens per tile (0: automatic), pair, K-slices.
std::atomic<int> g_force_bn{0}, g_force_pair{0}, g_force_splits{0};

}  // namespace

// Tile and split with the least estimated time, in clocks of one SM.  A stage
// of 128 of K costs the larger of its MMAs (tokens * 2: 8192 multiply-adds
// per clock) and its load from L2 (about 50 bytes per clock); a tile's start
// and end cost about 2500, its stores 8 per column, a split's exchange 1500.
Int8Plan plan_int8_mm(int64_t M, int64_t N, int64_t K) {
  const int kSms = 148;
  Int8Plan best{};
  double best_cost = 0;
  const int kblocks = (int)((K + kBK - 1) / kBK);
  const int fbn = g_force_bn.load(std::memory_order_relaxed);
  const int fpair = g_force_pair.load(std::memory_order_relaxed);
  const int fsplit = g_force_splits.load(std::memory_order_relaxed);
  for (int c = 0; c < 6; ++c) {
    const int bn = c < 4 ? 16 << c : 128 << (c - 4);
    const bool pair = c >= 4;
    if (fbn && (bn != fbn || pair != (fpair != 0))) continue;
    const int64_t chan = pair ? 2 * kBM : kBM;
    const int64_t tiles = ((M + bn - 1) / bn) * ((N + chan - 1) / chan);
    const int slots = pair ? kSms / 2 : bn <= 32 ? 2 * kSms : kSms;
    for (int s = 1; s <= (pair ? 1 : 8) && s <= kblocks; ++s) {
      if (s > 1 && (fsplit ? s > fsplit : tiles * s > slots)) break;
      const int kb = (kblocks + s - 1) / s;
      if ((kblocks + kb - 1) / kb != s) continue;        // an empty slice
      const double mma = 2.0 * (bn < 64 ? 64 : bn);
      const double load = (128.0 + (pair ? bn / 2 : bn)) * kBK / 50.0 * (bn <= 32 ? 2 : 1);
      const double waves = (double)((tiles * s + slots - 1) / slots);
      const double cost = waves * kb * (mma > load ? mma : load) + 2500.0 + 8.0 * bn +
                          (s > 1 ? 1500.0 : 0.0);
      if (best.bn == 0 || cost < best_cost || fsplit) {
        best_cost = cost;
        best.bn = bn;
        best.pair = pair;
        best.splits = s;
        best.kb_split = kb;
        best.groups = s > 1 ? tiles : (tiles < slots ? tiles : slots);
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
  return dtype == AQ_F16 ? by_plan<__half>(p, x_q, w_q, a, st)
                         : by_plan<__nv_bfloat16>(p, x_q, w_q, a, st);
}

cudaError_t read_device_error_int8(unsigned* out) {
  return cudaMemcpyFromSymbol(out, g_int8_device_error, sizeof(unsigned));
}

void testing_set_int8_plan(int bn, int pair, int splits) {
  g_force_bn.store(bn, std::memory_order_relaxed);
  g_force_pair.store(pair, std::memory_order_relaxed);
  g_force_splits.store(splits, std::memory_order_relaxed);
}

}  // namespace aq
