// moe_kernel.cuh — a mixture-of-experts layer for a few tokens in one kernel,
// over group-quantized expert weights.
//
//   l = x Wr^T;  (e, w) = top-k of softmax(l)           (or given e, w)
//   h = silu(x Wg[e]^T) * (x Wu[e]^T);  y = sum_slots w * (h Wd[e]^T)
//
// What bounds it: the packed weights of the experts chosen are read once,
// 3 I H codes each, while a token costs only one multiply-add per code; so the
// layer runs at the rate the weights stream from HBM, and for a token or two
// at the latency of its dependent steps.  Hence one cooperative kernel, one
// CTA per SM, with the steps separated by grid barriers instead of launches:
// router products, [barrier] top-k and plan (every CTA for itself), gate/up,
// [barrier] down, [barrier] weighted sums.  The down weights of a warp's
// first unit are already under way while it waits at the barrier before.
//
// A unit of work is a 16-row tile of weights times up to 8 of the tokens that
// chose its expert, done by one warp (or a team of warps that share K and add
// their sums in shared memory, when there are fewer units than warps): 8 gate
// rows and the same 8 up rows, so that a thread holds both factors of h, or
// 16 down rows.  A warp streams its rows by cp.async through a ring of its
// own in shared memory, so no unit waits for another warp.  The codes become
// the A operand of mma.m16n8k16 as exact small numbers (offset integers for
// affine codes, E2M1 values for FP4) and x the B operand; per group the
// products P and, with an A operand of ones, the sums X of x leave in fp32:
//   sum += s P' + (b - offset s) X,      P' = sum (offset + q) x.
// So w_hat is never rounded to T.  h is kept as two bf16 numbers (hi + lo, 16
// bits of significand), in the B operand's order, so that down's operand
// rounds far below T.  Each pair (token, slot) has its row of fp32 results;
// the last step adds them in slot order, so no atomics touch a sum and equal
// inputs give equal outputs.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "sm100.cuh"

namespace aq {
namespace moe {

using namespace sm100;

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxPairs = 1024;          // tokens * top_k
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 16;
constexpr int kCounterBytes = 65536;     // the workspace's shared counter area
constexpr uint64_t kWaitNs = 2000000000ull;

struct Params {
  MoeArgs a;
  double* logits;                        // [T, E]
  uint8_t* h;                            // [pairs][I / 32][4][hi 16 B, lo 16 B]
  float* part;                           // [pairs][H]
  unsigned* bars;                        // grid barrier counters (zero between calls)
  unsigned* error;
};

// ------------------------------------------------------------ code operands
enum class Order { kSplit, kPairs, kGroup16 };

template <int BITS, bool FP4, int GS>
struct Format {
  static constexpr int kBits = BITS;
  static constexpr int kGs = GS;
  static constexpr bool kFp4 = FP4;
  // Which of a thread's 8 codes of a 32-chunk form its operand words: halves
  // (j, j + 4) where masks take both at once, neighbours where codes are cut
  // out one by one; for groups of 16 a thread holds 4 codes of each group.
  static constexpr Order kOrder = GS == 16 ? Order::kGroup16
                                  : (BITS == 2 || BITS == 4) ? Order::kSplit : Order::kPairs;
  static constexpr int kStageK = BITS <= 4 ? 256 : 128;   // elements of K per ring stage
  static constexpr int kRowBytes = kStageK * BITS / 8;
  static constexpr int kRowPitch = kRowBytes + 16;        // spreads 8 rows over the banks
  static constexpr int kScaleSize = FP4 ? 1 : 2;
  static constexpr int kScaleBytes = kStageK / GS * kScaleSize;   // per row and stage
  // room for the aligned 4-byte words that hold a row's scales of a stage
  static constexpr int kScalePitch = (kScaleBytes + 4 + 7) / 8 * 8;
  static constexpr int kSlot = 16 * kRowPitch + (FP4 ? 1 : 2) * 16 * kScalePitch;
  static constexpr int kRingFit = 168 * 1024 / (kWarps * kSlot);
  static constexpr int kRing = kRingFit > 8 ? 8 : kRingFit;
  static_assert(kRing >= 3 && kSlot % 16 == 0, "ring");
};

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

template <typename O> struct Op;         // operand type of an mma
template <> struct Op<__half> {
  static constexpr uint32_t kMagic = 0x64006400u;         // 1024 + q
  static constexpr float kOffset = 0.0f;                  // taken off again, below
  static constexpr uint32_t kOnes = 0x3C003C00u;
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
        " {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};
template <> struct Op<__nv_bfloat16> {
  static constexpr uint32_t kMagic = 0x43004300u;         // 128 + q, q < 128
  static constexpr float kOffset = 128.0f;
  static constexpr uint32_t kOnes = 0x3F803F80u;
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7},"
        " {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};

// What the operand holds beside the code: P' = sum (offset + q) x.  8-bit
// codes do not fit bf16's 7 bits beside 128 and become q - 128 (exact).  With
// fp16's 1024 the products of the offset would cost up to 9 bits of the fp32
// sums (2-bit codes in groups of 128: 3.5e-4 instead of 2.1e-4 of error after
// rounding to fp16), so it is subtracted from the operand, which is exact.
template <typename O, typename F>
__host__ __device__ constexpr float code_offset() {
  return F::kFp4 ? 0.0f
         : (F::kBits == 8 && std::is_same<O, __nv_bfloat16>::value) ? -128.0f : Op<O>::kOffset;
}
// What the operand's values are multiplied with afterwards (FP4 in fp16: the
// code's bits are those of value * 2^-14).
template <typename O, typename F>
__host__ __device__ constexpr float product_scale() {
  return F::kFp4 && std::is_same<O, __half>::value ? 16384.0f : 1.0f;
}

// The operand word of two codes under the magic exponent.
template <typename O>
__device__ __forceinline__ uint32_t from_magic(uint32_t v) {
  if constexpr (std::is_same<O, __half>::value) {
    const uint32_t k = Op<O>::kMagic;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v),
                              *reinterpret_cast<const __half2*>(&k));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    return v;
  }
}

template <typename O>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t t) {   // codes in bits 0-3 and 16-19
  if constexpr (std::is_same<O, __half>::value) {
    return ((t & 0x00070007u) << 9) | ((t & 0x00080008u) << 12);
  } else {
    // bits of value * 2^-126 (subnormals are exact), times 2^126
    const uint32_t v = ((t & 0x00070007u) << 6) | ((t & 0x00080008u) << 12);
    const uint32_t k = 0x7E807E80u;
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                     *reinterpret_cast<const __nv_bfloat162*>(&k));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// The four operand words (two mma k-steps of two words) of a thread's 8 codes
// of one row's 32-chunk; `at` is the shared address of the row's chunk.
template <typename O, typename F>
__device__ __forceinline__ void operand(uint32_t at, int t, uint32_t (&r)[4]) {
  constexpr uint32_t magic = Op<O>::kMagic;
  if constexpr (F::kOrder == Order::kGroup16) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint32_t w = __byte_perm(lds16(at + 8 * g + 2 * t), 0u, 0x4140);
      r[2 * g] = e2m1_pair<O>(w & 0x000F000Fu);
      r[2 * g + 1] = e2m1_pair<O>((w >> 4) & 0x000F000Fu);
    }
  } else if constexpr (F::kBits == 4) {
    const uint32_t w = lds32(at + 4 * t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t q = (w >> (4 * i)) & 0x000F000Fu;
      r[i] = F::kFp4 ? e2m1_pair<O>(q) : from_magic<O>(q | magic);
    }
  } else if constexpr (F::kBits == 2) {
    const uint32_t w = __byte_perm(lds16(at + 2 * t), 0u, 0x4140);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = from_magic<O>(((w >> (2 * i)) & 0x00030003u) | magic);
  } else if constexpr (F::kBits == 8) {
    const uint2 w = lds64(at + 8 * t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = i < 2 ? w.x : w.y;
      const uint32_t sel = i & 1 ? 0x4342u : 0x4140u;
      if constexpr (std::is_same<O, __half>::value) {
        r[i] = from_magic<O>(__byte_perm(v, 0x64646464u, sel));   // 1024 + q
      } else {
        // 128 + (q & 127), minus 256 below 128 and 128 from there: q - 128
        const uint32_t q = __byte_perm(v, 0u, sel);
        const uint32_t m = (q & 0x007F007Fu) | 0x43004300u;
        const uint32_t d = (q & 0x00800080u) ^ 0x43804380u;
        const __nv_bfloat162 e = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                         *reinterpret_cast<const __nv_bfloat162*>(&d));
        r[i] = *reinterpret_cast<const uint32_t*>(&e);
      }
    }
  } else {
    // 3, 5, 6 bits: the thread's 8 codes are BITS bytes from byte BITS * t
    const uint32_t byte = F::kBits * t;
    const uint32_t w0 = lds32(at + (byte & ~3u)), w1 = lds32(at + (byte & ~3u) + 4);
    const uint32_t sh = (byte & 3u) * 8u;
    const uint32_t v[2] = {__funnelshift_r(w0, w1, sh), w1 >> sh};
    constexpr uint32_t mask = (1u << F::kBits) - 1u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t q[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int bit = F::kBits * (2 * i + j);
        q[j] = bit >= 32 ? v[1] >> (bit - 32) : __funnelshift_r(v[0], v[1], bit);
      }
      r[i] = from_magic<O>((q[0] & mask) | ((q[1] & mask) << 16) | magic);
    }
  }
}

// The words of x in the operand's order from a thread's 8 values of a chunk.
template <typename F>
__device__ __forceinline__ uint4 order_x(const uint4& v) {
  uint4 r = v;
  if constexpr (F::kOrder == Order::kSplit) {
    r.x = __byte_perm(v.x, v.z, 0x5410);
    r.y = __byte_perm(v.x, v.z, 0x7632);
    r.z = __byte_perm(v.y, v.w, 0x5410);
    r.w = __byte_perm(v.y, v.w, 0x7632);
  } else if constexpr (F::kOrder == Order::kGroup16) {
    r.x = __byte_perm(v.x, v.y, 0x5410);
    r.y = __byte_perm(v.x, v.y, 0x7632);
    r.z = __byte_perm(v.z, v.w, 0x5410);
    r.w = __byte_perm(v.z, v.w, 0x7632);
  }
  return r;
}
// Byte offset of element kk of h within a pair's row (its hi half).
template <typename F>
__device__ __forceinline__ uint32_t h_offset(int kk) {
  const int c = kk >> 5, r = kk & 31;
  int t, word, half;
  if constexpr (F::kOrder == Order::kGroup16) {
    t = (r & 15) >> 2;
    word = (r >> 4) * 2 + (r & 1);
    half = (r >> 1) & 1;
  } else {
    t = r >> 3;
    const int j = r & 7;
    word = F::kOrder == Order::kSplit ? (j & 3) : (j >> 1);
    half = F::kOrder == Order::kSplit ? (j >> 2) : (j & 1);
  }
  return (uint32_t)((c * 4 + t) * 32 + word * 4 + half * 2);
}

// ----------------------------------------------------------------- cp.async
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// --------------------------------------------------------------------- plan
struct Plan {
  float weight[kMaxPairs];
  int16_t expert[kMaxPairs];             // of a pair, -1: none
  int16_t rank[kMaxPairs];               // of a pair among its expert's
  int16_t order[kMaxPairs];              // pairs by expert
  int16_t tile_expert[kMaxPairs];
  int16_t tile_first[kMaxPairs];         // into order
  uint8_t tile_count[kMaxPairs];
  int count[kMaxExperts];
  int first[kMaxExperts];
  int scan[2][kWarps];
  int tiles;
  int abort;
};

template <typename F>
struct Smem {
  static constexpr int kPlanAt = 0;
  static constexpr int kExchangeAt = (sizeof(Plan) + 15) / 16 * 16;
  static constexpr int kRingAt = kExchangeAt + kWarps * 512;
  static constexpr int kBytes = kRingAt + kWarps * F::kRing * F::kSlot;
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
};

// Every CTA of the (cooperative, so co-resident) grid arrives; false after the
// time limit.
__device__ __forceinline__ bool grid_barrier(unsigned* counter, unsigned ctas, int* abort) {
  __syncthreads();
  if (threadIdx.x == 0) {
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(counter) : "memory");
    const uint64_t t0 = globaltimer_ns();
    for (unsigned it = 1;; ++it) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
      if (v >= ctas) break;
      if ((it & 255u) == 0u && globaltimer_ns() - t0 > kWaitNs) {
        *abort = 1;
        break;
      }
    }
    __threadfence();
  }
  __syncthreads();
  return *abort == 0;
}

// ------------------------------------------------------------------- router
// A warp per (token, expert): a product of two T is exact in fp32 and the
// sums are fp64, so that two logits are in the order of their exact values.
template <typename T>
__device__ __forceinline__ double dot8(const uint4& a, const uint4& b) {
  const T* pa = reinterpret_cast<const T*>(&a);
  const T* pb = reinterpret_cast<const T*>(&b);
  double s[2] = {0.0, 0.0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    s[i & 1] += (double)__fmul_rn(TT<T>::to_f(pa[i]), TT<T>::to_f(pb[i]));
  return s[0] + s[1];
}
template <typename T>
__device__ __forceinline__ void router_logits(const Params& p, int warp, int lane) {
  const int vecs = p.a.H / 8, tasks = p.a.T * p.a.E;
  for (int q = warp * (int)gridDim.x + (int)blockIdx.x; q < tasks; q += (int)gridDim.x * kWarps) {
    const int t = q / p.a.E, e = q - t * p.a.E;
    const uint4* x = reinterpret_cast<const uint4*>(p.a.x) + (int64_t)t * vecs;
    const uint4* w = reinterpret_cast<const uint4*>(p.a.w_router) + (int64_t)e * vecs;
    double acc = 0.0;
#pragma unroll 4
    for (int v = lane; v < vecs; v += 32) acc += dot8<T>(__ldg(x + v), __ldg(w + v));
#pragma unroll
    for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
    if (lane == 0) p.logits[t * p.a.E + e] = acc;
  }
}

// Unsigned order of doubles: 1 for NaN, above it every number from -inf on.
__device__ __forceinline__ unsigned long long order_key(double v) {
  const long long b = __double_as_longlong(v + 0.0);     // -0 counts as 0
  return v != v ? 1ull : b < 0 ? ~(unsigned long long)b : (unsigned long long)b | (1ull << 63);
}

// A warp per token: top_k logits (ties: the lowest index; NaN below all
// numbers) and their softmax weights, into the plan (and out, by CTA 0).
__device__ __forceinline__ void choose(const Params& p, Plan& plan, int warp, int lane) {
  const int E = p.a.E, k = p.a.top_k;
  constexpr int kPer = kMaxExperts / 32;
  for (int t = warp; t < p.a.T; t += kWarps) {
    double v[kPer];
    double top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = i * 32 + lane;
      if (i * 32 < E && e < E) {
        v[i] = __ldcg(p.logits + t * E + e);
        nan |= v[i] != v[i];
        top = fmax(top, v[i]);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i * 32 + lane < E) sum += expf((float)(v[i] - top));
    if (nan) sum = NAN;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    unsigned used = 0u;                                  // of this lane's experts
    int mine = 0;                                        // lane j holds slot j
    float mine_w = 0.0f, chosen = 0.0f;
    for (int j = 0; j < k; ++j) {
      unsigned long long best = 0ull;
      int at = 0;
      double bv = 0.0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i * 32 + lane < E && !((used >> i) & 1u)) {
          const unsigned long long key = order_key(v[i]);
          if (key > best) {
            best = key;
            at = i * 32 + lane;
            bv = v[i];
          }
        }
      const unsigned hi = (unsigned)(best >> 32), lo = (unsigned)best;
      const unsigned win_hi = __reduce_max_sync(0xFFFFFFFFu, hi);
      const unsigned win_lo = __reduce_max_sync(0xFFFFFFFFu, hi == win_hi ? lo : 0u);
      const bool wins = hi == win_hi && lo == win_lo;
      const int e = (int)__reduce_min_sync(0xFFFFFFFFu, wins ? (unsigned)at : 0x7FFFFFFFu);
      const float ex = expf((float)(__shfl_sync(0xFFFFFFFFu, bv, e & 31) - top));
      chosen += ex;
      if (lane == j) {
        mine = e;
        mine_w = ex;
      }
      if (lane == (e & 31)) used |= 1u << (e >> 5);
    }
    if (lane < k) {
      // a NaN among the logits shows in every weight
      const float w = sum != sum ? sum : __fdiv_rn(mine_w, p.a.normalize ? chosen : sum);
      plan.expert[t * k + lane] = (int16_t)mine;
      plan.weight[t * k + lane] = w;
      if (blockIdx.x == 0) {
        p.a.indices[t * k + lane] = mine;
        p.a.weights[t * k + lane] = w;
      }
    }
  }
}

// The pairs of each expert in their order, cut into tiles of up to 8: every
// CTA has to come to the same tiles.  One warp ranks the pairs, 32 at a time.
__device__ __forceinline__ void make_plan(const Params& p, Plan& plan) {
  const int E = p.a.E, P = p.a.T * p.a.top_k, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < E) plan.count[tid] = 0;
  __syncthreads();
  if (warp == 0) {
    for (int q = lane; q - lane < P; q += 32) {
      const int e = q < P ? plan.expert[q] : -1;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
      const int before = __popc(same & ((1u << lane) - 1u));
      const int base = e >= 0 ? plan.count[e] : 0;
      __syncwarp();
      if (e >= 0) {
        plan.rank[q] = (int16_t)(base + before);
        if (before == 0) plan.count[e] = base + __popc(same);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  const int c = tid < E ? plan.count[tid] : 0, n = (c + 7) / 8;
  int sc = c, sn = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int uc = __shfl_up_sync(0xFFFFFFFFu, sc, o), un = __shfl_up_sync(0xFFFFFFFFu, sn, o);
    if (lane >= o) {
      sc += uc;
      sn += un;
    }
  }
  if (lane == 31) {
    plan.scan[0][warp] = sc;
    plan.scan[1][warp] = sn;
  }
  __syncthreads();
  int bc = 0, bn = 0;
  for (int w = 0; w < warp; ++w) {
    bc += plan.scan[0][w];
    bn += plan.scan[1][w];
  }
  const int c0 = bc + sc - c, n0 = bn + sn - n;
  if (tid < E) plan.first[tid] = c0;
  for (int j = 0; j < n; ++j) {
    plan.tile_expert[n0 + j] = (int16_t)tid;
    plan.tile_first[n0 + j] = (int16_t)(c0 + 8 * j);
    plan.tile_count[n0 + j] = (uint8_t)min(8, c - 8 * j);
  }
  if (tid == kThreads - 1) plan.tiles = bn + sn;
  __syncthreads();
  for (int q = tid; q < P; q += kThreads) {
    const int e = plan.expert[q];
    if (e >= 0) plan.order[plan.first[e] + plan.rank[q]] = (int16_t)q;
  }
  __syncthreads();
}

// ------------------------------------------------------- gate/up and down
// PH 1: gate and up (8 rows each) over H; PH 2: down (16 rows) over I.
template <int PH, typename T, typename F>
struct Phase {
  using O = typename std::conditional<PH == 1, T, __nv_bfloat16>::type;
  static constexpr int kChunks = F::kStageK / 32;        // per stage
  static constexpr int kDepth = 4;                       // chunks of x loaded ahead
  static_assert(kChunks >= kDepth, "x runs at most one stage ahead");

  const Params& p;
  Plan& plan;
  const int lane, g, t;
  const uint32_t ring;
  int K, blocks, stages, units;                          // row blocks per tile, stages per unit
  int team, member, warps, ustride, unit0;               // warps of a team share a unit's K
  int64_t row_bytes, scale_row;
  bool vec16, vec8;
  // the next stage to copy
  int pu, ps;
  uint32_t pslot;
  int64_t prow;                                          // first row of its unit in the stack

  __device__ __forceinline__ Phase(const Params& pp, Plan& pl, uint32_t r, int warp, int ln)
      : p(pp), plan(pl), lane(ln), g(ln >> 2), t(ln & 3), ring(r) {
    K = PH == 1 ? p.a.H : p.a.I;
    blocks = PH == 1 ? p.a.I / 8 : p.a.H / 16;
    stages = (K + F::kStageK - 1) / F::kStageK;
    units = plan.tiles * blocks;
    row_bytes = (int64_t)K * F::kBits / 8;
    scale_row = (int64_t)(K / F::kGs) * F::kScaleSize;
    vec16 = row_bytes % 16 == 0;
    vec8 = F::kScaleBytes % 8 == 0 && scale_row % 8 == 0;
    // Team size with the fewest stages one after the other (and one more per
    // unit for its start and end).
    const int total = (int)gridDim.x * kWarps;
    warps = 1;
    int best = 0x7FFFFFFF;
    for (int s = 1; s <= 8 && s <= stages; s *= 2) {
      const int teams = total / s;
      const int cost = ((units + teams - 1) / teams) * ((stages + s - 1) / s + 1);
      if (cost < best) {
        best = cost;
        warps = s;
      }
    }
    team = warp / warps;
    member = warp - team * warps;
    unit0 = team * (int)gridDim.x + (int)blockIdx.x;
    ustride = (int)gridDim.x * (kWarps / warps);
    pu = unit0;
    ps = member;
    pslot = 0;
    place();
  }

  __device__ __forceinline__ void place() {
    if (pu < units) {
      const int tile = pu / blocks, rb = pu - tile * blocks;
      prow = (int64_t)plan.tile_expert[tile] * (PH == 1 ? p.a.I : p.a.H) + rb * (PH == 1 ? 8 : 16);
    }
  }
  // Row r (0..15) of a unit whose first row is `row` in a stack of matrices.
  static __device__ __forceinline__ int64_t row_of(int64_t row, int r) {
    return row + (PH == 1 ? (r & 7) : r);
  }
  __device__ __forceinline__ const MoeMatrix& matrix(int r) const {
    return PH == 2 ? p.a.down : r < 8 ? p.a.gate : p.a.up;
  }

  // Start the copy of the next stage (nothing when all are under way).
  __device__ __forceinline__ void issue() {
    if (pu < units) {
      const uint32_t slot = ring + pslot * F::kSlot;
      const int left = K - ps * F::kStageK;              // elements of this stage
      const int bytes = (left < F::kStageK ? left : F::kStageK) * F::kBits / 8;
      const int64_t at = (int64_t)ps * F::kRowBytes;
      if (vec16) {
        constexpr int kPer = F::kRowBytes / 16;
#pragma unroll
        for (int i = 0; i < (kPer + 1) / 2; ++i) {
          const int q = lane + 32 * i, r = q / kPer, c = (q - r * kPer) * 16;
          if (r < 16 && c < bytes)
            cp_async<16>(slot + r * F::kRowPitch + c,
                         matrix(r).w_q + row_of(prow, r) * row_bytes + at + c);
        }
      } else {
        constexpr int kPer = F::kRowBytes / 4;
#pragma unroll 4
        for (int q = lane; q < 16 * kPer; q += 32) {
          const int r = q / kPer, c = (q - r * kPer) * 4;
          if (c < bytes)
            cp_async<4>(slot + r * F::kRowPitch + c,
                        matrix(r).w_q + row_of(prow, r) * row_bytes + at + c);
        }
      }
      // scales and biases: the 4-byte words that hold this stage's, 8 bytes at
      // a time where the rows allow it
      const int groups = (left < F::kStageK ? left : F::kStageK) / F::kGs;
#pragma unroll
      for (int arr = 0; arr < (F::kFp4 ? 1 : 2); ++arr) {
        const uint32_t dst = slot + 16 * F::kRowPitch + arr * 16 * F::kScalePitch;
        if (vec8) {
          constexpr int kPer = F::kScaleBytes / 8 > 0 ? F::kScaleBytes / 8 : 1;
#pragma unroll
          for (int q = lane; q < 16 * kPer; q += 32) {
            const int r = q / kPer, c = (q - r * kPer) * 8;
            if (c < groups * F::kScaleSize)
              cp_async<8>(dst + r * F::kScalePitch + c,
                          base(matrix(r), arr) + row_of(prow, r) * scale_row +
                              (int64_t)ps * F::kScaleBytes + c);
          }
        } else {
          constexpr int kPer = F::kScalePitch / 4;
          for (int q = lane; q < 16 * kPer; q += 32) {
            const int r = q / kPer, c = (q - r * kPer) * 4;
            const uint8_t* first = base(matrix(r), arr) + row_of(prow, r) * scale_row +
                                   (int64_t)ps * F::kScaleBytes;
            const uint8_t* end = first + groups * F::kScaleSize;
            const uint8_t* src = first - ((uintptr_t)first & 3) + c;
            if (src < end) {
              const int n = end - src < 4 ? (int)(end - src) : 4;   // read no byte past the row
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                               dst + r * F::kScalePitch + c),
                           "l"(src), "r"(n)
                           : "memory");
            }
          }
        }
      }
      pslot = pslot + 1 == F::kRing ? 0 : pslot + 1;
      ps += warps;
      if (ps >= stages) {
        ps = member;
        pu += ustride;
        place();
      }
    }
    cp_commit();
  }
  static __device__ __forceinline__ const uint8_t* base(const MoeMatrix& m, int arr) {
    return arr ? m.biases : m.scales;
  }
  __device__ __forceinline__ void start() {
#pragma unroll
    for (int i = 0; i < F::kRing - 1; ++i) issue();
  }

  // x (or h) of this thread's column for 32-chunk c: PH 1 one vector (8
  // values of T), PH 2 two (hi, lo).  Columns past the tile's count are zero.
  struct X {
    uint4 v[PH];
  };
  __device__ __forceinline__ X load_x(const uint8_t* col, int c) const {
    X r;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (PH == 1) {
      if constexpr (F::kOrder == Order::kGroup16) {
        uint2 a = make_uint2(0u, 0u), b = a;
        if (col) {
          a = __ldg(reinterpret_cast<const uint2*>(col + (int64_t)c * 64 + t * 8));
          b = __ldg(reinterpret_cast<const uint2*>(col + (int64_t)c * 64 + 32 + t * 8));
        }
        r.v[0] = make_uint4(a.x, a.y, b.x, b.y);
      } else {
        r.v[0] = col ? __ldg(reinterpret_cast<const uint4*>(col + (int64_t)c * 64 + t * 16)) : zero;
      }
    } else {
      const uint4* h = reinterpret_cast<const uint4*>(col + (int64_t)c * 128 + t * 32);
      r.v[0] = col ? h[0] : zero;
      r.v[1] = col ? h[1] : zero;
    }
    return r;
  }

  __device__ __forceinline__ float scale_at(uint32_t at) const {
    if constexpr (F::kFp4) {
      uint32_t b;
      asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b) : "r"(at));
      return fp4_scale_t<T>(b, F::kGs);
    } else {
      const uint16_t b = (uint16_t)lds16(at);
      return TT<T>::to_f(*reinterpret_cast<const T*>(&b));
    }
  }

  __device__ __forceinline__ void run(float* exchange) {
    uint32_t slot_i = 0;
    for (int u = unit0; u < units; u += ustride) {
      const int tile = u / blocks, rb = u - tile * blocks;
      const int first = plan.tile_first[tile], count = plan.tile_count[tile];
      const int64_t row0 = (int64_t)plan.tile_expert[tile] * (PH == 1 ? p.a.I : p.a.H) +
                           rb * (PH == 1 ? 8 : 16);
      const uint8_t* col = nullptr;
      if (g < count) {
        const int pair = plan.order[first + g];
        col = PH == 1 ? static_cast<const uint8_t*>(p.a.x) + (int64_t)(pair / p.a.top_k) * K * 2
                      : p.h + (int64_t)pair * K * 4;
      }
      const int chunks = K / 32;
      float tot[4] = {0.f, 0.f, 0.f, 0.f};
      X xq[kDepth];
#pragma unroll
      for (int c = 0; c < kDepth; ++c) {
        const int cc = member * kChunks + c;
        xq[c] = load_x(cc < chunks ? col : nullptr, cc);
      }
      for (int s = member; s < stages; s += warps) {
        cp_wait<F::kRing - 2>();
        __syncwarp();
        issue();
        const uint32_t slot = ring + slot_i * F::kSlot;
        slot_i = slot_i + 1 == F::kRing ? 0 : slot_i + 1;
        // scales of rows g and g + 8: their offset within the copied words
        const int64_t so = (int64_t)s * F::kScaleBytes;
        const uint32_t dlo = (uint32_t)((row_of(row0, g) * scale_row + so) & 3);
        const uint32_t dhi = (uint32_t)((row_of(row0, g + 8) * scale_row + so) & 3);
        const uint32_t slo = slot + 16 * F::kRowPitch + g * F::kScalePitch + dlo;
        const uint32_t shi = slot + 16 * F::kRowPitch + (g + 8) * F::kScalePitch + dhi;
        const uint32_t wlo = slot + g * F::kRowPitch, whi = slot + (g + 8) * F::kRowPitch;
        float P[4] = {0.f, 0.f, 0.f, 0.f}, S[4] = {0.f, 0.f, 0.f, 0.f};
        auto flush = [&](int group) {
          const uint32_t o = group * F::kScaleSize;
          const float sl = scale_at(slo + o), sh = scale_at(shi + o);
          constexpr float scale = product_scale<O, F>();
          if constexpr (scale != 1.0f) {
#pragma unroll
            for (int i = 0; i < 4; ++i) P[i] *= scale;
          }
          tot[0] = fmaf(sl, P[0], tot[0]);
          tot[1] = fmaf(sl, P[1], tot[1]);
          tot[2] = fmaf(sh, P[2], tot[2]);
          tot[3] = fmaf(sh, P[3], tot[3]);
          if constexpr (!F::kFp4) {
            constexpr float off = code_offset<O, F>();
            const uint32_t bo = 16 * F::kScalePitch + o;
            const float bl = fmaf(-off, sl, scale_at(slo + bo)), bh = fmaf(-off, sh, scale_at(shi + bo));
            tot[0] = fmaf(bl, S[0], tot[0]);
            tot[1] = fmaf(bl, S[1], tot[1]);
            tot[2] = fmaf(bh, S[0], tot[2]);
            tot[3] = fmaf(bh, S[1], tot[3]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) P[i] = S[i] = 0.0f;
        };
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const int cc = s * kChunks + c;
          if (cc < chunks) {
            X x = xq[c % kDepth];
            {
              const int nx = c + kDepth < kChunks ? cc + kDepth
                                                  : (s + warps) * kChunks + c + kDepth - kChunks;
              xq[c % kDepth] = load_x(nx < chunks ? col : nullptr, nx);
            }
            if constexpr (PH == 1) x.v[0] = order_x<F>(x.v[0]);
            uint32_t lo[4], hi[4];
            operand<O, F>(wlo + c * 4 * F::kBits, t, lo);
            operand<O, F>(whi + c * 4 * F::kBits, t, hi);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
              for (int v = 0; v < PH; ++v) {
                const uint32_t b0 = half ? x.v[v].z : x.v[v].x, b1 = half ? x.v[v].w : x.v[v].y;
                Op<O>::mma(P, lo[2 * half], hi[2 * half], lo[2 * half + 1], hi[2 * half + 1], b0, b1);
                if constexpr (!F::kFp4)
                  Op<O>::mma(S, Op<O>::kOnes, Op<O>::kOnes, Op<O>::kOnes, Op<O>::kOnes, b0, b1);
              }
              if constexpr (F::kGs == 16) flush(2 * c + half);
            }
            if constexpr (F::kGs >= 32) {
              if ((c + 1) % (F::kGs / 32) == 0) flush(c / (F::kGs / 32));
            }
          }
        }
      }
      if (warps > 1) {
        float4* ex = reinterpret_cast<float4*>(exchange) + (team * warps) * 32;
        if (member) ex[member * 32 + lane] = make_float4(tot[0], tot[1], tot[2], tot[3]);
        named_barrier_sync(1 + team, 32 * warps);
        if (member == 0)
          for (int m = 1; m < warps; ++m) {
            const float4 v = ex[m * 32 + lane];
            tot[0] += v.x;
            tot[1] += v.y;
            tot[2] += v.z;
            tot[3] += v.w;
          }
        named_barrier_sync(1 + team, 32 * warps);
      }
      if (member == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (2 * t + j < count) {
            const int pair = plan.order[first + 2 * t + j];
            if constexpr (PH == 1) {
              const float gate = tot[j], up = tot[2 + j];
              const float h = __fdiv_rn(gate, 1.0f + expf(-gate)) * up;
              const __nv_bfloat16 hi = __float2bfloat16_rn(h);
              const float rest = h - __bfloat162float(hi);
              // an infinity or NaN is kept by the first part alone
              const __nv_bfloat16 lo = __float2bfloat16_rn(fabsf(rest) <= 3.0e38f ? rest : 0.0f);
              uint8_t* dst = p.h + (int64_t)pair * p.a.I * 4 + h_offset<F>(rb * 8 + g);
              *reinterpret_cast<__nv_bfloat16*>(dst) = hi;
              *reinterpret_cast<__nv_bfloat16*>(dst + 16) = lo;
            } else {
              float* dst = p.part + (int64_t)pair * p.a.H + rb * 16 + g;
              dst[0] = tot[j];
              dst[8] = tot[2 + j];
            }
          }
        }
      }
    }
  }
};

// y = sum over the slots of weight * result, in slot order; four columns per
// thread.
template <typename T>
__device__ __forceinline__ void weighted_sums(const Params& p, const Plan& plan) {
  const int vecs = p.a.H / 4, k = p.a.top_k, tasks = p.a.T * vecs;
  T* y = static_cast<T*>(p.a.y);
  for (int q = (int)blockIdx.x * kThreads + (int)threadIdx.x; q < tasks;
       q += (int)gridDim.x * kThreads) {
    const int tok = q / vecs, v = q - tok * vecs;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
      const int pair = tok * k + j;
      if (plan.expert[pair] >= 0) {
        const float w = plan.weight[pair];
        const float4 r = __ldcg(reinterpret_cast<const float4*>(p.part + (int64_t)pair * p.a.H) + v);
        s[0] = fmaf(w, r.x, s[0]);
        s[1] = fmaf(w, r.y, s[1]);
        s[2] = fmaf(w, r.z, s[2]);
        s[3] = fmaf(w, r.w, s[3]);
      }
    }
    T o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = TT<T>::from_f(s[i]);
    *reinterpret_cast<uint2*>(y + (int64_t)q * 4) = *reinterpret_cast<const uint2*>(o);
  }
}

template <typename T, typename F>
__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  using S = Smem<F>;
  Plan& plan = *reinterpret_cast<Plan*>(smem);
  float* exchange = reinterpret_cast<float*>(smem + S::kExchangeAt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem) + S::kRingAt + warp * F::kRing * F::kSlot;
  if (threadIdx.x == 0) plan.abort = 0;

  bool ok = true;
  if (p.a.w_router) {
    router_logits<T>(p, warp, lane);
    ok = grid_barrier(p.bars + 0, gridDim.x, &plan.abort);
    if (ok) choose(p, plan, warp, lane);
  } else {
    for (int q = threadIdx.x; q < p.a.T * p.a.top_k; q += kThreads) {
      const int e = p.a.indices[q];
      plan.expert[q] = e >= 0 && e < p.a.E ? (int16_t)e : (int16_t)-1;
      plan.weight[q] = p.a.weights[q];
    }
  }
  __syncthreads();
  if (ok) {
    make_plan(p, plan);
    {
      Phase<1, T, F> up(p, plan, ring, warp, lane);
      up.start();
      up.run(exchange);
    }
    __syncwarp();
    Phase<2, T, F> down(p, plan, ring, warp, lane);
    down.start();
    ok = grid_barrier(p.bars + 1, gridDim.x, &plan.abort);
    if (ok) {
      down.run(exchange);
      ok = grid_barrier(p.bars + 2, gridDim.x, &plan.abort);
      if (ok) weighted_sums<T>(p, plan);
    }
  }
  cp_wait<0>();
  if (threadIdx.x == 0) {
    if (!ok) {
      atomicOr(p.error, 1u);
    } else if (atomicAdd(p.bars + 3, 1u) == gridDim.x - 1) {
      // every CTA is past the last barrier: the counters are zero again
      p.bars[0] = p.bars[1] = p.bars[2] = p.bars[3] = 0u;
    }
  }
}

// -------------------------------------------------------------------- host
template <typename T, typename F>
cudaError_t launch(const Params& p, int sms, cudaStream_t st) {
  using S = Smem<F>;
  auto kern = moe_kernel<T, F>;
  static std::atomic<bool> attr_done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr_done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = S::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int BITS, bool FP4, int GS>
cudaError_t launch_gs(const Params& p, int sms, int dtype, cudaStream_t st) {
  using F = Format<BITS, FP4, GS>;
  return dtype == AQ_F16 ? launch<__half, F>(p, sms, st) : launch<__nv_bfloat16, F>(p, sms, st);
}
template <int BITS>
cudaError_t launch_affine(const Params& p, int sms, int dtype, cudaStream_t st) {
  switch (p.a.gs) {
    case 32: return launch_gs<BITS, false, 32>(p, sms, dtype, st);
    case 64: return launch_gs<BITS, false, 64>(p, sms, dtype, st);
    case 128: return launch_gs<BITS, false, 128>(p, sms, dtype, st);
    default: return cudaErrorInvalidValue;
  }
}

// One translation unit per width (they build in parallel).
cudaError_t launch_bits2(const Params& p, int sms, int dtype, cudaStream_t st);
cudaError_t launch_bits3(const Params& p, int sms, int dtype, cudaStream_t st);
cudaError_t launch_bits4(const Params& p, int sms, int dtype, cudaStream_t st);
cudaError_t launch_bits5(const Params& p, int sms, int dtype, cudaStream_t st);
cudaError_t launch_bits6(const Params& p, int sms, int dtype, cudaStream_t st);
cudaError_t launch_bits8(const Params& p, int sms, int dtype, cudaStream_t st);
cudaError_t launch_fp4(const Params& p, int sms, int dtype, cudaStream_t st);

}  // namespace moe
}  // namespace aq
