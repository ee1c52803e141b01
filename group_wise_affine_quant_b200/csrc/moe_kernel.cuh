// moe_kernel.cuh — a mixture-of-experts layer for a few tokens in one kernel,
// over group-quantized expert weights.
//
//   l = x Wr^T;  (e, w) = top-k of softmax(l)           (or given e, w)
//   h = silu(x Wg[e]^T) * (x Wu[e]^T);  y = sum_slots w * (h Wd[e]^T)
//
// What bounds it: the packed weights of the experts chosen are read once,
// 3 I H codes each, while a token costs only one multiply-add per code; so the
// floor is the rate the weights stream from HBM, and for a token or two the
// latency of the dependent steps.  Hence one cooperative kernel, one CTA per
// SM, with the steps separated by grid barriers instead of launches: router
// products, [barrier] top-k and plan (every CTA for itself), gate/up,
// [barrier] down, [barrier] weighted sums.  The first down weights are already
// under way while a CTA waits at the barrier before.
//
// Work is cut into row tiles of 16 rows (8 gate rows and the same 8 up rows, so
// that both factors of h meet in one place, or 16 down rows) times a token tile,
// up to 4 or 8 of the tokens that chose the expert.  A CTA takes neighbouring row
// tiles; a team of 2 to 16 of its warps shares the K of one, so each warp
// keeps its part of x in registers over all row tiles of a token tile and
// streams its part of the weight rows by cp.async through a ring of its own.
// The warps' sums meet in shared memory after four row tiles per team (16 tokens,
// 8 of 64 experts of 2048 x 1408 in 4 bits take 96 us, after two row tiles 105).
//
// Measured: that layer 96 us, 2.9 TB/s of its 275 MB (with token tiles of 8 only,
// 107): the issue slots and latencies of unpacking, about 53 instructions for
// 16 x 32 codes where the HBM rate leaves 45.  One token, 8 of 64 experts of
// 2048 x 768: 22 us (from HBM 24.5), most of it dependent steps.
//
// The codes become the A operand of mma.m16n8k16 as exact small numbers and x
// the B operand; per group the products P and the sums X of x leave in fp32:
//   sum += s P + (b - offset s) X,      P = sum (offset + q) x.
// So w_hat is never rounded to T.  In bf16 operands the offset is 128, which takes
// 4 (4 bits) to 6 (2 bits) of the 24 bits of these sums: the rest rounds far
// below T, and codes of up to 4 bits beside 16 instead of 128, three bits better,
// cost a shift a word (97.2 us instead of 95.9; the results are as far from the
// 64-bit values, 1.66e-3 of them in bf16, either way).  h is kept as two bf16
// numbers (hi + lo, 16 bits of significand), in the B operand's order, so that
// down's operand rounds far below T.  Each pair (token, slot) has its row of fp32 results;
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
constexpr int kBatch = 4;                // row tiles of a team between two barriers (even)
constexpr int kExchangeLanes = 33;       // a lane more, to spread the banks
constexpr int kCounterBytes = 65536;     // the workspace's shared counter area

struct Params {
  MoeArgs a;
  double* logits;                        // [T, E]
  uint8_t* h;                            // [pairs][I / 32][4][hi 16 B, lo 16 B]
  float* part;                           // [pairs][H]
  unsigned* bars;                        // grid barrier counters (zero between calls)
  unsigned* error;
  uint64_t wait_ns;                      // bound of a wait at a grid barrier
  uint64_t delay_ns;                     // test hook: start delay of one CTA (0: none)
};

// ------------------------------------------------------------ code operands
enum class Order { kSplit, kPairs, kGroup16 };

template <int BITS, bool FP4, int GS>
struct Format {
  static constexpr int kBits = BITS;
  static constexpr int kGs = GS;
  static constexpr bool kFp4 = FP4;
  // Which of a thread's 8 codes of a 32-chunk form its operand words: halves
  // (j, j + 4) where masks take both at once, neighbours for whole bytes; for
  // groups of 16 a thread holds 4 codes of each group.
  static constexpr Order kOrder = GS == 16 ? Order::kGroup16 : BITS == 8 ? Order::kPairs : Order::kSplit;
  static constexpr int kScaleSize = FP4 ? 1 : 2;
  // 32-chunks of x a warp holds with NB operands each: what the registers take,
  // and what lets three stages of its rows fit a warp's ring.
  template <int NB> static constexpr int kHeld = BITS <= 4 ? 8 / NB : 4;
  // A stage of a warp: its part of 16 rows.  A copied window starts at the 16
  // bytes (codes; rows start at multiples of 4 bytes, of 16 for 4 and 8 bits)
  // or 4 bytes (scales) below the part; pitches spread 8 rows over the banks.
  static constexpr int kCodeBytes = kHeld<1> * 4 * BITS;
  static constexpr int kPitch = 16 * (((kCodeBytes + (BITS == 4 || BITS == 8 ? 0 : 12) + 15) / 16) | 1);
  static constexpr int kScaleBytes = kHeld<1> * 32 / GS * kScaleSize;
  static constexpr int kScaleWords = (kScaleBytes + (FP4 ? 3 : 2) + 3) / 4;
  static constexpr int kScalePitch = (kScaleWords + 1) / 2 * 8;
  static constexpr int kSlot = 16 * kPitch + (FP4 ? 1 : 2) * 16 * kScalePitch;
  static_assert(kPitch <= 9 * 16 && kSlot % 16 == 0, "eight lanes copy a row");
};

template <int OFF>
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1+%2];" : "=r"(v) : "r"(a), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2+%3];" : "=r"(v.x), "=r"(v.y) : "r"(a), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1+%2];" : "=r"(v) : "r"(a), "n"(OFF));
  return v;
}

__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts_f4(uint32_t a, const float4& v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// (v & mask) | magic in one instruction, which takes one constant only: the
// other is kept in a register.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "n"(MASK), "r"(magic));
  return r;
}

template <typename O> struct Op;         // operand type of an mma
template <> struct Op<__half> {
  static constexpr uint32_t kMagic = 0u;                  // q * 2^-24, a subnormal
  static constexpr float kOffset = 0.0f;
  static constexpr uint32_t kOnes = 0x3C003C00u;
  // d = A B + {c0, c1, c2, c3}
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1, float c0,
                                             float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
        " {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  }
};
template <> struct Op<__nv_bfloat16> {
  static constexpr uint32_t kMagic = 0x43004300u;         // 128 + q, q < 128
  static constexpr float kOffset = 128.0f;
  static constexpr uint32_t kOnes = 0x3F803F80u;
  // d = A B + {c0, c1, c2, c3}
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1, float c0,
                                             float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
        " {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  }
};

// What the operand holds beside the code: P' = sum (offset + q) x.  In bf16 codes
// of 8 bits do not fit the 7 bits beside 128 and become q - 128 (exact).
// In fp16 the bits of a code are the subnormal q * 2^-24: no offset.
template <typename O, typename F>
__host__ __device__ constexpr float code_offset() {
  return F::kFp4 ? 0.0f
         : (F::kBits == 8 && std::is_same<O, __nv_bfloat16>::value) ? -128.0f : Op<O>::kOffset;
}
// What the operand's values are multiplied with afterwards (fp16: 2^24, or
// 2^14 for FP4, whose code's bits are those of value * 2^-14).
template <typename O, typename F>
__host__ __device__ constexpr float product_scale() {
  return !std::is_same<O, __half>::value ? 1.0f : F::kFp4 ? 16384.0f : 16777216.0f;
}

template <int BY>
__device__ __forceinline__ uint32_t shifted(uint32_t v) {
  if constexpr (BY >= 0) return v << BY;
  else return v >> -BY;
}
// The operand word of the E2M1 codes at bits AT and AT + 16 of w.
template <typename O, int AT>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w) {
  const uint32_t sign = shifted<12 - AT>(w) & 0x80008000u;
  if constexpr (std::is_same<O, __half>::value) {
    return (shifted<9 - AT>(w) & 0x0E000E00u) | sign;
  } else {
    // bits of value * 2^-126 (subnormals are exact), times 2^126
    const uint32_t v = (shifted<6 - AT>(w) & 0x01C001C0u) | sign;
    const uint32_t k = 0x7E807E80u;
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                     *reinterpret_cast<const __nv_bfloat162*>(&k));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// The four operand words (two mma k-steps of two words) of a thread's 8 codes
// of one row's 32-chunk, OFF bytes after the shared address `at`.
template <typename O, typename F, int OFF>
__device__ __forceinline__ void operand(uint32_t at, int t, uint32_t magic, uint32_t (&r)[4]) {
  if constexpr (F::kOrder == Order::kGroup16) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint32_t w = __byte_perm(g ? lds16<OFF + 8>(at + 2 * t) : lds16<OFF>(at + 2 * t), 0u, 0x4140);
      r[2 * g] = e2m1_pair<O, 0>(w);
      r[2 * g + 1] = e2m1_pair<O, 4>(w);
    }
  } else if constexpr (F::kBits == 4) {
    const uint32_t w = lds32<OFF>(at + 4 * t);
    if constexpr (F::kFp4) {
      r[0] = e2m1_pair<O, 0>(w);
      r[1] = e2m1_pair<O, 4>(w);
      r[2] = e2m1_pair<O, 8>(w);
      r[3] = e2m1_pair<O, 12>(w);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = and_or<0x000F000Fu>(w >> (4 * i), magic);
    }
  } else if constexpr (F::kBits == 2) {
    const uint32_t w = __byte_perm(lds16<OFF>(at + 2 * t), 0u, 0x4140);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = and_or<0x00030003u>(w >> (2 * i), magic);
  } else if constexpr (F::kBits == 8) {
    const uint2 w = lds64<OFF>(at + 8 * t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = i < 2 ? w.x : w.y;
      const uint32_t sel = i & 1 ? 0x4342u : 0x4140u;
      if constexpr (std::is_same<O, __half>::value) {
        r[i] = __byte_perm(v, 0u, sel);
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
    const uint32_t w0 = lds32<OFF>(at + (byte & ~3u)), w1 = lds32<OFF + 4>(at + (byte & ~3u));
    const uint32_t sh = (byte & 3u) * 8u;
    const uint32_t v = __funnelshift_r(w0, w1, sh);
    if constexpr (F::kBits == 3) {
      // codes 0-3 to the low half, 4-7 to the high one
      const uint32_t w = (v & 0x00000FFFu) | ((v << 4) & 0x0FFF0000u);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = and_or<0x00070007u>(w >> (3 * i), magic);
    } else {
      // codes 4-7 in a word of their own, then as many as fit 16 bits and the rest
      constexpr int kHalf = 4 * F::kBits, kFit = F::kBits == 5 ? 3 : 2, kSkip = kFit * F::kBits;
      constexpr uint32_t mask = F::kBits == 5 ? 0x001F001Fu : 0x003F003Fu;
      const uint32_t u = __funnelshift_r(v, w1 >> sh, kHalf);
      const uint32_t a = __byte_perm(v, u, 0x5410), b = __byte_perm(v >> kSkip, u >> kSkip, 0x5410);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r[i] = and_or<mask>(i < kFit ? a >> (F::kBits * i) : b >> (F::kBits * (i - kFit)), magic);
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
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most N of this thread's groups are under way.
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// --------------------------------------------------------------------- plan
struct Plan {
  float weight[kMaxPairs];
  int16_t expert[kMaxPairs];             // of a pair, -1: none
  int16_t rank[kMaxPairs];               // of a pair among its expert's
  int16_t order[kMaxPairs];              // pairs by expert
  int16_t tile_expert[kMaxPairs];
  int16_t tile_first[kMaxPairs + 1];     // into order; the next tile's is its end
  int16_t count[kMaxExperts];
  int16_t first[kMaxExperts];
  int scan[2][kWarps];
  int tiles;
  int wide;                              // tiles have up to 8 pairs, else up to 4
  int abort;
};

// Shared memory: plan, the sums that warps exchange, the ring.
constexpr int kExchangeAt = (int)((sizeof(Plan) + 15) / 16 * 16);
constexpr int kExchangeBytes = 2 * kBatch * kWarps * kExchangeLanes * 16;
constexpr int kRingAt = (kExchangeAt + kExchangeBytes + 127) / 128 * 128;
constexpr int kRingBytes = (227 * 1024 - kRingAt) / kWarps / 16 * 16;   // a warp's

// The CTA arrives at a barrier of the (cooperative, so co-resident) grid, with
// all its writes so far; what does not need the others goes before the wait.
__device__ __forceinline__ void grid_arrive(unsigned* counter) {
  __syncthreads();
  if (threadIdx.x == 0) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(counter) : "memory");
}
// Until every CTA has arrived; false after the time limit.
__device__ __forceinline__ bool grid_wait(unsigned* counter, unsigned ctas, int* abort, uint64_t wait_ns) {
  if (threadIdx.x == 0) {
    const uint64_t t0 = globaltimer_ns();
    for (unsigned it = 1;; ++it) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
      if (v >= ctas) break;
      if ((it & 255u) == 0u && globaltimer_ns() - t0 > wait_ns) {
        *abort = 1;
        break;
      }
    }
  }
  __syncthreads();                       // the acquire holds for the whole CTA
  return *(volatile int*)abort == 0;
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
// Experts per lane: PER, at least E / 32.
template <int PER>
__device__ __forceinline__ void choose_of(const Params& p, Plan& plan, int warp, int lane) {
  const int E = p.a.E, k = p.a.top_k;
  for (int t = warp; t < p.a.T; t += kWarps) {
    double v[PER];
    unsigned long long key[PER];
    double top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = i * 32 + lane;
      v[i] = e < E ? __ldcg(p.logits + t * E + e) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      key[i] = i * 32 + lane < E ? order_key(v[i]) : 0ull;
      nan |= v[i] != v[i];
      top = fmax(top, v[i]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    float sum = 0.0f;
    if (!p.a.normalize) {
#pragma unroll
      for (int i = 0; i < PER; ++i) sum += expf((float)(v[i] - top));
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
    int mine = 0;                                        // lane j holds slot j
    double logit = 0.0;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
      unsigned long long best = key[0];
      double bv = v[0];
      int at = 0;
#pragma unroll
      for (int i = 1; i < PER; ++i)
        if (key[i] > best) {
          best = key[i];
          bv = v[i];
          at = i;
        }
      const unsigned hi = (unsigned)(best >> 32), lo = (unsigned)best;
      const unsigned win_hi = __reduce_max_sync(0xFFFFFFFFu, hi);
      const unsigned ahead = __ballot_sync(0xFFFFFFFFu, hi == win_hi);
      int e;
      if ((ahead & (ahead - 1)) == 0) {                  // one lane has it
        e = __shfl_sync(0xFFFFFFFFu, at * 32 + lane, __ffs(ahead) - 1);
      } else {
        const unsigned win_lo = __reduce_max_sync(0xFFFFFFFFu, hi == win_hi ? lo : 0u);
        const bool wins = hi == win_hi && lo == win_lo;
        e = (int)__reduce_min_sync(0xFFFFFFFFu, wins ? (unsigned)(at * 32 + lane) : 0x7FFFFFFFu);
      }
      const double l = __shfl_sync(0xFFFFFFFFu, bv, e & 31);
      if (lane == j) {
        mine = e;
        logit = l;
      }
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e == i * 32 + lane) key[i] = 0ull;
    }
    const float ex = lane < k ? expf((float)(logit - top)) : 0.0f;
    if (p.a.normalize) {
      sum = ex;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
    if (__any_sync(0xFFFFFFFFu, nan)) sum = NAN;         // shows in every weight
    if (lane < k) {
      const float w = sum != sum ? sum : __fdiv_rn(ex, sum);
      plan.expert[t * k + lane] = (int16_t)mine;
      plan.weight[t * k + lane] = w;
      if (blockIdx.x == 0) {
        p.a.indices[t * k + lane] = mine;
        p.a.weights[t * k + lane] = w;
      }
    }
  }
}
__device__ __forceinline__ void choose(const Params& p, Plan& plan, int warp, int lane) {
  static_assert(kMaxExperts == 512, "experts per lane");
  if (p.a.E <= 64) choose_of<2>(p, plan, warp, lane);
  else if (p.a.E <= 128) choose_of<4>(p, plan, warp, lane);
  else choose_of<16>(p, plan, warp, lane);
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
  // Tiles of up to 8 pairs, or of 4 if that makes few more (their h fits one
  // operand, as hi and lo columns): scanned side by side.
  const int c = tid < E ? plan.count[tid] : 0, both = (c + 7) / 8 | (c + 3) / 4 << 16;
  int sc = c, sn = both;
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
  int bc = 0, bn = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int ac = plan.scan[0][w], an = plan.scan[1][w];
    total += an;
    if (w < warp) {
      bc += ac;
      bn += an;
    }
  }
  const bool wide = (total >> 16) * 8 > (total & 0xFFFF) * 9;
  const int cap = wide ? 8 : 4, shift = wide ? 0 : 16;
  const int c0 = bc + sc - c, n0 = ((bn + sn - both) >> shift) & 0xFFFF, n = (both >> shift) & 0xFFFF;
  if (tid < E) plan.first[tid] = c0;
  for (int j = 0; j < n; ++j) {
    plan.tile_expert[n0 + j] = (int16_t)tid;
    plan.tile_first[n0 + j] = (int16_t)(c0 + cap * j);
  }
  if (tid == kThreads - 1) {
    plan.tiles = (total >> shift) & 0xFFFF;
    plan.tile_first[plan.tiles] = (int16_t)(bc + sc);
    plan.wide = wide;
  }
  __syncthreads();
  for (int q = tid; q < P; q += kThreads) {
    const int e = plan.expert[q];
    if (e >= 0) plan.order[plan.first[e] + plan.rank[q]] = (int16_t)q;
  }
  __syncthreads();
}

// ------------------------------------------------------- gate/up and down
// a / b for 0 <= a < 2^24, b > 0: rounded division, put right by at most one.
__device__ __forceinline__ int quotient(int a, int b) {
  int q = (int)__fdividef((float)a, (float)b);
  const int r = a - q * b;
  return r < 0 ? q - 1 : r >= b ? q + 1 : q;
}

// The row tiles of one phase in a CTA, [m, end), in batches: up to `most`
// neighbouring row tiles of one token tile.
struct Cursor {
  int m, end, blocks, most;
  int tile, rb, nb;                      // token tile, first row tile, row tiles
  __device__ __forceinline__ Cursor(int begin, int e, int bl, int mo)
      : m(begin), end(e), blocks(bl), most(mo) {
    tile = quotient(begin, bl);
    rb = begin - tile * bl;
    size();
  }
  __device__ __forceinline__ void size() { nb = min(min(most, end - m), blocks - rb); }
  __device__ __forceinline__ bool more() const { return m < end; }
  __device__ __forceinline__ void next() {
    m += nb;
    rb += nb;
    if (rb == blocks) {
      rb = 0;
      ++tile;
    }
    size();
  }
};

// PH 1: gate and up (8 rows each) over H; PH 2: down (16 rows) over I.
template <int PH, typename T, typename F>
struct Phase {
  using O = typename std::conditional<PH == 1, T, __nv_bfloat16>::type;
  static constexpr int kGu = F::kGs >= 32 ? F::kGs / 32 : 1;     // chunks per group
  static constexpr int kParts = F::template kHeld<1> / kGu;      // groups held, at most
  // The sums of x over groups of 32 would take 16 registers more than there are:
  // they are made again with each row tile, by an MMA beside the codes'.
  static constexpr bool kSumsInPlace = !F::kFp4 && kParts > 4;
  static constexpr float kOffset = code_offset<O, F>();
  static constexpr float kScale = product_scale<O, F>();

  static constexpr int kRows = PH == 1 ? 8 : 16;         // rows of a matrix in a row tile
  static constexpr int kSlots = kRingBytes / F::kSlot < 6 ? kRingBytes / F::kSlot : 6;
  static_assert(kSlots >= 3, "ring");
  static constexpr uint32_t kBuffer = kBatch * kWarps * kExchangeLanes * 16;

  const Params& p;
  const Plan& plan;
  const uint32_t ring;                   // shared address, of the warp's
  const int warp, lane, g, t;
  uint32_t magic;                        // the operand's bits beside a code
  int K, chunks, blocks, row_bytes, scale_row;
  int held;                              // chunks of x a warp holds
  int shift, lt, team;                   // log2 of the warps of a team, of the teams
  int pass_chunks, passes;
  Cursor done;                           // batch to compute
  int turn;                              // batches computed
  uint32_t at, aat;                      // slots to read, to fill
  // the next stage to copy: token tile, the team's row tile (of `aend`), pass
  // and row tile of the batch; addresses and bytes from there on
  int atile, arb, aend, apass, ai;
  const uint8_t *pc, *ps;
  int csize, ssize;
  int tile;                              // whose x is held
  int first, count;                      // its pairs
  bool fresh;                            // it is still on its way
  // what a thread does the same way in every stage
  int from, n;                           // the warp's chunks of a pass
  const uint8_t *csrc, *ssrc;            // what it copies: codes, scales
  int64_t other;                         // from gate's to up's codes
  int cstep, sstep;                      // to the team's next row tile
  bool wide;                             // scales are copied 8 bytes at a time
  uint32_t cdst, sdst;
  uint32_t woff, soff;                   // row g's codes and scales in a slot
  uint32_t own, others;                  // where it puts sums, and gets them to add
  int jtile, jcol, jrow;                 // the sums it adds: row tile, column, row

  static __device__ __forceinline__ int blocks_of(const Params& p) {
    return PH == 1 ? p.a.I / 8 : p.a.H / 16;
  }
  // Where the share of the CTA with this fraction (of 2^32) of the grid before
  // it begins.
  static __device__ __forceinline__ int border(const Params& p, const Plan& plan, unsigned share) {
    return (int)__umulhi((unsigned)(plan.tiles * blocks_of(p)), share);
  }
  // log2 of the teams: as few warps to a team as hold K, but no more teams than
  // pairs of row tiles.
  static __device__ __forceinline__ int teams_of(int chunks, int held, int tiles) {
    int lt = chunks <= 2 * held ? 3 : chunks <= 4 * held ? 2 : chunks <= 8 * held ? 1 : 0;
    while (lt > 0 && tiles <= 1 << lt) --lt;
    return lt;
  }

  __device__ __forceinline__ Phase(const Params& pp, const Plan& pl, uint32_t ri, uint32_t exchange,
                                   int w, int ln, int begin, int end)
      : p(pp), plan(pl), ring(ri), warp(w), lane(ln), g(ln >> 2), t(ln & 3),
        K(PH == 1 ? pp.a.H : pp.a.I), chunks(K / 32), blocks(blocks_of(pp)),
        held(PH == 2 && pl.wide ? F::template kHeld<2> : F::template kHeld<1>),
        lt(teams_of(chunks, held, end - begin)), done(begin, end, blocks, kBatch << lt) {
    asm volatile("mov.b32 %0, %1;" : "=r"(magic) : "n"(Op<O>::kMagic));   // not a constant, see and_or
    shift = 4 - lt;
    team = warp >> shift;
    row_bytes = chunks * 4 * F::kBits;
    scale_row = K / F::kGs * F::kScaleSize;
    pass_chunks = held << shift;
    const int log = shift + (held == 8 ? 3 : 2);
    passes = (chunks + pass_chunks - 1) >> log;
    apass = ai = turn = 0;
    at = aat = ring;
    tile = -1;
    fresh = false;
    place(0, from, n);
    {
      // codes: eight lanes to a row, four rows at a time; scales and biases: a
      // lane to a row of each
      const int row = lane >> 3, srow = lane & 15, arr = F::kFp4 ? 0 : lane >> 4;
      csrc = (PH == 2 ? p.a.down : p.a.gate).w_q + row * row_bytes + (lane & 7) * 16;
      cdst = row * F::kPitch + (lane & 7) * 16;
      other = PH == 1 ? p.a.up.w_q - p.a.gate.w_q : 8 * (int64_t)row_bytes;
      const MoeMatrix& m = PH == 2 ? p.a.down : srow < 8 ? p.a.gate : p.a.up;
      ssrc = (arr ? m.biases : m.scales) + (PH == 1 ? srow & 7 : srow) * scale_row;
      sdst = 16 * F::kPitch + (arr * 16 + srow) * F::kScalePitch;
      cstep = (kRows << lt) * row_bytes;
      sstep = (kRows << lt) * scale_row;
    }
    settle();
    atile = done.tile;
    arb = done.rb + team;
    aend = min(blocks, end - atile * blocks);
    open();
    own = exchange + (warp * kExchangeLanes + lane) * 16;
    {
      // 64 pairs of numbers per row tile, each by 4 / teams lanes (one from 4
      // teams on) that add up to four warps' each
      const int spread = max(2 - lt, 0), item = (warp << (5 - spread)) + (lane >> spread);
      const int src = (item >> 1) & 31, part = lane & ((1 << spread) - 1);
      jtile = item >> 6;
      jcol = 2 * (src & 3) + (item & 1);
      jrow = src >> 2;
      const int first_warp = (jtile >> lt) * kWarps + ((jtile & ((1 << lt) - 1)) << shift) + part * 4;
      others = exchange + (first_warp * kExchangeLanes + src) * 16 + (item & 1) * 8;
      if (part) jtile |= 64;             // adds, but does not store
    }
  }

  // The warp's chunks of a pass: whole groups.
  __device__ __forceinline__ void place(int pass, int& from_, int& n_) const {
    const int member = warp & ((1 << shift) - 1);
    const int left = min(pass_chunks, chunks - pass * pass_chunks);
    const int per = ((left / kGu + (1 << shift) - 1) >> shift) * kGu;
    from_ = member * per;
    n_ = max(0, min(per, left - from_));
  }
  // Bytes from a row's start to the warp's part of it.
  __device__ __forceinline__ int code_at(int pass, int from_) const {
    return (pass * pass_chunks + from_) * 4 * F::kBits;
  }
  __device__ __forceinline__ int scale_at(int pass, int from_) const {
    return (pass * pass_chunks + from_) * 32 / F::kGs * F::kScaleSize;
  }
  // Where a thread finds row g (row g + 8 starts as far into its window).
  __device__ __forceinline__ void settle(int pass = 0) {
    woff = g * F::kPitch + ((uint32_t)(g * row_bytes + code_at(pass, from)) & 15u);
    soff = 16 * F::kPitch + g * F::kScalePitch + ((uint32_t)(g * scale_row + scale_at(pass, from)) & 3u);
  }

  // First row, in a stack, of a row tile.
  __device__ __forceinline__ int row0(int tl, int rb) const {
    return plan.tile_expert[tl] * (PH == 1 ? p.a.I : p.a.H) + rb * kRows;
  }
  // Row tile j of a batch is team j % teams'; a team has up to kBatch.
  __device__ __forceinline__ int mine(const Cursor& c) const {
    return min(kBatch, (c.nb - team + (1 << lt) - 1) >> lt);
  }

  // Move on to a token tile where the team has a row tile, if there is one.
  __device__ __forceinline__ void open() {
    while (arb >= aend && (atile + 1) * blocks < done.end) {
      ++atile;
      arb = team;
      aend = min(blocks, done.end - atile * blocks);
    }
    if (arb < aend) aim();
  }
  // Addresses of the stage: a row need not be aligned, the copy takes the
  // aligned window around the warp's part (a stack ends on a multiple of 16
  // bytes).
  __device__ __forceinline__ void aim() {
    int f = from, m = n;
    if (passes > 1) place(apass, f, m);
    const int row = row0(atile, arb + (ai << lt));
    const int off = code_at(apass, f), skew = ((lane >> 3) * row_bytes + off) & 15;
    pc = csrc + ((int64_t)row * row_bytes + (off - skew));
    csize = m > 0 ? skew + m * 4 * F::kBits - (lane & 7) * 16 : 0;
    ps = ssrc + ((int64_t)row * scale_row + scale_at(apass, f));
    ssize = F::kFp4 && lane >= 16 ? 0 : m * 32 / F::kGs * F::kScaleSize;
    wide = F::kScaleBytes % 8 == 0 && (scale_row | scale_at(apass, f)) % 8 == 0;
    if (!wide) {
      const int sk = (int)(reinterpret_cast<uintptr_t>(ps) & 3);
      ps -= sk;
      if (ssize) ssize += sk;
    }
  }

  // Start the copies of the warp's next stage: its part of a row tile.
  __device__ __forceinline__ void issue() {
    if (arb < aend) {
      if (csize > 0) {
        const uint32_t dst = aat + cdst;
        const uint8_t* far = pc + other;
        cp_async<16>(dst, pc);
        cp_async<16>(dst + 4 * F::kPitch, pc + 4 * row_bytes);
        cp_async<16>(dst + 8 * F::kPitch, far);
        cp_async<16>(dst + 12 * F::kPitch, far + 4 * row_bytes);
      }
      const uint32_t dst = aat + sdst;
      if (wide) {
#pragma unroll
        for (int u = 0; u < F::kScaleBytes; u += 8)
          if (u < ssize) cp_async<8>(dst + u, ps + u);
      } else {
#pragma unroll
        for (int u = 0; u < 4 * F::kScaleWords; u += 4)
          if (u < ssize) cp_async<4>(dst + u, ps + u);
      }
      aat = next(aat);
      if (passes == 1) {
        arb += 1 << lt;
        pc += cstep;
        ps += sstep;
        if (arb >= aend) open();
      } else {
        if (++ai == kBatch || arb + (ai << lt) >= aend) {
          ai = 0;
          if (++apass == passes) {
            apass = 0;
            arb += kBatch << lt;
          }
        }
        if (arb >= aend) open();
        else aim();
      }
    }
    cp_commit();
  }
  __device__ __forceinline__ uint32_t next(uint32_t slot) const {
    return slot == ring + (kSlots - 1) * F::kSlot ? ring : slot + F::kSlot;
  }
  __device__ __forceinline__ void start() {
#pragma unroll 1
    for (int i = 0; i < kSlots - 1; ++i) issue();
  }

  // x (or h) of this thread's column for the warp's chunks of a pass, in the
  // operand's order, and the sums of x over each group.  h is hi + lo: with up
  // to 4 pairs in a tile columns 0-3 hold the hi parts and 4-7 the lo parts of
  // one operand, else hi and lo are two operands.
  uint4 xv[F::template kHeld<PH> * PH];                       // of chunk c, operand b: c * NB + b
  float sum[kSumsInPlace ? 1 : kParts][2];

  template <int NB>
  __device__ __forceinline__ void load(int chunk) {
    const uint8_t* col = nullptr;
    const int at = PH == 2 && NB == 1 ? g & 3 : g;
    if (at < count) {
      const int pair = plan.order[first + at];
      col = PH == 1 ? static_cast<const uint8_t*>(p.a.x) + (int64_t)(pair / p.a.top_k) * K * 2
                    : p.h + (int64_t)pair * K * 4 + (NB == 1 ? (g >> 2) * 16 : 0);
    }
#pragma unroll
    for (int c = 0; c < F::template kHeld<NB>; ++c) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (col && c < n) {
          if constexpr (PH == 1 && F::kOrder == Order::kGroup16) {
            const uint2* q = reinterpret_cast<const uint2*>(col + (int64_t)(chunk + c) * 64) + t;
            const uint2 lo = __ldg(q), hi = __ldg(q + 4);
            v = make_uint4(lo.x, lo.y, hi.x, hi.y);
          } else if constexpr (PH == 1) {
            v = __ldg(reinterpret_cast<const uint4*>(col + (int64_t)(chunk + c) * 64) + t);
          } else {
            v = __ldcg(reinterpret_cast<const uint4*>(col + (int64_t)(chunk + c) * 128) + 2 * t + b);
          }
        }
        xv[c * NB + b] = v;
      }
    }
  }
  // What there is to do with it once it has come.
  template <int NB>
  __device__ __forceinline__ void prepare() {
#pragma unroll
    for (int k = 0; k < F::template kHeld<NB> / kGu; ++k) {
      float S[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = k * kGu; c < (k + 1) * kGu; ++c) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if constexpr (PH == 1) xv[c * NB + b] = order_x<F>(xv[c * NB + b]);
          if constexpr (!F::kFp4 && !kSumsInPlace) {
            const uint4& v = xv[c * NB + b];
            constexpr uint32_t one = Op<O>::kOnes;
            Op<O>::mma(S, one, one, one, one, v.x, v.y, S[0], S[1], S[2], S[3]);
            Op<O>::mma(S, one, one, one, one, v.z, v.w, S[0], S[1], S[2], S[3]);
          }
        }
      }
      if constexpr (!kSumsInPlace) {
        sum[k][0] = S[0] * (1.0f / kScale);
        sum[k][1] = S[1] * (1.0f / kScale);
      }
    }
  }

  template <int OFF>
  static __device__ __forceinline__ float scale_in(uint32_t at) {
    uint32_t b;
    if constexpr (F::kFp4) {
      asm volatile("ld.shared.u8 %0, [%1+%2];" : "=r"(b) : "r"(at), "n"(OFF));
      if constexpr (F::kGs == 16) {
        // E4M3 values are exact in both T
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
        return __half2float(__ushort_as_half((unsigned short)h));
      } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        return e8m0_to_float(b);                         // exact in bf16
      } else {
        return fp4_scale_t<T>(b, F::kGs);
      }
    } else {
      asm volatile("ld.shared.u16 %0, [%1+%2];" : "=r"(b) : "r"(at), "n"(OFF));
      if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(b << 16);
      else return __half2float(__ushort_as_half((unsigned short)b));
    }
  }

  // Sums of a row tile over the warp's N chunks (0: n of them): rows g (tot 0,
  // 1) and g + 8 (2, 3), columns 2 t and 2 t + 1.  `w`, `s`: row g's codes and
  // scales.
  template <int NB, int N, int C = 0>
  __device__ __forceinline__ void multiply(float (&tot)[4], float (&P)[4], uint32_t w, uint32_t s) {
    constexpr int k = C / kGu, kHigh = 8 * F::kScalePitch, kBias = 16 * F::kScalePitch;
    if constexpr (N == 0 && C % kGu == 0)
      if (C >= n) return;
    uint32_t lo[4], hi[4];
    operand<O, F, C * 4 * F::kBits>(w, t, magic, lo);
    operand<O, F, C * 4 * F::kBits + 8 * F::kPitch>(w, t, magic, hi);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4& v = xv[C * NB + b];
        const bool begin = b == 0 && (F::kGs == 16 || (half == 0 && C % kGu == 0));
        Op<O>::mma(P, lo[2 * half], hi[2 * half], lo[2 * half + 1], hi[2 * half + 1],
                   half ? v.z : v.x, half ? v.w : v.y, begin ? 0.0f : P[0], begin ? 0.0f : P[1],
                   begin ? 0.0f : P[2], begin ? 0.0f : P[3]);
      }
      if (F::kGs == 16 || (half == 1 && (C + 1) % kGu == 0)) {
        constexpr int o = F::kGs == 16 ? 2 * C : k * F::kScaleSize;
        const float sl = F::kGs == 16 && half ? scale_in<o + 1>(s) : scale_in<o>(s);
        const float sh = F::kGs == 16 && half ? scale_in<kHigh + o + 1>(s) : scale_in<kHigh + o>(s);
        tot[0] = fmaf(sl, P[0], tot[0]);
        tot[1] = fmaf(sl, P[1], tot[1]);
        tot[2] = fmaf(sh, P[2], tot[2]);
        tot[3] = fmaf(sh, P[3], tot[3]);
        if constexpr (!F::kFp4) {
          // the offset of the operand comes off with the bias
          const float bl = fmaf(-kOffset, sl, scale_in<kBias + o>(s));
          const float bh = fmaf(-kOffset, sh, scale_in<kBias + kHigh + o>(s));
          float x0, x1;
          if constexpr (kSumsInPlace) {
            // ones times 1 / kScale: 2^-24 is fp16's smallest number
            constexpr uint32_t one = kScale == 1.0f ? Op<O>::kOnes : 0x00010001u;
            float S[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const uint4& v = xv[C * NB + b];
              Op<O>::mma(S, one, one, one, one, v.x, v.y, S[0], S[1], S[2], S[3]);
              Op<O>::mma(S, one, one, one, one, v.z, v.w, S[0], S[1], S[2], S[3]);
            }
            x0 = S[0];
            x1 = S[1];
          } else {
            x0 = sum[k][0];
            x1 = sum[k][1];
          }
          tot[0] = fmaf(bl, x0, tot[0]);
          tot[1] = fmaf(bl, x1, tot[1]);
          tot[2] = fmaf(bh, x0, tot[2]);
          tot[3] = fmaf(bh, x1, tot[3]);
        }
      }
    }
    if constexpr (C + 1 < (N ? N : F::template kHeld<NB>)) multiply<NB, N, C + 1>(tot, P, w, s);
  }
  template <int NB>
  __device__ __forceinline__ void products(float (&tot)[4]) {
    constexpr int kFull = F::template kHeld<NB>, kMost = kFull * 3 / 4;
    const uint32_t w = at + woff, s = at + soff;
    float P[4];
    if (n == kFull) multiply<NB, kFull>(tot, P, w, s);
    else if (kMost % kGu == 0 && n == kMost) multiply<NB, kMost % kGu == 0 ? kMost : kFull>(tot, P, w, s);
    else multiply<NB, 0>(tot, P, w, s);
  }

  // The sums of a batch (its first row tile and how many, its pairs) over the
  // warps of each team.
  __device__ __forceinline__ void join(int rb, int nb, int first, int count) {
#pragma unroll 1
    for (int i = 0; i < kBatch && i << lt < nb; i += lt == 3 ? 1 : 2) {
      const int jt = jtile + (i << lt);
      const bool live = (jt & 63) < nb;
      float a = 0.0f, b = 0.0f;
      if (live) {
        const uint32_t o = others + (turn & 1) * kBuffer + i * (kWarps * kExchangeLanes * 16);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (lt == 3 && m >= 2) break;
          const float2 v = lds_f2(o + m * (kExchangeLanes * 16));
          a += v.x;
          b += v.y;
        }
      }
      if (lt < 2) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, 1);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, 1);
        if (lt < 1) {
          a += __shfl_xor_sync(0xFFFFFFFFu, a, 2);
          b += __shfl_xor_sync(0xFFFFFFFFu, b, 2);
        }
      }
      if (PH == 2 && count <= 4) {                       // columns of hi and lo
        a += __shfl_down_sync(0xFFFFFFFFu, a, max(16 >> lt, 4));
        b += __shfl_down_sync(0xFFFFFFFFu, b, max(16 >> lt, 4));
      }
      if (jt < nb && jcol < count) store(a, b, plan.order[first + jcol], rb + jt, jrow);
    }
  }

  // A pair of sums: (gate, up) of one h, or rows g and g + 8 of down's result.
  __device__ __forceinline__ void store(float a, float b, int pair, int rb, int gg) const {
    if constexpr (PH == 1) {
      const float h = __fdividef(a, 1.0f + expf(-a)) * b;
      const __nv_bfloat16 hi = __float2bfloat16_rn(h);
      const float rest = h - __bfloat162float(hi);
      // an infinity or NaN is kept by the first part alone
      const __nv_bfloat16 lo = __float2bfloat16_rn(fabsf(rest) <= 3.0e38f ? rest : 0.0f);
      uint8_t* dst = p.h + (int64_t)pair * p.a.I * 4 + h_offset<F>(rb * 8 + gg);
      *reinterpret_cast<__nv_bfloat16*>(dst) = hi;
      *reinterpret_cast<__nv_bfloat16*>(dst + 16) = lo;
    } else {
      float* dst = p.part + (int64_t)pair * p.a.H + rb * 16 + gg;
      dst[0] = a;
      dst[8] = b;
    }
  }

  // Ask for the batch's x: it comes while the warp waits for its copies.
  __device__ __forceinline__ void fetch(int pass) {
    if (!done.more()) return;
    tile = done.tile;
    first = plan.tile_first[tile];
    count = plan.tile_first[tile + 1] - first;
    if (passes > 1) {
      place(pass, from, n);
      settle(pass);
    }
    if (PH == 2 && count > 4) load<PH>(pass * pass_chunks + from);
    else load<1>(pass * pass_chunks + from);
    fresh = true;
  }

  // A warp waits for its own copies only, and all meet once per batch: the
  // barrier publishes the batch's sums, and the buffer of the batch after next
  // is written by warps past the next barrier.
  __device__ __forceinline__ void run() {
    while (done.more()) {
      const int nb = mine(done);
      for (int pass = 0; pass < passes; ++pass) {
        if (done.tile != tile || passes > 1) fetch(pass);
        uint32_t to = own + (turn & 1) * kBuffer;
        for (int i = 0; i < nb; ++i) {
          cp_wait<kSlots - 2>();
          __syncwarp();
          issue();
          if (fresh) {
            fresh = false;
            if (PH == 2 && count > 4) prepare<PH>();
            else prepare<1>();
          }
          float tot[4] = {0.f, 0.f, 0.f, 0.f};
          if (PH == 2 && count > 4) products<PH>(tot);
          else products<1>(tot);
          at = next(at);
          float4 v = make_float4(tot[0], tot[2], tot[1], tot[3]);
          if constexpr (kScale != 1.0f) {
            v.x *= kScale;
            v.y *= kScale;
            v.z *= kScale;
            v.w *= kScale;
          }
          if (pass) {
            const float4 o = lds_f4(to);
            v.x += o.x;
            v.y += o.y;
            v.z += o.z;
            v.w += o.w;
          }
          sts_f4(to, v);
          to += kWarps * kExchangeLanes * 16;
        }
      }
      const int rb = done.rb, nt = done.nb, of = first, pairs = count;
      done.next();
      if (done.tile != tile && passes == 1) fetch(0);    // the next x comes meanwhile
      __syncthreads();
      join(rb, nt, of, pairs);
      ++turn;
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
#pragma unroll 8
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
  extern __shared__ __align__(128) uint8_t smem[];
  Plan& plan = *reinterpret_cast<Plan*>(smem);
  // the shuffle tells the compiler that the warp's number is uniform
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t exchange = smem_u32(smem) + kExchangeAt;
  const uint32_t ring = smem_u32(smem) + kRingAt + warp * kRingBytes;
  if (threadIdx.x == 0) {
    plan.abort = 0;
    if (p.delay_ns && blockIdx.x == 0) {                 // test hook
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < p.delay_ns) {
      }
    }
  }

  // The grid's row tiles are cut at these fractions of 2^32 (the last CTA ends
  // with the last tile).
  const unsigned step = 0xFFFFFFFFu / gridDim.x;
  const unsigned share = step * blockIdx.x;
  const bool last = blockIdx.x == gridDim.x - 1;

  bool ok = true;
  if (p.a.w_router) {
    router_logits<T>(p, warp, lane);
    grid_arrive(p.bars + 0);
    ok = grid_wait(p.bars + 0, gridDim.x, &plan.abort, p.wait_ns);
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
    using Down = Phase<2, T, F>;
    {
      using Up = Phase<1, T, F>;
      Up up(p, plan, ring, exchange, warp, lane, Up::border(p, plan, share),
            last ? plan.tiles * Up::blocks_of(p) : Up::border(p, plan, share + step));
      up.fetch(0);
      up.start();
      up.run();
    }
    grid_arrive(p.bars + 1);             // h is written
    Down down(p, plan, ring, exchange, warp, lane, Down::border(p, plan, share),
              last ? plan.tiles * Down::blocks_of(p) : Down::border(p, plan, share + step));
    down.start();
    ok = grid_wait(p.bars + 1, gridDim.x, &plan.abort, p.wait_ns);
    if (ok) {
      down.run();
      grid_arrive(p.bars + 2);
      ok = grid_wait(p.bars + 2, gridDim.x, &plan.abort, p.wait_ns);
      if (ok) weighted_sums<T>(p, plan);
    }
  }
  cp_wait<0>();
  if (threadIdx.x == 0) {
    // Every CTA comes by here, one that gave up too: the last leaves the counters
    // at zero, so that a time-out does not spoil the calls to come.  Who has
    // passed all barriers has seen all arrivals; the fences order those of CTAs
    // that gave up before the zeros.
    if (!ok) {
      atomicOr(p.error, 1u);
      __threadfence();
    }
    if (atomicAdd(p.bars + 3, 1u) == gridDim.x - 1) {
      if (!ok) __threadfence();
      p.bars[0] = p.bars[1] = p.bars[2] = p.bars[3] = 0u;
    }
  }
}

// -------------------------------------------------------------------- host
template <typename T, typename F>
cudaError_t launch(const Params& p, int sms, cudaStream_t st) {
  auto kern = moe_kernel<T, F>;
  static std::atomic<bool> attr_done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr_done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingAt + kWarps * kRingBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kRingAt + kWarps * kRingBytes;
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
