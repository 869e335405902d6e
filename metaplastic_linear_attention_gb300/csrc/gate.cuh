// Shared by the gated scan's kernels (gate_fwd.cu, gate_bwd.cu): the tile they work on,
// and its gates.
#pragma once

#include <cooperative_groups.h>

#include "ssm.cuh"

namespace palimpsa {

constexpr int kPiece = kGateCheckpoint;  // tokens that a group of threads holds
constexpr int kGateCluster = 12;         // CTAs of a cluster, at most

// A tile of CH channels by a piece of tokens for each of the CTA's groups of threads, CPT
// channels a thread.
template <bool BF16, int CH_, int CPT, int THREADS>
struct GateTile {
  static constexpr int ES = BF16 ? 2 : 4, CH = CH_;
  static constexpr int group = CH / CPT, pieces = THREADS / group, threads = THREADS;
  static constexpr int tokens = kPiece * pieces;
  static constexpr int row = CH * ES;                 // bytes of a row
  static constexpr int bytes = tokens * row;          // of an array
  static constexpr int vecs = row / 16;               // 16-byte vectors of a row
  static constexpr int rows_at_once = threads / vecs; // rows that the CTA's threads copy in turn
  static_assert(tokens % rows_at_once == 0, "whole turns");
};

// How a batch is shared out: channels of a tile, and CTAs along time (a cluster's).
struct GatePlan {
  int channels, cluster;
  double us;  // the time that the model gives
};
struct GateCost {
  double round, cta, ends, hop;  // see gate_plan
};
// `tokens` of a CTA's tile of 64 channels (twice as many at `narrow`, the least channels of a tile),
// `resident` CTAs on an SM.
GatePlan gate_plan(const SeqRows& r, int D, int tokens, int resident, int narrow, const GateCost& c);
// Whether the batch's sequences are better walked by a thread (or a warp) each, `rate` channel-tokens a
// microsecond, than in tiles with plan p.
bool gate_short(const SeqRows& r, int D, const GatePlan& p, double rate);

#if defined(__CUDACC__)

__device__ __forceinline__ float fmin_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two neighbouring channels of the input type.
template <bool BF16>
__device__ __forceinline__ float2 load_pair(const void* p) {
  if constexpr (BF16) {
    const uint32_t u = *static_cast<const uint32_t*>(p);
    return make_float2(bf16_lo(u), bf16_hi(u));
  } else {
    return *static_cast<const float2*>(p);
  }
}
template <bool BF16>
__device__ __forceinline__ float2 read_pair(const void* p) {  // of what the kernel does not write
  if constexpr (BF16) {
    const uint32_t u = __ldg(static_cast<const unsigned int*>(p));
    return make_float2(bf16_lo(u), bf16_hi(u));
  } else {
    return __ldg(static_cast<const float2*>(p));
  }
}
template <bool BF16>
__device__ __forceinline__ void store_pair(void* p, float2 v) {
  if constexpr (BF16) *static_cast<uint32_t*>(p) = Vec<true>::two(v.x, v.y);
  else *static_cast<float2*>(p) = v;
}

__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 + e^-u and sigmoid(u) = 1 / (1 + e^-u), from x = -log2(e) u.
__device__ __forceinline__ float2 one_plus(float2 x) {
  return __fadd2_rn(make_float2(ex2_approx(x.x), ex2_approx(x.y)), make_float2(1.f, 1.f));
}
__device__ __forceinline__ float2 sigmoid_of(float2 x) {
  const float2 w = one_plus(x);
  return make_float2(rcp_approx(w.x), rcp_approx(w.y));
}
// The same with 1 - sigmoid(u) = e sigmoid(u), e = e^-u, which does not cancel. e is kept below
// 2^126, so that both stay finite (and sigmoid above 2^-127).
__device__ __forceinline__ float2 sigmoid_of(float2 x, float2* rest) {
  x = make_float2(fmin_nan(x.x, 126.f), fmin_nan(x.y, 126.f));
  const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
  const float2 w = __fadd2_rn(e, make_float2(1.f, 1.f));
  const float2 p = make_float2(rcp_approx(w.x), rcp_approx(w.y));
  *rest = __fmul2_rn(e, p);
  return p;
}

// The decay a = e^-w of a rate w >= 0 and 1 - a^2 = (1 - a)(1 + a). Slow channels have w of
// 1e-3 and below, where 1 - a from a rounded a has lost its digits, and a state of a long
// memory gathers a's own error over the tokens it remembers. So below 0.3 both come from
// m = 1 - a = w phi(w), with phi = (1 - e^-w) / w by the polynomial of degree 4 that is
// closest to it over [0, 0.3] (found by an exchange of its extrema; 6e-9 off at most). Above,
// a is the SFU's 2^x and 1 - a > 0.25 does not cancel. (1 - a^2 is kept at 4e-38 and above, a
// normal number, so that its root has a reciprocal.)
// left: what the rounding of a leaves out, (1 - m) - a exactly. It is up to 3e-8 of the state a token, the
// same way at every token where gates hardly change, 1e-3 over 32768 of them: so a state that is handed on
// from token to token, or from tile to tile, is a h + (left h + b).
__device__ __forceinline__ void decay_of(float2 w, float2* a, float2* rest, float2* left) {
  float2 m = make_float2(0.00735594891f, 0.00735594891f);
  m = __ffma2_rn(m, w, make_float2(-0.0414141268f, -0.0414141268f));
  m = __ffma2_rn(m, w, make_float2(0.166639641f, 0.166639641f));
  m = __ffma2_rn(m, w, make_float2(-0.499998987f, -0.499998987f));
  m = __ffma2_rn(m, w, make_float2(1.f, 1.f));
  m = __ffma2_rn(m, w, make_float2(2e-38f, 2e-38f));
  const float2 u = __fmul2_rn(w, make_float2(-kLog2e, -kLog2e));
  const float2 e = make_float2(ex2_approx(u.x), ex2_approx(u.y));
  const float2 far = __ffma2_rn(e, make_float2(-1.f, -1.f), make_float2(1.f, 1.f));
  const float2 near = __ffma2_rn(m, make_float2(-1.f, -1.f), make_float2(1.f, 1.f));
  const bool lx = w.x < 0.3f, ly = w.y < 0.3f;
  m = make_float2(lx ? m.x : far.x, ly ? m.y : far.y);
  *a = make_float2(lx ? near.x : e.x, ly ? near.y : e.y);
  *rest = __ffma2_rn(m, *a, m);
  *left = __fadd2_rn(__fadd2_rn(make_float2(1.f, 1.f), make_float2(-a->x, -a->y)), make_float2(-m.x, -m.y));
}
__device__ __forceinline__ void decay_of(float2 w, float2* a, float2* rest) {
  float2 left;
  decay_of(w, a, rest, &left);
}
// left h + b; b where h is infinite, so that an infinite state stays what a makes of it.
__device__ __forceinline__ float2 with_left(float2 left, float2 h, float2 b) {
  const float2 t = __ffma2_rn(left, h, b);
  return make_float2(fabsf(h.x) <= 3.4028235e38f ? t.x : b.x, fabsf(h.y) <= 3.4028235e38f ? t.y : b.y);
}
// sqrt(rest) x, from rest = 1 - a^2, and with the input gate p. In this order no product leaves fp32's
// range where the result does not.
__device__ __forceinline__ float2 input_of(float2 rest, float2 x) {
  return __fmul2_rn(__fmul2_rn(rest, make_float2(rsqrt_approx(rest.x), rsqrt_approx(rest.y))), x);
}
__device__ __forceinline__ float2 input_of(float2 rest, float2 p, float2 x) { return __fmul2_rn(input_of(rest, x), p); }
// The same from q = 1 + e^-u, for u >= kOpenGate: one reciprocal root for the root and the gate's quotient, as long
// as q^2 is finite. (A reciprocal for each gate instead takes 8 x 4096 x 1536 from 77 to 84 us, and looking
// for gates that are all but shut 77 to 79.)
constexpr float kOpenGate = -42.f;
__device__ __forceinline__ float2 open_input_of(float2 rest, float2 q, float2 x) {
  const float2 v = __fmul2_rn(__fmul2_rn(rest, q), q);
  return __fmul2_rn(__fmul2_rn(rest, make_float2(rsqrt_approx(v.x), rsqrt_approx(v.y))), x);
}

// The address of a shared object in another CTA of the cluster, 16 or 8 bytes stored there, counted
// on a barrier of that CTA, and the wait for them.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_async(uint32_t to, const float4& v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void st_async(uint32_t to, const float2& v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to),
               "f"(v.x), "f"(v.y), "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool cluster_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// false where the wait ran out.
__device__ __forceinline__ bool cluster_wait(uint64_t* bar, uint32_t parity, unsigned long long timeout_ns) {
  if (cluster_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (;;) {
    for (int i = 0; i < 64; ++i)
      if (cluster_try_wait(bar, parity)) return true;
    if (global_ns() - t0 >= timeout_ns) return cluster_try_wait(bar, parity);
  }
}
// Tests: until the others' waits have run out.
__device__ __forceinline__ void pass_the_limit(const GateArgs& a) {
  const unsigned long long t0 = global_ns(), late = 4 * min(a.wait_timeout_ns, 250000000ull) + 20000000ull;
  while (global_ns() - t0 < late) __nanosleep(1000);
}
// The end of a ring. An asynchronous store is seen to have landed by its barrier alone, not by a
// barrier of the cluster. A CTA whose waits have all held has seen every one of its states. Where a wait
// has run out, one that was merely late may still be under way; so each CTA tells the next one for how
// many rounds it has sent a state, and after the cluster's barrier, when no more are sent, the CTA's
// first thread waits (2 s at most) for those beyond the `good` rounds that it has seen. (Where the waits
// of some only of the threads that send a state have run out, the others have sent their parts, and these make
// up for theirs before they tell. A ring that breaks leaves two such states at most, one of them in a
// round for whose bytes this thread has not yet arrived.)
__device__ __forceinline__ void settle(uint64_t* bars, int good, int told, uint32_t bytes) {
  for (int k = good; k < told; ++k) {
    if (k > good) mbar_arrive_expect_tx(&bars[k & 1], bytes);
    if (!cluster_wait(&bars[k & 1], (k >> 1) & 1, 2000000000ull)) return;
  }
}

__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// Two neighbouring channels' parameters, or a value in their place.
__device__ __forceinline__ float2 pair_or(const float* p, int ch, bool in, float otherwise) {
  return p && in ? make_float2(p[ch], p[ch + 1]) : make_float2(otherwise, otherwise);
}

#endif

// f<BF16, with an input gate, with an output gate>(...)
#define PALIMPSA_GATE_DISPATCH(f, ...)                                                                            \
  if (a.bf16)                                                                                                     \
    return a.i ? (a.z ? f<true, true, true>(__VA_ARGS__) : f<true, true, false>(__VA_ARGS__))                     \
               : (a.z ? f<true, false, true>(__VA_ARGS__) : f<true, false, false>(__VA_ARGS__));                  \
  return a.i ? (a.z ? f<false, true, true>(__VA_ARGS__) : f<false, true, false>(__VA_ARGS__))                     \
             : (a.z ? f<false, false, true>(__VA_ARGS__) : f<false, false, false>(__VA_ARGS__));

}  // namespace palimpsa
