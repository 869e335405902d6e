// Shared by the gated scan's kernels (gate_fwd.cu, gate_bwd.cu): the tile they work on,
// and its gates.
#pragma once

#include <cooperative_groups.h>

#include "ssm.cuh"

namespace palimpsa {

// A tile is 64 channels (a lane holds two, a warp a row of them) by 8 tokens for each of
// the CTA's warps; the 8 tokens of a warp are a piece. 8 warps in bf16, 4 in fp32, whose
// rows are twice as long.
constexpr int kPiece = kGateCheckpoint;
constexpr int kGateChannels = 64;
constexpr int kGateCluster = 8;  // CTAs of a cluster, at most (the portable limit)

template <bool BF16>
struct GateTile {
  static constexpr int ES = BF16 ? 2 : 4;
  static constexpr int warps = BF16 ? 8 : 4;
  static constexpr int threads = 32 * warps;
  static constexpr int tokens = kPiece * warps;
  static constexpr int row = kGateChannels * ES;      // bytes of a row
  static constexpr int bytes = tokens * row;          // of an array
  static constexpr int vecs = row / 16;               // 16-byte vectors of a row
  static constexpr int rows_at_once = threads / vecs; // rows that the CTA's threads copy in turn
};

// A CTA's place: its sequence, rank in the cluster and channels.
inline long long gate_tiles(int D) { return (D + kGateChannels - 1) / kGateChannels; }

// CTAs of a cluster for tiles of `tokens` tokens, `slots` CTAs at once on the GPU.
int gate_cluster(const SeqRows& r, int D, int tokens, long long slots);

#if defined(__CUDACC__)

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
__device__ __forceinline__ void store_pair(void* p, float2 v) {
  if constexpr (BF16) *static_cast<uint32_t*>(p) = Vec<true>::two(v.x, v.y);
  else *static_cast<float2*>(p) = v;
}

// sigmoid(u) = 1 / (1 + e), e = e^-u, and 1 - sigmoid(u) = e sigmoid(u), which does not
// cancel. e is kept below 2^126, so that both stay finite (and sigmoid above 2^-127).
struct Sigmoid {
  float2 p, e;
  __device__ __forceinline__ explicit Sigmoid(float2 u) {
    const float2 x = __fmul2_rn(u, make_float2(-kLog2e, -kLog2e));
    e = make_float2(ex2_approx(fmin_nan(x.x)), ex2_approx(fmin_nan(x.y)));
    const float2 w = __fadd2_rn(e, make_float2(1.f, 1.f));
    p = make_float2(rcp_approx(w.x), rcp_approx(w.y));
  }
  __device__ __forceinline__ float2 rest() const { return __fmul2_rn(e, p); }  // 1 - p
  static __device__ __forceinline__ float fmin_nan(float x) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(126.f));
    return r;
  }
};

// The decay a = e^-w of a rate w >= 0 and 1 - a^2. Slow channels have w of 1e-3 and
// below, where 1 - a^2 from a rounded a has lost its digits, and a state of a long memory
// gathers a's own error over the tokens it remembers. So below 0.35 both come from
// m = 1 - e^-w by its series (up to w^7; what is left out is below 2e-8 of it): a = 1 - m,
// 1 - a^2 = m (2 - m). Above, a is the SFU's 2^x, and 1 - a^2 > 0.5 does not cancel.
__device__ __forceinline__ void decay_of(float2 w, float2* a, float2* rest) {
  float2 m = make_float2(1.f / 5040.f, 1.f / 5040.f);
  m = __ffma2_rn(m, w, make_float2(-1.f / 720.f, -1.f / 720.f));
  m = __ffma2_rn(m, w, make_float2(1.f / 120.f, 1.f / 120.f));
  m = __ffma2_rn(m, w, make_float2(-1.f / 24.f, -1.f / 24.f));
  m = __ffma2_rn(m, w, make_float2(1.f / 6.f, 1.f / 6.f));
  m = __ffma2_rn(m, w, make_float2(-0.5f, -0.5f));
  m = __ffma2_rn(m, w, make_float2(1.f, 1.f));
  m = __fmul2_rn(m, w);
  const float2 u = __fmul2_rn(w, make_float2(-kLog2e, -kLog2e));
  const bool lx = w.x < 0.35f, ly = w.y < 0.35f;
  a->x = lx ? 1.f - m.x : ex2_approx(u.x);
  a->y = ly ? 1.f - m.y : ex2_approx(u.y);
  rest->x = lx ? fmaf(-m.x, m.x, 2.f * m.x) : fmaf(-a->x, a->x, 1.f);
  rest->y = ly ? fmaf(-m.y, m.y, 2.f * m.y) : fmaf(-a->y, a->y, 1.f);
}
__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// The rate of a channel, or its refusal.
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
