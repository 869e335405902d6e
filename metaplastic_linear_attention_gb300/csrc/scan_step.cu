// Selective scan, one token: the state [batch, D, N] is read, decayed, written
// into and stored in place, and y read from it (formulas in scan_fwd.cu).
//
// A stream over the state: 8 bytes per state and about 7 operations, bound by
// memory (by L2 where the state fits its 129 MB). A lane owns 4 states of a
// channel (one 16-byte vector), N / 4 lanes a channel, and takes kPer channels with
// all their loads issued first; y's sum over the states is a butterfly over the
// channel's lanes.
#include "ssm.cuh"

namespace palimpsa {
namespace {

constexpr int kPer = 2;    // channels of a lane
constexpr int kWarps = 4;

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, long long i) {
  if constexpr (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ float4 load4(const void* p, long long i) {
  if constexpr (BF16) {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i);
    return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
  } else {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  }
}

template <bool BF16, int N>
__global__ void __launch_bounds__(32 * kWarps) palimpsa_scan_step_kernel(ScanArgs a, unsigned chunks) {
  constexpr int LPC = N / 4, CPW = 32 / LPC;  // lanes per channel, channels per warp and turn
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long n = blockIdx.x / chunks;  // sequence
  const int n0 = 4 * (lane % LPC);
  const int first = (int)(blockIdx.x % chunks) * (kWarps * kPer * CPW) + warp * (kPer * CPW) + lane / LPC;
  const int per_group = a.D / a.G;
  float* const hs = a.h_T + (n * a.D + first) * N + n0;
  const float* const As = a.A + (long long)first * N + n0;
  float4 h[kPer], A[kPer], B[kPer], C[kPer];
  float s[kPer], x[kPer], z[kPer], sk[kPer], bi[kPer];
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int d = first + k * CPW;
    if (d >= a.D) continue;
    h[k] = *reinterpret_cast<const float4*>(hs + k * CPW * N);
    A[k] = *reinterpret_cast<const float4*>(As + k * CPW * N);
    s[k] = load1<BF16>(a.dt, n * a.dt_ld + d);
    x[k] = load1<BF16>(a.x, n * a.x_ld + d);
    z[k] = a.z ? load1<BF16>(a.z, n * a.z_ld + d) : 0.f;
    bi[k] = a.dt_bias ? a.dt_bias[d] : 0.f;
    sk[k] = a.skip ? a.skip[d] : 0.f;
    const int g = a.G == 1 ? 0 : d / per_group;
    B[k] = load4<BF16>(a.B, n * a.B_ld + g * N + n0);
    C[k] = load4<BF16>(a.C, n * a.C_ld + g * N + n0);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int d = first + k * CPW;
    const bool in = d < a.D;
    float y = 0.f;
    if (in) {
      s[k] += bi[k];
      if (a.softplus) s[k] = softplus_fast(s[k]);
      bad |= !(nonneg_finite(s[k]) && pos_finite(A[k].x) && pos_finite(A[k].y) && pos_finite(A[k].z) &&
               pos_finite(A[k].w));
      const float m = -kLog2e * s[k], w = s[k] * x[k];
      h[k].x = fmaf(ex2_approx(fmaf(m, A[k].x, kDecayShift)), h[k].x, w * B[k].x);
      h[k].y = fmaf(ex2_approx(fmaf(m, A[k].y, kDecayShift)), h[k].y, w * B[k].y);
      h[k].z = fmaf(ex2_approx(fmaf(m, A[k].z, kDecayShift)), h[k].z, w * B[k].z);
      h[k].w = fmaf(ex2_approx(fmaf(m, A[k].w, kDecayShift)), h[k].w, w * B[k].w);
      *reinterpret_cast<float4*>(hs + k * CPW * N) = h[k];
      y = fmaf(h[k].x, C[k].x, fmaf(h[k].y, C[k].y, fmaf(h[k].z, C[k].z, h[k].w * C[k].w)));
    }
#pragma unroll
    for (int m = LPC / 2; m > 0; m /= 2) y += __shfl_xor_sync(0xffffffffu, y, m);
    if (in && lane % LPC == 0) {
      y = fmaf(sk[k], x[k], y);
      if (a.z) y *= silu_fast(z[k]);
      if constexpr (BF16) static_cast<__nv_bfloat16*>(a.y)[n * a.D + d] = __float2bfloat16_rn(y);
      else static_cast<float*>(a.y)[n * a.D + d] = y;
    }
  }
  if (bad) latch_status(a.status, kStatusDomain);
}

template <int N>
cudaError_t run(const ScanArgs& a, cudaStream_t s) {
  const int per_block = kWarps * kPer * (32 / (N / 4));
  const long long chunks = (a.D + per_block - 1) / per_block, blocks = chunks * a.rows.n_seq;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  if (a.bf16) palimpsa_scan_step_kernel<true, N><<<(unsigned)blocks, 32 * kWarps, 0, s>>>(a, (unsigned)chunks);
  else palimpsa_scan_step_kernel<false, N><<<(unsigned)blocks, 32 * kWarps, 0, s>>>(a, (unsigned)chunks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan_step(const ScanArgs& a, cudaStream_t s) {
  switch (a.N) {
    case 8: return run<8>(a, s);
    case 16: return run<16>(a, s);
    case 32: return run<32>(a, s);
    case 64: return run<64>(a, s);
    default: return run<128>(a, s);
  }
}

}  // namespace palimpsa
