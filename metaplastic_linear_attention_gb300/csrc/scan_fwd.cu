// Selective scan, forward. Per channel d (of group g) and state n:
//   s_t = softplus(dt_t + dt_bias)   (or dt_t + dt_bias as it is)
//   h_t = exp(-A s_t) h_{t-1} + (s_t x_t) B_t,    A = A[d, n] > 0, B_t = B_t[g, n]
//   y_t = (sum_n C_t[g, n] h_t + skip x_t) silu(z_t).
//
// What bounds it: each state-token costs one 2^x on the SFU (32 per clock and SM)
// and four FP32 operations (s A, (s x) B, the update, the readout; 128 per clock
// and SM), 8 bytes of HBM per channel-token in bf16. At N = 16 that is half a
// clock per channel-token and SM on either pipe and a third of one on HBM, so
// the kernel feeds the SFU and the FP32 pipe together and keeps everything else
// off them:
// * a lane holds 4 channels x 4 states (4 x 2 at N = 8) in registers, as f32x2 pairs.
//   Lanes that share 4 states are neighbours (8 lanes, 32 channels), so a B or C
//   load is one broadcast per quarter warp, shared by 4 channels; a step size
//   serves 4 states;
// * step sizes, s x and B, C become fp32 in shared memory once per chunk of 16
//   tokens, each value by one lane;
// * y's sum over a warp's 16 states is a reduce-scatter over its 4 lane groups (3
//   shuffles for 4 channels); more than 16 states are shared out over warps and
//   summed with the gate and the skip term when the chunk is stored;
// * inputs arrive through a ring of asynchronous 16-byte copies, two chunks ahead.
// A tile is 32 channels of one group, all states, one sequence (or a segment of
// one), by one CTA of N / 16 warps.
//
// Time split. Where the tiles are too few for the GPU, each sequence is cut into
// segments: pass A runs the recurrence of every segment but the last from zero
// and keeps its end state and the sum of its step sizes (the segment's decay is
// exp(-A sum)); the carry kernel folds them into start states; pass C runs every
// segment from its own.
//
// Rounding: states, sums and step sizes are fp32; y is rounded to the input
// type once. 2^x is the SFU's (measured bias about -2e-8 a token for decays near
// 1, so a state with a window of w tokens is off by about 2e-8 w).
#include <algorithm>
#include <mutex>

#include "ssm.cuh"

namespace palimpsa {
namespace {

constexpr int kChunk = 16;   // tokens staged together
constexpr int kStages = 3;   // chunks in the ring
constexpr int CH = kScanChannels;

// Shared memory of a CTA, bytes (all parts 16-byte aligned).
struct Smem {
  int rx, rdt, rz, rB, rC, raw;  // one stage
  int s, sx, B, C, y, par, total;
  __host__ __device__ Smem(int N, int W, int es, int mode) {
    const bool summary = mode != 0;
    rx = 0;
    rdt = rx + kChunk * CH * es;
    rz = rdt + kChunk * CH * es;
    rB = mode == 1 ? rz : rz + kChunk * CH * es;
    rC = rB + kChunk * N * es;
    raw = summary ? rC : rC + kChunk * N * es;
    s = kStages * raw;
    sx = s + kChunk * CH * 4;
    B = sx + kChunk * CH * 4;
    C = B + kChunk * N * 4;
    y = summary ? C : C + kChunk * N * 4;
    par = summary ? y : y + W * kChunk * CH * 4;
    total = par + 2 * CH * 4;
  }
};

// What a launch computes: the scan; pass A of its time split; or pass A of the
// backward's, which runs from the last token to the first with dy silu(z) in the
// place of s x and C in the place of B: g <- exp(-A s_t) (g + C_t dpre_t).
enum Mode { kForward, kSummary, kReverseSummary };

// NS states per lane (2 or 4), W warps: N = 4 NS W.
template <bool BF16, int NS, int W, int MODE>
__global__ void __launch_bounds__(32 * W) palimpsa_scan_kernel(ScanArgs a, int tiles) {
  using V = Vec<BF16>;
  constexpr int VN = V::n, ES = V::bytes, N = 4 * NS * W, NP = NS / 2;
  constexpr int VPR = CH / VN;        // vectors in a row of the tile
  constexpr int BPR = (N + VN - 1) / VN;  // vectors in a row of B or C
  constexpr int NT = 32 * W;
  constexpr bool SUMMARY = MODE != kForward, REV = MODE == kReverseSummary;
  extern __shared__ __align__(128) unsigned char smem[];
  const Smem L(N, W, ES, MODE);
  float* const fs = reinterpret_cast<float*>(smem + L.s);
  float* const fsx = reinterpret_cast<float*>(smem + L.sx);
  float* const fB = reinterpret_cast<float*>(smem + L.B);
  float* const fC = reinterpret_cast<float*>(smem + L.C);
  float* const fy = reinterpret_cast<float*>(smem + L.y);
  float* const fbias = reinterpret_cast<float*>(smem + L.par);
  float* const fskip = fbias + CH;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = (int)(blockIdx.x % tiles);
  const long long rest = blockIdx.x / tiles;
  // Pass A leaves out the segment that no other follows.
  const int nseg = SUMMARY ? a.nseg - 1 : a.nseg;
  const int seg = (int)(rest % nseg) + (REV ? 1 : 0);
  const long long n = rest / nseg;
  const int per_group = a.D / a.G, tpg = (per_group + CH - 1) / CH;
  const int g = tile / tpg, ch0 = g * per_group + (tile % tpg) * CH;
  const int nch = min(CH, (g + 1) * per_group - ch0);  // a multiple of 8
  const int nv = nch / VN;
  long long row0;
  int len;
  if (!seq_rows(a.rows, n, &row0, &len)) {
    if (tile == 0 && tid == 0) latch_status(a.status, kStatusDomain);
    return;
  }
  const int tb = seg * a.seg_len, te = min(len, tb + a.seg_len);
  const bool last = te >= len;
  // Segments past the end have nothing to do, nor has the forward's pass A on the last.
  if ((tb >= len && seg > 0) || (MODE == kSummary && last)) return;
  const int tn = te - tb, nchunk = (tn + kChunk - 1) / kChunk;

  // A lane's channels 4 cl .. 4 cl + 3 of the tile, and states n0 .. n0 + NS - 1.
  const int cl = lane & 7, sl = lane >> 3;
  const int n0 = warp * 4 * NS + sl * NS;
  bool bad = false;
  float2 A2[4][NP], h[4][NP];  // A scaled by -log2(e): exp(-A s) = 2^(A2 s)
  float2 dsum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int d = 4 * cl + c;
    const bool in = d < nch;
    const size_t an = ((size_t)(ch0 + d)) * N + n0;
    const float* h0 = nullptr;
    if (!SUMMARY && in) {
      if (a.nseg > 1) h0 = a.seg_state + ((size_t)(n * a.nseg + seg) * a.D + ch0 + d) * N + n0;
      else if (a.h0) h0 = a.h0 + ((size_t)n * a.D + ch0 + d) * N + n0;
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const float2 v = in ? *reinterpret_cast<const float2*>(a.A + an + 2 * p) : make_float2(1.f, 1.f);
      bad |= !(pos_finite(v.x) && pos_finite(v.y));
      A2[c][p] = make_float2(-kLog2e * v.x, -kLog2e * v.y);
      h[c][p] = h0 ? *reinterpret_cast<const float2*>(h0 + 2 * p) : make_float2(0.f, 0.f);
    }
  }
  for (int c = tid; c < CH; c += NT) {
    fbias[c] = c < nch && a.dt_bias ? a.dt_bias[ch0 + c] : 0.f;
    fskip[c] = c < nch && a.skip ? a.skip[ch0 + c] : 0.f;
  }

  const long long x_ld = REV ? a.dy_ld : a.x_ld, B_ld = REV ? a.C_ld : a.B_ld;
  const char* const gx = static_cast<const char*>(REV ? a.dy : a.x) + ((row0 + tb) * x_ld + ch0) * ES;
  const char* const gdt = static_cast<const char*>(a.dt) + ((row0 + tb) * a.dt_ld + ch0) * ES;
  const char* const gz = a.z ? static_cast<const char*>(a.z) + ((row0 + tb) * a.z_ld + ch0) * ES : nullptr;
  const char* const gB = static_cast<const char*>(REV ? a.C : a.B) + ((row0 + tb) * B_ld + g * N) * ES;
  const char* const gC = SUMMARY ? nullptr : static_cast<const char*>(a.C) + ((row0 + tb) * a.C_ld + g * N) * ES;
  auto stage = [&](int c) {  // copies of chunk c, as one group
    if (c < nchunk) {
      unsigned char* const st = smem + (c % kStages) * L.raw;
      const int t0 = (REV ? nchunk - 1 - c : c) * kChunk, nt = min(kChunk, tn - t0);
      for (int i = tid; i < kChunk * VPR; i += NT) {
        const int t = i / VPR, v = i % VPR;
        if (t >= nt || v >= nv) continue;
        const int o = (t * CH + v * VN) * ES;
        const long long r = t0 + t, b = (long long)v * 16;
        cp_async16(st + L.rx + o, gx + r * x_ld * ES + b);
        cp_async16(st + L.rdt + o, gdt + r * a.dt_ld * ES + b);
        if (MODE != kSummary && gz) cp_async16(st + L.rz + o, gz + r * a.z_ld * ES + b);
      }
      for (int i = tid; i < kChunk * BPR; i += NT) {
        const int t = i / BPR, v = i % BPR;
        if (t >= nt) continue;
        const int o = (t * N + v * VN) * ES;
        const long long r = t0 + t, b = (long long)v * 16;
        cp_async16(st + L.rB + o, gB + r * B_ld * ES + b);
        if (!SUMMARY) cp_async16(st + L.rC + o, gC + r * a.C_ld * ES + b);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int c = 0; c < kStages - 1; ++c) stage(c);

  for (int c = 0; c < nchunk; ++c) {
    const int t0 = (REV ? nchunk - 1 - c : c) * kChunk, nt = min(kChunk, tn - t0);
    cp_async_wait<kStages - 2>();
    __syncthreads();  // chunk c is here; the last chunk's stage and y are free
    stage(c + kStages - 1);
    const unsigned char* const st = smem + (c % kStages) * L.raw;
    for (int i = tid; i < kChunk * VPR; i += NT) {
      const int t = i / VPR, v = i % VPR;
      if (t >= nt) continue;
      float s[VN], x[VN];
      if (v < nv) {
        V::unpack(*reinterpret_cast<const uint4*>(st + L.rdt + (t * CH + v * VN) * ES), s);
        V::unpack(*reinterpret_cast<const uint4*>(st + L.rx + (t * CH + v * VN) * ES), x);
#pragma unroll
        for (int k = 0; k < VN; ++k) {
          s[k] += fbias[v * VN + k];
          if (a.softplus) s[k] = softplus_fast(s[k]);
          bad |= !nonneg_finite(s[k]);
          if (!REV) x[k] *= s[k];
        }
        if (REV && gz) {
          float z[VN];
          V::unpack(*reinterpret_cast<const uint4*>(st + L.rz + (t * CH + v * VN) * ES), z);
#pragma unroll
          for (int k = 0; k < VN; ++k) x[k] *= silu_fast(z[k]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < VN; ++k) s[k] = x[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < VN; k += 4) {
        *reinterpret_cast<float4*>(fs + t * CH + v * VN + k) = make_float4(s[k], s[k + 1], s[k + 2], s[k + 3]);
        *reinterpret_cast<float4*>(fsx + t * CH + v * VN + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
      }
    }
    for (int i = tid; i < kChunk * BPR; i += NT) {
      const int t = i / BPR;
      if (t >= nt) continue;
      float f[VN];
      V::unpack(reinterpret_cast<const uint4*>(st + L.rB)[i], f);
#pragma unroll
      for (int k = 0; k < VN; k += 4)
        *reinterpret_cast<float4*>(fB + i * VN + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
      if (!SUMMARY) {
        V::unpack(reinterpret_cast<const uint4*>(st + L.rC)[i], f);
#pragma unroll
        for (int k = 0; k < VN; k += 4)
          *reinterpret_cast<float4*>(fC + i * VN + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
      }
    }
    __syncthreads();

    if (!SUMMARY && a.ckpt && (tb + t0) % kScanCheckpoint == 0) {
      float* const ck = a.ckpt + (scan_ckpt_row0(a.rows, n, row0) + (tb + t0) / kScanCheckpoint) * a.D * N;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (4 * cl + k < nch)
#pragma unroll
          for (int p = 0; p < NP; ++p)
            *reinterpret_cast<float2*>(ck + (size_t)(ch0 + 4 * cl + k) * N + n0 + 2 * p) = h[k][p];
    }

    auto token = [&](int t) {
      const float4 s4 = *reinterpret_cast<const float4*>(fs + t * CH + 4 * cl);
      const float4 x4 = *reinterpret_cast<const float4*>(fsx + t * CH + 4 * cl);
      const float sv[4] = {s4.x, s4.y, s4.z, s4.w}, xv[4] = {x4.x, x4.y, x4.z, x4.w};
      float2 b[NP], cc[NP];
#pragma unroll
      for (int p = 0; p < NP; ++p) b[p] = *reinterpret_cast<const float2*>(fB + t * N + n0 + 2 * p);
      if (!SUMMARY)
#pragma unroll
        for (int p = 0; p < NP; ++p) cc[p] = *reinterpret_cast<const float2*>(fC + t * N + n0 + 2 * p);
      float y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const float2 u = __fmul2_rn(make_float2(sv[k], sv[k]), A2[k][p]);
          const float2 e = make_float2(ex2_approx(u.x), ex2_approx(u.y));
          if (REV) h[k][p] = __fmul2_rn(e, __ffma2_rn(make_float2(xv[k], xv[k]), b[p], h[k][p]));
          else h[k][p] = __ffma2_rn(e, h[k][p], __fmul2_rn(make_float2(xv[k], xv[k]), b[p]));
          if (!SUMMARY) acc = p == 0 ? __fmul2_rn(h[k][p], cc[p]) : __ffma2_rn(h[k][p], cc[p], acc);
        }
        y[k] = acc.x + acc.y;
      }
      if (SUMMARY) {
        dsum[0] = __fadd2_rn(dsum[0], make_float2(sv[0], sv[1]));
        dsum[1] = __fadd2_rn(dsum[1], make_float2(sv[2], sv[3]));
      } else {
        // Reduce-scatter over the 4 lane groups: lane (cl, sl) ends with channel 4 cl + sl.
        const bool hi = sl & 2, odd = sl & 1;
        const float k0 = hi ? y[2] : y[0], k1 = hi ? y[3] : y[1];
        const float r0 = k0 + __shfl_xor_sync(0xffffffffu, hi ? y[0] : y[2], 16);
        const float r1 = k1 + __shfl_xor_sync(0xffffffffu, hi ? y[1] : y[3], 16);
        const float r = (odd ? r1 : r0) + __shfl_xor_sync(0xffffffffu, odd ? r0 : r1, 8);
        fy[(warp * kChunk + t) * CH + 4 * cl + sl] = r;
      }
    };
    if (nt == kChunk) {
#pragma unroll 4
      for (int t = 0; t < kChunk; ++t) token(REV ? kChunk - 1 - t : t);
    } else {
      for (int t = 0; t < nt; ++t) token(REV ? nt - 1 - t : t);
    }

    if (!SUMMARY) {
      __syncthreads();
      for (int i = tid; i < kChunk * VPR; i += NT) {
        const int t = i / VPR, v = i % VPR;
        if (t >= nt || v >= nv) continue;
        float o[VN], x[VN];
        V::unpack(*reinterpret_cast<const uint4*>(st + L.rx + (t * CH + v * VN) * ES), x);
#pragma unroll
        for (int k = 0; k < VN; ++k) {
          o[k] = fskip[v * VN + k] * x[k];
#pragma unroll
          for (int w = 0; w < W; ++w) o[k] += fy[(w * kChunk + t) * CH + v * VN + k];
        }
        if (gz) {
          V::unpack(*reinterpret_cast<const uint4*>(st + L.rz + (t * CH + v * VN) * ES), x);
#pragma unroll
          for (int k = 0; k < VN; ++k) o[k] *= silu_fast(x[k]);
        }
        *reinterpret_cast<uint4*>(static_cast<char*>(a.y) + ((row0 + tb + t0 + t) * a.D + ch0 + v * VN) * ES) =
            V::pack(o);
      }
    }
  }
  if (bad) latch_status(a.status, kStatusDomain);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (4 * cl + c >= nch) continue;
    float* out = nullptr;
    if (SUMMARY) out = a.seg_state + ((size_t)(n * a.nseg + seg) * a.D + ch0 + 4 * cl + c) * N + n0;
    else if (last && a.h_T) out = a.h_T + ((size_t)n * a.D + ch0 + 4 * cl + c) * N + n0;
    if (out)
#pragma unroll
      for (int p = 0; p < NP; ++p) *reinterpret_cast<float2*>(out + 2 * p) = h[c][p];
  }
  if (SUMMARY && warp == 0 && sl == 0) {
    const float v[4] = {dsum[0].x, dsum[0].y, dsum[1].x, dsum[1].y};
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (4 * cl + c < nch) a.seg_dt[(size_t)(n * a.nseg + seg) * a.D + ch0 + 4 * cl + c] = v[c];
  }
}

// Start states of the segments, in place over their summaries: one thread per
// (sequence, channel, state).
__global__ void __launch_bounds__(256) palimpsa_scan_carry_kernel(ScanArgs a, bool reverse) {
  const long long per = (long long)a.D * a.N, i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= per * a.rows.n_seq) return;
  const long long n = i / per, e = i % per;
  const int d = (int)(e / a.N);
  long long row0;
  int len;
  if (!seq_rows(a.rows, n, &row0, &len)) return;
  const int ns = max(1, (len + a.seg_len - 1) / a.seg_len);
  const float A = -kLog2e * a.A[e];
  const float* const init = reverse ? a.dh_T : a.h0;
  float h = init ? init[n * per + e] : 0.f;
  float* const st = a.seg_state + n * a.nseg * per + e;
  const float* const sd = a.seg_dt + n * a.nseg * a.D + d;
  for (int k = 0; k < ns; ++k) {
    const int s = reverse ? ns - 1 - k : k;
    const float add = k + 1 < ns ? st[s * per] : 0.f;
    const float dec = k + 1 < ns ? ex2_approx(A * sd[(long long)s * a.D]) : 0.f;
    st[s * per] = h;
    h = fmaf(dec, h, add);
  }
}

template <bool BF16, int NS, int W, int MODE>
cudaError_t run(const ScanArgs& a, cudaStream_t s) {
  const Smem L(4 * NS * W, W, Vec<BF16>::bytes, MODE);
  const long long tiles = scan_tiles(a), blocks = tiles * a.rows.n_seq * (MODE != kForward ? a.nseg - 1 : a.nseg);
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  if (L.total > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(palimpsa_scan_kernel<BF16, NS, W, MODE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, L.total);
    if (e != cudaSuccess) return e;
  }
  palimpsa_scan_kernel<BF16, NS, W, MODE><<<(unsigned)blocks, 32 * W, L.total, s>>>(a, (int)tiles);
  return cudaGetLastError();
}

template <int MODE>
cudaError_t dispatch(const ScanArgs& a, cudaStream_t s) {
  switch (a.N) {
    case 8: return a.bf16 ? run<true, 2, 1, MODE>(a, s) : run<false, 2, 1, MODE>(a, s);
    case 16: return a.bf16 ? run<true, 4, 1, MODE>(a, s) : run<false, 4, 1, MODE>(a, s);
    case 32: return a.bf16 ? run<true, 4, 2, MODE>(a, s) : run<false, 4, 2, MODE>(a, s);
    case 64: return a.bf16 ? run<true, 4, 4, MODE>(a, s) : run<false, 4, 4, MODE>(a, s);
    default: return a.bf16 ? run<true, 4, 8, MODE>(a, s) : run<false, 4, 8, MODE>(a, s);
  }
}

}  // namespace

cudaError_t plan_scan(const ScanArgs& a, bool backward, int* nseg, int* seg_len) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const long long warps = scan_tiles(a) * a.rows.n_seq * std::max(1, a.N / 16);
  const long long slots = 4ll * sms;  // one warp per scheduler
  const int len = a.rows.max_len;
  *nseg = 1;
  *seg_len = std::max(len, 1);
  // Forward: the split does about twice the work, so it pays below half a warp
  // per scheduler; it then aims at three. Backward: pass A is a small part of the
  // work, so the split pays below the two warps that a scheduler's registers hold.
  if (backward ? warps < 2 * slots : 2 * warps <= slots) {
    const int shortest = backward ? 64 : 128;  // tokens of a segment, at least
    long long want = backward ? 2 * slots / warps : (3 * slots + warps - 1) / warps;
    want = std::min<long long>(want, len / shortest);
    if (want >= (backward ? 2 : 3)) {
      const int per = (int)((len + want - 1) / want);
      *seg_len = (per + kScanCheckpoint - 1) / kScanCheckpoint * kScanCheckpoint;
      *nseg = (len + *seg_len - 1) / *seg_len;
    }
  }
  return cudaSuccess;
}

cudaError_t launch_scan_carry(const ScanArgs& a, bool reverse, cudaStream_t s) {
  const long long blocks = ((long long)a.rows.n_seq * a.D * a.N + 255) / 256;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  palimpsa_scan_carry_kernel<<<(unsigned)blocks, 256, 0, s>>>(a, reverse);
  return cudaGetLastError();
}

cudaError_t launch_scan_forward(const ScanArgs& a, cudaStream_t s) {
  if (a.nseg > 1) {
    cudaError_t e = dispatch<kSummary>(a, s);
    if (e == cudaSuccess) e = launch_scan_carry(a, false, s);
    if (e != cudaSuccess) return e;
  }
  return dispatch<kForward>(a, s);
}

cudaError_t launch_scan_reverse_summary(const ScanArgs& a, cudaStream_t s) { return dispatch<kReverseSummary>(a, s); }

}  // namespace palimpsa
