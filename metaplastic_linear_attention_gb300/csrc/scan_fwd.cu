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
// * inputs arrive in chunks of 8 tokens by asynchronous 16-byte copies, a chunk ahead;
//   step sizes and s x become fp32 in shared memory once, each by one lane (B and C stay
//   as they came: a lane unpacks its 4);
// * the lane groups' parts of y (4 states each, of all warps) are stored after the chunk's
//   tokens and summed, with the skip term and the gate, when y is written. (Shuffles in
//   place of these stores took twice the time: their latency stood in every token.)
// A tile is 32 channels of one group, all states, one sequence (or a segment of
// one), by one CTA of N / 16 warps; a single warp needs no barriers. 16 warps of 128
// registers fill an SM. Tried and slower: 8 channels a lane (11 warps), the next
// chunk's conversion among this one's tokens, warps of their own for the conversions.
// Measured (GB300, bf16, N = 16, gate): 1.3 clocks per channel-token and SM for the
// scan itself and 0.9 for pass A, two thirds of the issue slots busy: 298 and 204 us at
// 1 x 32768 x 2048, where half a clock would be 113.
//
// Time split. Where the tiles are too few for the GPU, each sequence is cut into
// segments: pass A runs the recurrence of every segment but the last from zero
// and keeps its end state and the sum of its step sizes (the segment's decay is
// exp(-A sum)); pass C runs every segment, from the state that it folds from the
// summaries before it (or a kernel between them, where the segments are many).
//
// Rounding: states, sums and step sizes are fp32; y is rounded to the input type once.
#include <algorithm>

#include "ssm.cuh"

namespace palimpsa {
namespace {

constexpr int kChunk = 8;    // tokens staged together
constexpr int kStages = 2;   // chunks in the ring of raw inputs
constexpr int CH = kScanChannels;
constexpr int kGroup = 8;    // tokens whose y is stored together
constexpr int kWarpsPerSM = 16;

// What a launch computes: the scan; pass A of its time split; or pass A of the
// backward's, which runs from the last token to the first with dy silu(z) in the
// place of s x and C in the place of B: g <- exp(-A s_t) (g + C_t dpre_t).
enum Mode { kForward, kSummary, kReverseSummary };

// Shared memory of a CTA, bytes (all parts 16-byte aligned).
struct Smem {
  int rx, rdt, rz, rB, rC, raw;  // one stage of raw inputs
  int s, sx, par, y, total;      // step sizes, s x, dt_bias and skip, the lane groups' parts of y
  __host__ __device__ constexpr Smem(int N, int groups, int es, int mode)
      : rx(0),
        rdt(kChunk * CH * es),
        rz(2 * kChunk * CH * es),
        rB(mode == kSummary ? rz : rz + kChunk * CH * es),
        rC(rB + kChunk * N * es),
        raw(mode == kForward ? rC + kChunk * N * es : rC),
        s(kStages * raw),
        sx(s + kChunk * CH * 4),
        par(sx + kChunk * CH * 4),
        y(par + 2 * CH * 4),
        total(mode == kForward ? y + groups * kChunk * CH * 4 : y) {}
};

// 4 values of the input type.
template <bool BF16>
__device__ __forceinline__ void load4(float* f, const unsigned char* p) {
  if constexpr (BF16) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x); f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
  } else {
    const float4 u = *reinterpret_cast<const float4*>(p);
    f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
  }
}
// NS values of a row of B or C as they came, each twice (for two channels).
template <bool BF16, int NS>
__device__ __forceinline__ void load_states(float2* f, const unsigned char* p) {
  float v[NS];
  if constexpr (NS == 4) {
    load4<BF16>(v, p);
  } else if constexpr (BF16) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    v[0] = bf16_lo(u); v[1] = bf16_hi(u);
  } else {
    const float2 u = *reinterpret_cast<const float2*>(p);
    v[0] = u.x; v[1] = u.y;
  }
#pragma unroll
  for (int j = 0; j < NS; ++j) f[j] = make_float2(v[j], v[j]);
}

// NS states per lane (2 or 4), W warps: N = 4 NS W.
template <bool BF16, int NS, int W, int MODE>
__global__ void __launch_bounds__(32 * W, kWarpsPerSM / W) palimpsa_scan_kernel(ScanArgs a, int tiles) {
  using V = Vec<BF16>;
  constexpr int VN = V::n, ES = V::bytes, N = 4 * NS * W, NT = 32 * W;
  constexpr int VPR = CH / VN;  // vectors in a row of the tile
  constexpr int BPR = N / VN;   // vectors in a row of B or C
  constexpr bool FWD = MODE == kForward, REV = MODE == kReverseSummary;
  constexpr Smem L(N, 4 * W, ES, MODE);
  extern __shared__ __align__(128) unsigned char smem[];
  float* const fs = reinterpret_cast<float*>(smem + L.s);
  float* const fsx = reinterpret_cast<float*>(smem + L.sx);
  float* const fy = reinterpret_cast<float*>(smem + L.y);
  float* const fpar = reinterpret_cast<float*>(smem + L.par);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = (int)(blockIdx.x % tiles);
  const long long rest = blockIdx.x / tiles;
  // Pass A leaves out the segment that no other follows.
  int n, seg;
  if (FWD || a.slots.starts) {
    if (!slot_place(a.rows, a.slots, rest, &n, &seg) || (REV && seg == 0)) return;
  } else {
    seg = (int)(rest % (a.nseg - 1)) + (REV ? 1 : 0);
    n = (int)(rest / (a.nseg - 1));
  }
  const int per_group = a.D / a.G, tpg = (per_group + CH - 1) / CH;
  const int g = tile / tpg, ch0 = g * per_group + (tile % tpg) * CH;
  const int nch = min(CH, (g + 1) * per_group - ch0);  // a multiple of 8
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
  // (A chunk's tokens past the end have steps of size 0 and B = C = 0: they change nothing.)
  const int tn = te - tb, nchunk = (tn + kChunk - 1) / kChunk;
  auto first_token = [&](int c) { return (REV ? nchunk - 1 - c : c) * kChunk; };

  // A thread copies in, converts and finishes the same vectors of x, dt and z; their
  // place v in a row is the same for all of them. The copies' addresses move on by a
  // chunk each time.
  constexpr int VPT = (kChunk * VPR + NT - 1) / NT, BPT = (kChunk * BPR + NT - 1) / NT;
  const int v = tid % VPR, vt = tid / VPR, bv = tid % BPR, bt = tid / BPR;
  const bool vin = v * VN < nch, gated = a.z && MODE != kSummary;
  const long long x_ld = (REV ? a.dy_ld : a.x_ld) * ES, dt_ld = a.dt_ld * ES, z_ld = a.z_ld * ES;
  const long long B_ld = (REV ? a.C_ld : a.B_ld) * ES, C_ld = a.C_ld * ES;
  const long long rb = row0 + tb;
  const int t_first = first_token(0);
  const char* gx = static_cast<const char*>(REV ? a.dy : a.x) + (rb + t_first + vt) * x_ld + ch0 * ES + v * 16;
  const char* gdt = static_cast<const char*>(a.dt) + (rb + t_first + vt) * dt_ld + ch0 * ES + v * 16;
  const char* gz = gated ? static_cast<const char*>(a.z) + (rb + t_first + vt) * z_ld + ch0 * ES + v * 16 : nullptr;
  const char* gB = static_cast<const char*>(REV ? a.C : a.B) + (rb + t_first + bt) * B_ld + g * N * ES + bv * 16;
  const char* gC = FWD ? static_cast<const char*>(a.C) + (rb + t_first + bt) * C_ld + g * N * ES + bv * 16 : nullptr;
  auto stage = [&](int c) {  // copies of chunk c (the next in order), as one group
    if (c < nchunk) {
      unsigned char* const st = smem + (c % kStages) * L.raw;
      const int nt = min(kChunk, tn - first_token(c));
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int i = tid + k * NT;
        if (k * (NT / VPR) + vt >= nt || !vin) continue;
        cp_async16(st + L.rx + 16 * i, gx + k * (NT / VPR) * x_ld);
        cp_async16(st + L.rdt + 16 * i, gdt + k * (NT / VPR) * dt_ld);
        if (gated) cp_async16(st + L.rz + 16 * i, gz + k * (NT / VPR) * z_ld);
      }
#pragma unroll
      for (int k = 0; k < BPT; ++k) {
        const int i = tid + k * NT;
        if (i >= kChunk * BPR) continue;
        const bool in = k * NT / BPR + bt < nt;  // rows past the end are filled with zeros
        cp_async16(st + L.rB + 16 * i, in ? gB + k * (NT / BPR) * B_ld : gB - bt * B_ld, in);
        if (FWD) cp_async16(st + L.rC + 16 * i, in ? gC + k * (NT / BPR) * C_ld : gC - bt * C_ld, in);
      }
      constexpr int step = REV ? -kChunk : kChunk;
      gx += step * x_ld;
      gdt += step * dt_ld;
      gB += step * B_ld;
      if (FWD) gC += step * C_ld;
      if (gated) gz += step * z_ld;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int c = 0; c < kStages - 1; ++c) stage(c);

  for (int c = tid; c < CH; c += NT) {
    fpar[c] = c < nch && a.dt_bias ? a.dt_bias[ch0 + c] : 0.f;
    fpar[CH + c] = FWD && c < nch && a.skip ? a.skip[ch0 + c] : 0.f;
  }
  // A lane's channels 4 cl .. 4 cl + 3 of the tile, as two pairs, and its states from n0 on.
  // In rows of fp32 values per channel (s, s x, y parts) the quads of 4 channels of odd
  // tokens change places in pairs, so that the threads that hold 8 channels each (two
  // quads) and those that hold one reach all banks alike.
  const int cl = lane & 7, ng = warp * 4 + (lane >> 3), n0 = ng * NS;
  const int cq0 = 4 * cl, cq1 = 4 * (cl ^ 1);
  float2 A2[2][NS], h[2][NS];  // A scaled by -log2(e): exp(-A s) = 2^(A2 s)
  float2 dsum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const size_t at = (size_t)(ch0 + 4 * cl) * N + n0;  // of the first channel in [D, N]
  // The start state. With a time split, segment 0's pass A has put h0 into the slot of the
  // sequence's last segment, which no summary takes: h_T may be h0, and another CTA may have
  // written it.
  int slot0 = FWD || a.slots.starts ? (int)rest - seg : n * a.nseg;  // of the sequence
  asm("" : "+r"(slot0));  // (left to form it anew from the grid's indices, the compiler spills: 2 % of the time)
  const int nsegs = len > a.seg_len ? (len + a.seg_len - 1) / a.seg_len : 1;
  float* const slots = a.nseg > 1 ? a.seg_state + (size_t)slot0 * a.D * N : nullptr;
  float* const spare = a.nseg > 1 ? slots + (size_t)(nsegs - 1) * a.D * N : nullptr;
  const float* h0 = nullptr;
  if (FWD && a.carried) h0 = slots + (size_t)seg * a.D * N;
  else if (FWD && a.h0) h0 = last && seg == 0 ? a.h0 + (size_t)n * a.D * N : spare;
  bool bad = false;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const bool in = 4 * cl + c < nch;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const float A = in ? a.A[at + c * N + j] : 1.f;
      bad |= !pos_finite(A);
      (c & 1 ? A2[c / 2][j].y : A2[c / 2][j].x) = decay_rate(A);
      (c & 1 ? h[c / 2][j].y : h[c / 2][j].x) = in && h0 ? h0[at + c * N + j] : 0.f;
    }
  }
  if (FWD && seg > 0 && !a.carried && 4 * cl < nch)
    fold_segments<4, NS>(h, A2, slots + at, a.seg_dt + (size_t)slot0 * a.D + ch0 + 4 * cl, seg, 1, a.D, N);
  if (MODE == kSummary && seg == 0 && a.h0 && !a.carried && 4 * cl < nch) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float q[NS];
      load_own<NS>(q, reinterpret_cast<const unsigned char*>(a.h0 + (size_t)n * a.D * N + at + c * N));
      store_own<NS>(reinterpret_cast<unsigned char*>(spare + at + c * N), q);
    }
  }
  // The lane's part of a [D, N] array, stored.
  auto store_state = [&](float* out) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (4 * cl + c < nch) {
        float q[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) q[j] = c & 1 ? h[c / 2][j].y : h[c / 2][j].x;
        store_own<NS>(reinterpret_cast<unsigned char*>(out + at + c * N), q);
      }
  };
  // One token; y gets this lane's part of its channels' y.
  auto token = [&](const unsigned char* st, int t, float2* y) {
    const float4 s4 = *reinterpret_cast<const float4*>(fs + t * CH + (t & 1 ? cq1 : cq0));
    const float4 x4 = *reinterpret_cast<const float4*>(fsx + t * CH + (t & 1 ? cq1 : cq0));
    const float2 s[2] = {make_float2(s4.x, s4.y), make_float2(s4.z, s4.w)};
    const float2 x[2] = {make_float2(x4.x, x4.y), make_float2(x4.z, x4.w)};
    float2 b[NS], cc[NS];
    load_states<BF16, NS>(b, st + L.rB + (t * N + n0) * ES);
    if (FWD) load_states<BF16, NS>(cc, st + L.rC + (t * N + n0) * ES);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        float2& hh = h[p][j];
        const float2 u = decay_exponent(s[p], A2[p][j]);
        const float2 e = make_float2(ex2_approx(u.x), ex2_approx(u.y));
        if (REV) hh = __fmul2_rn(e, __ffma2_rn(x[p], b[j], hh));
        else hh = __ffma2_rn(e, hh, __fmul2_rn(x[p], b[j]));
        if (FWD) y[p] = j == 0 ? __fmul2_rn(hh, cc[j]) : __ffma2_rn(hh, cc[j], y[p]);
      }
    if (!FWD)
#pragma unroll
      for (int p = 0; p < 2; ++p) dsum[p] = __fadd2_rn(dsum[p], s[p]);
  };

  float least = 0.f, most = 0.f;  // of the step sizes
  for (int c = 0; c < nchunk; ++c) {
    const int t0 = first_token(c), nt = min(kChunk, tn - t0);
    unsigned char* const st = smem + (c % kStages) * L.raw;
    cp_async_wait<kStages - 2>();
    cta_sync<W>();  // chunk c is here, and the last one's stage, operands and y are free
    stage(c + kStages - 1);
#pragma unroll
    for (int i = tid; i < kChunk * VPR; i += NT) {
      float s[VN], x[VN];
      if (vin && i / VPR < nt) {
        float bias[VN];
#pragma unroll
        for (int k = 0; k < VN; k += 4)
          *reinterpret_cast<float4*>(bias + k) = *reinterpret_cast<const float4*>(fpar + v * VN + k);
        V::unpack(*reinterpret_cast<const uint4*>(st + L.rdt + 16 * i), s);
        V::unpack(*reinterpret_cast<const uint4*>(st + L.rx + 16 * i), x);
        if (REV && gated) {
          float z[VN];
          V::unpack(*reinterpret_cast<const uint4*>(st + L.rz + 16 * i), z);
#pragma unroll
          for (int k = 0; k < VN; k += 2) {
            const float2 d = __fmul2_rn(make_float2(x[k], x[k + 1]), silu_fast(make_float2(z[k], z[k + 1])));
            x[k] = d.x;
            x[k + 1] = d.y;
          }
        }
#pragma unroll
        for (int k = 0; k < VN; k += 2) {
          float2 u = __fadd2_rn(make_float2(s[k], s[k + 1]), make_float2(bias[k], bias[k + 1]));
          if (a.softplus) u = softplus_fast(u);
          else least = fminf(least, fminf(u.x, u.y));
          most = fmax_nan(most, fmax_nan(u.x, u.y));
          s[k] = u.x;
          s[k + 1] = u.y;
          if (!REV) {
            const float2 sx = __fmul2_rn(u, make_float2(x[k], x[k + 1]));
            x[k] = sx.x;
            x[k + 1] = sx.y;
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < VN; ++k) s[k] = x[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < VN; k += 4) {
        const int o = i / VPR * CH + ((v * VN + k) ^ 4 * (i / VPR & 1));
        *reinterpret_cast<float4*>(fs + o) = make_float4(s[k], s[k + 1], s[k + 2], s[k + 3]);
        *reinterpret_cast<float4*>(fsx + o) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
      }
    }
    cta_sync<W>();

    if (FWD && a.ckpt && (tb + t0) % kScanCheckpoint == 0)
      store_state(a.ckpt + (scan_ckpt_row0(a.rows, n, row0) + (tb + t0) / kScanCheckpoint) * a.D * N);
    // y is stored after a group of tokens: a store between two tokens would hold back
    // the loads of the second, which the compiler cannot tell from it.
#pragma unroll 1
    for (int tg = 0; tg < kChunk; tg += kGroup) {
      float2 y[kGroup][2];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) token(st, REV ? kChunk - 1 - tg - i : tg + i, y[i]);
      if (FWD)
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
          *reinterpret_cast<float4*>(fy + (ng * kChunk + tg + i) * CH + ((tg + i) & 1 ? cq1 : cq0)) =
              make_float4(y[i][0].x, y[i][0].y, y[i][1].x, y[i][1].y);
    }

    if (FWD) {
      cta_sync<W>();
#pragma unroll
      for (int i = tid; i < kChunk * VPR; i += NT) {
        const int t = i / VPR;
        if (t >= nt || !vin) continue;
        float o[VN], x[VN], skip[VN];
        V::unpack(*reinterpret_cast<const uint4*>(st + L.rx + 16 * i), x);
#pragma unroll
        for (int k = 0; k < VN; k += 4) {
          *reinterpret_cast<float4*>(skip + k) = *reinterpret_cast<const float4*>(fpar + CH + v * VN + k);
          float2 y0 = __fmul2_rn(make_float2(skip[k], skip[k + 1]), make_float2(x[k], x[k + 1]));
          float2 y1 = __fmul2_rn(make_float2(skip[k + 2], skip[k + 3]), make_float2(x[k + 2], x[k + 3]));
#pragma unroll
          for (int w = 0; w < 4 * W; ++w) {
            const float4 p =
                *reinterpret_cast<const float4*>(fy + (w * kChunk + t) * CH + ((v * VN + k) ^ 4 * (t & 1)));
            y0 = __fadd2_rn(y0, make_float2(p.x, p.y));
            y1 = __fadd2_rn(y1, make_float2(p.z, p.w));
          }
          o[k] = y0.x; o[k + 1] = y0.y; o[k + 2] = y1.x; o[k + 3] = y1.y;
        }
        if (gated) {
          V::unpack(*reinterpret_cast<const uint4*>(st + L.rz + 16 * i), x);
#pragma unroll
          for (int k = 0; k < VN; k += 2) {
            const float2 y = __fmul2_rn(make_float2(o[k], o[k + 1]), silu_fast(make_float2(x[k], x[k + 1])));
            o[k] = y.x;
            o[k + 1] = y.y;
          }
        }
        *reinterpret_cast<uint4*>(static_cast<char*>(a.y) + ((rb + t0 + t) * a.D + ch0 + v * VN) * ES) = V::pack(o);
      }
    }
  }
  if (bad || !(nonneg_finite(least) && nonneg_finite(most))) latch_status(a.status, kStatusDomain);
  if (!FWD) store_state(a.seg_state + (size_t)(slot0 + seg) * a.D * N);
  else if (last) store_state(a.h_T + (size_t)n * a.D * N);
  if (!FWD && ng == 0)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (4 * cl + c < nch)
        a.seg_dt[(size_t)(slot0 + seg) * a.D + ch0 + 4 * cl + c] = c & 1 ? dsum[c / 2].y : dsum[c / 2].x;
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
  const long long slot0 = first_slot(a.slots, n) + (reverse ? ns - 1 : 0);
  if (a.slots.starts && a.slots.starts[n + 1] - a.slots.starts[n] != ns) return;  // it has none
  const float A = decay_rate(a.A[e]);
  const float* const init = reverse ? a.dh_T : a.h0;
  float h = init ? init[n * per + e] : 0.f;
  // 8 segments at a time, their loads first: a store would hold back the next segment's.
  const long long step = reverse ? -1 : 1;
  float* st = a.seg_state + slot0 * per + e;
  const float* sd = a.seg_dt + slot0 * a.D + d;
  for (int k0 = 0; k0 < ns; k0 += 8) {
    float add[8], sum[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool more = k0 + k + 1 < ns;  // the last one's summary is not needed (nor there)
      add[k] = more ? st[k * step * per] : 0.f;
      sum[k] = more ? sd[k * step * a.D] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k0 + k >= ns) break;
      st[k * step * per] = h;
      h = fmaf(ex2_approx(A * sum[k]), h, add[k]);
    }
    st += 8 * step * per;
    sd += 8 * step * a.D;
  }
}

template <bool BF16, int NS, int W, int MODE>
cudaError_t run(const ScanArgs& a, cudaStream_t s) {
  constexpr Smem L(4 * NS * W, 4 * W, Vec<BF16>::bytes, MODE);
  const bool all = MODE == kForward || a.slots.starts;
  const long long tiles = scan_tiles(a), blocks = tiles * (all ? a.slots.count : a.rows.n_seq * (a.nseg - 1ll));
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

cudaError_t plan_scan(ScanArgs* a, bool backward, bool* close) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int len = a->rows.max_len;
  a->nseg = 1;
  a->seg_len = std::max(len, 1);
  // CTAs that an SM holds, and CTAs with work: of a packed batch, as many sequences of the
  // longest's length as its rows make.
  const int held = backward ? scan_backward_resident(*a) : kWarpsPerSM / std::max(1, a->N / 16);
  if (held < 1) return cudaErrorInvalidConfiguration;
  const long long slots = (long long)held * sms, tiles = scan_tiles(*a);
  const long long seqs = a->rows.cu ? std::max(1, (int)(((long long)a->rows.T + len - 1) / std::max(len, 1))) : a->rows.n_seq;
  // Segments for one wave of CTAs (in fp32 at N = 16 an SM's shared memory holds 14 of the 16
  // that this counts on, and the last of them make a second wave); the backward for two, whose pass A then has CTAs
  // enough (35 us against 45 at 4 x 2048 x 1024, the rest alike). The forward's split does
  // nearly twice the work and pays from 3 segments on (N = 16, 1 x 32768 x 2048: 0.52 ms
  // against 6.4; 8 x 4096 x 1536: 0.41 against 0.97). Pass A is a small part of a backward.
  long long want = (backward ? 2 : 1) * slots / (tiles * seqs);
  if (!backward && want < 3) want = 1;
  want = std::min<long long>(want, len / 32);
  if (want >= 2) {
    const int per = (int)((len + want - 1) / want);
    a->seg_len = (per + kScanCheckpoint - 1) / kScanCheckpoint * kScanCheckpoint;
    a->nseg = (len + a->seg_len - 1) / a->seg_len;
    a->carried = a->nseg > kFoldSegments;
  }
  a->slots = slots_of(a->rows, a->seg_len);
  const long long least = close_slots(a->rows, a->seg_len);
  long long idle = (a->slots.count - least) * tiles;
  if (backward) idle += ((long long)a->rows.n_seq * len - a->rows.T) * a->G / 256 * (2 * a->N / 4);  // of the sums
  *close = close_pays(a->rows, idle);
  if (*close) a->slots.count = least;
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
    if (e == cudaSuccess && a.carried) e = launch_scan_carry(a, false, s);
    if (e != cudaSuccess) return e;
  }
  return dispatch<kForward>(a, s);
}

cudaError_t launch_scan_reverse_summary(const ScanArgs& a, cudaStream_t s) { return dispatch<kReverseSummary>(a, s); }

}  // namespace palimpsa
