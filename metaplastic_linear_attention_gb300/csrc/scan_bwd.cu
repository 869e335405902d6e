// Selective scan, backward (formulas of the forward in scan_fwd.cu). With
// dpre_t = dy_t silu(z_t), a_t = exp(-A s_t) and g_t the gradient of h_t:
//   g_t   = C_t dpre_t + a_{t+1} g_{t+1}          (g after the last token: dh_T)
//   dC_t  = sum_d h_t dpre_t,     dB_t = sum_d g_t s_t x_t
//   w_t   = sum_n g_t B_t         (the gradient of s_t x_t)
//   p_t   = g_t a_t h_{t-1}       (the gradient of -A s_t)
//   dA    = -sum_t p_t s_t
//   ds_t  = w_t x_t - sum_n p_t A,  ddt_t = ds_t sigmoid(dt_t + dt_bias)
//   dx_t  = w_t s_t + dpre_t skip,  dskip = sum_t dpre_t x_t
//   dz_t  = dy_t (sum_n C_t h_t + skip x_t) silu'(z_t),  ddt_bias = sum_t ddt_t.
//
// The states come from the forward's checkpoints, one every 16 tokens. A CTA has a tile
// of 32 channels with all states and walks its tokens from the last chunk of 16 to the
// first; a lane holds a pair of channels x 4 states (two pairs at N = 128), a warp 16
// channels x 16 states. In a chunk, a first sweep from the checkpoint leaves the states
// before tokens 4, 8 and 12 in shared memory; then, from the last window of 4 tokens to
// the first, a second sweep fills the window's a_t and a_t h_{t-1} into registers (64 of
// them), the tokens are taken in reverse, and their sums are reduced together.
// What bounds it: about 16 FP32 operations and 2 exponentials per state-token (2 clocks
// per channel-token and SM at N = 16), and as much again for operands, reductions and the
// token arrays: issue slots, 61 % busy. Measured (GB300, bf16, N = 16, gate, 4 x 2048 x
// 1024): 169 us, 6 clocks, in the two waves of segments that are planned (158 in one, whose
// pass A takes 10 more). At N = 64 and 128, where an SM holds one CTA of 8 warps (230 to 255
// registers, spills at 128), 743 and 1415 us. Before: two pairs a lane (255 registers, 7 warps an SM) 231,
// reductions token by token 393; with 14 warps of 128 registers it spills (202).
//
// Sums. w, sum p A and sum C h go over the 4 lane groups by halves and over warps in
// shared memory; dB_t and dC_t over 8 lanes by halves and over the tile's two halves in
// shared memory, then to a row of scratch per tile; dA stays in registers, dskip and
// ddt_bias in shared memory until the segment's end, and go to scratch. One more kernel
// adds tiles and segments up in a fixed order: no atomics, the same bits every time. All
// sums are fp32; gradients of token arrays are rounded to the input type once.
#include <algorithm>
#include <atomic>

#include "ssm.cuh"

namespace palimpsa {
namespace {

constexpr int kChunk = kScanCheckpoint;
constexpr int kWin = 4;
constexpr int kWins = kChunk / kWin;
constexpr int kStages = 2;
constexpr int kWarpsPerSM = 12;  // up to N = 32
constexpr int CH = kScanChannels;

// Channel pairs of a lane: 1 (two warps share a tile's channels), or 2 at N = 128, where
// 16 warps of the former's registers do not fit an SM.
__host__ __device__ constexpr int pairs(int N) { return N == 128 ? 2 : 1; }
__host__ __device__ constexpr int parts(int N) { return CH / (16 * pairs(N)); }
__host__ __device__ constexpr int states(int N) { return N == 8 ? 2 : 4; }  // of a lane
__host__ __device__ constexpr int warps(int N) { return N / (4 * states(N)) * parts(N); }

// Shared memory of a CTA, bytes (all parts 16-byte aligned).
struct Smem {
  int rx, rdt, rz, rdy, rB, rC, rck, raw;  // one stage of raw inputs and a checkpoint
  int s, sx, dp;                           // fp32 operands
  int win;                                 // per warp and window: a state, then the window's sums
  int bc, acc, par, total;
  __host__ __device__ constexpr Smem(int N, int es)
      : rx(0),
        rdt(kChunk * CH * es),
        rz(2 * kChunk * CH * es),
        rdy(3 * kChunk * CH * es),
        rB(4 * kChunk * CH * es),
        rC(rB + kChunk * N * es),
        rck(rC + kChunk * N * es),
        raw(rck + CH * N * 4),
        s(kStages * raw),
        sx(s + kChunk * CH * 4),
        dp(sx + kChunk * CH * 4),
        win(dp + kChunk * CH * 4),
        bc(win + kWins * warps(N) * slot(N)),
        acc(bc + (parts(N) > 1 ? parts(N) * kChunk * 2 * N * 4 : 0)),
        par(acc + 32 * warps(N) * 2 * (16 / es) * 4),
        total(par + 2 * CH * 4) {}
  // Bytes of a warp's slot: the states of its lanes, or 3 sums of 4 tokens of its channels.
  static __host__ __device__ constexpr int slot(int N) {
    return 32 * 2 * pairs(N) * states(N) * 4 > 3 * kWin * 16 * pairs(N) * 4 ? 32 * 2 * pairs(N) * states(N) * 4
                                                                          : 3 * kWin * 16 * pairs(N) * 4;
  }
};

struct Partials {  // parts of the backward's scratch
  float* bc;   // [tiles][rows][2][N]: dB, dC
  long long rows;
  float* dA;   // [slots, D, N]
  float* par;  // [slots, 2, D]: dskip, ddt_bias
};

// NS values of a row of B or C as they came, each twice (for two channels).
template <bool BF16, int NS>
__device__ __forceinline__ void load_states(float2* f, const unsigned char* p) {
  float v[NS];
  if constexpr (BF16 && NS == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
  } else if constexpr (BF16) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    v[0] = bf16_lo(u); v[1] = bf16_hi(u);
  } else if constexpr (NS == 4) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  } else {
    const float2 u = *reinterpret_cast<const float2*>(p);
    v[0] = u.x; v[1] = u.y;
  }
#pragma unroll
  for (int j = 0; j < NS; ++j) f[j] = make_float2(v[j], v[j]);
}
// 2 CP values, as pairs.
template <int CP>
__device__ __forceinline__ void load_pairs(float2* f, const float* p) {
  if constexpr (CP == 2) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = make_float2(v.x, v.y);
    f[1] = make_float2(v.z, v.w);
  } else {
    f[0] = *reinterpret_cast<const float2*>(p);
  }
}
// The kept half of two vectors plus the partner's copy of it (the partner keeps the other).
template <int M>
__device__ __forceinline__ void halve(float* out, const float* a, const float* b, bool second, int lane_mask) {
#pragma unroll
  for (int k = 0; k < M; ++k)
    out[k] = (second ? b[k] : a[k]) + __shfl_xor_sync(0xffffffffu, second ? a[k] : b[k], lane_mask);
}

template <bool BF16, int N>
__global__ void __launch_bounds__(32 * warps(N), N == 128 ? 1 : kWarpsPerSM / warps(N))
palimpsa_scan_bwd_kernel(ScanArgs a, Partials part, int tiles) {
  using V = Vec<BF16>;
  constexpr int VN = V::n, ES = V::bytes, NS = states(N), CP = pairs(N), CPC = 2 * CP, W = warps(N), NT = 32 * W;
  constexpr int VPR = CH / VN, BPR = N / VN, kParts = parts(N);
  constexpr Smem L(N, ES);
  extern __shared__ __align__(128) unsigned char smem[];
  float* const fs = reinterpret_cast<float*>(smem + L.s);
  float* const fsx = reinterpret_cast<float*>(smem + L.sx);
  float* const fdp = reinterpret_cast<float*>(smem + L.dp);
  float4* const facc = reinterpret_cast<float4*>(smem + L.acc) + threadIdx.x;
  float* const fpar = reinterpret_cast<float*>(smem + L.par);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = (int)(blockIdx.x % tiles);
  const long long rest = blockIdx.x / tiles;
  int n, seg;
  if (!slot_place(a.rows, a.slots, rest, &n, &seg)) return;
  const int per_group = a.D / a.G, tpg = (per_group + CH - 1) / CH;
  const int g = tile / tpg, ch0 = g * per_group + (tile % tpg) * CH;
  const int nch = min(CH, (g + 1) * per_group - ch0);
  long long row0;
  int len;
  if (!seq_rows(a.rows, n, &row0, &len)) {
    if (tile == 0 && seg == 0 && tid == 0) latch_status(a.status, kStatusDomain);
    return;
  }
  const int tb = seg * a.seg_len, te = min(len, tb + a.seg_len);
  if (tb >= len && seg > 0) return;
  const int tn = te - tb, nchunk = (tn + kChunk - 1) / kChunk;

  // A lane's CPC channels of the tile from d0 on, as pairs, and its states from n0 on. Quads
  // of 4 channels of odd tokens change places in pairs in shared memory, as in the forward.
  const int cl = lane & 7, sl = lane >> 3, wpart = warp % kParts, n0 = (warp / kParts * 4 + sl) * NS;
  const int d0 = wpart * 16 * CP + CPC * cl, cq0 = d0, cq1 = d0 ^ 4;
  const size_t at = (size_t)(ch0 + d0) * N + n0;  // of the first channel in [D, N]
  bool bad = false;
  float2 A2[CP][NS], gh[CP][NS], dA[CP][NS];
  const float* g0 = nullptr;
  const long long slot0 = rest - seg;  // of the sequence
  if (a.carried) g0 = a.seg_state + (size_t)rest * a.D * N;
  else if (a.dh_T) g0 = a.dh_T + (size_t)n * a.D * N;
#pragma unroll
  for (int c = 0; c < CPC; ++c) {
    const bool in = d0 + c < nch;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const float A = in ? a.A[at + c * N + j] : 1.f;
      bad |= !pos_finite(A);
      (c & 1 ? A2[c / 2][j].y : A2[c / 2][j].x) = decay_rate(A);
      (c & 1 ? gh[c / 2][j].y : gh[c / 2][j].x) = in && g0 ? g0[at + c * N + j] : 0.f;
      dA[c / 2][j] = make_float2(0.f, 0.f);
    }
  }
  const int nsegs = (len + a.seg_len - 1) / a.seg_len;  // the sequence's; the ones after this one's summaries
  if (seg + 1 < nsegs && !a.carried && d0 < nch)
    fold_segments<CPC, NS>(gh, A2, a.seg_state + (size_t)(slot0 + nsegs - 1) * a.D * N + at,
                           a.seg_dt + (size_t)(slot0 + nsegs - 1) * a.D + ch0 + d0, nsegs - 1 - seg, -1, a.D, N);
  for (int c = tid; c < CH; c += NT) {
    fpar[c] = c < nch && a.dt_bias ? a.dt_bias[ch0 + c] : 0.f;
    fpar[CH + c] = c < nch && a.skip ? a.skip[ch0 + c] : 0.f;
  }
  // Sums over tokens of dskip and ddt_bias of the channels that a thread stores: 2 VN
  // floats, each thread's own.
#pragma unroll
  for (int k = 0; k < VN / 2; ++k) facc[k * NT] = make_float4(0.f, 0.f, 0.f, 0.f);

  // Copies, from the last chunk to the first. A thread copies in, converts and finishes
  // the same vectors; their place v in a row is the same for all of them.
  const long long rb = row0 + tb;
  const int v = tid % VPR;
  const bool vin = v * VN < nch, gated = a.z != nullptr;
  const char* const gx = static_cast<const char*>(a.x) + (rb * a.x_ld + ch0) * ES + v * 16;
  const char* const gdt = static_cast<const char*>(a.dt) + (rb * a.dt_ld + ch0) * ES + v * 16;
  const char* const gz = gated ? static_cast<const char*>(a.z) + (rb * a.z_ld + ch0) * ES + v * 16 : nullptr;
  const char* const gdy = static_cast<const char*>(a.dy) + (rb * a.dy_ld + ch0) * ES + v * 16;
  const char* const gB = static_cast<const char*>(a.B) + (rb * a.B_ld + g * N) * ES;
  const char* const gC = static_cast<const char*>(a.C) + (rb * a.C_ld + g * N) * ES;
  const float* const gck =
      a.ckpt_in + (scan_ckpt_row0(a.rows, n, row0) + tb / kScanCheckpoint) * a.D * N + at;
  auto stage = [&](int c) {  // copies of the c-th chunk from the end, as one group
    if (c < nchunk) {
      unsigned char* const st = smem + (c % kStages) * L.raw;
      const int ci = nchunk - 1 - c, t0 = ci * kChunk, nt = min(kChunk, tn - t0);
#pragma unroll
      for (int i = tid; i < kChunk * VPR; i += NT) {
        const int t = i / VPR;
        if (t >= nt || !vin) continue;
        const long long r = (long long)(t0 + t) * ES;
        cp_async16(st + L.rx + 16 * i, gx + r * a.x_ld);
        cp_async16(st + L.rdt + 16 * i, gdt + r * a.dt_ld);
        if (gated) cp_async16(st + L.rz + 16 * i, gz + r * a.z_ld);
        cp_async16(st + L.rdy + 16 * i, gdy + r * a.dy_ld);
      }
#pragma unroll
      for (int i = tid; i < kChunk * BPR; i += NT) {
        const int t = i / BPR, o = i % BPR * 16;
        const long long r = (long long)(t0 + min(t, nt - 1)) * ES;
        cp_async16(st + L.rB + 16 * i, gB + r * a.B_ld + o, t < nt);
        cp_async16(st + L.rC + 16 * i, gC + r * a.C_ld + o, t < nt);
      }
      // each lane its own part of the checkpoint
      const float* const ck = gck + (long long)ci * a.D * N;
#pragma unroll
      for (int k = 0; k < CPC; ++k)
        if (d0 + k < nch) cp_async_states<NS>(st + L.rck + (k * NT + tid) * NS * 4, ck + k * N);
    }
    cp_async_commit();
  };
  stage(0);

  for (int c = 0; c < nchunk; ++c) {
    const int ci = nchunk - 1 - c, t0 = ci * kChunk, nt = min(kChunk, tn - t0);
    cp_async_wait<0>();
    cta_sync<W>();  // chunk c is here; the other stage, the operands and the sums are free
    stage(c + 1);
    const unsigned char* const st = smem + (c % kStages) * L.raw;
    // Tokens past the end and channels past the tile count as s = s x = dpre = 0 (and B = C
    // = 0): they change nothing.
#pragma unroll
    for (int i = tid; i < kChunk * VPR; i += NT) {
      const int t = i / VPR;
      float s[VN], x[VN], d[VN];
      if (t < nt && vin) {
        V::unpack(*reinterpret_cast<const uint4*>(st + L.rdt + 16 * i), s);
        V::unpack(*reinterpret_cast<const uint4*>(st + L.rx + 16 * i), x);
        V::unpack(*reinterpret_cast<const uint4*>(st + L.rdy + 16 * i), d);
#pragma unroll
        for (int k = 0; k < VN; k += 2) {
          float2 u = __fadd2_rn(make_float2(s[k], s[k + 1]), *reinterpret_cast<const float2*>(fpar + v * VN + k));
          if (a.softplus) u = softplus_fast(u);
          bad |= !(nonneg_finite(u.x) && nonneg_finite(u.y));
          const float2 sx = __fmul2_rn(u, make_float2(x[k], x[k + 1]));
          s[k] = u.x;
          s[k + 1] = u.y;
          x[k] = sx.x;
          x[k + 1] = sx.y;
        }
        if (gated) {
          float z[VN];
          V::unpack(*reinterpret_cast<const uint4*>(st + L.rz + 16 * i), z);
#pragma unroll
          for (int k = 0; k < VN; k += 2) {
            const float2 e = __fmul2_rn(make_float2(d[k], d[k + 1]), silu_fast(make_float2(z[k], z[k + 1])));
            d[k] = e.x;
            d[k + 1] = e.y;
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < VN; ++k) s[k] = x[k] = d[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < VN; k += 4) {
        const int o = t * CH + ((v * VN + k) ^ 4 * (t & 1));
        *reinterpret_cast<float4*>(fs + o) = make_float4(s[k], s[k + 1], s[k + 2], s[k + 3]);
        *reinterpret_cast<float4*>(fsx + o) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
        *reinterpret_cast<float4*>(fdp + o) = make_float4(d[k], d[k + 1], d[k + 2], d[k + 3]);
      }
    }
    cta_sync<W>();

    float2 h[CP][NS];
    // A lane's states in its own places of shared memory (CPC channels of NS states).
    auto load_h = [&](const unsigned char* p) {
#pragma unroll
      for (int k = 0; k < CPC; ++k) {
        float q[NS];
        load_own<NS>(q, p + (k * NT + tid) * NS * 4);
#pragma unroll
        for (int j = 0; j < NS; ++j) (k & 1 ? h[k / 2][j].y : h[k / 2][j].x) = d0 + k < nch ? q[j] : 0.f;
      }
    };
    unsigned char* const slots = smem + L.win + warp * (kWins * L.slot(N));
    auto slot_h = [&](int w) { return slots + w * L.slot(N) + lane * NS * 4; };
    // First sweep: the states before tokens 4, 8, 12.
    load_h(st + L.rck);
#pragma unroll 1
    for (int w = 0; w < kWins - 1; ++w) {
#pragma unroll
      for (int i = 0; i < kWin; ++i) {
        const int t = w * kWin + i, q = i & 1 ? cq1 : cq0;
        float2 s[CP], x[CP], b[NS];
        load_pairs<CP>(s, fs + t * CH + q);
        load_pairs<CP>(x, fsx + t * CH + q);
        load_states<BF16, NS>(b, st + L.rB + (t * N + n0) * ES);
#pragma unroll
        for (int p = 0; p < CP; ++p)
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            const float2 u = decay_exponent(s[p], A2[p][j]);
            const float2 e = make_float2(ex2_approx(u.x), ex2_approx(u.y));
            h[p][j] = __ffma2_rn(x[p], b[j], __fmul2_rn(e, h[p][j]));
          }
      }
#pragma unroll
      for (int k = 0; k < CPC; ++k) {
        float q[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) q[j] = k & 1 ? h[k / 2][j].y : h[k / 2][j].x;
        store_own<NS>(slot_h(w + 1) + k * 32 * NS * 4, q);
      }
    }

    // Windows, last to first.
#pragma unroll 1
    for (int w = kWins - 1; w >= 0; --w) {
      if (w == 0) {
        load_h(st + L.rck);
      } else {
#pragma unroll
        for (int k = 0; k < CPC; ++k) {
          float q[NS];
          load_own<NS>(q, slot_h(w) + k * 32 * NS * 4);
#pragma unroll
          for (int j = 0; j < NS; ++j) (k & 1 ? h[k / 2][j].y : h[k / 2][j].x) = q[j];
        }
      }
      float2 al[kWin][CP][NS], ah[kWin][CP][NS];  // a_t and a_t h_{t-1}
#pragma unroll
      for (int i = 0; i < kWin; ++i) {
        const int t = w * kWin + i, q = i & 1 ? cq1 : cq0;
        float2 s[CP], x[CP], b[NS];
        load_pairs<CP>(s, fs + t * CH + q);
        load_pairs<CP>(x, fsx + t * CH + q);
        load_states<BF16, NS>(b, st + L.rB + (t * N + n0) * ES);
#pragma unroll
        for (int p = 0; p < CP; ++p)
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            const float2 u = decay_exponent(s[p], A2[p][j]);
            al[i][p][j] = make_float2(ex2_approx(u.x), ex2_approx(u.y));
            ah[i][p][j] = __fmul2_rn(al[i][p][j], h[p][j]);
            h[p][j] = __ffma2_rn(x[p], b[j], ah[i][p][j]);
          }
      }
      // Sums of a token over the lane's channels (dB, dC) and states (w, sum p A, sum C h).
      float db[kWin][NS], dc[kWin][NS], sum[3][kWin][CPC];
#pragma unroll
      for (int i = kWin - 1; i >= 0; --i) {
        const int t = w * kWin + i, q = i & 1 ? cq1 : cq0;
        float2 s[CP], x[CP], d[CP], b[NS], cc[NS];
        load_pairs<CP>(s, fs + t * CH + q);
        load_pairs<CP>(x, fsx + t * CH + q);
        load_pairs<CP>(d, fdp + t * CH + q);
        load_states<BF16, NS>(b, st + L.rB + (t * N + n0) * ES);
        load_states<BF16, NS>(cc, st + L.rC + (t * N + n0) * ES);
        float2 ws[CP], qs[CP], ys[CP];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          float2 dcj, dbj;
#pragma unroll
          for (int p = 0; p < CP; ++p) {
            const float2 carried = ah[i][p][j];
            const float2 ht = __ffma2_rn(x[p], b[j], carried);
            const float2 gt = __ffma2_rn(cc[j], d[p], gh[p][j]);
            const float2 pt = __fmul2_rn(gt, carried);
            dcj = p == 0 ? __fmul2_rn(ht, d[p]) : __ffma2_rn(ht, d[p], dcj);
            dbj = p == 0 ? __fmul2_rn(gt, x[p]) : __ffma2_rn(gt, x[p], dbj);
            ws[p] = j == 0 ? __fmul2_rn(gt, b[j]) : __ffma2_rn(gt, b[j], ws[p]);
            qs[p] = j == 0 ? __fmul2_rn(pt, A2[p][j]) : __ffma2_rn(pt, A2[p][j], qs[p]);
            ys[p] = j == 0 ? __fmul2_rn(ht, cc[j]) : __ffma2_rn(ht, cc[j], ys[p]);
            dA[p][j] = __ffma2_rn(pt, s[p], dA[p][j]);
            gh[p][j] = __fmul2_rn(gt, al[i][p][j]);
          }
          dc[i][j] = dcj.x + dcj.y;
          db[i][j] = dbj.x + dbj.y;
        }
#pragma unroll
        for (int p = 0; p < CP; ++p) {
          sum[0][i][2 * p] = ws[p].x; sum[0][i][2 * p + 1] = ws[p].y;
          sum[1][i][2 * p] = qs[p].x; sum[1][i][2 * p + 1] = qs[p].y;
          sum[2][i][2 * p] = ys[p].x; sum[2][i][2 * p + 1] = ys[p].y;
        }
      }
      if (nch < CH && d0 >= nch) {  // lanes past the tile's channels: 0, whatever B and C hold
#pragma unroll
        for (int i = 0; i < kWin; ++i)
#pragma unroll
          for (int j = 0; j < NS; ++j) db[i][j] = dc[i][j] = 0.f;
      }
      // Over the 4 lane groups: group sl ends with token sl, CPC channels a lane.
      __syncwarp();  // every lane has read its states from the slot
      float* const sm = reinterpret_cast<float*>(slots + w * L.slot(N)) + sl * 16 * CP + CPC * cl;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        float two[2 * CPC], one[CPC];
        halve<2 * CPC>(two, &sum[k][0][0], &sum[k][2][0], sl & 2, 16);
        halve<CPC>(one, two, two + CPC, sl & 1, 8);
        store_own<CPC>(reinterpret_cast<unsigned char*>(sm + k * kWin * 16 * CP), one);
      }
      // Over the 8 lanes that share states: lane cl ends with token cl & 3 of dC (cl & 4)
      // or dB, NS states.
      {
        float four[4 * NS], two[2 * NS], one[NS];
        halve<4 * NS>(four, &db[0][0], &dc[0][0], cl & 4, 4);
        halve<2 * NS>(two, four, four + 2 * NS, cl & 2, 2);
        halve<NS>(one, two, two + NS, cl & 1, 1);
        const int t = w * kWin + (cl & 3);
        if constexpr (kParts > 1) {
          store_own<NS>(smem + L.bc + (((wpart * kChunk + t) * 2 + (cl >> 2)) * N + n0) * 4, one);
        } else if (t < nt) {
          store_own<NS>(reinterpret_cast<unsigned char*>(
                            part.bc + ((tile * part.rows + rb + t0 + t) * 2 + (cl >> 2)) * N + n0),
                        one);
        }
      }
    }
    cta_sync<W>();

    if constexpr (kParts > 1) {  // dB, dC of the tile: the parts' rows lie as the scratch's do
      float4* const out = reinterpret_cast<float4*>(part.bc + (tile * part.rows + rb + t0) * 2 * N);
      const float4* const in = reinterpret_cast<const float4*>(smem + L.bc);
      for (int i = tid; i < nt * 2 * N / 4; i += NT) {
        float4 q = in[i];
#pragma unroll
        for (int k = 1; k < kParts; ++k) {
          const float4 e = in[k * kChunk * 2 * N / 4 + i];
          q.x += e.x; q.y += e.y; q.z += e.z; q.w += e.w;
        }
        out[i] = q;
      }
    }
    // Gradients of the tokens' arrays.
#pragma unroll
    for (int i = tid; i < kChunk * VPR; i += NT) {
      const int t = i / VPR;
      if (t >= nt || !vin) continue;
      float x[VN], dt[VN], dy[VN], z[VN], dx[VN], ddt[VN];
      V::unpack(*reinterpret_cast<const uint4*>(st + L.rx + 16 * i), x);
      V::unpack(*reinterpret_cast<const uint4*>(st + L.rdt + 16 * i), dt);
      V::unpack(*reinterpret_cast<const uint4*>(st + L.rdy + 16 * i), dy);
      if (gated) V::unpack(*reinterpret_cast<const uint4*>(st + L.rz + 16 * i), z);
#pragma unroll
      for (int k0 = 0; k0 < VN; k0 += 4) {
        const int o = (v * VN + k0) ^ 4 * (t & 1);
        float sums[3][4] = {};
#pragma unroll
        for (int wp = 0; wp < W / kParts; ++wp)  // the warps of the channels' part
#pragma unroll
          for (int r = 0; r < 3; ++r) {
            const int dd = v * VN + k0;
            const float4 q = *reinterpret_cast<const float4*>(
                smem + L.win + ((wp * kParts + dd / (16 * CP)) * kWins + t / kWin) * L.slot(N) +
                ((r * kWin + t % kWin) * 16 * CP + dd % (16 * CP)) * 4);
            sums[r][0] += q.x; sums[r][1] += q.y; sums[r][2] += q.z; sums[r][3] += q.w;
          }
        const float4 s4 = *reinterpret_cast<const float4*>(fs + t * CH + o);
        const float4 d4 = *reinterpret_cast<const float4*>(fdp + t * CH + o);
        const float sv[4] = {s4.x, s4.y, s4.z, s4.w}, dv[4] = {d4.x, d4.y, d4.z, d4.w};
        float4 a0 = facc[(k0 / 2) * NT], a1 = facc[(k0 / 2 + 1) * NT];  // dskip, ddt_bias
        float *const s0 = &a0.x, *const s1 = &a1.x;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int k = k0 + m;
          const float skip = fpar[CH + v * VN + k];
          dx[k] = fmaf(sums[0][m], sv[m], dv[m] * skip);
          // the second sum holds -log2(e) sum p A
          ddt[k] = fmaf(sums[0][m], x[k], sums[1][m] * 0.6931471805599453f);
          if (a.softplus) ddt[k] *= sigmoid_fast(dt[k] + fpar[v * VN + k]);
          s0[m] = fmaf(dv[m], x[k], s0[m]);
          s1[m] += ddt[k];
          if (gated) {
            const float q = sigmoid_fast(z[k]);
            z[k] = dy[k] * fmaf(skip, x[k], sums[2][m]) * (q * fmaf(z[k], 1.f - q, 1.f));
          }
        }
        facc[(k0 / 2) * NT] = a0;
        facc[(k0 / 2 + 1) * NT] = a1;
      }
      const long long to = ((rb + t0 + t) * a.D + ch0 + v * VN) * ES;
      *reinterpret_cast<uint4*>(static_cast<char*>(a.dx) + to) = V::pack(dx);
      *reinterpret_cast<uint4*>(static_cast<char*>(a.ddt) + to) = V::pack(ddt);
      if (gated) *reinterpret_cast<uint4*>(static_cast<char*>(a.dz) + to) = V::pack(z);
    }
  }
  if (bad) latch_status(a.status, kStatusDomain);

  const size_t ns = (size_t)rest;
#pragma unroll
  for (int c = 0; c < CPC; ++c) {
    if (d0 + c >= nch) continue;
    float q[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) q[j] = -(c & 1 ? dA[c / 2][j].y : dA[c / 2][j].x);
    store_own<NS>(reinterpret_cast<unsigned char*>(part.dA + ns * a.D * N + at + c * N), q);
    if (tb == 0 && a.dh0) {
#pragma unroll
      for (int j = 0; j < NS; ++j) q[j] = c & 1 ? gh[c / 2][j].y : gh[c / 2][j].x;
      store_own<NS>(reinterpret_cast<unsigned char*>(a.dh0 + (size_t)n * a.D * N + at + c * N), q);
    }
  }
  // dskip, ddt_bias of the segment: the threads of a vector, added up in thread order.
  __syncthreads();
  for (int e = tid; e < 2 * nch; e += NT) {
    const int which = e / nch, ch = e % nch, vv = ch / VN, k = ch % VN;
    const float* const f = reinterpret_cast<const float*>(smem + L.acc) + (k / 4 * 2 + which) * NT * 4 + k % 4;
    float s = 0.f;
    for (int t = vv; t < NT; t += VPR) s += f[t * 4];
    part.par[(ns * 2 + which) * a.D + ch0 + ch] = s;
  }
}

// The sums that the tiles and segments left, in one launch: CTAs 0 .. bc_ctas - 1 add
// up dB and dC over the tiles of a group (one thread per 4 values of a row's [2][N]),
// the next dA_ctas add up dA over sequences and segments, the rest dskip and ddt_bias.
template <bool BF16>
__device__ __forceinline__ void sum_bc(const ScanArgs& a, const Partials& part, int tpg, long long i) {
  const int per = 2 * a.N / 4;  // threads of a row and group
  const int q = (int)(i % per), g = (int)(i / per % a.G);
  const long long r = i / per / a.G;
  long long row0;
  int n, t, len;
  if (r >= a.row_slots.count || !slot_place(a.rows, a.row_slots, r, &n, &t)) return;
  if (!seq_rows(a.rows, n, &row0, &len) || t >= len) return;
  const long long row = row0 + t;
  const float* const p = part.bc + ((long long)g * tpg * part.rows + row) * 2 * a.N + 4 * q;
  const long long stride = part.rows * 2 * a.N;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 16
  for (int k = 0; k < tpg; ++k) {
    const float4 v = *reinterpret_cast<const float4*>(p + k * stride);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  const int half = q >= per / 2;
  const long long at = (row * a.G + g) * a.N + 4 * q - (half ? a.N : 0);
  void* const out = half ? a.dC : a.dB;
  if constexpr (BF16)
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
        make_uint2(Vec<true>::two(s.x, s.y), Vec<true>::two(s.z, s.w));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = s;
}

// The `per` values of one (sequence, segment) lie together in p, the first `split` of
// them for out and the others for out2 (either may be null). 32 values by 8 slices of the
// sum to a CTA.
__device__ __forceinline__ void sum_segments(const ScanArgs& a, long long block, const float* p, long long per,
                                             long long split, float* out, float* out2) {
  __shared__ float red[8][33];
  const int cx = threadIdx.x % 32, sy = threadIdx.x / 32;
  const long long e = block * 32 + cx;
  float s = 0.f;
  if (e < per && a.slots.starts) {
    const int count = a.slots.starts[a.rows.n_seq];
#pragma unroll 4
    for (int i = sy; i < count; i += 8) s += p[i * per + e];
  } else if (e < per) {
#pragma unroll 4
    for (long long i = sy; i < a.slots.count; i += 8) {
      long long row0;
      int len;
      // (an empty sequence has its first segment's zeros; a skipped one has nothing)
      if (!seq_rows(a.rows, i / a.nseg, &row0, &len)) continue;
      const long long k = i % a.nseg;
      if (k == 0 || k * a.seg_len < len) s += p[i * per + e];
    }
  }
  red[sy][cx] = s;
  __syncthreads();
  if (sy || e >= per) return;
  for (int k = 1; k < 8; ++k) s += red[k][cx];
  if (e >= split) out = out2 ? out2 - split : nullptr;
  if (out) out[e] = s;
}

template <bool BF16>
__global__ void __launch_bounds__(256) palimpsa_scan_bwd_sum_kernel(ScanArgs a, Partials part, int tpg, unsigned bc_ctas,
                                                                    unsigned dA_ctas) {
  const unsigned b = blockIdx.x;
  const long long dn = (long long)a.D * a.N;
  if (b < bc_ctas) sum_bc<BF16>(a, part, tpg, (long long)b * 256 + threadIdx.x);
  else if (b < bc_ctas + dA_ctas) sum_segments(a, b - bc_ctas, part.dA, dn, dn, a.dA, nullptr);
  else sum_segments(a, b - bc_ctas - dA_ctas, part.par, 2ll * a.D, a.D, a.dskip, a.ddt_bias);
}

long long total_rows(const ScanArgs& a) { return a.rows.cu ? a.rows.T : (long long)a.rows.n_seq * a.rows.T; }

template <bool BF16, int N>
cudaError_t prepare() {
  constexpr Smem L(N, Vec<BF16>::bytes);
  if (L.total <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(palimpsa_scan_bwd_kernel<BF16, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              L.total);
}

// CTAs that an SM holds (from the occupancy calculator, once per kernel); 0 on failure.
template <bool BF16, int N>
int resident() {
  static std::atomic<int> known{0};
  int r = known.load(std::memory_order_relaxed);
  if (r > 0) return r;
  constexpr Smem L(N, Vec<BF16>::bytes);
  if (prepare<BF16, N>() != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&r, palimpsa_scan_bwd_kernel<BF16, N>, 32 * warps(N), L.total) !=
          cudaSuccess)
    return 0;
  known.store(r, std::memory_order_relaxed);
  return r;
}

template <bool BF16, int N>
cudaError_t run(const ScanArgs& a, const Partials& part, cudaStream_t s) {
  constexpr Smem L(N, Vec<BF16>::bytes);
  const long long tiles = scan_tiles(a), blocks = tiles * a.slots.count;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaError_t e = prepare<BF16, N>();
  if (e != cudaSuccess) return e;
  palimpsa_scan_bwd_kernel<BF16, N><<<(unsigned)blocks, 32 * warps(N), L.total, s>>>(a, part, (int)tiles);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long bc_ctas = (a.row_slots.count * a.G * (2 * a.N / 4) + 255) / 256;
  const long long dA_ctas = ((long long)a.D * a.N + 31) / 32, par_ctas = (2 * a.D + 31) / 32;
  if (bc_ctas + dA_ctas + par_ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  palimpsa_scan_bwd_sum_kernel<BF16><<<(unsigned)(bc_ctas + dA_ctas + par_ctas), 256, 0, s>>>(
      a, part, (int)(tiles / a.G), (unsigned)bc_ctas, (unsigned)dA_ctas);
  return cudaGetLastError();
}

size_t bc_floats(const ScanArgs& a) { return (size_t)scan_tiles(a) * total_rows(a) * 2 * a.N; }

}  // namespace

size_t scan_backward_scratch_floats(const ScanArgs& a) {
  const size_t ns = (size_t)a.slots.count;
  return bc_floats(a) + ns * a.D * a.N + ns * 2 * a.D;
}

cudaError_t launch_scan_backward(const ScanArgs& a, float* scratch, cudaStream_t s) {
  Partials part;
  part.bc = scratch;
  part.rows = total_rows(a);
  part.dA = part.bc + bc_floats(a);
  part.par = part.dA + (size_t)a.slots.count * a.D * a.N;
  if (a.nseg > 1) {
    cudaError_t e = launch_scan_reverse_summary(a, s);
    if (e == cudaSuccess && a.carried) e = launch_scan_carry(a, true, s);
    if (e != cudaSuccess) return e;
  }
  switch (a.N) {
    case 8: return a.bf16 ? run<true, 8>(a, part, s) : run<false, 8>(a, part, s);
    case 16: return a.bf16 ? run<true, 16>(a, part, s) : run<false, 16>(a, part, s);
    case 32: return a.bf16 ? run<true, 32>(a, part, s) : run<false, 32>(a, part, s);
    case 64: return a.bf16 ? run<true, 64>(a, part, s) : run<false, 64>(a, part, s);
    default: return a.bf16 ? run<true, 128>(a, part, s) : run<false, 128>(a, part, s);
  }
}

int scan_backward_resident(const ScanArgs& a) {
  switch (a.N) {
    case 8: return a.bf16 ? resident<true, 8>() : resident<false, 8>();
    case 16: return a.bf16 ? resident<true, 16>() : resident<false, 16>();
    case 32: return a.bf16 ? resident<true, 32>() : resident<false, 32>();
    case 64: return a.bf16 ? resident<true, 64>() : resident<false, 64>();
    default: return a.bf16 ? resident<true, 128>() : resident<false, 128>();
  }
}

}  // namespace palimpsa
