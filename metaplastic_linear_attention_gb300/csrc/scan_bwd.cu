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
// The states come from the forward's checkpoints, one every 16 tokens. A CTA has
// the forward's tile (32 channels, all states, N / 16 warps; a lane 4 channels x
// 4 states) and walks its tokens from the last chunk of 16 to the first. In a
// chunk, a first sweep from the checkpoint leaves the state before tokens 4, 8
// and 12 in shared memory; then, from the last window of 4 tokens to the first, a
// second sweep fills the window's a_t and a_t h_{t-1} into registers (128 of them)
// and the tokens are taken in reverse. The windows hold 4 tokens because two
// values x 16 states x 4 tokens are half of a lane's registers: two CTA warps per
// scheduler stay resident.
// What bounds it: about 16 FP32 operations and 2 exponentials per state-token,
// 2 clocks per channel-token and SM at N = 16, and as much of the shared-memory
// and shuffle pipe.
//
// Sums. w, sum p A and sum C h go over the 4 lane groups by reduce-scatter and over
// warps in shared memory; dB_t and dC_t over the 32 channels by reduce-scatter, then
// to a row of scratch per tile; dA, dskip, ddt_bias stay in registers until the
// segment's end and go to scratch. Small kernels add tiles and segments up in a
// fixed order: no atomics, the same bits every time. All sums are fp32; gradients
// of token arrays are rounded to the input type once.
#include <algorithm>

#include "ssm.cuh"

namespace palimpsa {
namespace {

constexpr int kChunk = kScanCheckpoint;
constexpr int kWin = 4;
constexpr int kStages = 2;
constexpr int CH = kScanChannels;

struct Smem {
  int rx, rdt, rz, rdy, rB, rC, rck, raw;
  int s, sx, dp, B, C, sub, sum, par, total;
  __host__ __device__ Smem(int N, int W, int es) {
    const int row = kChunk * CH * es;
    rx = 0;
    rdt = rx + row;
    rz = rdt + row;
    rdy = rz + row;
    rB = rdy + row;
    rC = rB + kChunk * N * es;
    rck = rC + kChunk * N * es;
    raw = rck + CH * N * 4;
    s = kStages * raw;
    sx = s + kChunk * CH * 4;
    dp = sx + kChunk * CH * 4;
    B = dp + kChunk * CH * 4;
    C = B + kChunk * N * 4;
    sub = C + kChunk * N * 4;
    sum = sub + (kChunk / kWin - 1) * CH * N * 4;
    par = sum + 3 * W * kChunk * CH * 4;
    total = par + 2 * CH * 4;
  }
};

struct Partials {  // parts of the backward's scratch
  float* bc;   // [tiles][rows][2][N]: dB, dC
  long long rows;
  float* dA;   // [n_seq, nseg, D, N]
  float* par;  // [n_seq, nseg, 2, D]: dskip, ddt_bias
};

// Sum over the 4 lane groups of 4 channels' values: lane (cl, sl) ends with
// channel 4 cl + sl.
__device__ __forceinline__ float scatter_groups(const float* y, int sl) {
  const bool hi = sl & 2, odd = sl & 1;
  const float k0 = hi ? y[2] : y[0], k1 = hi ? y[3] : y[1];
  const float r0 = k0 + __shfl_xor_sync(0xffffffffu, hi ? y[0] : y[2], 16);
  const float r1 = k1 + __shfl_xor_sync(0xffffffffu, hi ? y[1] : y[3], 16);
  return (odd ? r1 : r0) + __shfl_xor_sync(0xffffffffu, odd ? r0 : r1, 8);
}

template <bool BF16, int NS>
__global__ void __launch_bounds__(256) palimpsa_scan_bwd_kernel(ScanArgs a, Partials part, int tiles, int W) {
  using V = Vec<BF16>;
  constexpr int VN = V::n, ES = V::bytes, NP = NS / 2;
  constexpr int VPR = CH / VN;
  const int N = 4 * NS * W, NT = 32 * W, BPR = N / VN;
  extern __shared__ __align__(128) unsigned char smem[];
  const Smem L(N, W, ES);
  float* const fs = reinterpret_cast<float*>(smem + L.s);
  float* const fsx = reinterpret_cast<float*>(smem + L.sx);
  float* const fdp = reinterpret_cast<float*>(smem + L.dp);
  float* const fB = reinterpret_cast<float*>(smem + L.B);
  float* const fC = reinterpret_cast<float*>(smem + L.C);
  float* const fsum = reinterpret_cast<float*>(smem + L.sum);
  float* const fbias = reinterpret_cast<float*>(smem + L.par);
  float* const fskip = fbias + CH;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = (int)(blockIdx.x % tiles);
  const long long rest = blockIdx.x / tiles;
  const int seg = (int)(rest % a.nseg);
  const long long n = rest / a.nseg;
  const int per_group = a.D / a.G, tpg = (per_group + CH - 1) / CH;
  const int g = tile / tpg, ch0 = g * per_group + (tile % tpg) * CH;
  const int nch = min(CH, (g + 1) * per_group - ch0);
  const int nv = nch / VN;
  long long row0;
  int len;
  if (!seq_rows(a.rows, n, &row0, &len)) {
    if (tile == 0 && seg == 0 && tid == 0) latch_status(a.status, kStatusDomain);
    return;
  }
  const int tb = seg * a.seg_len, te = min(len, tb + a.seg_len);
  if (tb >= len && seg > 0) return;
  const int tn = te - tb, nchunk = (tn + kChunk - 1) / kChunk;

  const int cl = lane & 7, sl = lane >> 3;
  const int n0 = warp * 4 * NS + sl * NS;
  bool bad = false;
  float2 A2[4][NP], gh[4][NP], dA[4][NP];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int d = 4 * cl + c;
    const bool in = d < nch;
    const float* g0 = nullptr;
    if (in) {
      if (a.nseg > 1) g0 = a.seg_state + ((size_t)(n * a.nseg + seg) * a.D + ch0 + d) * N + n0;
      else if (a.dh_T) g0 = a.dh_T + ((size_t)n * a.D + ch0 + d) * N + n0;
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const float2 v = in ? *reinterpret_cast<const float2*>(a.A + (size_t)(ch0 + d) * N + n0 + 2 * p)
                          : make_float2(1.f, 1.f);
      bad |= !(pos_finite(v.x) && pos_finite(v.y));
      A2[c][p] = make_float2(-kLog2e * v.x, -kLog2e * v.y);
      gh[c][p] = g0 ? *reinterpret_cast<const float2*>(g0 + 2 * p) : make_float2(0.f, 0.f);
      dA[c][p] = make_float2(0.f, 0.f);
    }
  }
  for (int c = tid; c < CH; c += NT) {
    fbias[c] = c < nch && a.dt_bias ? a.dt_bias[ch0 + c] : 0.f;
    fskip[c] = c < nch && a.skip ? a.skip[ch0 + c] : 0.f;
  }

  const long long rb = row0 + tb;
  const char* const gx = static_cast<const char*>(a.x) + (rb * a.x_ld + ch0) * ES;
  const char* const gdt = static_cast<const char*>(a.dt) + (rb * a.dt_ld + ch0) * ES;
  const char* const gz = a.z ? static_cast<const char*>(a.z) + (rb * a.z_ld + ch0) * ES : nullptr;
  const char* const gdy = static_cast<const char*>(a.dy) + (rb * a.dy_ld + ch0) * ES;
  const char* const gB = static_cast<const char*>(a.B) + (rb * a.B_ld + g * N) * ES;
  const char* const gC = static_cast<const char*>(a.C) + (rb * a.C_ld + g * N) * ES;
  const float* const gck =
      a.ckpt_in + ((scan_ckpt_row0(a.rows, n, row0) + tb / kScanCheckpoint) * a.D + ch0) * N;
  auto stage = [&](int c) {  // copies of the c-th chunk from the end, as one group
    if (c < nchunk) {
      unsigned char* const st = smem + (c % kStages) * L.raw;
      const int ci = nchunk - 1 - c, t0 = ci * kChunk, nt = min(kChunk, tn - t0);
      for (int i = tid; i < kChunk * VPR; i += NT) {
        const int t = i / VPR, v = i % VPR;
        if (t >= nt || v >= nv) continue;
        const int o = (t * CH + v * VN) * ES;
        const long long r = t0 + t, b = (long long)v * 16;
        cp_async16(st + L.rx + o, gx + r * a.x_ld * ES + b);
        cp_async16(st + L.rdt + o, gdt + r * a.dt_ld * ES + b);
        if (gz) cp_async16(st + L.rz + o, gz + r * a.z_ld * ES + b);
        cp_async16(st + L.rdy + o, gdy + r * a.dy_ld * ES + b);
      }
      for (int i = tid; i < kChunk * BPR; i += NT) {
        const int t = i / BPR, v = i % BPR;
        if (t >= nt) continue;
        const int o = (t * N + v * VN) * ES;
        const long long r = t0 + t, b = (long long)v * 16;
        cp_async16(st + L.rB + o, gB + r * a.B_ld * ES + b);
        cp_async16(st + L.rC + o, gC + r * a.C_ld * ES + b);
      }
      const float* const ck = gck + (long long)ci * a.D * N;
      for (int i = tid; i < nch * N / 4; i += NT) cp_async16(st + L.rck + 16 * i, ck + 4 * i);
    }
    cp_async_commit();
  };
  stage(0);

  // Sums over tokens of the channels that a thread stores (its vector's place in
  // the row never changes: the threads are a multiple of the vectors).
  float sskip[VN], sbias[VN];
#pragma unroll
  for (int k = 0; k < VN; ++k) sskip[k] = sbias[k] = 0.f;

  for (int c = 0; c < nchunk; ++c) {
    const int ci = nchunk - 1 - c, t0 = ci * kChunk, nt = min(kChunk, tn - t0);
    cp_async_wait<0>();
    __syncthreads();  // chunk c is here; the other stage and the sums are free
    stage(c + 1);
    const unsigned char* const st = smem + (c % kStages) * L.raw;
    // Tokens past the end and channels past the tile count as s = s x = dpre = 0: they
    // change nothing.
    for (int i = tid; i < kChunk * VPR; i += NT) {
      const int t = i / VPR, v = i % VPR;
      float s[VN], x[VN], d[VN];
      if (t < nt && v < nv) {
        const int o = (t * CH + v * VN) * ES;
        V::unpack(*reinterpret_cast<const uint4*>(st + L.rdt + o), s);
        V::unpack(*reinterpret_cast<const uint4*>(st + L.rx + o), x);
        V::unpack(*reinterpret_cast<const uint4*>(st + L.rdy + o), d);
#pragma unroll
        for (int k = 0; k < VN; ++k) {
          s[k] += fbias[v * VN + k];
          if (a.softplus) s[k] = softplus_fast(s[k]);
          bad |= !nonneg_finite(s[k]);
          x[k] *= s[k];
        }
        if (gz) {
          float z[VN];
          V::unpack(*reinterpret_cast<const uint4*>(st + L.rz + o), z);
#pragma unroll
          for (int k = 0; k < VN; ++k) d[k] *= silu_fast(z[k]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < VN; ++k) s[k] = x[k] = d[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < VN; k += 4) {
        const int o = t * CH + v * VN + k;
        *reinterpret_cast<float4*>(fs + o) = make_float4(s[k], s[k + 1], s[k + 2], s[k + 3]);
        *reinterpret_cast<float4*>(fsx + o) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
        *reinterpret_cast<float4*>(fdp + o) = make_float4(d[k], d[k + 1], d[k + 2], d[k + 3]);
      }
    }
    for (int i = tid; i < kChunk * BPR; i += NT) {
      float fb[VN], fc[VN];
      if (i / BPR < nt) {
        V::unpack(reinterpret_cast<const uint4*>(st + L.rB)[i], fb);
        V::unpack(reinterpret_cast<const uint4*>(st + L.rC)[i], fc);
      } else {
#pragma unroll
        for (int k = 0; k < VN; ++k) fb[k] = fc[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < VN; k += 4) {
        *reinterpret_cast<float4*>(fB + i * VN + k) = make_float4(fb[k], fb[k + 1], fb[k + 2], fb[k + 3]);
        *reinterpret_cast<float4*>(fC + i * VN + k) = make_float4(fc[k], fc[k + 1], fc[k + 2], fc[k + 3]);
      }
    }
    __syncthreads();

    // First sweep: the states before tokens 4, 8, 12 (each lane keeps its own).
    float2 h[4][NP];
    const float* const ck = reinterpret_cast<const float*>(st + L.rck);
    float2* const sub = reinterpret_cast<float2*>(smem + L.sub) + tid;
    auto load_ckpt = [&]() {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int p = 0; p < NP; ++p)
          h[k][p] = 4 * cl + k < nch ? *reinterpret_cast<const float2*>(ck + (4 * cl + k) * N + n0 + 2 * p)
                                     : make_float2(0.f, 0.f);
    };
    load_ckpt();
#pragma unroll 1
    for (int w = 0; w < kChunk / kWin - 1; ++w) {
#pragma unroll
      for (int i = 0; i < kWin; ++i) {
        const int t = w * kWin + i;
        const float4 s4 = *reinterpret_cast<const float4*>(fs + t * CH + 4 * cl);
        const float4 x4 = *reinterpret_cast<const float4*>(fsx + t * CH + 4 * cl);
        const float sv[4] = {s4.x, s4.y, s4.z, s4.w}, xv[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const float2 b = *reinterpret_cast<const float2*>(fB + t * N + n0 + 2 * p);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 u = decay_exponent(make_float2(sv[k], sv[k]), A2[k][p]);
            h[k][p] = __ffma2_rn(make_float2(xv[k], xv[k]), b,
                                 __fmul2_rn(make_float2(ex2_approx(u.x), ex2_approx(u.y)), h[k][p]));
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int p = 0; p < NP; ++p) sub[((w * 4 + k) * NP + p) * NT] = h[k][p];
    }

    // Windows, last to first.
#pragma unroll 1
    for (int w = kChunk / kWin - 1; w >= 0; --w) {
      if (w == 0) {
        load_ckpt();
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int p = 0; p < NP; ++p) h[k][p] = sub[(((w - 1) * 4 + k) * NP + p) * NT];
      }
      float2 al[kWin][4][NP], ah[kWin][4][NP];  // a_t and a_t h_{t-1}
#pragma unroll
      for (int i = 0; i < kWin; ++i) {
        const int t = w * kWin + i;
        const float4 s4 = *reinterpret_cast<const float4*>(fs + t * CH + 4 * cl);
        const float4 x4 = *reinterpret_cast<const float4*>(fsx + t * CH + 4 * cl);
        const float sv[4] = {s4.x, s4.y, s4.z, s4.w}, xv[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const float2 b = *reinterpret_cast<const float2*>(fB + t * N + n0 + 2 * p);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 u = decay_exponent(make_float2(sv[k], sv[k]), A2[k][p]);
            al[i][k][p] = make_float2(ex2_approx(u.x), ex2_approx(u.y));
            ah[i][k][p] = __fmul2_rn(al[i][k][p], h[k][p]);
            h[k][p] = __ffma2_rn(make_float2(xv[k], xv[k]), b, ah[i][k][p]);
          }
        }
      }
#pragma unroll
      for (int i = kWin - 1; i >= 0; --i) {
        const int t = w * kWin + i;
        const float4 s4 = *reinterpret_cast<const float4*>(fs + t * CH + 4 * cl);
        const float4 x4 = *reinterpret_cast<const float4*>(fsx + t * CH + 4 * cl);
        const float4 d4 = *reinterpret_cast<const float4*>(fdp + t * CH + 4 * cl);
        const float sv[4] = {s4.x, s4.y, s4.z, s4.w}, xv[4] = {x4.x, x4.y, x4.z, x4.w},
                    dv[4] = {d4.x, d4.y, d4.z, d4.w};
        float2 db[NP], dc[NP], ws[4], qs[4], ys[4];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const float2 b = *reinterpret_cast<const float2*>(fB + t * N + n0 + 2 * p);
          const float2 cc = *reinterpret_cast<const float2*>(fC + t * N + n0 + 2 * p);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 s2 = make_float2(sv[k], sv[k]), x2 = make_float2(xv[k], xv[k]), d2 = make_float2(dv[k], dv[k]);
            const float2 ht = __ffma2_rn(x2, b, ah[i][k][p]);
            const float2 gt = __ffma2_rn(cc, d2, gh[k][p]);
            const float2 pt = __fmul2_rn(gt, ah[i][k][p]);
            dc[p] = k == 0 ? __fmul2_rn(ht, d2) : __ffma2_rn(ht, d2, dc[p]);
            db[p] = k == 0 ? __fmul2_rn(gt, x2) : __ffma2_rn(gt, x2, db[p]);
            ys[k] = p == 0 ? __fmul2_rn(ht, cc) : __ffma2_rn(ht, cc, ys[k]);
            ws[k] = p == 0 ? __fmul2_rn(gt, b) : __ffma2_rn(gt, b, ws[k]);
            qs[k] = p == 0 ? __fmul2_rn(pt, A2[k][p]) : __ffma2_rn(pt, A2[k][p], qs[k]);
            dA[k][p] = __ffma2_rn(pt, s2, dA[k][p]);
            gh[k][p] = __fmul2_rn(gt, al[i][k][p]);
          }
        }
        float v[4];
        float* const sm = fsum + (warp * kChunk + t) * CH + 4 * cl + sl;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = ws[k].x + ws[k].y;
        sm[0] = scatter_groups(v, sl);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = qs[k].x + qs[k].y;
        sm[W * kChunk * CH] = scatter_groups(v, sl);
        if (gz) {
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = ys[k].x + ys[k].y;
          sm[2 * W * kChunk * CH] = scatter_groups(v, sl);
        }
        // dB, dC over the 8 lanes that share states: lane cl ends with one value, of dC
        // where cl & 4, else of dB.
        const bool b4 = cl & 4, b2 = cl & 2, b1 = cl & 1;
        float2 keep[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const float2 give = b4 ? db[p] : dc[p];
          keep[p] = b4 ? dc[p] : db[p];
          keep[p].x += __shfl_xor_sync(0xffffffffu, give.x, 4);
          keep[p].y += __shfl_xor_sync(0xffffffffu, give.y, 4);
        }
        float* const out = part.bc + ((tile * part.rows + rb + t0 + t) * 2 + (b4 ? 1 : 0)) * N + n0;
        if constexpr (NS == 4) {
          float2 k2 = b2 ? keep[1] : keep[0];
          const float2 give = b2 ? keep[0] : keep[1];
          k2.x += __shfl_xor_sync(0xffffffffu, give.x, 2);
          k2.y += __shfl_xor_sync(0xffffffffu, give.y, 2);
          const float r = (b1 ? k2.y : k2.x) + __shfl_xor_sync(0xffffffffu, b1 ? k2.x : k2.y, 1);
          if (t < nt) out[(b2 ? 2 : 0) + (b1 ? 1 : 0)] = r;
        } else {
          float r = (b2 ? keep[0].y : keep[0].x) + __shfl_xor_sync(0xffffffffu, b2 ? keep[0].x : keep[0].y, 2);
          r += __shfl_xor_sync(0xffffffffu, r, 1);
          if (t < nt && !b1) out[b2 ? 1 : 0] = r;
        }
      }
    }
    __syncthreads();

    // Gradients of the tokens' arrays.
    for (int i = tid; i < kChunk * VPR; i += NT) {
      const int t = i / VPR, v = i % VPR;
      if (t >= nt || v >= nv) continue;
      const int o = (t * CH + v * VN) * ES;
      float x[VN], dt[VN], dy[VN], z[VN], dx[VN], ddt[VN];
      V::unpack(*reinterpret_cast<const uint4*>(st + L.rx + o), x);
      V::unpack(*reinterpret_cast<const uint4*>(st + L.rdt + o), dt);
      V::unpack(*reinterpret_cast<const uint4*>(st + L.rdy + o), dy);
      if (gz) V::unpack(*reinterpret_cast<const uint4*>(st + L.rz + o), z);
#pragma unroll
      for (int k = 0; k < VN; ++k) {
        const int e = t * CH + v * VN + k;
        float ws = 0.f, qs = 0.f, ys = 0.f;
        for (int w = 0; w < W; ++w) {
          ws += fsum[w * kChunk * CH + e];
          qs += fsum[(W + w) * kChunk * CH + e];
          if (gz) ys += fsum[(2 * W + w) * kChunk * CH + e];
        }
        const float skip = fskip[v * VN + k], dpre = fdp[e];
        dx[k] = fmaf(ws, fs[e], dpre * skip);
        // qs holds -log2(e) sum p A
        ddt[k] = fmaf(ws, x[k], qs * 0.6931471805599453f);
        if (a.softplus) ddt[k] *= sigmoid_fast(dt[k] + fbias[v * VN + k]);
        sskip[k] = fmaf(dpre, x[k], sskip[k]);
        sbias[k] += ddt[k];
        if (gz) {
          const float q = sigmoid_fast(z[k]);
          z[k] = dy[k] * fmaf(skip, x[k], ys) * (q * fmaf(z[k], 1.f - q, 1.f));
        }
      }
      const long long at = ((rb + t0 + t) * a.D + ch0 + v * VN) * ES;
      *reinterpret_cast<uint4*>(static_cast<char*>(a.dx) + at) = V::pack(dx);
      *reinterpret_cast<uint4*>(static_cast<char*>(a.ddt) + at) = V::pack(ddt);
      if (gz) *reinterpret_cast<uint4*>(static_cast<char*>(a.dz) + at) = V::pack(z);
    }
  }
  if (bad) latch_status(a.status, kStatusDomain);

  const size_t ns = (size_t)(n * a.nseg + seg);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (4 * cl + c >= nch) continue;
    const size_t e = (size_t)(ch0 + 4 * cl + c) * N + n0;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      *reinterpret_cast<float2*>(part.dA + ns * a.D * N + e + 2 * p) = make_float2(-dA[c][p].x, -dA[c][p].y);
      if (tb == 0 && a.dh0) *reinterpret_cast<float2*>(a.dh0 + (size_t)n * a.D * N + e + 2 * p) = gh[c][p];
    }
  }
  // dskip, ddt_bias of the segment: the threads of a vector, added up in thread order.
  __syncthreads();
  float* const red = fs;  // 2 x NT x VN values fit the chunk's arrays
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < VN; ++k) red[tid * VN + k] = which ? sbias[k] : sskip[k];
    __syncthreads();
    for (int e = tid; e < nch; e += NT) {
      const int v = e / VN, k = e % VN;
      float s = 0.f;
      for (int t = v; t < NT; t += VPR) s += red[t * VN + k];
      part.par[(ns * 2 + which) * a.D + ch0 + e] = s;
    }
  }
}

// dB, dC: sum over the tiles of a group, in the input type. One thread per 4
// values of a row's [2][N].
template <bool BF16>
__global__ void __launch_bounds__(256) palimpsa_scan_bwd_bc_kernel(ScanArgs a, Partials part, int tpg) {
  const int per = 2 * a.N / 4;  // threads of a row and group
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int q = (int)(i % per), g = (int)(i / per % a.G);
  const long long r = i / per / a.G;
  if (r >= (long long)a.rows.n_seq * a.rows.max_len) return;
  const long long n = r / a.rows.max_len;
  const int t = (int)(r % a.rows.max_len);
  long long row0;
  int len;
  if (!seq_rows(a.rows, n, &row0, &len) || t >= len) return;
  const long long row = row0 + t;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < tpg; ++k) {
    const float4 v = *reinterpret_cast<const float4*>(part.bc + ((g * tpg + k) * part.rows + row) * 2 * a.N + 4 * q);
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

// dA, or dskip and ddt_bias: sum over sequences and segments. The `per` values of
// one (sequence, segment) lie together in `p`, the first `split` of them for out and
// the others for out2 (either may be null). 32 values by 8 slices of the sum to a CTA.
__global__ void __launch_bounds__(256) palimpsa_scan_bwd_par_kernel(ScanArgs a, const float* p, long long per,
                                                                    long long split, float* out, float* out2) {
  __shared__ float red[8][33];
  const int cx = threadIdx.x % 32, sy = threadIdx.x / 32;
  const long long e = (long long)blockIdx.x * 32 + cx;
  float s = 0.f;
  for (long long n = sy; n < a.rows.n_seq; n += 8) {
    long long row0;
    int len;
    if (!seq_rows(a.rows, n, &row0, &len)) continue;
    const int ns = max(1, (len + a.seg_len - 1) / a.seg_len);
    if (e < per)
      for (int k = 0; k < ns; ++k) s += p[(n * a.nseg + k) * per + e];
  }
  red[sy][cx] = s;
  __syncthreads();
  if (sy || e >= per) return;
  for (int k = 1; k < 8; ++k) s += red[k][cx];
  if (e >= split) out = out2 ? out2 - split : nullptr;
  if (out) out[e] = s;
}

long long total_rows(const ScanArgs& a) { return a.rows.cu ? a.rows.T : (long long)a.rows.n_seq * a.rows.T; }

template <bool BF16, int NS>
cudaError_t run(const ScanArgs& a, const Partials& part, cudaStream_t s) {
  const int W = a.N / (4 * NS);
  const Smem L(a.N, W, Vec<BF16>::bytes);
  const long long tiles = scan_tiles(a), blocks = tiles * a.rows.n_seq * a.nseg;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  if (L.total > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(palimpsa_scan_bwd_kernel<BF16, NS>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, L.total);
    if (e != cudaSuccess) return e;
  }
  palimpsa_scan_bwd_kernel<BF16, NS><<<(unsigned)blocks, 32 * W, L.total, s>>>(a, part, (int)tiles, W);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long bct = (long long)a.rows.n_seq * a.rows.max_len * a.G * (2 * a.N / 4);
  if (bct > 0) {
    const long long bb = (bct + 255) / 256;
    if (bb > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    palimpsa_scan_bwd_bc_kernel<BF16>
        <<<(unsigned)bb, 256, 0, s>>>(a, part, (int)(tiles / a.G));
  }
  const long long dn = (long long)a.D * a.N;
  palimpsa_scan_bwd_par_kernel<<<(unsigned)((dn + 31) / 32), 256, 0, s>>>(a, part.dA, dn, dn, a.dA, nullptr);
  palimpsa_scan_bwd_par_kernel<<<(unsigned)((2 * a.D + 31) / 32), 256, 0, s>>>(a, part.par, 2ll * a.D, a.D,
                                                                             a.dskip, a.ddt_bias);
  return cudaGetLastError();
}

size_t bc_floats(const ScanArgs& a) { return (size_t)scan_tiles(a) * total_rows(a) * 2 * a.N; }

}  // namespace

size_t scan_backward_scratch_floats(const ScanArgs& a) {
  const size_t ns = (size_t)a.rows.n_seq * a.nseg;
  return bc_floats(a) + ns * a.D * a.N + ns * 2 * a.D;
}

cudaError_t launch_scan_backward(const ScanArgs& a, float* scratch, cudaStream_t s) {
  Partials part;
  part.bc = scratch;
  part.rows = total_rows(a);
  part.dA = part.bc + bc_floats(a);
  part.par = part.dA + (size_t)a.rows.n_seq * a.nseg * a.D * a.N;
  if (a.nseg > 1) {
    cudaError_t e = launch_scan_reverse_summary(a, s);
    if (e == cudaSuccess) e = launch_scan_carry(a, true, s);
    if (e != cudaSuccess) return e;
  }
  if (a.N == 8) return a.bf16 ? run<true, 2>(a, part, s) : run<false, 2>(a, part, s);
  return a.bf16 ? run<true, 4>(a, part, s) : run<false, 4>(a, part, s);
}

}  // namespace palimpsa
