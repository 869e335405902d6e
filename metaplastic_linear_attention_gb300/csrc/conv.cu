// Short causal convolution over tokens, one filter of W taps per channel
// (depthwise), with bias and optional SiLU:
//   u_t = bias + sum_{j < W} w_j x_{t - (W-1) + j},   y_t = silu(u_t) or u_t,
// where x_{-1}, ..., x_{-(W-1)} are the sequence's state (zeros without one):
// the last W - 1 inputs before its first token, oldest first, in the input
// type (they are copies of inputs, so a prompt cut in two gives the same bits).
//
// A value is read once and written once, against 2 W + 6 operations: the kernels
// are bound by HBM. A thread owns 4 channels (8 bytes of bf16, 16 of fp32) and a
// run of tokens, which it walks in batches of 8; the batches come by asynchronous
// copies into a ring of three in shared memory, each thread its own column (held in
// registers instead, one batch ahead, they left HBM at two thirds of its rate). The
// W - 1 rows before a run are read again. Long runs also spread the loads of the taps,
// which are far apart in memory for neighbouring threads. Sums are fp32; y is rounded
// once. Measured (GB300, bf16, W = 4, SiLU): 30 us at 8 x 4096 x 1536, the time of a
// copy of as many bytes; backward 17 to 19 us at 4 x 2048 x 1024 and 67 at 8 x 4096 x 1536
// (7 and 44 for their bytes; its window of W inputs and W gradients holds it to 16 warps an
// SM), and 3 to 4 for the sums over CTAs.
#include <algorithm>
#include <cooperative_groups.h>

#include "ssm.cuh"

namespace palimpsa {
namespace {

constexpr int kBatch = 8;      // tokens loaded together
constexpr int kRing = 3;       // batches in the ring
constexpr int kThreads = 128;
constexpr int kMinRun = 16;   // tokens of a run, at least
constexpr int kCtas = 5;      // of an SM, in bf16; of fp32's rings (48 KB) 4 fit, and the waves are planned with 5 all the same

// Parameters of a thread's 4 channels, as pairs: 4 W neighbouring floats, by 16-byte
// loads where the array allows it (it only has to be aligned to 4 bytes).
template <int W>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int ch, float2 (*w)[2], float2* b) {
  const float* const k = a.weight + (size_t)ch * W;
  float f[4 * W];
  if ((reinterpret_cast<uintptr_t>(a.weight) & 15) == 0) {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float4 v = reinterpret_cast<const float4*>(k)[j];
      f[4 * j] = v.x; f[4 * j + 1] = v.y; f[4 * j + 2] = v.z; f[4 * j + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4 * W; ++j) f[j] = k[j];
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][p] = make_float2(f[2 * p * W + j], f[(2 * p + 1) * W + j]);
    b[p] = a.bias ? make_float2(a.bias[ch + 2 * p], a.bias[ch + 2 * p + 1]) : make_float2(0.f, 0.f);
  }
}

template <bool BF16>
__device__ __forceinline__ typename Quad<BF16>::Raw load_quad(const void* p, long long i) {
  return *reinterpret_cast<const typename Quad<BF16>::Raw*>(static_cast<const char*>(p) + i * Vec<BF16>::bytes);
}
template <bool BF16>
__device__ __forceinline__ void cp_async_quad(void* dst, const void* src) {
  if constexpr (BF16) cp_async8(dst, src);
  else cp_async16(dst, src);
}
template <bool BF16>
__device__ __forceinline__ void store_quad(void* p, long long i, const typename Quad<BF16>::Raw& v) {
  *reinterpret_cast<typename Quad<BF16>::Raw*>(static_cast<char*>(p) + i * Vec<BF16>::bytes) = v;
}

// Input row p of a sequence (p may be negative: the state).
template <bool BF16, int W>
__device__ __forceinline__ typename Quad<BF16>::Raw input_row(const ConvArgs& a, long long n, long long row0, int p,
                                                              int ch) {
  if (p >= 0) return load_quad<BF16>(a.x, (row0 + p) * a.x_ld + ch);
  if (!a.state0) return Quad<BF16>::zero();
  return load_quad<BF16>(a.state0, (n * (W - 1) + (W - 1 + p)) * a.D + ch);
}

template <bool BF16, int W>
__global__ void __launch_bounds__(kThreads, kCtas) palimpsa_conv_kernel(ConvArgs a) {
  using Q = Quad<BF16>;
  using Raw = typename Q::Raw;
  const int nvec = a.D / 4;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int ch = (int)(i % nvec) * 4;
  long long row0;
  int seq, run, len;
  if (i >= nvec * a.slots.count || !slot_place(a.rows, a.slots, i / nvec, &seq, &run)) return;
  const long long n = seq;
  if (!seq_rows(a.rows, n, &row0, &len)) {
    if (run == 0 && ch == 0) latch_status(a.status, kStatusDomain);
    return;
  }
  const int t0 = run * a.run, t1 = min(len, t0 + a.run);
  if (t0 >= t1 && run > 0) return;
  // A ring of batches in shared memory, each thread its own column: no barriers.
  extern __shared__ __align__(16) unsigned char smem[];
  Raw* const ring = reinterpret_cast<Raw*>(smem) + threadIdx.x;
  const long long ld = a.x_ld * Vec<BF16>::bytes;
  const char* px = static_cast<const char*>(a.x) + (row0 + t0) * ld + ch * Vec<BF16>::bytes;
  int t_next = t0, slot = 0;  // of the next batch to copy in
  auto fetch = [&]() {
    Raw* const to = ring + slot * (kBatch * kThreads);
    if (t_next + kBatch <= t1) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) cp_async_quad<BF16>(to + k * kThreads, px + k * ld);
    } else {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (t_next + k < t1) cp_async_quad<BF16>(to + k * kThreads, px + k * ld);
    }
    cp_async_commit();
    px += kBatch * ld;
    t_next += kBatch;
    slot = slot + 1 == kRing ? 0 : slot + 1;
  };
  float2 win[W - 1][2];  // the W - 1 inputs before the next token
  {
    Raw old[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) old[j] = input_row<BF16, W>(a, n, row0, t0 - (W - 1) + j, ch);
#pragma unroll
    for (int r = 0; r < kRing - 1; ++r) fetch();
#pragma unroll
    for (int j = 0; j < W - 1; ++j) Q::unpack(old[j], win[j]);
  }
  // The state after the sequence: the last W - 1 of (state0, inputs). The thread that
  // holds the first run has read the state before it writes, so state_T may be state0.
  if (run == 0 && a.state_T) {
    Raw last[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) last[j] = input_row<BF16, W>(a, n, row0, len - (W - 1) + j, ch);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_quad<BF16>(a.state_T, (n * (W - 1) + j) * a.D + ch, last[j]);
  }
  float2 w[W][2], b[2];
  load_taps<W>(a, ch, w, b);
  const long long yd = (long long)a.D * Vec<BF16>::bytes;
  char* py = static_cast<char*>(a.y) + (row0 + t0) * yd + ch * Vec<BF16>::bytes;
  int at = 0;  // slot of the batch at hand
  for (int t = t0; t < t1; t += kBatch) {
    cp_async_wait<kRing - 2>();
    Raw cur[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) cur[k] = ring[(at * kBatch + k) * kThreads];
    at = at + 1 == kRing ? 0 : at + 1;
    fetch();  // into the slot of the batch before
    auto token = [&](int k) {
      float2 x[2], out[2];
      Q::unpack(cur[k], x);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float2 u = __ffma2_rn(w[W - 1][p], x[p], b[p]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) u = __ffma2_rn(w[j][p], win[j][p], u);
        out[p] = a.silu ? silu_fast(u) : u;
#pragma unroll
        for (int j = 0; j < W - 2; ++j) win[j][p] = win[j + 1][p];
        win[W - 2][p] = x[p];
      }
      *reinterpret_cast<Raw*>(py + k * yd) = Q::pack(out);
    };
    if (t + kBatch <= t1) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) token(k);
    } else {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (t + k < t1) token(k);
    }
    py += kBatch * yd;
  }
}

// One token: the state's W - 1 rows and the new input give y, and the state
// moves on by one row.
template <bool BF16, int W>
__global__ void __launch_bounds__(kThreads) palimpsa_conv_step_kernel(ConvArgs a) {
  using Q = Quad<BF16>;
  const int nvec = a.D / 4;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (long long)nvec * a.rows.n_seq) return;
  const int ch = (int)(i % nvec) * 4;
  const long long n = i / nvec, st = n * (W - 1) * a.D + ch;
  typename Q::Raw raw[W];
  raw[W - 1] = load_quad<BF16>(a.x, n * a.x_ld + ch);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) raw[j] = load_quad<BF16>(a.state_T, st + (long long)j * a.D);
  float2 w[W][2], u[2];
  load_taps<W>(a, ch, w, u);
#pragma unroll
  for (int k = 0; k < W; ++k) {  // the newest input first, as a prompt sums
    const int j = (k + W - 1) % W;
    float2 x[2];
    Q::unpack(raw[j], x);
#pragma unroll
    for (int p = 0; p < 2; ++p) u[p] = __ffma2_rn(w[j][p], x[p], u[p]);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_quad<BF16>(a.state_T, st + (long long)j * a.D, raw[j + 1]);
#pragma unroll
  for (int p = 0; p < 2; ++p) u[p] = a.silu ? silu_fast(u[p]) : u[p];
  store_quad<BF16>(a.y, n * a.D + ch, Q::pack(u));
}

// ------------------------------------------------------------------ backward
//
//   du_t = dy_t silu'(u_t),  silu'(u) = p (1 + u (1 - p)),  p = sigmoid(u)
//   dx_t = sum_j w_j du_{t + (W-1) - j}   (+ dstate_T for the last W - 1 inputs)
//   dw_j = sum_t du_t x_{t - (W-1) + j},  dbias = sum_t du_t.
// u is recomputed from x. A CTA owns 16 quads of channels and 16 runs of tokens (of any
// sequences), one run to a thread; each thread walks its run in batches of 3 or 4 tokens through a ring
// like the forward's, with the last W inputs and du's in registers, and looks W - 1
// tokens past its end for the dx of its last ones. The parameter sums go over
// the CTA's runs in shared memory and then, in a fixed order, over CTAs in a second
// kernel: no atomics, the same bits every time. An SM holds two CTAs (one in fp32 with W = 4,
// 184 registers; the waves are planned with two).
constexpr int kBwdVecs = 16, kBwdRuns = 16, kBwdCtas = 2, kBwdRing = 3;

template <bool BF16, int W>
__global__ void __launch_bounds__(kBwdVecs* kBwdRuns, BF16 || W < 4 ? kBwdCtas : 1)
palimpsa_conv_bwd_kernel(ConvArgs a, float* partial) {
  using Q = Quad<BF16>;
  using Raw = typename Q::Raw;
  constexpr int ES = Vec<BF16>::bytes;
  const int nvec = a.D / 4, vtiles = (nvec + kBwdVecs - 1) / kBwdVecs;
  const int vx = threadIdx.x % kBwdVecs, ry = threadIdx.x / kBwdVecs;
  const long long blk = blockIdx.x / vtiles;  // of kBwdRuns slots, over all sequences
  const int vec = (int)(blockIdx.x % vtiles) * kBwdVecs + vx;
  const int ch = vec * 4;
  long long row0 = 0;
  int seq = 0, place = 0, len = 0;
  const long long slot = blk * kBwdRuns + ry;
  bool live = vec < nvec && slot < a.slots.count && slot_place(a.rows, a.slots, slot, &seq, &place);
  const long long n = seq;
  if (live && !seq_rows(a.rows, n, &row0, &len)) {
    live = false;
    latch_status(a.status, kStatusDomain);
  }
  const int t0 = place * a.run;
  const int t1 = min(len, t0 + a.run);  // this run's tokens are [t0, t1)
  const float2 zero = make_float2(0.f, 0.f);

  float2 gw[W][2], gb[2] = {zero, zero};
#pragma unroll
  for (int j = 0; j < W; ++j) gw[j][0] = gw[j][1] = zero;
  // The run at the sequence's start also owns the gradient of the state rows
  // (places -(W-1) .. -1); with an empty sequence they pass dstate_T through.
  const bool first = t0 == 0;
  if (live && (t0 < t1 || first)) {
    float2 w[W][2], b[2];
    load_taps<W>(a, ch, w, b);
    // The inputs and du's of the last W tokens, by place modulo W (a batch is a whole
    // number of turns, so a token's slot is known at compile time).
    constexpr int NB = W == 3 ? 3 : 4;
    float2 x[W][2], du[W][2];
#pragma unroll
    for (int j = 0; j < W; ++j) du[j][0] = du[j][1] = x[j][0] = x[j][1] = zero;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) Q::unpack(input_row<BF16, W>(a, n, row0, t0 - (W - 1) + k, ch), x[k + 1]);
    // Token t0 + s brings in its x and dy and finishes the gradient of place t0 + s -
    // (W-1), all of whose W du's are then known.
    const int steps = max(t1 - t0, 0) + W - 1, stop = min(len, t0 + steps);
    const long long xl = a.x_ld * ES, yl = a.dy_ld * ES, dl = (long long)a.D * ES;
    const char* px = static_cast<const char*>(a.x) + (row0 + t0) * xl + ch * ES;
    const char* pg = static_cast<const char*>(a.dy) + (row0 + t0) * yl + ch * ES;
    char* pd = static_cast<char*>(a.dx) + (row0 + t0 - (W - 1)) * dl + ch * ES;  // of the finished place
    extern __shared__ __align__(16) unsigned char smem[];  // the ring, each thread its own column
    Raw* const ring = reinterpret_cast<Raw*>(smem) + threadIdx.x;
    constexpr int kCol = kBwdVecs * kBwdRuns;
    int t_next = t0, slot = 0;  // of the next batch to copy in
    auto fetch = [&]() {
      Raw* const to = ring + slot * (2 * NB * kCol);
#pragma unroll
      for (int k = 0; k < NB; ++k)
        if (t_next + k < stop) {
          cp_async_quad<BF16>(to + k * kCol, px + k * xl);
          cp_async_quad<BF16>(to + (NB + k) * kCol, pg + k * yl);
        }
      cp_async_commit();
      px += NB * xl;
      pg += NB * yl;
      t_next += NB;
      slot = slot + 1 == kBwdRing ? 0 : slot + 1;
    };
#pragma unroll
    for (int r = 0; r < kBwdRing - 1; ++r) fetch();
    int from = 0;  // slot of the batch at hand
    for (int s0 = 0; s0 < steps; s0 += NB) {
      cp_async_wait<kBwdRing - 2>();
      Raw rx[NB], rd[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const bool in = t0 + s0 + k < stop;
        rx[k] = in ? ring[(from * 2 * NB + k) * kCol] : Q::zero();
        rd[k] = in ? ring[(from * 2 * NB + NB + k) * kCol] : Q::zero();
      }
      from = from + 1 == kBwdRing ? 0 : from + 1;
      fetch();  // into the slot of the batch before
      // Takes in token t (its sums too, if it is the run's own) and forms the gradient of
      // place t - (W-1): w_j du_{t - j}.
      auto token = [&](int k, bool inside, bool own, float2* d) {
        float2 g[2];
        Q::unpack(rd[k], g);
        Q::unpack(rx[k], x[k % W]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float2 u = b[q];
#pragma unroll
          for (int j = 0; j < W; ++j) u = __ffma2_rn(w[j][q], x[(k + 1 + j) % W][q], u);
          if (a.silu) {
            const float2 sg = make_float2(sigmoid_fast(u.x), sigmoid_fast(u.y));
            const float2 m = __ffma2_rn(make_float2(-sg.x, -sg.y), u, u);  // u (1 - p)
            g[q] = __fmul2_rn(g[q], __ffma2_rn(sg, m, sg));
          }
          if (!inside) g[q] = zero;
          du[k % W][q] = g[q];
          if (own) {
            gb[q] = __fadd2_rn(gb[q], g[q]);
#pragma unroll
            for (int j = 0; j < W; ++j) gw[j][q] = __ffma2_rn(g[q], x[(k + 1 + j) % W][q], gw[j][q]);
          }
          d[q] = __fmul2_rn(w[0][q], g[q]);
#pragma unroll
          for (int j = 1; j < W; ++j) d[q] = __ffma2_rn(w[j][q], du[(k + W - j) % W][q], d[q]);
        }
      };
      const int t = t0 + s0, p = t - (W - 1);
      // All four tokens the run's own, and their places inside the run and before the
      // part of it that dstate_T reaches.
      if (t + NB <= t1 && p >= t0 && (!a.dstate_T || p + NB <= len - (W - 1))) {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          float2 d[2];
          token(k, true, true, d);
          *reinterpret_cast<Raw*>(pd + k * dl) = Q::pack(d);
        }
      } else {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          if (s0 + k >= steps) continue;
          float2 d[2];
          token(k, t + k < len, t + k < t1, d);  // tokens past the run only finish its dx
          if (p + k < t0 && !first) continue;
          const int back = p + k - (len - (W - 1));  // place in state_T, if >= 0
          if (a.dstate_T && back >= 0) {
            float2 e[2];
            Q::unpack(load_quad<BF16>(a.dstate_T, (n * (W - 1) + back) * a.D + ch), e);
            d[0] = __fadd2_rn(d[0], e[0]);
            d[1] = __fadd2_rn(d[1], e[1]);
          }
          if (p + k >= 0) *reinterpret_cast<Raw*>(pd + k * dl) = Q::pack(d);
          else if (a.dstate0) store_quad<BF16>(a.dstate0, (n * (W - 1) + (W - 1 + p + k)) * a.D + ch, Q::pack(d));
        }
      }
      pd += NB * dl;
    }
  }
  // Parameter sums over the CTA's runs, value by value.
  __shared__ float4 red[kBwdRuns][kBwdVecs];
#pragma unroll
  for (int v = 0; v <= W; ++v) {
    __syncthreads();
    const float2 *const g = v == W ? gb : gw[v < W ? v : 0];
    red[ry][vx] = make_float4(g[0].x, g[0].y, g[1].x, g[1].y);
    __syncthreads();
    if (ry == v % kBwdRuns && vec < nvec) {
      float4 s = red[0][vx];
#pragma unroll
      for (int r = 1; r < kBwdRuns; ++r) {
        const float4 e = red[r][vx];
        s.x += e.x; s.y += e.y; s.z += e.z; s.w += e.w;
      }
      *reinterpret_cast<float4*>(partial + (blk * (W + 1) + v) * a.D + ch) = s;
    }
  }
}

// Sums the token blocks' partials [blocks, W + 1, D]; block y = v, 32 channels by 8
// slices of the blocks.
__global__ void __launch_bounds__(256) palimpsa_conv_bwd_sum_kernel(const float* partial, long long blocks, int W,
                                                                    int D, float* dweight, float* dbias) {
  __shared__ float red[8][33];
  const int cx = threadIdx.x % 32, sy = threadIdx.x / 32, ch = blockIdx.x * 32 + cx, v = blockIdx.y;
  float s = 0.f;
  if (ch < D)
    for (long long b = sy; b < blocks; b += 8) s += partial[(b * (W + 1) + v) * D + ch];
  red[sy][cx] = s;
  __syncthreads();
  if (sy == 0 && ch < D) {
    for (int k = 1; k < 8; ++k) s += red[k][cx];
    if (v < W) dweight[(size_t)ch * W + v] = s;
    else if (dbias) dbias[ch] = s;
  }
}

// Where an offset is below the one before it, sequences may overlap, and those that do not
// fit the close slots are skipped, which only the kernel that lays the slots knows:
// everything is zeroed then. Every CTA looks all offsets over; with many sequences the 8 CTAs
// of a cluster do so together (SHARED): 28 us against 390 for 2^20 sequences, the same for
// 4096, and for 24, where the whole takes 4 us, 1.7 more.
constexpr int kZeroCtas = 152, kZeroCluster = 8, kZeroAlone = 4096;
template <bool SHARED>
__global__ void __launch_bounds__(SHARED ? 512 : 256) palimpsa_zero_outside_kernel(ZeroArgs a, int arrays) {
  namespace cg = cooperative_groups;
  constexpr int kZeroThreads = SHARED ? 512 : 256;
  const int* const cu = a.rows.cu;
  const long long T = a.rows.T, n_seq = a.rows.n_seq;
  const long long first = min(max((long long)cu[0], 0ll), T), last = min(max((long long)cu[n_seq], first), T);
  bool down = false;
  const int part = SHARED ? blockIdx.x % kZeroCluster : 0, parts = SHARED ? kZeroCluster : 1;
#pragma unroll 8
  for (long long n = part * kZeroThreads + threadIdx.x; n < n_seq; n += parts * kZeroThreads) down |= cu[n + 1] < cu[n];
  down = __syncthreads_or(down);
  if constexpr (SHARED) {
    __shared__ int seen;  // by any CTA of the cluster
    const cg::cluster_group cluster = cg::this_cluster();
    if (threadIdx.x == 0) seen = 0;
    cluster.sync();  // every CTA of the cluster is there, its flag clear
    if (down && threadIdx.x < kZeroCluster) *cluster.map_shared_rank(&seen, threadIdx.x) = 1;
    cluster.sync();
    down = seen;
  }

  const long long step = (long long)gridDim.x * kZeroThreads, i0 = (long long)blockIdx.x * kZeroThreads + threadIdx.x;
  const int lane = threadIdx.x & 31;
  for (int k = 0; k < arrays; ++k) {
    const bool per_token = k < a.row_arrays;
    const long long rows = per_token ? T : n_seq, w = a.width[k] / 16;
    long long lo = 0, hi = rows;  // rows [lo, hi) are left to the sequences
    if (down) {
      lo = rows;
    } else if (per_token) {
      lo = first;
      hi = last;
    }
    uint4* const p = static_cast<uint4*>(a.p[k]);
    for (long long i = i0; i < lo * w; i += step) p[i] = make_uint4(0, 0, 0, 0);
    for (long long i = hi * w + i0; i < rows * w; i += step) p[i] = make_uint4(0, 0, 0, 0);
    if (down) continue;
    // Sequences that are skipped for their offsets, each by the warp that finds it.
    for (long long n0 = i0 - lane; n0 < n_seq; n0 += step) {
      const long long n = n0 + lane;
      int from = 0, to = 0;
      if (n < n_seq) {
        const long long s0 = cu[n], s1 = cu[n + 1];
        if (s0 < 0 || s1 > T || s1 - s0 > a.rows.max_len) {
          from = per_token ? (int)min(max(s0, 0ll), T) : (int)n;
          to = per_token ? (int)min(max(s1, 0ll), T) : (int)n + 1;
        }
      }
      for (unsigned left = __ballot_sync(~0u, to > from); left; left &= left - 1) {
        const long long r0 = __shfl_sync(~0u, from, __ffs(left) - 1), r1 = __shfl_sync(~0u, to, __ffs(left) - 1);
        for (long long i = r0 * w + lane; i < r1 * w; i += 32) p[i] = make_uint4(0, 0, 0, 0);
      }
    }
  }
}

// The slots' starts, by one CTA: sums over the sequences before, 1024 at a time. (In 64 bits:
// offsets out of order can make valid sequences that overlap, and sums past the bounds.)
__global__ void __launch_bounds__(1024) palimpsa_slot_starts_kernel(SeqRows r, int piece, int* starts, int* row_starts,
                                                                    unsigned* status) {
  __shared__ long long sums[2][32];
  __shared__ int fit[2];  // ends of the sequences that have slots
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long bound = r.T / piece + (long long)r.n_seq;
  long long before[2] = {0, 0};
  if (tid < 2) fit[tid] = 0;
  for (int base = 0; base < r.n_seq; base += 1024) {
    const bool in = tid < r.n_seq - base;
    long long row0;
    int len = 0;
    const bool ok = in && seq_rows(r, base + tid, &row0, &len);
    const long long own[2] = {ok ? max(1, (len + piece - 1) / piece) : 0, ok ? len : 0};
    long long upto[2] = {own[0], own[1]};
    for (int d = 1; d < 32; d *= 2)
      for (int q = 0; q < 2; ++q) {
        const long long o = __shfl_up_sync(~0u, upto[q], d);
        if (lane >= d) upto[q] += o;
      }
    __syncthreads();  // the last round's sums are read
    if (lane == 31)
      for (int q = 0; q < 2; ++q) sums[q][warp] = upto[q];
    __syncthreads();
    long long all[2] = {0, 0};
    for (int q = 0; q < 2; ++q)
      for (int w = 0; w < 32; ++w) {
        if (w == warp) upto[q] += before[q] + all[q];
        all[q] += sums[q][w];
      }
    const bool fits = upto[0] <= bound && upto[1] <= r.T;
    if (in && fits)
      for (int q = 0; q < 2; ++q) atomicMax(&fit[q], (int)upto[q]);
    __syncthreads();
    if (in) {
      starts[base + tid] = fits ? (int)(upto[0] - own[0]) : fit[0];
      if (row_starts) row_starts[base + tid] = fits ? (int)(upto[1] - own[1]) : fit[1];
      if (!ok || !fits) latch_status(status, kStatusDomain);
    }
    for (int q = 0; q < 2; ++q) before[q] += all[q];
  }
  if (tid == 0) {
    starts[r.n_seq] = fit[0];
    if (row_starts) row_starts[r.n_seq] = fit[1];
  }
}

// Tokens of a run, a multiple of 8: long runs read fewer rows twice and load the taps
// less often (together about 8 tokens' worth), short ones make CTAs enough, and the CTAs
// should fill whole waves of the SMs' slots: the cheapest of waves x (run + 8). (With
// runs of 64, 8 x 4096 x 1536 took 1536 CTAs on 760 slots, a third wave for the last 16.)
// `threads` of a CTA take a run of 4 channels each.
int run_len_of(const ConvArgs& a, long long threads, int slots, int shortest) {
  // Runs with work: of a packed batch, its rows' and one cut short for every sequence.
  const long long rows = a.rows.cu ? a.rows.T : a.rows.max_len, seqs = a.rows.cu ? 1 : a.rows.n_seq;
  long long best = 0;
  int run = shortest;
  for (int r = shortest; r <= 128; r += 8) {
    const long long runs = seqs * ((rows + r - 1) / r) + (a.rows.cu ? a.rows.n_seq : 0);
    const long long ctas = (runs * (a.D / 4) + threads - 1) / threads;
    const long long cost = (ctas + slots - 1) / slots * (r + 8);
    if (r == shortest || cost < best) {
      best = cost;
      run = r;
    }
  }
  return run;
}
int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 152;
  return sms;
}
int bwd_vtiles(const ConvArgs& a) { return (a.D / 4 + kBwdVecs - 1) / kBwdVecs; }
long long bwd_blocks(const ConvArgs& a) { return (a.slots.count + kBwdRuns - 1) / kBwdRuns; }
size_t partial_floats(const ConvArgs& a) { return (size_t)bwd_blocks(a) * (a.W + 1) * a.D; }

template <bool BF16, int W>
cudaError_t backward(const ConvArgs& a, float* scratch, cudaStream_t s) {
  const long long blocks = bwd_blocks(a), ctas = blocks * bwd_vtiles(a);
  if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  constexpr int bytes = kBwdRing * 2 * (W == 3 ? 3 : 4) * kBwdVecs * kBwdRuns * (int)sizeof(typename Quad<BF16>::Raw);
  const cudaError_t e = cudaFuncSetAttribute(palimpsa_conv_bwd_kernel<BF16, W>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  palimpsa_conv_bwd_kernel<BF16, W><<<(unsigned)ctas, kBwdVecs * kBwdRuns, bytes, s>>>(a, scratch);
  palimpsa_conv_bwd_sum_kernel<<<dim3((a.D + 31) / 32, W + 1), 256, 0, s>>>(scratch, blocks, W, a.D, a.dweight,
                                                                            a.dbias);
  return cudaGetLastError();
}

template <bool BF16, int W>
cudaError_t forward(const ConvArgs& a, cudaStream_t s) {
  const long long blocks = (a.D / 4 * a.slots.count + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  constexpr int bytes = kRing * kBatch * kThreads * (int)sizeof(typename Quad<BF16>::Raw);
  palimpsa_conv_kernel<BF16, W><<<(unsigned)blocks, kThreads, bytes, s>>>(a);
  return cudaGetLastError();
}

// The slots' starts, if they lie close, in scratch behind `floats` floats.
cudaError_t place_slots(ConvArgs* a, float* scratch, size_t floats, cudaStream_t s) {
  if (!a->slots.starts) return cudaSuccess;
  int* const starts = reinterpret_cast<int*>(scratch + floats);
  a->slots.starts = starts;
  return launch_slot_starts(a->rows, a->run, starts, nullptr, a->status, s);
}

template <bool BF16, int W>
cudaError_t step(const ConvArgs& a, cudaStream_t s) {
  const long long n = (long long)(a.D / 4) * a.rows.n_seq, blocks = (n + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  palimpsa_conv_step_kernel<BF16, W><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

#define PALIMPSA_CONV_DISPATCH(f, ...)                                     \
  switch (a.W) {                                                           \
    case 2: return a.bf16 ? f<true, 2>(__VA_ARGS__) : f<false, 2>(__VA_ARGS__); \
    case 3: return a.bf16 ? f<true, 3>(__VA_ARGS__) : f<false, 3>(__VA_ARGS__); \
    default: return a.bf16 ? f<true, 4>(__VA_ARGS__) : f<false, 4>(__VA_ARGS__); \
  }

cudaError_t launch_slot_starts(const SeqRows& r, int piece, int* starts, int* row_starts, unsigned* status,
                               cudaStream_t s) {
  palimpsa_slot_starts_kernel<<<1, 1024, 0, s>>>(r, piece, starts, row_starts, status);
  return cudaGetLastError();
}
cudaError_t launch_zero_outside(const ZeroArgs& a, int arrays, cudaStream_t s) {
  if (arrays == 0) return cudaSuccess;
  if (a.rows.n_seq <= kZeroAlone) {
    palimpsa_zero_outside_kernel<false><<<kZeroCtas, 256, 0, s>>>(a, arrays);
    return cudaGetLastError();
  }
  cudaLaunchAttribute cluster = {};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = kZeroCluster;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(kZeroCtas);
  c.blockDim = dim3(512);
  c.stream = s;
  c.attrs = &cluster;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, palimpsa_zero_outside_kernel<true>, a, arrays);
}
size_t plan_conv(ConvArgs* a, bool backward) {
  const int sms = sm_count();
  a->run = backward ? run_len_of(*a, kBwdVecs * kBwdRuns, kBwdCtas * sms, 8)
                    : run_len_of(*a, kThreads, kCtas * sms, kMinRun);
  a->slots = slots_of(a->rows, a->run);
  const long long close = close_slots(a->rows, a->run), idle = a->slots.count - close;
  const bool lie_close = close_pays(a->rows, idle * (a->D / 4) / (backward ? kBwdRuns * kBwdVecs : kThreads));
  if (lie_close) {
    a->slots.count = close;
    a->slots.starts = a->rows.cu;  // until the launch has a place for them
  }
  return (backward ? partial_floats(*a) * sizeof(float) : 0) + (lie_close ? (a->rows.n_seq + 1ull) * sizeof(int) : 0);
}
cudaError_t launch_conv_forward(const ConvArgs& given, float* scratch, cudaStream_t s) {
  ConvArgs a = given;
  const cudaError_t e = place_slots(&a, scratch, 0, s);
  if (e != cudaSuccess) return e;
  PALIMPSA_CONV_DISPATCH(forward, a, s)
}
cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t s) { PALIMPSA_CONV_DISPATCH(step, a, s) }
cudaError_t launch_conv_backward(const ConvArgs& given, float* scratch, cudaStream_t s) {
  ConvArgs a = given;
  const cudaError_t e = place_slots(&a, scratch, partial_floats(a), s);
  if (e != cudaSuccess) return e;
  PALIMPSA_CONV_DISPATCH(backward, a, scratch, s)
}

}  // namespace palimpsa
