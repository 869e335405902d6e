// Short causal convolution over tokens, one filter of W taps per channel
// (depthwise), with bias and optional SiLU:
//   u_t = bias + sum_{j < W} w_j x_{t - (W-1) + j},   y_t = silu(u_t) or u_t,
// where x_{-1}, ..., x_{-(W-1)} are the sequence's state (zeros without one):
// the last W - 1 inputs before its first token, oldest first, in the input
// type (they are copies of inputs, so a prompt cut in two gives the same bits).
//
// A value is read once and written once, against 2 W + 6 operations: the
// kernels are bound by HBM. A thread owns one 16-byte vector of channels (8 bf16
// or 4 fp32) and a short run of tokens, with the W - 1 rows before it read again
// (they hit in L1/L2: the neighbouring run reads them at the same time). All its
// loads are issued before any arithmetic. Sums are fp32; y is rounded once.
#include <algorithm>

#include "ssm.cuh"

namespace palimpsa {
namespace {

constexpr int kRun = 8;        // tokens of a thread, forward
constexpr int kThreads = 256;

// Parameters of a thread's channels.
template <int VN, int W>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int ch, float (*w)[W], float* b) {
#pragma unroll
  for (int i = 0; i < VN; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[i][j] = a.weight[(size_t)(ch + i) * W + j];
    b[i] = a.bias ? a.bias[ch + i] : 0.f;
  }
}

// Input row p of a sequence (p may be negative: the state) as a raw vector.
template <bool BF16, int W>
__device__ __forceinline__ uint4 input_row(const ConvArgs& a, long long n, long long row0, int p, int ch) {
  constexpr int ES = Vec<BF16>::bytes;
  if (p >= 0)
    return *reinterpret_cast<const uint4*>(static_cast<const char*>(a.x) + ((row0 + p) * a.x_ld + ch) * ES);
  if (!a.state0) return make_uint4(0, 0, 0, 0);
  return *reinterpret_cast<const uint4*>(static_cast<const char*>(a.state0) +
                                         ((n * (W - 1) + (W - 1 + p)) * a.D + ch) * (long long)ES);
}

template <bool BF16, int W>
__global__ void __launch_bounds__(kThreads) palimpsa_conv_kernel(ConvArgs a, int runs) {
  using V = Vec<BF16>;
  constexpr int VN = V::n, ES = V::bytes;
  const int nvec = a.D / VN;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (long long)nvec * runs * a.rows.n_seq) return;
  const int ch = (int)(i % nvec) * VN;
  const long long r = i / nvec;
  const int run = (int)(r % runs);
  const long long n = r / runs;
  long long row0;
  int len;
  if (!seq_rows(a.rows, n, &row0, &len)) {
    if (run == 0 && ch == 0) latch_status(a.status, kStatusDomain);
    return;
  }
  const int t0 = run * kRun, nt = min(kRun, len - t0);
  if (nt <= 0 && run > 0) return;
  uint4 raw[kRun + W - 1];
#pragma unroll
  for (int k = 0; k < kRun + W - 1; ++k)
    if (k < nt + W - 1) raw[k] = input_row<BF16, W>(a, n, row0, t0 - (W - 1) + k, ch);
  // The state after the sequence: the last W - 1 of (state0, inputs). The
  // thread that holds the first run reads what it needs before it writes, so
  // state_T may be state0.
  if (run == 0 && a.state_T) {
    uint4 last[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) last[j] = input_row<BF16, W>(a, n, row0, len - (W - 1) + j, ch);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      *reinterpret_cast<uint4*>(static_cast<char*>(a.state_T) + ((n * (W - 1) + j) * a.D + ch) * (long long)ES) =
          last[j];
  }
  if (nt <= 0) return;
  float w[VN][W], b[VN];
  load_taps<VN, W>(a, ch, w, b);
  float win[W][VN];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) V::unpack(raw[k], win[k]);
#pragma unroll
  for (int t = 0; t < kRun; ++t) {
    if (t >= nt) break;
    V::unpack(raw[t + W - 1], win[(t + W - 1) % W]);
    float out[VN];
#pragma unroll
    for (int c = 0; c < VN; ++c) {
      float u = b[c];
#pragma unroll
      for (int j = 0; j < W; ++j) u = fmaf(w[c][j], win[(t + j) % W][c], u);
      out[c] = a.silu ? silu_fast(u) : u;
    }
    *reinterpret_cast<uint4*>(static_cast<char*>(a.y) + ((row0 + t0 + t) * a.D + ch) * (long long)ES) =
        V::pack(out);
  }
}

// One token: the state's W - 1 rows and the new input give y, and the state
// moves on by one row.
template <bool BF16, int W>
__global__ void __launch_bounds__(128) palimpsa_conv_step_kernel(ConvArgs a) {
  using V = Vec<BF16>;
  constexpr int VN = V::n, ES = V::bytes;
  const int nvec = a.D / VN;
  const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
  if (i >= (long long)nvec * a.rows.n_seq) return;
  const int ch = (int)(i % nvec) * VN;
  const long long n = i / nvec;
  char* st = static_cast<char*>(a.state_T) + (n * (W - 1) * a.D + ch) * (long long)ES;
  uint4 raw[W];
  raw[W - 1] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.x) + (n * a.x_ld + ch) * ES);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) raw[j] = *reinterpret_cast<const uint4*>(st + (long long)j * a.D * ES);
  float w[VN][W], u[VN];
  load_taps<VN, W>(a, ch, w, u);
#pragma unroll
  for (int j = 0; j < W; ++j) {
    float v[VN];
    V::unpack(raw[j], v);
#pragma unroll
    for (int c = 0; c < VN; ++c) u[c] = fmaf(w[c][j], v[c], u[c]);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) *reinterpret_cast<uint4*>(st + (long long)j * a.D * ES) = raw[j + 1];
#pragma unroll
  for (int c = 0; c < VN; ++c) u[c] = a.silu ? silu_fast(u[c]) : u[c];
  *reinterpret_cast<uint4*>(static_cast<char*>(a.y) + (n * a.D + ch) * (long long)ES) = V::pack(u);
}

// ------------------------------------------------------------------ backward
//
//   du_t = dy_t silu'(u_t),  silu'(u) = p (1 + u (1 - p)),  p = sigmoid(u)
//   dx_t = sum_j w_j du_{t + (W-1) - j}   (+ dstate_T for the last W - 1 inputs)
//   dw_j = sum_t du_t x_{t - (W-1) + j},  dbias = sum_t du_t.
// u is recomputed from x. A CTA owns 16 vectors of channels and 16 runs of
// tokens, one run to a thread; each thread walks its run with the last W inputs
// and W du's in registers, and looks W - 1 tokens past its end for the dx of its
// last ones. The parameter sums go over the CTA's runs in shared memory and then,
// in a fixed order, over CTAs in a second kernel: no atomics, the same bits
// every time.
constexpr int kBwdVecs = 16, kBwdRuns = 16;

template <bool BF16, int W>
__global__ void __launch_bounds__(kBwdVecs* kBwdRuns)
palimpsa_conv_bwd_kernel(ConvArgs a, int run_len, int blocks_per_seq, float* partial) {
  using V = Vec<BF16>;
  constexpr int VN = V::n, ES = V::bytes;
  const int nvec = a.D / VN, vtiles = (nvec + kBwdVecs - 1) / kBwdVecs;
  const int vx = threadIdx.x % kBwdVecs, ry = threadIdx.x / kBwdVecs;
  const long long blk = blockIdx.x / vtiles;  // token block, over all sequences
  const int vec = (int)(blockIdx.x % vtiles) * kBwdVecs + vx;
  const int ch = vec * VN;
  const long long n = blk / blocks_per_seq;
  const int t0 = ((int)(blk % blocks_per_seq) * kBwdRuns + ry) * run_len;
  long long row0;
  int len;
  const bool ok = seq_rows(a.rows, n, &row0, &len);
  if (!ok && threadIdx.x == 0) latch_status(a.status, kStatusDomain);
  const bool live = ok && vec < nvec;
  const int t1 = min(len, t0 + run_len);  // this run's tokens are [t0, t1)

  float gw[VN][W], gb[VN];
#pragma unroll
  for (int c = 0; c < VN; ++c) {
    gb[c] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) gw[c][j] = 0.f;
  }
  // The run at the sequence's start also owns the gradient of the state rows
  // (places -(W-1) .. -1); with an empty sequence they pass dstate_T through.
  const bool first = t0 == 0;
  if (live && (t0 < t1 || first)) {
    float w[VN][W], b[VN];
    load_taps<VN, W>(a, ch, w, b);
    const char* gdy = static_cast<const char*>(a.dy);
    float x[W][VN], du[W][VN];  // rings by place modulo W
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int c = 0; c < VN; ++c) du[j][c] = 0.f;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) V::unpack(input_row<BF16, W>(a, n, row0, t0 - (W - 1) + k, ch), x[k]);
    // Step s brings in token t0 + s (its x and dy) and finishes the gradient of
    // place t0 + s - (W-1): all W of its du's are then known.
    const int steps = (t1 - t0 > 0 ? t1 - t0 : 0) + W - 1;
    for (int s0 = 0; s0 < steps; s0 += W) {
      // Both rows of the next W tokens are loaded before any is used.
      uint4 rx[W], rd[W];
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const int t = t0 + s0 + k;
        const bool in = s0 + k < steps && t < len;
        rx[k] = in ? input_row<BF16, W>(a, n, row0, t, ch) : make_uint4(0, 0, 0, 0);
        rd[k] = in ? *reinterpret_cast<const uint4*>(gdy + ((row0 + t) * a.dy_ld + ch) * ES) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < W; ++k) {
        if (s0 + k >= steps) break;
        const int t = t0 + s0 + k, p = t - (W - 1);
        const bool own = t < t1;  // later tokens only finish this run's dx
        float g[VN];
        V::unpack(rx[k], x[(k + W - 1) % W]);
        V::unpack(rd[k], g);
#pragma unroll
        for (int c = 0; c < VN; ++c) {
          float u = b[c];
#pragma unroll
          for (int j = 0; j < W; ++j) u = fmaf(w[c][j], x[(k + j) % W][c], u);
          if (a.silu) {
            const float q = sigmoid_fast(u);
            g[c] *= q * fmaf(u, 1.f - q, 1.f);
          }
          if (t >= len) g[c] = 0.f;
          du[k][c] = g[c];
          if (own) {
            gb[c] += g[c];
#pragma unroll
            for (int j = 0; j < W; ++j) gw[c][j] = fmaf(g[c], x[(k + j) % W][c], gw[c][j]);
          }
        }
        // place p takes w_j du_{p + (W-1) - j} = w_j du_{t - j}
        if (p < t0 && !first) continue;
        float d[VN];
#pragma unroll
        for (int c = 0; c < VN; ++c) {
          d[c] = 0.f;
#pragma unroll
          for (int j = 0; j < W; ++j) d[c] = fmaf(w[c][j], du[(k - j + W) % W][c], d[c]);
        }
        const int back = p - (len - (W - 1));  // place in state_T, if >= 0
        if (a.dstate_T && back >= 0) {
          float e[VN];
          V::unpack(*reinterpret_cast<const uint4*>(static_cast<const char*>(a.dstate_T) +
                                                    ((n * (W - 1) + back) * a.D + ch) * (long long)ES), e);
#pragma unroll
          for (int c = 0; c < VN; ++c) d[c] += e[c];
        }
        if (p >= 0)
          *reinterpret_cast<uint4*>(static_cast<char*>(a.dx) + ((row0 + p) * a.D + ch) * (long long)ES) = V::pack(d);
        else if (a.dstate0)
          *reinterpret_cast<uint4*>(static_cast<char*>(a.dstate0) +
                                    ((n * (W - 1) + (W - 1 + p)) * a.D + ch) * (long long)ES) = V::pack(d);
      }
    }
  }
  // Parameter sums over the CTA's runs, value by value.
  __shared__ float red[kBwdRuns][kBwdVecs * VN + 1];
  for (int v = 0; v <= W; ++v) {
    __syncthreads();
#pragma unroll
    for (int c = 0; c < VN; ++c) {
      float g = gb[c];
#pragma unroll
      for (int j = 0; j < W; ++j) g = v == j ? gw[c][j] : g;
      red[ry][vx * VN + c] = g;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < kBwdVecs * VN; c += kBwdVecs * kBwdRuns) {
      const int cc = (int)(blockIdx.x % vtiles) * kBwdVecs * VN + c;
      if (cc >= a.D) continue;
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < kBwdRuns; ++r) s += red[r][c];
      partial[(blk * (W + 1) + v) * a.D + cc] = s;
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

// Run length of the backward: long runs waste less on the W - 1 tokens past the
// end and on partials, short ones make enough threads. From 64 down to 8 until
// there are 512 threads for each of 152 SMs.
int bwd_run_len(const ConvArgs& a) {
  const long long vecs = a.D / (a.bf16 ? 8 : 4);
  int r = 64;
  while (r > 8 && (long long)a.rows.n_seq * ((a.rows.max_len + r - 1) / r) * vecs < 152ll * 512) r /= 2;
  return r;
}
int bwd_blocks_per_seq(const ConvArgs& a, int run) {
  const int per = run * kBwdRuns;
  return std::max(1, (a.rows.max_len + per - 1) / per);
}

template <bool BF16, int W>
cudaError_t backward(const ConvArgs& a, float* scratch, cudaStream_t s) {
  const int run = bwd_run_len(a), bps = bwd_blocks_per_seq(a, run);
  const int nvec = a.D / Vec<BF16>::n, vtiles = (nvec + kBwdVecs - 1) / kBwdVecs;
  const long long blocks = (long long)bps * a.rows.n_seq;
  if (blocks * vtiles > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  palimpsa_conv_bwd_kernel<BF16, W>
      <<<(unsigned)(blocks * vtiles), kBwdVecs * kBwdRuns, 0, s>>>(a, run, bps, scratch);
  palimpsa_conv_bwd_sum_kernel<<<dim3((a.D + 31) / 32, W + 1), 256, 0, s>>>(scratch, blocks, W, a.D, a.dweight,
                                                                            a.dbias);
  return cudaGetLastError();
}

template <bool BF16, int W>
cudaError_t forward(const ConvArgs& a, cudaStream_t s) {
  const int runs = std::max(1, (a.rows.max_len + kRun - 1) / kRun);
  const long long n = (long long)(a.D / Vec<BF16>::n) * runs * a.rows.n_seq, blocks = (n + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  palimpsa_conv_kernel<BF16, W><<<(unsigned)blocks, kThreads, 0, s>>>(a, runs);
  return cudaGetLastError();
}

template <bool BF16, int W>
cudaError_t step(const ConvArgs& a, cudaStream_t s) {
  const long long n = (long long)(a.D / Vec<BF16>::n) * a.rows.n_seq, blocks = (n + 127) / 128;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  palimpsa_conv_step_kernel<BF16, W><<<(unsigned)blocks, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

#define PALIMPSA_CONV_DISPATCH(f, ...)                                     \
  switch (a.W) {                                                           \
    case 2: return a.bf16 ? f<true, 2>(__VA_ARGS__) : f<false, 2>(__VA_ARGS__); \
    case 3: return a.bf16 ? f<true, 3>(__VA_ARGS__) : f<false, 3>(__VA_ARGS__); \
    default: return a.bf16 ? f<true, 4>(__VA_ARGS__) : f<false, 4>(__VA_ARGS__); \
  }

cudaError_t launch_conv_forward(const ConvArgs& a, cudaStream_t s) { PALIMPSA_CONV_DISPATCH(forward, a, s) }
cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t s) { PALIMPSA_CONV_DISPATCH(step, a, s) }
size_t conv_backward_scratch_bytes(const ConvArgs& a) {
  return (size_t)bwd_blocks_per_seq(a, bwd_run_len(a)) * a.rows.n_seq * (a.W + 1) * a.D * sizeof(float);
}
cudaError_t launch_conv_backward(const ConvArgs& a, float* scratch, cudaStream_t s) {
  PALIMPSA_CONV_DISPATCH(backward, a, scratch, s)
}

}  // namespace palimpsa
