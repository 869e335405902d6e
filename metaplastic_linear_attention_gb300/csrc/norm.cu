// Layer norm of rows of D values, forward and backward.
//   s = x + residual (rounded to the type: the rows that are normalised are the ones that are
//   kept), m = mean(s), q = 1 / sqrt(mean((s - m)^2) + eps), y = (s - m) q w + b
//   ds' = q (u - mean(u) - t mean(u t)) + ds,  u = dy w,  t = (s - m) q;  dw = sum dy t, db = sum dy
// (ds: the gradient that reaches s past the norm; x and residual both receive ds'.)
//
// Bound by HBM: 4 bytes a value in bf16 (8 with a residual), backward 6 (8), against some 15 and
// 20 operations. A thread owns 8 columns (16 for rows of more than 4096) of many rows, so
// that weights and the parameters' sums stay in registers; a row's team of threads is
// part of a warp (8 lanes up to 64 columns, a whole one up to 256) or a CTA. A grid of as many
// CTAs as the GPU holds walks the rows, two at a time in bf16; the next ones come by
// asynchronous copies into a ring in shared memory, each thread its own columns, so the
// copies need no barrier. A forward row costs one exchange between warps: each has the
// mean and the squares about its own mean of its part, and these are joined exactly
// (the squares about the row's mean are those about the warp's plus count (mean_w - m)^2),
// so nothing cancels, however far the row is off centre.
//
// Rounding: sums and statistics are fp32; outputs are rounded to the input type once.
#include <algorithm>

#include "ssm.cuh"

namespace palimpsa {
namespace {

constexpr int kCols = 8;             // columns of a thread's vector
constexpr int kThreadsPerSm = 1024;  // which all of a launch's CTAs on an SM come to, at most
constexpr int kWarps = 8;            // of a CTA of several teams

// Rows at a time and stages of the ring: at most 192 bytes a thread and vector.
template <bool BF16>
constexpr int kRows = BF16 ? 2 : 1;
template <int ARRAYS>
constexpr int kRing = ARRAYS == 1 ? 4 : ARRAYS == 2 ? 3 : 2;

template <bool BF16>
struct Cols {  // 8 values of the input type, in 16-byte vectors
  static constexpr int halves = BF16 ? 1 : 2;
  static __device__ __forceinline__ void unpack(const uint4* u, float* f) {
#pragma unroll
    for (int k = 0; k < halves; ++k) Vec<BF16>::unpack(u[k], f + k * Vec<BF16>::n);
  }
  static __device__ __forceinline__ void pack(const float* f, uint4* u) {
#pragma unroll
    for (int k = 0; k < halves; ++k) u[k] = Vec<BF16>::pack(f + k * Vec<BF16>::n);
  }
};

// A thread's place: its team, its vectors' columns, the rows it walks.
template <bool BF16, int LANES, bool MULTI, int V, int ARRAYS>
struct Walk {
  static constexpr int R = kRows<BF16>, S = kRing<ARRAYS>, H = Cols<BF16>::halves;
  int tid, t, team_size;
  long long first, stride, rows;
  int batches, nv;
  uint4* ring;
  __device__ __forceinline__ Walk(long long rows_, int D, unsigned char* smem) : rows(rows_), nv(D / kCols) {
    tid = threadIdx.x;
    t = MULTI ? tid : tid % LANES;
    team_size = MULTI ? blockDim.x : LANES;
    const int teams = MULTI ? 1 : blockDim.x / LANES;
    first = (long long)blockIdx.x * teams + (MULTI ? 0 : tid / LANES);
    stride = (long long)gridDim.x * teams;
    batches = (int)((rows + stride * R - 1) / (stride * R));  // the same for every team
    ring = reinterpret_cast<uint4*>(smem) + tid;
  }
  __device__ __forceinline__ int vec(int v) const { return v * team_size + t; }
  __device__ __forceinline__ bool has(int v) const { return vec(v) < nv; }
  __device__ __forceinline__ long long row(int b, int j) const { return ((long long)b * R + j) * stride + first; }
  __device__ __forceinline__ uint4* slot(int b, int array, int j, int v) const {
    return ring + ((((b % S) * ARRAYS + array) * R + j) * V + v) * H * (int)blockDim.x;
  }
  // Copies of a batch of rows of an array.
  __device__ __forceinline__ void fetch(int b, int array, const void* p, long long ld) const {
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (row(b, j) < rows && has(v)) {
          const char* from = static_cast<const char*>(p) + (row(b, j) * ld + vec(v) * kCols) * Vec<BF16>::bytes;
          uint4* const to = slot(b, array, j, v);
#pragma unroll
          for (int h = 0; h < H; ++h) cp_async16(to + h * blockDim.x, from + 16 * h);
        }
  }
  // 8 values of the ring (zeros where there are none).
  __device__ __forceinline__ void read(int b, int array, int j, int v, float* f) const {
    uint4 u[H];
#pragma unroll
    for (int h = 0; h < H; ++h) u[h] = slot(b, array, j, v)[h * blockDim.x];
    Cols<BF16>::unpack(u, f);
    if (!has(v) || row(b, j) >= rows)
#pragma unroll
      for (int c = 0; c < kCols; ++c) f[c] = 0.f;
  }
  __device__ __forceinline__ void write(void* p, int D, int b, int j, int v, const float* f) const {
    if (row(b, j) >= rows || !has(v)) return;
    uint4 u[H];
    Cols<BF16>::pack(f, u);
    uint4* const to =
        reinterpret_cast<uint4*>(static_cast<char*>(p) + (row(b, j) * D + vec(v) * kCols) * Vec<BF16>::bytes);
#pragma unroll
    for (int h = 0; h < H; ++h) to[h] = u[h];
  }
  // A thread's columns of a parameter.
  __device__ __forceinline__ void param(const float* p, float otherwise, int v, float* f) const {
#pragma unroll
    for (int c = 0; c < kCols; ++c) f[c] = p && has(v) ? p[vec(v) * kCols + c] : otherwise;
  }
};

template <int LANES>
__device__ __forceinline__ float team_sum(float x) {
#pragma unroll
  for (int d = LANES / 2; d > 0; d /= 2) x += __shfl_xor_sync(~0u, x, d);
  return x;
}

template <bool BF16, int LANES, bool MULTI, int V, bool RES>
__global__ void __launch_bounds__(512) palimpsa_norm_kernel(NormArgs a) {
  using W = Walk<BF16, LANES, MULTI, V, 1 + RES>;
  constexpr int R = W::R;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float2 parts[2][R][16];  // of the warps: mean and squares about it
  const W at(a.rows, a.D, smem);
  const int warp = at.tid / 32, lane = at.tid % 32, warps = blockDim.x / 32;
  auto stage = [&](int b) {
    if (b < at.batches) {
      at.fetch(b, 0, a.x, a.x_ld);
      if (RES) at.fetch(b, 1, a.residual, a.residual_ld);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < W::S - 1; ++k) stage(k);
  float wt[V][kCols], bias[V][kCols];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    at.param(a.weight, 1.f, v, wt[v]);
    at.param(a.bias, 0.f, v, bias[v]);
  }
  // Values of warp w of the row.
  auto count = [&](int w) {
    int n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) n += min(max(at.nv - (v * (int)blockDim.x + 32 * w), 0), 32);
    return (float)(n * kCols);
  };
  const float D = (float)a.D, own = MULTI ? count(warp) : D;

  for (int b = 0; b < at.batches; ++b) {
    cp_async_wait<W::S - 2>();
    float s[R][V][kCols], mean[R], rstd[R];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        at.read(b, 0, j, v, s[j][v]);
        if (RES) {
          float r[kCols];
          at.read(b, 1, j, v, r);
#pragma unroll
          for (int c = 0; c < kCols; ++c) r[c] += s[j][v][c];
          uint4 u[W::H];
          Cols<BF16>::pack(r, u);
          Cols<BF16>::unpack(u, s[j][v]);
          at.write(a.sum, a.D, b, j, v, s[j][v]);
        }
      }
    stage(b + W::S - 1);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int c = 0; c < kCols; ++c) sum += s[j][v][c];
      mean[j] = __fdiv_rn(team_sum<LANES>(sum), own);
      float sq = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (at.has(v))
#pragma unroll
          for (int c = 0; c < kCols; ++c) sq = fmaf(s[j][v][c] - mean[j], s[j][v][c] - mean[j], sq);
      rstd[j] = team_sum<LANES>(sq);
      if (MULTI && lane == 0) parts[b & 1][j][warp] = make_float2(mean[j], rstd[j]);
    }
    if (MULTI) {
      __syncthreads();  // (two sets of parts: the last batch's may still be read)
#pragma unroll
      for (int j = 0; j < R; ++j) {
        float m = 0.f, q = 0.f;
        for (int w = 0; w < warps; ++w) m = fmaf(count(w), parts[b & 1][j][w].x, m);
        m = __fdiv_rn(m, D);
        for (int w = 0; w < warps; ++w) {
          const float2 p = parts[b & 1][j][w];
          q += fmaf(count(w) * (p.x - m), p.x - m, p.y);
        }
        mean[j] = m;
        rstd[j] = q;
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      rstd[j] = __frsqrt_rn(__fdiv_rn(rstd[j], D) + a.eps);
      if (a.stats && at.t == 0 && at.row(b, j) < at.rows)
        reinterpret_cast<float2*>(a.stats)[at.row(b, j)] = make_float2(mean[j], rstd[j]);
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          s[j][v][c] = fmaf((s[j][v][c] - mean[j]) * rstd[j], wt[v][c], bias[v][c]);
        at.write(a.y, a.D, b, j, v, s[j][v]);
      }
    }
  }
}

// sums: [CTAs, 2, D], the CTAs' parts of dweight and dbias, or null.
template <bool BF16, int LANES, bool MULTI, int V, bool DS>
__global__ void __launch_bounds__(512) palimpsa_norm_bwd_kernel(NormArgs a, float* sums) {
  using W = Walk<BF16, LANES, MULTI, V, 2 + DS>;
  constexpr int R = W::R;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float2 parts[2][R][16];
  const W at(a.rows, a.D, smem);
  const int warp = at.tid / 32, lane = at.tid % 32, warps = blockDim.x / 32;
  float2 next[R];  // the statistics of the next batch's rows
  auto stage = [&](int b) {
    if (b < at.batches) {
      at.fetch(b, 0, a.x, a.x_ld);
      at.fetch(b, 1, a.dy, a.dy_ld);
      if (DS) at.fetch(b, 2, a.ds, a.ds_ld);
    }
    cp_async_commit();
  };
  auto load_stats = [&](int b) {
#pragma unroll
    for (int j = 0; j < R; ++j)
      next[j] = at.row(b, j) < at.rows ? reinterpret_cast<const float2*>(a.stats)[at.row(b, j)] : make_float2(0.f, 0.f);
  };
  load_stats(0);
#pragma unroll
  for (int k = 0; k < W::S - 1; ++k) stage(k);
  float wt[V][kCols], gw[V][kCols], gb[V][kCols];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    at.param(a.weight, 1.f, v, wt[v]);
#pragma unroll
    for (int c = 0; c < kCols; ++c) gw[v][c] = gb[v][c] = 0.f;
  }
  const float inv = __frcp_rn((float)a.D);

  for (int b = 0; b < at.batches; ++b) {
    float2 st[R], tot[R];
#pragma unroll
    for (int j = 0; j < R; ++j) st[j] = next[j];
    cp_async_wait<W::S - 2>();
    stage(b + W::S - 1);
    load_stats(b + 1);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float x[kCols], dy[kCols];
        at.read(b, 0, j, v, x);
        at.read(b, 1, j, v, dy);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const float t = (x[c] - st[j].x) * st[j].y, u = dy[c] * wt[v][c];
          gw[v][c] = fmaf(dy[c], t, gw[v][c]);
          gb[v][c] += dy[c];
          s1 += u;
          s2 = fmaf(u, t, s2);
        }
      }
      tot[j] = make_float2(team_sum<LANES>(s1), team_sum<LANES>(s2));
      if (MULTI && lane == 0) parts[b & 1][j][warp] = tot[j];
    }
    if (MULTI) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < R; ++j) {
        tot[j] = parts[b & 1][j][0];
        for (int w = 1; w < warps; ++w) {
          const float2 p = parts[b & 1][j][w];
          tot[j].x += p.x;
          tot[j].y += p.y;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float x[kCols], dy[kCols], ds[kCols];
        at.read(b, 0, j, v, x);
        at.read(b, 1, j, v, dy);
        if (DS) at.read(b, 2, j, v, ds);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const float t = (x[c] - st[j].x) * st[j].y;
          const float u = fmaf(dy[c], wt[v][c], -tot[j].x * inv);
          const float d = fmaf(-t, tot[j].y * inv, u);
          x[c] = DS ? fmaf(st[j].y, d, ds[c]) : st[j].y * d;
        }
        at.write(a.dx, a.D, b, j, v, x);
      }
  }
  if (!sums) return;
  float* const out = sums + (long long)blockIdx.x * 2 * a.D;
  if (MULTI) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at.has(v)) {
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          float* const p = out + at.vec(v) * kCols + c;
          *reinterpret_cast<float4*>(p) = make_float4(gw[v][c], gw[v][c + 1], gw[v][c + 2], gw[v][c + 3]);
          *reinterpret_cast<float4*>(p + a.D) = make_float4(gb[v][c], gb[v][c + 1], gb[v][c + 2], gb[v][c + 3]);
        }
      }
  } else {
    // The CTA's teams, through the ring's memory (its copies are done: the last groups are empty).
    cp_async_wait<0>();
    float* const red = reinterpret_cast<float*>(smem);
    const int teams = blockDim.x / LANES, team = at.tid / LANES, cols = LANES * kCols;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kCols; ++c) red[(team * kCols + c) * LANES + at.t] = q ? gb[0][c] : gw[0][c];
      __syncthreads();
      for (int k = at.tid; k < cols; k += blockDim.x) {
        float s = 0.f;
        for (int m = 0; m < teams; ++m) s += red[m * cols + k];
        const int col = k % LANES * kCols + k / LANES;
        if (col < a.D) out[q * a.D + col] = s;
      }
    }
  }
}

// Sums the CTAs' parts [rows, 2, D]: 32 columns by 32 slices of the rows; block y = 0 dweight, 1 dbias.
__global__ void __launch_bounds__(1024) palimpsa_norm_bwd_sum_kernel(const float* sums, int rows, int D, float* dweight,
                                                                     float* dbias) {
  __shared__ float red[32][33];
  const int cx = threadIdx.x % 32, sy = threadIdx.x / 32, col = blockIdx.x * 32 + cx, v = blockIdx.y;
  float* const out = v ? dbias : dweight;
  if (!out) return;
  float s = 0.f;
  if (col < D)
#pragma unroll 4
    for (int b = sy; b < rows; b += 32) s += sums[((long long)b * 2 + v) * D + col];
  red[sy][cx] = s;
  __syncthreads();
  s = red[cx][sy];  // column sy
#pragma unroll
  for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(~0u, s, d);
  if (cx == 0 && blockIdx.x * 32 + sy < D) out[blockIdx.x * 32 + sy] = s;
}

// Threads of a CTA and its teams for rows of D values.
struct Shape {
  int threads, teams, ctas;  // ctas: as the rows need, and the GPU holds
};
Shape shape_of(const NormArgs& a) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 152;
  const int nv = a.D / kCols;
  Shape p;
  if (nv <= 32) {
    p.threads = 32 * kWarps;
    p.teams = p.threads / (nv <= 8 ? 8 : 32);
  } else {
    const int per = nv <= 512 ? nv : (nv + 1) / 2;
    p.threads = (per + 31) / 32 * 32;
    p.teams = 1;
  }
  const long long held = (long long)std::max(1, kThreadsPerSm / p.threads) * sms;
  p.ctas = (int)std::min(held, (a.rows + p.teams - 1) / p.teams);
  return p;
}

template <bool BF16, int LANES, bool MULTI, int V, bool MORE>
cudaError_t run_forward(const NormArgs& a, const Shape& p, cudaStream_t s) {
  using W = Walk<BF16, LANES, MULTI, V, 1 + MORE>;
  const int bytes = p.threads * 16 * W::S * (1 + MORE) * W::R * V * W::H;
  const auto kernel = palimpsa_norm_kernel<BF16, LANES, MULTI, V, MORE>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  kernel<<<p.ctas, p.threads, bytes, s>>>(a);
  return cudaGetLastError();
}

template <bool BF16, int LANES, bool MULTI, int V, bool MORE>
cudaError_t run_backward(const NormArgs& a, const Shape& p, float* sums, cudaStream_t s) {
  using W = Walk<BF16, LANES, MULTI, V, 2 + MORE>;
  const int bytes = p.threads * 16 * W::S * (2 + MORE) * W::R * V * W::H;
  const auto kernel = palimpsa_norm_bwd_kernel<BF16, LANES, MULTI, V, MORE>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  kernel<<<p.ctas, p.threads, bytes, s>>>(a, sums);
  return cudaGetLastError();
}

}  // namespace

#define PALIMPSA_NORM_TEAM(f, BF16, MORE, ...)                                                    \
  (a.D <= 64 ? f<BF16, 8, false, 1, MORE>(__VA_ARGS__)                                            \
   : a.D <= 256 ? f<BF16, 32, false, 1, MORE>(__VA_ARGS__)                                        \
   : a.D <= 4096 ? f<BF16, 32, true, 1, MORE>(__VA_ARGS__) : f<BF16, 32, true, 2, MORE>(__VA_ARGS__))
#define PALIMPSA_NORM_DISPATCH(f, more, ...)                                                      \
  (a.bf16 ? ((more) ? PALIMPSA_NORM_TEAM(f, true, true, __VA_ARGS__) : PALIMPSA_NORM_TEAM(f, true, false, __VA_ARGS__)) \
          : ((more) ? PALIMPSA_NORM_TEAM(f, false, true, __VA_ARGS__) : PALIMPSA_NORM_TEAM(f, false, false, __VA_ARGS__)))

cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  const Shape p = shape_of(a);
  return PALIMPSA_NORM_DISPATCH(run_forward, a.residual, a, p, s);
}

size_t norm_backward_scratch_floats(const NormArgs& a) {
  return a.dweight || a.dbias ? (size_t)shape_of(a).ctas * 2 * a.D : 0;
}

cudaError_t launch_norm_backward(const NormArgs& a, float* scratch, cudaStream_t s) {
  const Shape p = shape_of(a);
  if (a.rows > 0) {
    const cudaError_t e = PALIMPSA_NORM_DISPATCH(run_backward, a.ds, a, p, scratch, s);
    if (e != cudaSuccess) return e;
  }
  if (!a.dweight && !a.dbias) return cudaSuccess;
  palimpsa_norm_bwd_sum_kernel<<<dim3((a.D + 31) / 32, 2), 1024, 0, s>>>(scratch, a.rows > 0 ? p.ctas : 0, a.D,
                                                                         a.dweight, a.dbias);
  return cudaGetLastError();
}

}  // namespace palimpsa
