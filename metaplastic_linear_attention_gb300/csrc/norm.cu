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

constexpr int kCols = 8, kPairs = 4;  // columns of a thread's vector
constexpr int kWarps = 8;            // of a CTA of several teams

// Rows at a time and stages of the ring: at most 192 bytes a thread and vector (and 16 to
// spread the threads over the banks).
template <bool BF16>
constexpr int kRows = BF16 ? 2 : 1;
template <int ARRAYS>
constexpr int kRing = ARRAYS == 1 ? 4 : ARRAYS == 2 ? 3 : 2;

// A thread's place: its team, its vectors' columns, the rows it walks, and its part of the
// ring: [stage][array][row][vector][half] of 16 bytes, an odd number in all.
template <bool BF16, int LANES, bool MULTI, int V, int ARRAYS>
struct Walk {
  static constexpr int R = kRows<BF16>, S = kRing<ARRAYS>, H = BF16 ? 1 : 2, ES = Vec<BF16>::bytes;
  static constexpr int planes = ARRAYS * R * V * H, units = S * planes | 1;
  int t, team_size, batches, nv;
  long long rows, first, stride;  // the team's first row, and how far apart its rows are
  unsigned char* ring;
  __device__ __forceinline__ Walk(long long rows_, int D, unsigned char* smem) : nv(D / kCols), rows(rows_) {
    const int tid = threadIdx.x, teams = MULTI ? 1 : blockDim.x / LANES;
    t = MULTI ? tid : tid % LANES;
    team_size = MULTI ? blockDim.x : LANES;
    first = (long long)blockIdx.x * teams + (MULTI ? 0 : tid / LANES);
    stride = (long long)gridDim.x * teams;
    batches = (int)((rows + stride * R - 1) / (stride * R));  // the same for every team
    ring = smem + tid * units * 16;
    // Columns past D are zeros: no copy goes there.
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!has(v))
        for (int k = 0; k < S * ARRAYS * R; ++k)
#pragma unroll
          for (int h = 0; h < H; ++h) *reinterpret_cast<uint4*>(ring + ((k * V + v) * H + h) * 16) = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ int col(int v) const { return (v * team_size + t) * kCols; }
  __device__ __forceinline__ bool has(int v) const { return v * team_size + t < nv; }
  // The byte offset of the team's first row, and from a row to the next, in an array.
  __device__ __forceinline__ long long start(long long ld) const { return (first * ld + t * kCols) * ES; }
  __device__ __forceinline__ long long apart(long long ld) const { return stride * ld * ES; }
  // A batch's rows of an array, from row on, p their place in the first; rows past the end as
  // zeros.
  __device__ __forceinline__ void fetch(int stage, int array, const char* p, long long next, long long row) const {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool in = row + j * stride < rows;
      const char* const q = in ? p + j * next : p;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (has(v))
#pragma unroll
          for (int h = 0; h < H; ++h)
            cp_async16(ring + (stage * planes + ((array * R + j) * V + v) * H + h) * 16,
                       q + (long long)v * team_size * (kCols * ES) + 16 * h, in);
    }
  }
  // 8 values of the ring, as pairs.
  __device__ __forceinline__ void read(int stage, int array, int j, int v, float2* f) const {
#pragma unroll
    for (int h = 0; h < H; ++h)
      unpack(*reinterpret_cast<const uint4*>(ring + (stage * planes + ((array * R + j) * V + v) * H + h) * 16), f + 2 * h);
  }
  // Rounds 8 values to the type, stores them at p and, if kept, leaves them rounded in f.
  __device__ __forceinline__ void write(char* p, int v, float2* f, bool in, bool keep) const {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      uint4 u;
      if constexpr (BF16) {
        u = make_uint4(Vec<true>::two(f[0].x, f[0].y), Vec<true>::two(f[1].x, f[1].y), Vec<true>::two(f[2].x, f[2].y),
                       Vec<true>::two(f[3].x, f[3].y));
      } else {
        u = make_uint4(__float_as_uint(f[2 * h].x), __float_as_uint(f[2 * h].y), __float_as_uint(f[2 * h + 1].x),
                       __float_as_uint(f[2 * h + 1].y));
      }
      if (in) *reinterpret_cast<uint4*>(p + (long long)v * team_size * (kCols * ES) + 16 * h) = u;
      if (keep && BF16) unpack(u, f);
    }
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float2* f) {
    if constexpr (BF16) {
      f[0] = make_float2(bf16_lo(u.x), bf16_hi(u.x));
      f[1] = make_float2(bf16_lo(u.y), bf16_hi(u.y));
      f[2] = make_float2(bf16_lo(u.z), bf16_hi(u.z));
      f[3] = make_float2(bf16_lo(u.w), bf16_hi(u.w));
    } else {
      f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
      f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
  }
  // A thread's columns of a parameter.
  __device__ __forceinline__ void param(const float* p, float otherwise, int v, float2* f) const {
#pragma unroll
    for (int c = 0; c < kPairs; ++c)
      f[c] = p && has(v) ? make_float2(p[col(v) + 2 * c], p[col(v) + 2 * c + 1]) : make_float2(otherwise, otherwise);
  }
};

// Sums over teams of LANES of N values. Each step halves what a lane goes on with, as long as
// there are several: lane l of the team ends up with the sum of value l N / LANES.
template <int LANES, int N>
__device__ __forceinline__ float team_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int d = LANES / 2;
#pragma unroll
  for (int n = N; n > 1; n /= 2, d /= 2) {
    const bool upper = lane & d;
#pragma unroll
    for (int k = 0; k < n / 2; ++k) {
      const float keep = upper ? v[k + n / 2] : v[k], send = upper ? v[k] : v[k + n / 2];
      v[k] = keep + __shfl_xor_sync(~0u, send, d);
    }
  }
#pragma unroll
  for (; d > 0; d /= 2) v[0] += __shfl_xor_sync(~0u, v[0], d);
  return v[0];
}
// All N sums in every lane, from what team_sums left.
template <int LANES, int N>
__device__ __forceinline__ void spread(float mine, float (&v)[N]) {
  const int first = (threadIdx.x & 31) & ~(LANES - 1);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = __shfl_sync(~0u, mine, first + k * (LANES / N));
}
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
  for (int d = 8; d > 0; d /= 2) x += __shfl_xor_sync(~0u, x, d);
  return x;
}
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }
// 1 / sqrt(x): the SFU's, with one step of Newton's method.
__device__ __forceinline__ float rsqrt_of(float x) {
  const float y = rsqrtf(x);
  return y * fmaf(-0.5f * x * y, y, 1.5f);
}

template <bool BF16, int LANES, bool MULTI, int V, bool RES>
__global__ void __launch_bounds__(MULTI ? 512 : 32 * kWarps, MULTI ? 3 - V : 4) palimpsa_norm_kernel(NormArgs a) {
  using W = Walk<BF16, LANES, MULTI, V, 1 + RES>;
  constexpr int R = W::R;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float2 parts[2][R][16];  // of the warps: sums, and squares about their means
  const W at(a.rows, a.D, smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  const long long nx = at.apart(a.x_ld), nr = at.apart(a.residual_ld), ny = at.apart(a.D);
  const char* px = static_cast<const char*>(a.x) + at.start(a.x_ld);
  const char* pr = static_cast<const char*>(a.residual) + at.start(a.residual_ld);
  char* py = static_cast<char*>(a.y) + at.start(a.D);
  char* ps = static_cast<char*>(a.sum) + at.start(a.D);
  long long ahead = at.first, row = at.first;  // the next batch's rows to fetch, and at hand
  int to = 0;
  auto stage = [&]() {
    at.fetch(to, 0, px, nx, ahead);
    if (RES) at.fetch(to, 1, pr, nr, ahead);
    cp_async_commit();
    px += R * nx;
    if (RES) pr += R * nr;
    ahead += R * at.stride;
    to = to + 1 == W::S ? 0 : to + 1;
  };
#pragma unroll
  for (int k = 0; k < W::S - 1; ++k) stage();
  float2 wt[V][kPairs], bias[V][kPairs];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    at.param(a.weight, 1.f, v, wt[v]);
    at.param(a.bias, 0.f, v, bias[v]);
  }
  // Values of warp w's part of a row.
  auto count = [&](int w) {
    int n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) n += min(max(at.nv - (v * (int)blockDim.x + 32 * w), 0), 32);
    return (float)(n * kCols);
  };
  const float whole = __frcp_rn((float)a.D), own = MULTI ? __frcp_rn(count(warp)) : whole;
  const int part = lane & 15;  // the warp whose part of a row (the second half warp: of the second row) a lane joins
  const float parts_n = MULTI && part < warps ? count(part) : 0.f, parts_inv = parts_n ? __frcp_rn(parts_n) : 0.f;

  int from = 0;
  for (int b = 0; b < at.batches; ++b) {
    cp_async_wait<W::S - 2>();
    float2 s[R][V][kPairs];
    float sum[R], sq[R], mean[R], rstd[R];
    bool live[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      live[j] = row + j * at.stride < at.rows;
      float2 t = two(0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        at.read(from, 0, j, v, s[j][v]);
        if (RES) {
          float2 r[kPairs];
          at.read(from, 1, j, v, r);
#pragma unroll
          for (int c = 0; c < kPairs; ++c) s[j][v][c] = __fadd2_rn(s[j][v][c], r[c]);
          at.write(ps + j * ny, v, s[j][v], live[j] && at.has(v), true);
        }
#pragma unroll
        for (int c = 0; c < kPairs; ++c) t = __fadd2_rn(t, s[j][v][c]);
      }
      sum[j] = t.x + t.y;
    }
    from = from + 1 == W::S ? 0 : from + 1;
    stage();  // into the stage of the batch before
    const float sums = team_sums<LANES>(sum);
    spread<LANES>(sums, sum);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      mean[j] = sum[j] * own;
      float2 t = two(0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float2 q = two(0.f);
#pragma unroll
        for (int c = 0; c < kPairs; ++c) {
          const float2 d = __fadd2_rn(s[j][v][c], two(-mean[j]));
          q = __ffma2_rn(d, d, q);
        }
        if (at.has(v)) t = __fadd2_rn(t, q);
      }
      sq[j] = t.x + t.y;
    }
    const float squares = team_sums<LANES>(sq);
    if (MULTI) {
      if (lane % (32 / R) == 0) parts[b & 1][lane / (32 / R)][warp] = make_float2(sums, squares);
      __syncthreads();  // (two sets of parts: the last batch's may still be read)
      const float2 p = part < warps ? parts[b & 1][R == 2 ? lane / 16 : 0][part] : make_float2(0.f, 0.f);
      const float m = sum16(p.x) * whole, d = fmaf(p.x, parts_inv, -m);
      const float q = sum16(fmaf(parts_n * d, d, p.y));
      const float r = rsqrt_of(fmaf(q, whole, a.eps));
#pragma unroll
      for (int j = 0; j < R; ++j) {
        mean[j] = __shfl_sync(~0u, m, 16 * j);
        rstd[j] = __shfl_sync(~0u, r, 16 * j);
      }
    } else {
      spread<LANES>(rsqrt_of(fmaf(squares, whole, a.eps)), rstd);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (a.stats && live[j] && at.t == 0)
        reinterpret_cast<float2*>(a.stats)[row + j * at.stride] = make_float2(mean[j], rstd[j]);
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int c = 0; c < kPairs; ++c) {
          const float2 t = __fmul2_rn(__fadd2_rn(s[j][v][c], two(-mean[j])), two(rstd[j]));
          s[j][v][c] = __ffma2_rn(t, wt[v][c], bias[v][c]);
        }
        at.write(py + j * ny, v, s[j][v], live[j] && at.has(v), false);
      }
    }
    __syncwarp();
    row += R * at.stride;
    py += R * ny;
    if (RES) ps += R * ny;
  }
}

// sums: [CTAs, 2, D], the CTAs' parts of dweight and dbias, or null.
template <bool BF16, int LANES, bool MULTI, int V, bool DS>
__global__ void __launch_bounds__(MULTI ? 512 : 32 * kWarps, MULTI ? 3 - V : 3) palimpsa_norm_bwd_kernel(NormArgs a, float* sums) {
  using W = Walk<BF16, LANES, MULTI, V, 2 + DS>;
  constexpr int R = W::R;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float parts[2][2 * R][16];  // of the warps: mean(u), mean(u t), each for every row
  const W at(a.rows, a.D, smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  const long long nx = at.apart(a.x_ld), ny = at.apart(a.dy_ld), ns = at.apart(a.ds_ld), nd = at.apart(a.D);
  const char* px = static_cast<const char*>(a.x) + at.start(a.x_ld);
  const char* py = static_cast<const char*>(a.dy) + at.start(a.dy_ld);
  const char* ps = static_cast<const char*>(a.ds) + at.start(a.ds_ld);
  char* pd = static_cast<char*>(a.dx) + at.start(a.D);
  const float2* const stats = reinterpret_cast<const float2*>(a.stats);
  long long ahead = at.first, row = at.first;
  int to = 0;
  auto stage = [&]() {
    at.fetch(to, 0, px, nx, ahead);
    at.fetch(to, 1, py, ny, ahead);
    if (DS) at.fetch(to, 2, ps, ns, ahead);
    cp_async_commit();
    px += R * nx;
    py += R * ny;
    if (DS) ps += R * ns;
    ahead += R * at.stride;
    to = to + 1 == W::S ? 0 : to + 1;
  };
  float2 next[R];  // the statistics of the next batch's rows
  auto load_stats = [&](long long r) {
#pragma unroll
    for (int j = 0; j < R; ++j) next[j] = r + j * at.stride < at.rows ? stats[r + j * at.stride] : make_float2(0.f, 0.f);
  };
  load_stats(row);
#pragma unroll
  for (int k = 0; k < W::S - 1; ++k) stage();
  float2 wt[V][kPairs], gw[V][kPairs], gb[V][kPairs];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    at.param(a.weight, 1.f, v, wt[v]);
#pragma unroll
    for (int c = 0; c < kPairs; ++c) gw[v][c] = gb[v][c] = two(0.f);
  }
  const float inv = __frcp_rn((float)a.D);

  int from = 0;
  for (int b = 0; b < at.batches; ++b) {
    float2 st[R];
    float tot[2 * R];
    bool live[R];
#pragma unroll
    for (int j = 0; j < R; ++j) st[j] = next[j];
    cp_async_wait<W::S - 2>();
    stage();  // into the stage of the batch before
    load_stats(row + R * at.stride);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      live[j] = row + j * at.stride < at.rows;
      float2 s1 = two(0.f), s2 = two(0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float2 x[kPairs], dy[kPairs];
        at.read(from, 0, j, v, x);
        at.read(from, 1, j, v, dy);
#pragma unroll
        for (int c = 0; c < kPairs; ++c) {
          const float2 t = __fmul2_rn(__fadd2_rn(x[c], two(-st[j].x)), two(st[j].y)), u = __fmul2_rn(dy[c], wt[v][c]);
          gw[v][c] = __ffma2_rn(dy[c], t, gw[v][c]);
          gb[v][c] = __fadd2_rn(gb[v][c], dy[c]);
          s1 = __fadd2_rn(s1, u);
          s2 = __ffma2_rn(u, t, s2);
        }
      }
      tot[2 * j] = s1.x + s1.y;
      tot[2 * j + 1] = s2.x + s2.y;
    }
    constexpr int per = LANES / (2 * R);  // lanes that share a sum
    float mine = team_sums<LANES>(tot) * inv;
    if (MULTI) {
      if (lane % per == 0) parts[b & 1][lane / per][warp] = mine;
      __syncthreads();
      const int half = lane / 16, w = lane & 15;
#pragma unroll
      for (int j = 0; j < R; ++j) {  // a half warp adds up each of the row's two sums
        const float all = sum16(w < warps ? parts[b & 1][2 * j + half][w] : 0.f);
        tot[2 * j] = __shfl_sync(~0u, all, 0);
        tot[2 * j + 1] = __shfl_sync(~0u, all, 16);
      }
    } else {
      spread<LANES>(mine, tot);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float2 x[kPairs], dy[kPairs], ds[kPairs];
        at.read(from, 0, j, v, x);
        at.read(from, 1, j, v, dy);
        if (DS) at.read(from, 2, j, v, ds);
#pragma unroll
        for (int c = 0; c < kPairs; ++c) {
          const float2 t = __fmul2_rn(__fadd2_rn(x[c], two(-st[j].x)), two(st[j].y));
          const float2 d = __ffma2_rn(t, two(-tot[2 * j + 1]), __ffma2_rn(dy[c], wt[v][c], two(-tot[2 * j])));
          x[c] = DS ? __ffma2_rn(two(st[j].y), d, ds[c]) : __fmul2_rn(two(st[j].y), d);
        }
        at.write(pd + j * nd, v, x, live[j] && at.has(v), false);
      }
    }
    __syncwarp();
    from = from + 1 == W::S ? 0 : from + 1;
    row += R * at.stride;
    pd += R * nd;
  }
  if (!sums) return;
  float* const out = sums + (long long)blockIdx.x * 2 * a.D;
  if (MULTI) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at.has(v)) {
#pragma unroll
        for (int c = 0; c < kPairs; c += 2) {
          float* const p = out + at.col(v) + 2 * c;
          *reinterpret_cast<float4*>(p) = make_float4(gw[v][c].x, gw[v][c].y, gw[v][c + 1].x, gw[v][c + 1].y);
          *reinterpret_cast<float4*>(p + a.D) = make_float4(gb[v][c].x, gb[v][c].y, gb[v][c + 1].x, gb[v][c + 1].y);
        }
      }
  } else {
    // The CTA's teams, through the ring's memory (its copies are done: the last groups are empty).
    cp_async_wait<0>();
    float* const red = reinterpret_cast<float*>(smem);
    const int teams = blockDim.x / LANES, team = threadIdx.x / LANES, cols = LANES * kCols;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const float2 g = q ? gb[0][c / 2] : gw[0][c / 2];
        red[(team * kCols + c) * LANES + at.t] = c & 1 ? g.y : g.x;
      }
      __syncthreads();
      for (int k = threadIdx.x; k < cols; k += blockDim.x) {
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
Shape shape_of(const NormArgs& a, bool backward) {
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
  // (The backward of narrow rows needs 80 registers a thread, the others 64.)
  const int per_sm = backward && p.teams > 1 ? 768 : 1024;
  const long long held = (long long)std::max(1, per_sm / p.threads) * sms;
  p.ctas = (int)std::min(held, (a.rows + p.teams - 1) / p.teams);
  return p;
}

template <bool BF16, int LANES, bool MULTI, int V, bool MORE>
cudaError_t run_forward(const NormArgs& a, const Shape& p, cudaStream_t s) {
  using W = Walk<BF16, LANES, MULTI, V, 1 + MORE>;
  const int bytes = p.threads * 16 * W::units;
  const auto kernel = palimpsa_norm_kernel<BF16, LANES, MULTI, V, MORE>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  kernel<<<p.ctas, p.threads, bytes, s>>>(a);
  return cudaGetLastError();
}

template <bool BF16, int LANES, bool MULTI, int V, bool MORE>
cudaError_t run_backward(const NormArgs& a, const Shape& p, float* sums, cudaStream_t s) {
  using W = Walk<BF16, LANES, MULTI, V, 2 + MORE>;
  const int bytes = p.threads * 16 * W::units;
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
  const Shape p = shape_of(a, false);
  return PALIMPSA_NORM_DISPATCH(run_forward, a.residual, a, p, s);
}

size_t norm_backward_scratch_floats(const NormArgs& a) {
  return a.dweight || a.dbias ? (size_t)shape_of(a, true).ctas * 2 * a.D : 0;
}

cudaError_t launch_norm_backward(const NormArgs& a, float* scratch, cudaStream_t s) {
  const Shape p = shape_of(a, true);
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
