// Layer norm of rows of D values, forward and backward.
//   s = x + residual (rounded to the type: the rows that are normalised are the ones that are
//   kept), m = mean(s), q = 1 / sqrt(mean((s - m)^2) + eps), y = (s - m) q w + b
//   ds' = q (u - mean(u) - t mean(u t)) + ds,  u = dy w,  t = (s - m) q;  dw = sum dy t, db = sum dy
// (ds: the gradient that reaches s past the norm; x and residual both receive ds'.)
//
// Bound by HBM: 4 bytes a value in bf16 (8 with a residual), backward 6 (8), against some 15 and
// 20 operations. A row's team of threads, each with 8 to 64 columns, is 2 to 32 lanes (forward up to 2048
// columns, backward up to 512 and in bf16 1024) or a CTA.
// A grid of as many CTAs as the GPU holds walks the rows; the next ones come by asynchronous
// copies into a ring in shared memory, each thread its own columns, so the copies need no barrier.
// The squares are summed about the row's mean m, which is known by then to the roundings of a sum; so is what m
// leaves out, e = mean(s - m), and the variance is mean((s - m)^2) - e^2 and the mean m + e. Where a row is a
// CTA's, each warp does this about the mean m_w of its own part, and the parts are joined by
//   n variance = sum over warps of n_w (variance_w + (m_w + e_w - mean)^2)
// with one exchange, the means taken relative to the first warp's: nothing cancels, however far the row and its parts are
// off centre. Above 1024 columns in bf16 (512 in fp32) the backward's rows are a CTA's: a thread
// keeps the parameters' sums of its columns in registers over all its rows. CTAs leave theirs for a second
// kernel, which adds them in a fixed order: no atomics, the same bits every time.
//
// Measured (GB300): 70 us at 32768 x 1536 in bf16 with a residual (5.8 TB/s, 59 at the rate of a
// copy), backward 61; rows of 16 to 2048 columns run at 0.7 to 0.9 of a copy's rate (the backward in bf16
// at 0.55 to 0.85), wider ones at 0.7 to 0.9 in fp32 and 0.65 to 0.9 in bf16.
//
// Rounding: sums and statistics are fp32; outputs are rounded to the input type once.
#include <algorithm>

#include "ssm.cuh"

namespace palimpsa {
namespace {

// A thread's place: its team, the rows it walks (R at a time), its columns (V vectors of 16 bytes,
// a team's width apart), and its part of the ring, [stage][array][row][vector][thread]: lanes
// that are neighbours in HBM are so there too (with each thread's vectors next to each other
// in the ring instead, a copy asks for every sector twice: 88 us against 71 at 32768 x 1536 with a
// residual).
template <bool BF16, int LANES, bool MULTI, int COLS, int R_, int ARRAYS>
struct Walk {
  static constexpr int R = R_, ES = Vec<BF16>::bytes, N = Vec<BF16>::n, V = COLS / N, P = N / 2;  // P: pairs of a vector
  static constexpr int planes = ARRAYS * R * V, S = planes <= 4 ? 4 : planes <= 6 ? 3 : 2;
  int t, team_size, batches, nv;
  long long rows, first, stride;  // the team's first row, and how far apart its rows are
  unsigned char* ring;
  __device__ __forceinline__ Walk(long long rows_, int D, unsigned char* smem) : nv(D / N), rows(rows_) {
    const int tid = threadIdx.x, teams = MULTI ? 1 : blockDim.x / LANES;
    t = MULTI ? tid : tid % LANES;
    team_size = MULTI ? blockDim.x : LANES;
    first = (long long)blockIdx.x * teams + (MULTI ? 0 : tid / LANES);
    stride = (long long)gridDim.x * teams;
    batches = (int)((rows + stride * R - 1) / (stride * R));  // the same for every team
    ring = smem + tid * 16;
    // Columns past D are zeros: no copy goes there.
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!has(v))
        for (int k = 0; k < S * ARRAYS * R; ++k) *reinterpret_cast<uint4*>(ring + plane(k * V + v)) = make_uint4(0, 0, 0, 0);
  }
  static __device__ __forceinline__ int plane(int k) { return k * (int)blockDim.x * 16; }
  __device__ __forceinline__ int col(int v) const { return (v * team_size + t) * N; }
  __device__ __forceinline__ bool has(int v) const { return v * team_size + t < nv; }
  // Bytes from a thread's first vector to another.
  __device__ __forceinline__ int across(int v) const { return v * team_size * 16; }
  // The byte offset of the team's first row, and from a row to the next, in an array.
  __device__ __forceinline__ long long start(long long ld) const { return first * ld * ES + t * 16; }
  __device__ __forceinline__ long long apart(long long ld) const { return stride * ld * ES; }
  // A batch's rows of an array, from row on, p their place in the first; rows past the end as
  // zeros.
  __device__ __forceinline__ void fetch(int stage, int array, const char* p, long long next, long long row) const {
    unsigned char* const to = ring + plane(stage * planes + array * R * V);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool in = row + j * stride < rows;
      const char* const q = in ? p + j * next : p;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (has(v)) cp_async16(to + plane(j * V + v), q + across(v), in);
    }
  }
  // A vector of the ring, as pairs.
  __device__ __forceinline__ void read(int stage, int array, int j, int v, float2* f) const {
    unpack(*reinterpret_cast<const uint4*>(ring + plane(stage * planes + (array * R + j) * V + v)), f);
  }
  // Rounds a vector to the type, stores it at p and, if kept, leaves it rounded in f.
  __device__ __forceinline__ void write(char* p, int v, float2* f, bool in, bool keep) const {
    uint4 u;
    if constexpr (BF16) {
      u = make_uint4(Vec<true>::two(f[0].x, f[0].y), Vec<true>::two(f[1].x, f[1].y), Vec<true>::two(f[2].x, f[2].y),
                     Vec<true>::two(f[3].x, f[3].y));
    } else {
      u = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    }
    if (in) *reinterpret_cast<uint4*>(p + across(v)) = u;
    if (keep && BF16) unpack(u, f);
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
};

// A thread's columns of a parameter vector: in registers, or, where a thread has more than 16, in
// shared memory, where all the CTA's teams read them: [vector][4 of its columns][thread of the team].
template <class W, bool SHARED>
struct Param {
  float2 f[SHARED ? 1 : W::V][W::P];
  const float4* at;
  int size;
  __device__ __forceinline__ Param(const W& w, const float* p, float otherwise, float4* shared) {
    if constexpr (SHARED) {
      constexpr int Q = W::N / 4;
      for (int k = threadIdx.x; k < W::V * w.team_size * Q; k += blockDim.x) {
        const int c = k * 4, unit = k / Q;  // 4 columns, of the row's vector `unit`
        float4 u = make_float4(otherwise, otherwise, otherwise, otherwise);
        if (p && c < w.nv * W::N) u = make_float4(p[c], p[c + 1], p[c + 2], p[c + 3]);
        shared[(unit / w.team_size * Q + k % Q) * w.team_size + unit % w.team_size] = u;
      }
      at = shared + w.t;
      size = w.team_size;
    } else {
#pragma unroll
      for (int v = 0; v < W::V; ++v)
#pragma unroll
        for (int c = 0; c < W::P; ++c)
          f[v][c] = p && w.has(v) ? make_float2(p[w.col(v) + 2 * c], p[w.col(v) + 2 * c + 1])
                                  : make_float2(otherwise, otherwise);
    }
  }
  __device__ __forceinline__ void get(int v, float2* out) const {
    if constexpr (SHARED) {
      constexpr int Q = W::N / 4;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const float4 u = at[(v * Q + q) * size];
        out[2 * q] = make_float2(u.x, u.y);
        out[2 * q + 1] = make_float2(u.z, u.w);
      }
    } else {
#pragma unroll
      for (int c = 0; c < W::P; ++c) out[c] = f[v][c];
    }
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
  if constexpr (N == 1) {
    v[0] = mine;
  } else {
    const int first = (threadIdx.x & 31) & ~(LANES - 1);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __shfl_sync(~0u, mine, first + k * (LANES / N));
  }
}
// All sums of both in every lane; in one go where the team has lanes enough.
template <int LANES, int N>
__device__ __forceinline__ void all_sums(float (&a)[N], float (&b)[N]) {
  if constexpr (2 * N <= LANES) {
    float v[2 * N];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = a[k], v[N + k] = b[k];
    spread<LANES>(team_sums<LANES>(v), v);
#pragma unroll
    for (int k = 0; k < N; ++k) a[k] = v[k], b[k] = v[N + k];
  } else {
    spread<LANES>(team_sums<LANES>(a), a);
    spread<LANES>(team_sums<LANES>(b), b);
  }
}
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }
// The variance from the mean square about a rounded mean and what that mean leaves out.
__device__ __forceinline__ float variance(float square, float rest) {
  return square <= 3.4e38f ? fmaxf(fmaf(-rest, rest, square), 0.f) : square;
}
// 1 / sqrt(x): the SFU's, with one step of Newton's method (0 where x has overflowed). x y is the root, a
// normal number where x, and half of it, are not.
__device__ __forceinline__ float rsqrt_of(float x) {
  const float y = rsqrtf(x);
  return x <= 3.4e38f ? y * fmaf(x * y * -0.5f, y, 1.5f) : y;
}

template <int COLS>
constexpr bool kSharedParams = COLS > 16;

template <bool BF16, int LANES, bool MULTI, int COLS, int R, bool RES>
__global__ void __launch_bounds__(MULTI ? 8192 / COLS : COLS > 16 ? 128 : 256, MULTI ? 2 : COLS == 16 ? 3 : 4)
palimpsa_norm_kernel(NormArgs a) {
  using W = Walk<BF16, LANES, MULTI, COLS, R, 1 + RES>;
  constexpr int V = W::V, P = W::P;
  // Whether what a mean's sum leaves out of it is added up from the deviations and put right. (With 8 columns a
  // thread the sum has 8 roundings at most, and that takes 131072 x 64 in fp32 from 7.9 us to 9.9.)
  constexpr bool kCorrected = COLS > 8;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float4 parts[2][16][R];  // of the warps: means, what they leave out, squares about them
  __shared__ float2 shares[16];       // of the warps in a row's values, and one value's in theirs
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
    if (ahead < at.rows) {
      at.fetch(to, 0, px, nx, ahead);
      if (RES) at.fetch(to, 1, pr, nr, ahead);
    }
    cp_async_commit();
    px += R * nx;
    if (RES) pr += R * nr;
    ahead += R * at.stride;
    to = to + 1 == W::S ? 0 : to + 1;
  };
#pragma unroll
  for (int k = 0; k < W::S - 1; ++k) stage();
  constexpr bool kShared = kSharedParams<COLS>;
  float4* const shared = reinterpret_cast<float4*>(smem + W::plane(W::S * W::planes));
  const Param<W, kShared> weight(at, a.weight, 1.f, shared), bias(at, a.bias, 0.f, shared + COLS / 4 * at.team_size);
  if (kShared) __syncthreads();
  // Values of warp w's part of a row.
  auto count = [&](int w) {
    int n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) n += min(max(at.nv - (v * (int)blockDim.x + 32 * w), 0), 32);
    return (float)(n * W::N);
  };
  const float whole = __frcp_rn((float)a.D), own = MULTI ? __frcp_rn(count(warp)) : whole;
  if (MULTI && lane == 0) shares[warp] = make_float2(count(warp) * whole, own);  // (read behind the first batch's barrier)

  int from = 0;
  for (int b = 0; b < at.batches; ++b) {
    cp_async_wait<W::S - 2>();
    float2 s[R][V][P];
    float mean[R], sq[R], rest[R], rstd[R];
    bool live[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      live[j] = row + j * at.stride < at.rows;
      float2 t = two(0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        at.read(from, 0, j, v, s[j][v]);
        if (RES) {
          float2 r[P];
          at.read(from, 1, j, v, r);
#pragma unroll
          for (int c = 0; c < P; ++c) s[j][v][c] = __fadd2_rn(s[j][v][c], r[c]);
          at.write(ps + j * ny, v, s[j][v], live[j] && at.has(v), true);
        }
        // (Each value's part of the mean: the sum may pass fp32's range.)
#pragma unroll
        for (int c = 0; c < P; ++c) t = __ffma2_rn(s[j][v][c], two(own), t);
      }
      mean[j] = t.x + t.y;
    }
    from = from + 1 == W::S ? 0 : from + 1;
    stage();  // into the stage of the batch before
    spread<LANES>(team_sums<LANES>(mean), mean);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float2 t = two(0.f), u = two(0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float2 q = two(0.f);
        const float part = at.has(v) ? own : 0.f;
        if (!kCorrected || v * at.team_size < at.nv) {
#pragma unroll
          for (int c = 0; c < P; ++c) {
            const float2 d = __fadd2_rn(s[j][v][c], two(-mean[j]));
            q = __ffma2_rn(d, d, q);
            if (kCorrected) u = __ffma2_rn(d, two(part), u);
          }
          if (at.has(v)) t = __fadd2_rn(t, q);
        }
      }
      sq[j] = t.x + t.y;
      rest[j] = u.x + u.y;
    }
    if constexpr (MULTI) {
      float both[2 * R];
#pragma unroll
      for (int j = 0; j < R; ++j) both[j] = rest[j], both[R + j] = sq[j];
      const float mine = team_sums<LANES>(both);
      constexpr int per = LANES / (2 * R);
      float* const p = &parts[b & 1][warp][0].x;
      if (lane % per == 0) p[lane / per % R * 4 + 1 + lane / per / R] = mine;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (lane == j) p[j * 4] = mean[j];
      __syncthreads();  // (two sets of parts: the last batch's may still be read)
#pragma unroll
      for (int j = 0; j < R; ++j) {
        // Means relative to the first warp's, m the row's.
        const float first = parts[b & 1][0][j].x;
        float m = 0.f, q = 0.f;
        for (int w = 0; w < warps; ++w) {
          const float4 p = parts[b & 1][w][j];
          m = fmaf((p.x - first) + p.y, shares[w].x, m);
        }
        for (int w = 0; w < warps; ++w) {
          const float4 p = parts[b & 1][w][j];
          const float2 share = shares[w];
          const float d = ((p.x - first) + p.y) - m;
          q = fmaf(fmaf(d, d, variance(p.z * share.y, p.y)), share.x, q);
        }
        mean[j] = first + m;
        rstd[j] = rsqrt_of(q + a.eps);
      }
    } else if constexpr (kCorrected) {
      all_sums<LANES>(sq, rest);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        rstd[j] = rsqrt_of(variance(sq[j] * own, rest[j]) + a.eps);
        mean[j] += rest[j];
      }
    } else {
      spread<LANES>(rsqrt_of(fmaf(team_sums<LANES>(sq), own, a.eps)), rstd);
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (a.stats && live[j] && at.t == 0)
        reinterpret_cast<float2*>(a.stats)[row + j * at.stride] = make_float2(mean[j], rstd[j]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float2 wt[P], add[P];
      weight.get(v, wt);
      bias.get(v, add);
#pragma unroll
      for (int j = 0; j < R; ++j) {
#pragma unroll
        for (int c = 0; c < P; ++c) {
          const float2 t = __fmul2_rn(__fadd2_rn(s[j][v][c], two(-mean[j])), two(rstd[j]));
          s[j][v][c] = __ffma2_rn(t, wt[c], add[c]);
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
template <bool BF16, int LANES, bool MULTI, int COLS, int R, bool DS>
__global__ void __launch_bounds__(MULTI ? 8192 / COLS : COLS > 16 ? 128 : 256, MULTI ? 1 : COLS == 16 ? 2 : 3)
palimpsa_norm_bwd_kernel(NormArgs a, float* sums) {
  using W = Walk<BF16, LANES, MULTI, COLS, R, 2 + DS>;
  constexpr int V = W::V, P = W::P;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float parts[2][16][2 * R];  // of the warps: mean(u), mean(u t), each for every row
  const W at(a.rows, a.D, smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  const long long nx = at.apart(a.x_ld), ny = at.apart(a.dy_ld), ns = at.apart(a.ds_ld), nd = at.apart(a.D);
  const char* px = static_cast<const char*>(a.x) + at.start(a.x_ld);
  const char* py = static_cast<const char*>(a.dy) + at.start(a.dy_ld);
  const char* ps = static_cast<const char*>(a.ds) + at.start(a.ds_ld);
  char* pd = static_cast<char*>(a.dx) + at.start(a.D);
  const float2* stats = reinterpret_cast<const float2*>(a.stats) + at.first;
  long long ahead = at.first, row = at.first;
  int to = 0;
  auto stage = [&]() {
    if (ahead < at.rows) {
      at.fetch(to, 0, px, nx, ahead);
      at.fetch(to, 1, py, ny, ahead);
      if (DS) at.fetch(to, 2, ps, ns, ahead);
    }
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
    for (int j = 0; j < R; ++j) next[j] = r + j * at.stride < at.rows ? stats[j * at.stride] : make_float2(0.f, 0.f);
    stats += R * at.stride;
  };
  load_stats(row);
#pragma unroll
  for (int k = 0; k < W::S - 1; ++k) stage();
  const Param<W, false> weight(at, a.weight, 1.f, nullptr);
  float2 gw[V][P], gb[V][P];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int c = 0; c < P; ++c) gw[v][c] = gb[v][c] = two(0.f);
  const float inv = __frcp_rn((float)a.D);

  int from = 0;
  for (int b = 0; b < at.batches; ++b) {
    // (A team of a warp may have no row left while others have: it goes on, its ring then
    // holding anything.)
    if (MULTI && row >= at.rows) break;
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
      if (live[0])
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float2 x[P], dy[P];
          at.read(from, 0, j, v, x);
          at.read(from, 1, j, v, dy);
          const float scale = at.has(v) ? st[j].y : 0.f;  // (columns past D: a mean may be past fp32's range of it)
#pragma unroll
          for (int c = 0; c < P; ++c) {
            const float2 t = __fmul2_rn(__fadd2_rn(x[c], two(-st[j].x)), two(scale)), u = __fmul2_rn(dy[c], weight.f[v][c]);
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
    const float mine = team_sums<LANES>(tot) * inv;
    if (MULTI) {
      if (lane % per == 0) parts[b & 1][warp][lane / per] = mine;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 2 * R; ++j) tot[j] = parts[b & 1][0][j];
      for (int w = 1; w < warps; ++w)
#pragma unroll
        for (int j = 0; j < 2 * R; ++j) tot[j] += parts[b & 1][w][j];
    } else {
      spread<LANES>(mine, tot);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float2 x[P], dy[P], ds[P];
        at.read(from, 0, j, v, x);
        at.read(from, 1, j, v, dy);
        if (DS) at.read(from, 2, j, v, ds);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          const float2 t = __fmul2_rn(__fadd2_rn(x[c], two(-st[j].x)), two(st[j].y));
          const float2 d = __ffma2_rn(t, two(-tot[2 * j + 1]), __ffma2_rn(dy[c], weight.f[v][c], two(-tot[2 * j])));
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
        for (int c = 0; c < P; c += 2) {
          float* const p = out + at.col(v) + 2 * c;
          *reinterpret_cast<float4*>(p) = make_float4(gw[v][c].x, gw[v][c].y, gw[v][c + 1].x, gw[v][c + 1].y);
          *reinterpret_cast<float4*>(p + a.D) = make_float4(gb[v][c].x, gb[v][c].y, gb[v][c + 1].x, gb[v][c + 1].y);
        }
      }
  } else {
    // The CTA's teams, through the ring's memory (its copies are done: the last groups are empty).
    cp_async_wait<0>();
    float* const red = reinterpret_cast<float*>(smem);
    constexpr int N = W::N, cols = LANES * N;
    const int teams = blockDim.x / LANES, team = threadIdx.x / LANES;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float2 g = q ? gb[v][c / 2] : gw[v][c / 2];
          red[(team * N + c) * LANES + at.t] = c & 1 ? g.y : g.x;
        }
        __syncthreads();
        for (int k = threadIdx.x; k < cols; k += blockDim.x) {
          float s = 0.f;
          for (int m = 0; m < teams; ++m) s += red[m * cols + k];
          const int col = v * cols + k % LANES * N + k / LANES;
          if (col < a.D) out[q * a.D + col] = s;
        }
      }
  }
}

// A launch: as many CTAs as the rows need and the GPU holds.
struct Shape {
  int threads, bytes, ctas;
};
struct Held {
  HeldCtas ctas;
  SharedBytes allowed;
};
template <class K>
cudaError_t shape_of(K kernel, const NormArgs& a, int threads, int teams, int bytes, Held* known, Shape* p) {
  cudaError_t e = allow_shared(kernel, bytes, &known->allowed);
  if (e != cudaSuccess) return e;
  int held;
  if ((e = held_ctas(kernel, threads, bytes, &known->ctas, &held)) != cudaSuccess) return e;
  const long long most = (long long)held * sms_of_device();
  *p = {threads, bytes, (int)std::max<long long>(1, std::min(most, (a.rows + teams - 1) / teams))};
  return cudaSuccess;
}
// Threads of a CTA that a row takes for itself, each with COLS columns.
template <int COLS>
int row_threads(const NormArgs& a) {
  return (a.D + COLS * 32 - 1) / (COLS * 32) * 32;
}

template <bool BF16, int LANES, bool MULTI, int COLS, int R, bool MORE>
cudaError_t forward(const NormArgs& a, cudaStream_t s) {
  using W = Walk<BF16, LANES, MULTI, COLS, R, 1 + MORE>;
  constexpr bool kShared = kSharedParams<COLS>;
  const auto kernel = palimpsa_norm_kernel<BF16, LANES, MULTI, COLS, R, MORE>;
  const int threads = MULTI ? row_threads<COLS>(a) : kShared ? 128 : 256;
  static Held known;
  Shape p;
  const cudaError_t e = shape_of(kernel, a, threads, MULTI ? 1 : threads / LANES,
                                 threads * 16 * W::S * W::planes + (kShared ? 8 * COLS * (MULTI ? threads : LANES) : 0), &known, &p);
  if (e != cudaSuccess) return e;
  kernel<<<p.ctas, p.threads, p.bytes, s>>>(a);
  return cudaGetLastError();
}

template <bool BF16, int LANES, bool MULTI, int COLS, int R, bool MORE>
cudaError_t backward(const NormArgs& a, float* sums, int* ctas, cudaStream_t s) {
  using W = Walk<BF16, LANES, MULTI, COLS, R, 2 + MORE>;
  const auto kernel = palimpsa_norm_bwd_kernel<BF16, LANES, MULTI, COLS, R, MORE>;
  const int threads = MULTI ? row_threads<COLS>(a) : COLS > 16 ? 128 : 256;
  static Held known;
  Shape p;
  const cudaError_t e = shape_of(kernel, a, threads, MULTI ? 1 : threads / LANES, threads * 16 * W::S * W::planes,
                                 &known, &p);
  if (e != cudaSuccess) return e;
  if (ctas) {
    *ctas = p.ctas;
    return cudaSuccess;
  }
  kernel<<<p.ctas, p.threads, p.bytes, s>>>(a, sums);
  return cudaGetLastError();
}

// (Few lanes with many columns each: a lane without columns does the same work, and sums over lanes take
// steps. 136, 264 and 384 columns in bf16 with 8 or 16 lanes of 24: 40, 38 and 37 us for 96 MB; with a warp of
// 8 or 16 each: 56, 57 and 44. 64 columns with 2 lanes of 32: 41, with 8 of 8: 37. In bf16 without a residual
// 520 and 640 columns with a warp of 24: 40 and 35, with 32 each 47 and 41; with one 71 and 70, 69 and 64.)
// (Two rows at a time in a CTA halve its barriers: 4096 columns in bf16 without a residual 47 us -> 43 for
// 96 MB; in fp32, whose rows are twice as long, 38.7 -> 39.9. Above 4096, one row with 64 columns a thread:
// 8192 66 -> 52; with a residual 82 -> 83. Since then 4096 columns have come to 38 and 8192 to 44.)
template <bool BF16, bool MORE>
cudaError_t forward_by_width(const NormArgs& a, cudaStream_t s) {
  if (a.D <= (BF16 ? 16 : 8)) return forward<BF16, 2, false, 8, 2, MORE>(a, s);
  if (a.D <= 32) return forward<BF16, 4, false, 8, 2, MORE>(a, s);
  if (a.D <= 64) return forward<BF16, 8, false, 8, 2, MORE>(a, s);
  if (a.D <= 96) return forward<BF16, 4, false, 24, 2, MORE>(a, s);
  if (a.D <= 128) return forward<BF16, 4, false, 32, 2, MORE>(a, s);
  if (a.D <= 192) return forward<BF16, 8, false, 24, 2, MORE>(a, s);
  if (a.D <= 256) return forward<BF16, 8, false, 32, 2, MORE>(a, s);
  if (a.D <= 384) return forward<BF16, 16, false, 24, 2, MORE>(a, s);
  if (a.D <= 512) return forward<BF16, 16, false, 32, 2, MORE>(a, s);
  if constexpr (BF16 && !MORE)
    if (a.D <= 768) return forward<true, 32, false, 24, 1, false>(a, s);
  if (a.D <= 1024) return forward<BF16, 32, false, 32, 1, MORE>(a, s);
  if (a.D <= 1536) return forward<BF16, 32, false, 48, 1, MORE>(a, s);
  if (a.D <= 2048) return forward<BF16, 32, false, 64, 1, MORE>(a, s);
  if constexpr (BF16 && !MORE)
    if (a.D > 4096) return forward<true, 32, true, 64, 1, false>(a, s);
  return forward<BF16, 32, true, 32, BF16 && !MORE ? 2 : 1, MORE>(a, s);
}
// (As in the forward: 72, 136, 264 columns in bf16 78, 70 and 68 us; with 16 lanes or a warp of 8 or 16 columns
// each 97, 99 and 82.)
// (In bf16 a CTA a row with 16 columns a thread has too little to do between its barriers: 520, 768 and
// 1024 columns 92, 70 and 61 us for 96 MB, with a warp a row 68, 57 and 57; 8192 with 32 columns a
// thread 77 -> 69. From 1032 to 2048 a warp a row, its weight in shared memory, is no faster.)
template <bool BF16, bool MORE>
cudaError_t backward_by_width(const NormArgs& a, float* sums, int* ctas, cudaStream_t s) {
  if (a.D <= (BF16 ? 16 : 8)) return backward<BF16, 2, false, 8, 1, MORE>(a, sums, ctas, s);
  if (a.D <= 32) return backward<BF16, 4, false, 8, BF16 ? 2 : 1, MORE>(a, sums, ctas, s);
  if (a.D <= 64) return backward<BF16, BF16 ? 4 : 8, false, BF16 ? 16 : 8, BF16 ? 2 : 1, MORE>(a, sums, ctas, s);
  if (a.D <= 96) return backward<BF16, 4, false, 24, BF16 ? 2 : 1, MORE>(a, sums, ctas, s);
  if (a.D <= 128) return backward<BF16, 8, false, 16, BF16 ? 2 : 1, MORE>(a, sums, ctas, s);
  if (a.D <= 192) return backward<BF16, 8, false, 24, BF16 ? 2 : 1, MORE>(a, sums, ctas, s);
  if (a.D <= 256) return backward<BF16, 16, false, 16, BF16 ? 2 : 1, MORE>(a, sums, ctas, s);
  if (a.D <= 384) return backward<BF16, 16, false, 24, BF16 ? 2 : 1, MORE>(a, sums, ctas, s);
  if (a.D <= 512) return backward<BF16, 32, false, 16, BF16 ? 2 : 1, MORE>(a, sums, ctas, s);
  if constexpr (BF16) {
    if (a.D <= 768) return backward<true, 32, false, 24, 2, MORE>(a, sums, ctas, s);
    if (a.D <= 1024) return backward<true, 32, false, 32, 2, MORE>(a, sums, ctas, s);
    if (a.D >= 4096) return backward<true, 32, true, 32, 1, MORE>(a, sums, ctas, s);
  }
  return backward<BF16, 32, true, 16, BF16 ? 2 : 1, MORE>(a, sums, ctas, s);
}
cudaError_t backward_any(const NormArgs& a, float* sums, int* ctas, cudaStream_t s) {
  if (a.bf16) return a.ds ? backward_by_width<true, true>(a, sums, ctas, s) : backward_by_width<true, false>(a, sums, ctas, s);
  return a.ds ? backward_by_width<false, true>(a, sums, ctas, s) : backward_by_width<false, false>(a, sums, ctas, s);
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  if (a.bf16) return a.residual ? forward_by_width<true, true>(a, s) : forward_by_width<true, false>(a, s);
  return a.residual ? forward_by_width<false, true>(a, s) : forward_by_width<false, false>(a, s);
}

cudaError_t plan_norm_backward(NormArgs* a, size_t* floats) {
  *floats = 0;
  a->ctas = 0;
  if (a->rows == 0) return cudaSuccess;
  const cudaError_t e = backward_any(*a, nullptr, &a->ctas, nullptr);
  if (a->dweight || a->dbias) *floats = (size_t)a->ctas * 2 * a->D;
  return e;
}

cudaError_t launch_norm_backward(const NormArgs& a, float* scratch, cudaStream_t s) {
  if (a.rows > 0) {
    const cudaError_t e = backward_any(a, scratch, nullptr, s);
    if (e != cudaSuccess) return e;
  }
  if (!a.dweight && !a.dbias) return cudaSuccess;
  float* const out[2] = {a.dweight, a.dbias};
  return launch_row_sums(scratch, a.ctas, 2, a.D, out, s);
}

}  // namespace palimpsa
