// Gated scan, forward and one token. Per channel d:
//   s_t = sigmoid(r_t + r_bias),  w_t = A s_t,  a_t = exp(-w_t),        A = A[d] > 0
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t + i_bias) x_t        (without i: its gate is 1)
//   y_t = h_t silu(z_t)                                                  (without z: h_t)
// The input's factor keeps the state's variance at the input's, whatever the decay.
//
// What bounds it: HBM. A channel-token moves 8 bytes in bf16 (10 with z), 0.37 clocks
// (0.47) of an SM's share of the measured 6.77 TB/s, against 3 2^x, a reciprocal and a
// reciprocal root on the SFU (0.22 clocks; a 2^x and a reciprocal more with z) and about 30 FP32
// operations. So every input is read once: a thread takes 8 tokens of 4 channels (a piece),
// forms their decays and inputs a, b in registers and runs them from 0, keeping for each token
// the product P of the a's and the state H so far; with the state h before the piece known, the
// states are P h + H. The last P and H and the sum of the rates are the piece's summary. (4 tokens and twice the threads
// took 1.3 times as long: what a round costs a thread besides its tokens is a fifth of it.) The
// summaries of a CTA's pieces (groups of 16 or 8 threads, along time) pass through shared
// memory, every thread folds the ones before its own, and the last group works out the state
// behind the tile, which goes to the next round by shared memory too. A CTA walks its sequence in rounds of
// such tiles, the next round's inputs coming by asynchronous copies meanwhile. Where the CTAs are
// too few, those of a cluster take turns along time: each gets the state before its tile from
// the one before it and hands on the state after it, as an asynchronous store into the next
// one's shared memory that a barrier there counts. (A ring: with all summaries sent to all, the
// CTAs of a cluster went in step, and 8 x 4096 x 1536 took 83 us, where the ring took 78.)
// Measured (GB300, bf16): 78 us at 8 x 4096 x 1536 without z (5.2 TB/s, 59 at the rate of a
// copy), 166 at 1 x 32768 x 2048 with z (4.0 TB/s, 99), 230 at 256 x 256 x 2048 (5.8 TB/s), where
// CTAs are many; in fp32 157 at 8 x 4096 x 1536 with z, 0.95 of a copy's rate. The warp schedulers issue in 50 to
// 60 % of their cycles, with the 16 warps an SM that 128 registers and two stages of inputs allow.
//
// Rounding: gates, decays and states are fp32; y is rounded to the input type once.
#include <algorithm>
#include <cmath>

#include "gate.cuh"

namespace palimpsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kResident = 4;  // CTAs of an SM

// Tiles of 64 channels, or 32 where those are too few; in fp32 half the threads, since rows are
// twice as long.
template <bool BF16, int CH>
using Tile = GateTile<BF16, CH, 4, BF16 ? 128 : 64>;

// Shared memory: two stages of x, r and i, then two states of the tile's channels before it. A
// piece's summary takes the place of its first rows of x. Where rows are 64 bytes, those of odd
// pieces change places in pairs, so that the two that a half warp reads at once lie in different
// banks.
template <bool BF16, bool IN>
constexpr int kStageBytes = (2 + IN) * Tile<BF16, 64>::bytes;  // the same for 32

// h <- P h + H over 4 channels.
struct Four {
  float2 v[2];
  __device__ __forceinline__ void fold(const float4& P, const float4& H) {
    v[0] = ffma2(make_float2(P.x, P.y), v[0], make_float2(H.x, H.y));
    v[1] = ffma2(make_float2(P.z, P.w), v[1], make_float2(H.z, H.w));
  }
  __device__ __forceinline__ void add(const float4& f) {
    v[0] = __fadd2_rn(v[0], make_float2(f.x, f.y));
    v[1] = __fadd2_rn(v[1], make_float2(f.z, f.w));
  }
  // v + P h + L h
  __device__ __forceinline__ void fold_after(const Four& P, const Four& L, const Four& h) {
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = ffma2(P.v[j], h.v[j], with_left(L.v[j], h.v[j], v[j]));
  }
  __device__ __forceinline__ float4 all() const { return make_float4(v[0].x, v[0].y, v[1].x, v[1].y); }
};
__device__ __forceinline__ Four four(const float4& f) { return {make_float2(f.x, f.y), make_float2(f.z, f.w)}; }
__device__ __forceinline__ Four four(float v) { return {make_float2(v, v), make_float2(v, v)}; }

template <bool BF16, bool IN, bool GATE, bool CLUSTER, int CH>
__global__ void __launch_bounds__(BF16 ? 128 : 64, kResident) palimpsa_gate_kernel(GateArgs a, int tiles) {
  using G = Tile<BF16, CH>;
  using Q = Quad<BF16>;
  using Raw = typename Q::Raw;
  constexpr int ES = G::ES, RT = G::tokens, NP = G::pieces, LG = G::group, kStage = kStageBytes<BF16, IN>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t bars[2];
  __shared__ int told, held[G::group + 1];  // see settle; the rounds whose wait has held, for the last group's threads and the first
  const int tid = threadIdx.x, piece = tid / LG, lane = tid % LG;
  const int cs = CLUSTER ? a.cluster : 1;
  const int rank = CLUSTER ? (int)(blockIdx.x % cs) : 0;
  const long long rest = CLUSTER ? blockIdx.x / cs : blockIdx.x;
  const int ch0 = (int)(rest % tiles) * CH, ch = ch0 + 4 * lane;
  const bool in = ch < a.D;
  const long long n = rest / tiles;
  long long row0;
  int len;
  if (!seq_rows(a.rows, n, &row0, &len)) {
    if (tid == 0) latch_status(a.status, kStatusDomain);
    return;  // (the whole cluster)
  }
  const int step = cs * RT, rounds = (len + step - 1) / step;

  // Copies of a round's x, r and i, as one group: a thread takes the same vector of rows
  // rows_at_once apart. Rows past the end and channels past D are left as they are.
  const int vec = tid % G::vecs, vrow = tid / G::vecs;
  constexpr bool kFlip = G::row == 64;
  static_assert(!kFlip || G::rows_at_once % (2 * kPiece) == 0, "a thread's rows are all of odd or all of even pieces");
  const int flip = kFlip ? (vrow / kPiece) & 1 : 0, slot0 = ((vrow ^ flip) * G::vecs + vec) * 16;
  const bool vin = ch0 * ES + vec * 16 < a.D * ES;
  auto stage = [&](int k) {
    const int t0 = k * step + rank * RT, nt = min(RT, len - t0);
    if (k < rounds && vin) {
      unsigned char* const to = smem + (k & 1) * kStage + slot0;
      const long long first = row0 + t0 + vrow, col = (long long)ch0 * ES + vec * 16;
      auto copy = [&](const void* from, long long ld, int slot) {
        const char* p = static_cast<const char*>(from) + first * ld * ES + col;
        const long long next = G::rows_at_once * ld * ES;
        if (nt == RT) {
#pragma unroll
          for (int j = 0; j < RT / G::rows_at_once; ++j, p += next)
            cp_async16(to + slot * G::bytes + j * G::threads * 16, p);
        } else {
#pragma unroll
          for (int j = 0; j < RT / G::rows_at_once; ++j, p += next)
            if (j * G::rows_at_once + vrow < nt) cp_async16(to + slot * G::bytes + j * G::threads * 16, p);
        }
      };
      copy(a.x, a.x_ld, 0);
      copy(a.r, a.r_ld, 1);
      if (IN) copy(a.i, a.i_ld, 2);
    }
    cp_async_commit();
  };
  stage(0);
  if (IN && !vin)  // gates behind D that are open: with chance ones 8 x 4096 x 520 took 56 us, now 47
    for (int k = 0; k < 2 * RT / G::rows_at_once; ++k)
      *reinterpret_cast<uint4*>(smem + (k & 1) * kStage + 2 * G::bytes + slot0 + (k >> 1) * G::threads * 16) = make_uint4(0, 0, 0, 0);

  if (CLUSTER && tid == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    fence_mbar_init();
  }
  if (CLUSTER && piece == NP - 1) held[lane] = rounds;
  if (CLUSTER && tid == 0) held[LG] = rounds;
  // Parameters, the gates' biases as their exponents' addends.
  float2 A[2], rb[2], ib[2];
  // The states before this CTA's rounds, two places in turn.
  float4* const states = reinterpret_cast<float4*>(smem + 2 * kStage) + lane;
  if (rank == 0 && piece == 0)
    states[0] = a.h0 && in ? *reinterpret_cast<const float4*>(a.h0 + n * a.D + ch) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    A[j] = pair_or(a.A, ch + 2 * j, in, 1.f);
    if (!pos_finite(A[j].x) || !pos_finite(A[j].y)) latch_status(a.status, kStatusDomain);
    rb[j] = __fmul2_rn(pair_or(a.r_bias, ch + 2 * j, in, 0.f), make_float2(-kLog2e, -kLog2e));
    if (IN) ib[j] = __fmul2_rn(pair_or(a.i_bias, ch + 2 * j, in, 0.f), make_float2(-kLog2e, -kLog2e));
  }
  bool waits = true;
  constexpr unsigned kLast = ~0u << (32 - LG);  // the last group's lanes
  if (CLUSTER) cg::this_cluster().sync();  // every CTA has started, its barriers set: it may be written to
  if (CLUSTER && a.late && rank == 0) pass_the_limit(a);

  const long long yd = (long long)a.D * ES;
  for (int k = 0; k < rounds; ++k) {
    const int tp = k * step + rank * RT + piece * kPiece;  // the piece's first token
    const int np = min(kPiece, len - tp);                  // its tokens (0 or less: none)
    unsigned char* const tile = smem + (k & 1) * kStage;
    const unsigned char* const raw = tile + piece * kPiece * G::row + lane * 4 * ES;
    const int odd = kFlip ? piece & 1 : 0;
    // A piece's summary: products and states of the lane's channels.
    auto sums_of = [&](int p) { return reinterpret_cast<float4*>(tile + p * kPiece * G::row) + lane; };
    cp_async_wait<0>();
    if (CLUSTER && tid == 0 && waits) mbar_arrive_expect_tx(&bars[k & 1], k + rank > 0 ? LG * 16 : 0);
    __syncthreads();  // the round's inputs are here; the other stage and the summaries are free
    stage(k + 1);

    float2 da[kPiece][2], b[kPiece][2];
    Four W = four(0.f);  // the rates' sum
    auto token = [&](int t, bool open) {
      float2 x[2], r[2], i[2];
      Q::unpack(*reinterpret_cast<const Raw*>(raw + (t ^ odd) * G::row), x);
      Q::unpack(*reinterpret_cast<const Raw*>(raw + G::bytes + (t ^ odd) * G::row), r);
      if (IN) Q::unpack(*reinterpret_cast<const Raw*>(raw + 2 * G::bytes + (t ^ odd) * G::row), i);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 s = sigmoid_of(ffma2(r[j], make_float2(-kLog2e, -kLog2e), rb[j]));
        float2 sq;
        const float2 w = __fmul2_rn(A[j], s);
        W.v[j] = __fadd2_rn(W.v[j], w);
        decay_of(w, &da[t][j], &sq);
        const float2 u = IN ? ffma2(i[j], make_float2(-kLog2e, -kLog2e), ib[j]) : make_float2(0.f, 0.f);
        b[t][j] = !IN ? input_of(sq, x[j]) : open ? open_input_of(sq, one_plus(u), x[j]) : input_of(sq, sigmoid_of(u), x[j]);
      }
    };
    // Whole pieces whose input gates are open far enough; others token by token.
    bool open = true;
    if (IN && np == kPiece) {
      float2 low[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int t = 0; t < kPiece; ++t) {
        float2 i[2];
        Q::unpack(*reinterpret_cast<const Raw*>(raw + 2 * G::bytes + (t ^ odd) * G::row), i);
#pragma unroll
        for (int j = 0; j < 2; ++j) low[j] = make_float2(fminf(low[j].x, i[j].x), fminf(low[j].y, i[j].y));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 u = ffma2(low[j], make_float2(-kLog2e, -kLog2e), ib[j]);
        open = open && u.x <= -kLog2e * kOpenGate && u.y <= -kLog2e * kOpenGate;
      }
    }
    if (np == kPiece && open) {
#pragma unroll
      for (int t = 0; t < kPiece; ++t) token(t, true);
    } else {
#pragma unroll
      for (int t = 0; t < kPiece; ++t) {
        da[t][0] = da[t][1] = make_float2(1.f, 1.f);
        b[t][0] = b[t][1] = make_float2(0.f, 0.f);
        if (t < np) token(t, false);
      }
    }
    Four P = four(1.f), H = four(0.f);
#pragma unroll
    for (int t = 0; t < kPiece; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // (In their places: the state after the token is then P h + H, with h the one before the piece.)
        b[t][j] = H.v[j] = ffma2(da[t][j], H.v[j], b[t][j]);
        da[t][j] = P.v[j] = __fmul2_rn(P.v[j], da[t][j]);
      }
    __syncwarp();  // the piece's rows of x are read
    sums_of(piece)[0] = P.all();
    sums_of(piece)[LG] = H.all();
    sums_of(piece)[2 * LG] = W.all();
    Raw z[kPiece];  // on their way during the exchange
    if (GATE && in) {
      const char* p = static_cast<const char*>(a.z) + ((row0 + tp) * a.z_ld + ch) * ES;
#pragma unroll
      for (int t = 0; t < kPiece; ++t, p += a.z_ld * ES)
        if (t < np) z[t] = *reinterpret_cast<const Raw*>(p);
    }
    __syncthreads();

    // The last group works out the CTA's summary, and hands on the state behind the tile: the decay from the
    // rates' sum, so that no state gathers the roundings of products. (Two places for it. A cluster's are each
    // written again only after this CTA's next state has gone round.)
    const bool last = piece == NP - 1;
    Four Hc = four(0.f), Pc, Lc;
    if (last) {
      Four Wc = four(0.f);
#pragma unroll 4  // (in full it wants more registers than there are: 1 x 32768 x 2048 takes 177 us, 166 so)
      for (int w = 0; w < NP; ++w) {
        Hc.fold(sums_of(w)[0], sums_of(w)[LG]);
        Wc.add(sums_of(w)[2 * LG]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float2 rest;
        decay_of(Wc.v[j], &Pc.v[j], &rest, &Lc.v[j]);
      }
    }
    if (CLUSTER && waits && !cluster_wait(&bars[k & 1], (k >> 1) & 1, a.wait_timeout_ns)) {
      waits = false;
      if (tid == 0) held[LG] = k;
      if (last) held[lane] = k;
      latch_status(a.status, kStatusTimeout);
    }
    Four h = four(states[(k & 1) * LG]);
    if (last) {
      Hc.fold_after(Pc, Lc, h);
      const int next = rank + 1 == cs ? k + 1 : k;  // its round
      if (next >= rounds) {
        if (in) *reinterpret_cast<float4*>(a.h_T + n * a.D + ch) = Hc.all();
      } else if (!CLUSTER) {
        states[(next & 1) * LG] = Hc.all();
      } else {
        const int to = rank + 1 == cs ? 0 : rank + 1;
        // (Where a wait has run out, nothing more is handed on: the others' waits run out too.)
        if (waits && !(a.withhold && k + rank == 0))
          st_async(cluster_addr(states + (next & 1) * LG, to), Hc.all(), cluster_addr(&bars[next & 1], to));
      }
    }
    for (int w = 0; w < piece; ++w) h.fold(sums_of(w)[0], sums_of(w)[LG]);
    if (in && np > 0) {
      if (a.ckpt)
        *reinterpret_cast<float4*>(a.ckpt + (gate_ckpt_row0(a.rows, n, row0) + tp / kPiece) * a.D + ch) = h.all();
      char* py = static_cast<char*>(a.y) + (row0 + tp) * yd + ch * ES;
      auto out = [&](int t) {
        float2 y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) y[j] = ffma2(da[t][j], h.v[j], b[t][j]);
        if (GATE) {
          float2 f[2];
          Q::unpack(z[t], f);
#pragma unroll
          for (int j = 0; j < 2; ++j) y[j] = __fmul2_rn(y[j], silu_fast(f[j]));
        }
        *reinterpret_cast<Raw*>(py) = Q::pack(y);
        py += yd;
      };
      if (np == kPiece) {
#pragma unroll
        for (int t = 0; t < kPiece; ++t) out(t);
      } else {
#pragma unroll
        for (int t = 0; t < kPiece; ++t)
          if (t < np) out(t);
      }
    }
    __syncwarp();
  }
  if (rounds == 0 && rank == 0 && piece == 0 && in) *reinterpret_cast<float4*>(a.h_T + n * a.D + ch) = states[0];
  __syncwarp();
  if (CLUSTER) {
    // Nobody hands anything to a CTA that has left.
    if (piece == NP - 1) {
      const int to = rank + 1 == cs ? 0 : rank + 1, on = rank + 1 == cs;
      const int mine = a.withhold && rank == 0 ? 0 : held[lane], sent = __reduce_max_sync(kLast, mine);
      for (int k = mine + on; k < min(sent + on, rounds); ++k)
        st_async(cluster_addr(states + (k & 1) * LG, to), make_float4(0.f, 0.f, 0.f, 0.f), cluster_addr(&bars[k & 1], to));
      if (lane == 0) *cg::this_cluster().map_shared_rank(&told, to) = min(sent + on, rounds);
    }
    cg::this_cluster().sync();
    if (tid == 0) settle(bars, held[LG], told, LG * 16);
  }
}

// Short sequences, many of them: a thread takes 4 channels of a sequence and walks its tokens, with
// nothing to exchange (in the kernel above a sequence of 8 tokens leaves seven of eight groups of
// threads idle). kBatch tokens' loads go out together.
constexpr int kBatch = 4;
template <bool BF16, bool IN, bool GATE>
__global__ void __launch_bounds__(128, BF16 ? 5 : 4) palimpsa_gate_short_kernel(GateArgs a) {
  using Q = Quad<BF16>;
  using Raw = typename Q::Raw;
  constexpr int ES = Vec<BF16>::bytes;
  const int quads = a.D / 4;
  const long long k = (long long)blockIdx.x * 128 + threadIdx.x;
  if (k >= quads * (long long)a.rows.n_seq) return;
  const long long n = k / quads;
  const int ch = (int)(k % quads) * 4;
  long long row0;
  int len;
  if (!seq_rows(a.rows, n, &row0, &len)) {
    if (ch == 0) latch_status(a.status, kStatusDomain);
    return;
  }
  const float2 scale = make_float2(-kLog2e, -kLog2e);
  float2 A[2], rb[2], ib[2];
  Four h = four(0.f);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    A[j] = pair_or(a.A, ch + 2 * j, true, 1.f);
    if (!pos_finite(A[j].x) || !pos_finite(A[j].y)) latch_status(a.status, kStatusDomain);
    rb[j] = __fmul2_rn(pair_or(a.r_bias, ch + 2 * j, true, 0.f), scale);
    if (IN) ib[j] = __fmul2_rn(pair_or(a.i_bias, ch + 2 * j, true, 0.f), scale);
  }
  if (a.h0) h = four(*reinterpret_cast<const float4*>(a.h0 + n * a.D + ch));
  float* ckpt = a.ckpt ? a.ckpt + gate_ckpt_row0(a.rows, n, row0) * a.D + ch : nullptr;
  auto at = [&](const void* p, long long ld) { return static_cast<const char*>(p) + (row0 * ld + ch) * ES; };
  const char *px = at(a.x, a.x_ld), *pr = at(a.r, a.r_ld), *pi = at(a.i, a.i_ld), *pz = at(a.z, a.z_ld);
  char* py = static_cast<char*>(a.y) + (row0 * a.D + ch) * ES;
  for (int t0 = 0; t0 < len; t0 += kBatch) {
    Raw x[kBatch], r[kBatch], i[kBatch], z[kBatch];
#pragma unroll
    for (int t = 0; t < kBatch; ++t)
      if (t0 + t < len) {
        x[t] = *reinterpret_cast<const Raw*>(px + t * a.x_ld * ES);
        r[t] = *reinterpret_cast<const Raw*>(pr + t * a.r_ld * ES);
        if (IN) i[t] = *reinterpret_cast<const Raw*>(pi + t * a.i_ld * ES);
        if (GATE) z[t] = *reinterpret_cast<const Raw*>(pz + t * a.z_ld * ES);
      }
    if (ckpt && t0 % kPiece == 0) {
      *reinterpret_cast<float4*>(ckpt) = h.all();
      ckpt += a.D;
    }
#pragma unroll
    for (int t = 0; t < kBatch; ++t)
      if (t0 + t < len) {
        float2 fx[2], fr[2], fi[2], fz[2], y[2];
        Q::unpack(x[t], fx);
        Q::unpack(r[t], fr);
        if (IN) Q::unpack(i[t], fi);
        if (GATE) Q::unpack(z[t], fz);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float2 da, sq, left;
          decay_of(__fmul2_rn(A[j], sigmoid_of(ffma2(fr[j], scale, rb[j]))), &da, &sq, &left);
          const float2 b = IN ? input_of(sq, sigmoid_of(ffma2(fi[j], scale, ib[j])), fx[j]) : input_of(sq, fx[j]);
          h.v[j] = ffma2(da, h.v[j], with_left(left, h.v[j], b));
          y[j] = GATE ? __fmul2_rn(h.v[j], silu_fast(fz[j])) : h.v[j];
        }
        *reinterpret_cast<Raw*>(py + (long long)t * a.D * ES) = Q::pack(y);
      }
    px += kBatch * a.x_ld * ES;
    pr += kBatch * a.r_ld * ES;
    pi += kBatch * a.i_ld * ES;
    pz += kBatch * a.z_ld * ES;
    py += (long long)kBatch * a.D * ES;
  }
  *reinterpret_cast<float4*>(a.h_T + n * a.D + ch) = h.all();
}

// One token: a thread takes 4 channels of a sequence. A few bytes each way: latency alone.
template <bool BF16, bool IN, bool GATE>
__global__ void __launch_bounds__(128) palimpsa_gate_step_kernel(GateArgs a) {
  using Q = Quad<BF16>;
  constexpr int ES = Vec<BF16>::bytes;
  const int quads = a.D / 4;
  const long long k = (long long)blockIdx.x * 128 + threadIdx.x;
  if (k >= quads * (long long)a.rows.n_seq) return;
  const long long n = k / quads;
  const int ch = (int)(k % quads) * 4;
  auto load = [&](const void* p, long long ld, float2* f) {
    Q::unpack(*reinterpret_cast<const typename Q::Raw*>(static_cast<const char*>(p) + (n * ld + ch) * ES), f);
  };
  float2 x[2], r[2], i[2], z[2], y[2];
  float4* const state = reinterpret_cast<float4*>(a.h_T + n * a.D + ch);
  const float4 h4 = *state;
  load(a.x, a.x_ld, x);
  load(a.r, a.r_ld, r);
  if (IN) load(a.i, a.i_ld, i);
  if (GATE) load(a.z, a.z_ld, z);
  float2 h[2] = {make_float2(h4.x, h4.y), make_float2(h4.z, h4.w)};
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float2 A = pair_or(a.A, ch + 2 * j, true, 1.f);
    bad |= !pos_finite(A.x) || !pos_finite(A.y);
    const float2 scale = make_float2(-kLog2e, -kLog2e);
    const float2 s = sigmoid_of(__fmul2_rn(__fadd2_rn(r[j], pair_or(a.r_bias, ch + 2 * j, true, 0.f)), scale));
    float2 da, sq, left;
    decay_of(__fmul2_rn(A, s), &da, &sq, &left);
    const float2 b =
        IN ? input_of(sq, sigmoid_of(__fmul2_rn(__fadd2_rn(i[j], pair_or(a.i_bias, ch + 2 * j, true, 0.f)), scale)), x[j])
           : input_of(sq, x[j]);
    h[j] = ffma2(da, h[j], with_left(left, h[j], b));
    y[j] = GATE ? __fmul2_rn(h[j], silu_fast(z[j])) : h[j];
  }
  *state = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
  *reinterpret_cast<typename Q::Raw*>(static_cast<char*>(a.y) + (n * a.D + ch) * ES) = Q::pack(y);
  if (bad) latch_status(a.status, kStatusDomain);
}

template <bool BF16, bool IN, bool GATE, bool CLUSTER, int CH>
cudaError_t run(const GateArgs& a, cudaStream_t s) {
  using G = Tile<BF16, CH>;
  const long long tiles = (a.D + CH - 1) / CH, blocks = tiles * a.rows.n_seq * a.cluster;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  constexpr int bytes = 2 * kStageBytes<BF16, IN> + 2 * G::group * 16;
  const auto kernel = palimpsa_gate_kernel<BF16, IN, GATE, CLUSTER, CH>;
  static SharedBytes allowed;
  const cudaError_t e = allow_shared(kernel, bytes, &allowed, CLUSTER);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute cluster = {};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = a.cluster;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)blocks);
  c.blockDim = dim3(G::threads);
  c.dynamicSmemBytes = bytes;
  c.stream = s;
  c.attrs = &cluster;
  c.numAttrs = CLUSTER ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, a, (int)tiles);
}

template <bool BF16, bool IN, bool GATE>
cudaError_t forward(const GateArgs& given, cudaStream_t s) {
  GateArgs a = given;
  const GatePlan p = gate_plan(a.rows, a.D, Tile<BF16, 64>::tokens, kResident, 32, {1.8, 0.55, 0.5, 0.06});
  if (gate_short(a.rows, a.D, p, BF16 ? 430e3 : 330e3)) {
    const long long blocks = ((long long)(a.D / 4) * a.rows.n_seq + 127) / 128;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    palimpsa_gate_short_kernel<BF16, IN, GATE><<<(unsigned)blocks, 128, 0, s>>>(a);
    return cudaGetLastError();
  }
  a.cluster = p.cluster;
  if (p.channels == 32)
    return a.cluster > 1 ? run<BF16, IN, GATE, true, 32>(a, s) : run<BF16, IN, GATE, false, 32>(a, s);
  return a.cluster > 1 ? run<BF16, IN, GATE, true, 64>(a, s) : run<BF16, IN, GATE, false, 64>(a, s);
}

template <bool BF16, bool IN, bool GATE>
cudaError_t step(const GateArgs& a, cudaStream_t s) {
  const long long blocks = ((long long)(a.D / 4) * a.rows.n_seq + 127) / 128;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  palimpsa_gate_step_kernel<BF16, IN, GATE><<<(unsigned)blocks, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

// The cheapest of 1 to 12 CTAs a cluster and of 64 or 32 channels a tile, by a model of the time (its
// constants fitted to 44 sweeps of both passes, from 2 x 3000 x 520 to 8 x 4096 x 2048; what it takes
// is within 2 % of the best on average, and within 12). A round of a CTA with c CTAs on its SM takes
// c `cta` us and a `round` besides, and a CTA `ends` rounds besides its own. Clusters leave some SMs
// short of CTAs (larger than 12, a quarter of them; powers of two fewer). Where there is one wave, the SMs with the most
// CTAs set its pace, half the way from the mean; in the last of several less so. Handing the state
// on takes `hop` a tile. A tile of 32 channels has twice the pieces to fold: 12 % more. A packed
// batch's CTAs have the mean of the rounds (and half of one lost) and fill the slots as they come free;
// what the longest sequence has beyond the mean comes behind that, by 0.9 of it (6 ragged batches:
// within 3 % of the best on average, and within 11).
// Measured for the fit, 8 x 4096 x 1536 with clusters of 1, 2, 3, 4 and 8: 111, 90, 78 (taken: 576 CTAs
// where 584 fit), 90 and 87 us; 8 x 4096 x 2048 166, 139, 147, 127 (taken) and 134; 1 x 32768 x 512 in tiles of
// 32 channels with 6, 8, 12 and 16: 110, 103, 81 (taken) and 80, backward 240, 171, 136 and 149. For one
// sequence of 32768 tokens and 1024 or 2048 channels the forward was faster with 16 than with the 12 or 8 that are taken, 94
// us against 99 (fp32 115 against 128) and 154 against 165, the backward slower: 260 against 189, 406 against 297.
GatePlan gate_plan(const SeqRows& r, int D, int tokens, int resident, int narrow, const GateCost& c) {
  const int sms = sms_of_device();
  GatePlan best = {64, 1, 0};
  for (int ch = 64; ch >= narrow; ch /= 2) {
    const double tiles = (D + ch - 1) / ch;
    for (int cs = 1; cs <= kGateCluster; ++cs) {
      const long long per = (long long)cs * tokens * (64 / ch);
      const double longest = (double)((r.max_len + per - 1) / per);
      const double rounds = r.cu ? std::min(longest, (double)r.T / per / r.n_seq + 0.5) : longest;
      const double slots = (cs == 1 ? 1 : cs > 8 ? 0.84 : cs & (cs - 1) ? 0.95 : 0.96) * resident * sms;
      const double ctas = tiles * r.n_seq * cs, waves = std::floor(ctas / slots), rest = ctas - waves * slots;
      const double mean = rest / sms, load = mean + (waves > 0 ? 0.4 : 0.5) * (std::ceil(mean) - mean);
      const double full = c.round + c.cta * resident, some = rest > 0 ? c.round + c.cta * load : 0;
      const double one = waves > 0 ? full : some;
      double us = (rounds + c.ends) * (waves * full + some);
      if (r.cu) us = (rounds + c.ends) * (waves > 0 ? ctas / slots * full : some) + 0.9 * (longest - rounds) * one;
      if (cs > 1) us += longest * cs * c.hop;
      if (ch < 64) us *= 1.12;
      if ((ch == 64 && cs == 1) || us < best.us) best = {ch, cs, us};
    }
  }
  return best;
}

// A token takes a thread 0.35 to 0.45 us at least, and the GPU's threads together come to `rate`. Measured for the fit
// in bf16 with both gates, threads against tiles: 256 x 4 x 2048 8.5 us and 41, 256 x 16 20.7 and 45,
// 256 x 64 76 and 72 (threads are taken), 256 x 256 274 and 226; backward, warps against tiles, 19 and
// 84, 45 and 107, 150 and 154, 575 and 497. In fp32 512 x 32 x 2048 105 and 124, 256 x 256 389 and 391;
// backward 217 and 236, 829 and 785. Where the sequences differ, the threads of the longest end last: 300
// of 1 to 581 tokens, 218 on average, x 1536, backward 774 and 428.
bool gate_short(const SeqRows& r, int D, const GatePlan& p, double rate) {
  const double rows = r.cu ? r.T : (double)r.n_seq * r.T, uneven = r.max_len - rows / r.n_seq;
  return std::max(rows * D / rate, 0.45 * r.max_len) + 0.35 * std::max(uneven, 0.0) < p.us;
}

cudaError_t launch_gate_forward(const GateArgs& a, cudaStream_t s) { PALIMPSA_GATE_DISPATCH(forward, a, s) }
cudaError_t launch_gate_step(const GateArgs& a, cudaStream_t s) { PALIMPSA_GATE_DISPATCH(step, a, s) }

}  // namespace palimpsa
