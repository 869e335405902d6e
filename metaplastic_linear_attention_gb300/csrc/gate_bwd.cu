// Gated scan, backward. With g_t the gradient with respect to h_t and u_t = p_t x_t, p the
// input gate, n_t = sqrt(1 - a_t^2) (formulas of the forward in gate_fwd.cu):
//   g_t = dy_t silu(z_t) + a_{t+1} g_{t+1}        (dh_T comes in behind the last token)
//   dx = g n p,  di = g n x p (1 - p),  dz = dy h silu'(z),  dh0 = a_0 g_0
//   dw = g (u a^2 / n - a h_{t-1}),  dr = dw A s (1 - s),  dA = sum_t dw s
// and the biases' gradients are the sums of dr and di over the tokens.
//
// As in the forward, one pass over the data: HBM bounds it, 18 bytes a channel-token in
// bf16 with both gates (0.84 clocks of an SM's share) and half a byte of checkpoints. The
// forward leaves the state before every 8th token, so a thread recomputes the states of its
// piece by itself (8 tokens of 2 channels), with the factors of g_t in dx, di, dr and dA; a first
// run over the piece from the back, from a gradient of 0, gives its summary, and with the
// gradient behind the piece known, a second run gives the results. (Kept products and sums instead
// of the second run, as in the forward: 1 % slower.) The rounds go from the back to the front, and
// in a cluster the gradient goes round the other way.
// The parameters' sums wait in shared memory from round to round, each thread's in its own place; they
// are added up over the CTA's pieces and over CTAs by a second kernel, in a fixed order: no atomics, the
// same bits every time. (In registers they spilled: 8 x 4096 x 2048 267 us, now 249.)
// Measured (GB300, bf16, both gates): 191 us at 8 x 4096 x 1536 (138 for its bytes at the rate of a
// copy), 41 at 4 x 2048 x 1024 with the sums (23); fp32 292 at 8 x 4096 x 1536, 0.95 of that rate. What a token keeps
// (the decay, four factors, its part of g_t) takes 96 of the 128 registers that 16 warps an SM allow.
#include <algorithm>

#include "gate.cuh"

namespace palimpsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kResident = 2;  // CTAs of an SM

// Warps a CTA: in fp32 half as many, whose rows are twice as long.
template <bool BF16>
using Tile = GateTile<BF16, 64, 2, BF16 ? 256 : 128>;

// Shared memory: the ring of raw inputs (and the states before the pieces), then the pieces'
// summaries and two gradients that the CTA behind hands over.
template <bool BF16, bool IN, bool GATE>
struct BwdSmem {
  static constexpr int h = (3 + IN + GATE) * Tile<BF16>::bytes, stage = h + Tile<BF16>::pieces * Tile<BF16>::CH * 4;
  static constexpr int agg = 2 * stage, rates = agg + Tile<BF16>::pieces * 512,
                       given = rates + Tile<BF16>::pieces * 256, own = given + 512,
                       bytes = own + Tile<BF16>::threads * 8 * (2 + IN);
};

// A thread's piece: 8 tokens of two neighbouring channels.
template <bool BF16, bool IN, bool GATE>
struct Piece {
  // The decays, the factors of g_t in dx, di, dr and dA, and dy silu(z).
  float2 da[kPiece], fx[kPiece], fi[IN ? kPiece : 1], fr[kPiece], fA[kPiece], gy[kPiece];
  float2 W = make_float2(0.f, 0.f);  // the rates' sum

  __device__ __forceinline__ void no_token(int t) {
    da[t] = make_float2(1.f, 1.f);
    fx[t] = fr[t] = fA[t] = gy[t] = make_float2(0.f, 0.f);
    if (IN) fi[t] = make_float2(0.f, 0.f);
  }
  // Takes in token t, with the state before it in h, which moves on; returns dz. (rb, ib: the biases
  // times -log2(e).)
  __device__ __forceinline__ float2 token(int t, float2 x, float2 r, float2 dy, float2 i, float2 z, float2 A, float2 rb,
                                          float2 ib, float2* h) {
    const float2 scale = make_float2(-kLog2e, -kLog2e);
    float2 closed;  // 1 - s
    const float2 s = sigmoid_of(ffma2(r, scale, rb), &closed);
    gy[t] = dy;
    const float2 w = __fmul2_rn(A, s);
    float2 q;  // 1 - a^2
    decay_of(w, &da[t], &q);
    W = __fadd2_rn(W, w);
    // (A rate of 0 has 1 / n of 5e18, and no gradient: the factor w of dr, or s of dA, is 0 too.)
    const float2 ni = make_float2(rsqrt_approx(q.x), rsqrt_approx(q.y));
    fx[t] = __fmul2_rn(q, ni);
    float2 u = x;
    if (IN) {
      float2 shut;  // 1 - p
      const float2 p = sigmoid_of(ffma2(i, scale, ib), &shut);
      fx[t] = __fmul2_rn(fx[t], p);
      fi[t] = __fmul2_rn(__fmul2_rn(fx[t], x), shut);
      u = __fmul2_rn(x, p);
    }
    const float2 old = __fmul2_rn(da[t], *h);
    // dw / g = u a^2 / n - a h
    const float2 aa = __fmul2_rn(__fmul2_rn(da[t], da[t]), ni);
    const float2 dw = ffma2(u, aa, make_float2(-old.x, -old.y));
    fA[t] = __fmul2_rn(dw, s);
    fr[t] = __fmul2_rn(__fmul2_rn(dw, w), closed);
    *h = ffma2(fx[t], x, old);
    if (!GATE) return dy;
    float2 rest;
    const float2 c = sigmoid_of(__fmul2_rn(z, scale), &rest);
    const float2 m = ffma2(z, rest, make_float2(1.f, 1.f));  // silu' = c (1 + z (1 - c))
    gy[t] = __fmul2_rn(dy, __fmul2_rn(z, c));
    return __fmul2_rn(__fmul2_rn(dy, *h), __fmul2_rn(c, m));
  }
};

// A thread's sums of dA, dr_bias and di_bias, and where its results go, from the back: `last` bytes into
// each array, `yd` bytes a token.
template <bool BF16, bool IN, bool GATE>
struct Results {
  float2 sA = make_float2(0.f, 0.f), sr = sA, si = sA;
  // The results of a piece's np tokens; c comes in from behind it, and what goes on to the token before it
  // comes out.
  __device__ __forceinline__ float2 finish(const GateArgs& a, const Piece<BF16, IN, GATE>& p, int np, long long last,
                                           long long yd, float2 c) {
    float2 pA = make_float2(0.f, 0.f), pr = pA, pi = pA;  // the piece's sums
    char *px = static_cast<char*>(a.dx) + last, *pg = static_cast<char*>(a.dr) + last, *pp = static_cast<char*>(a.di) + last;
    auto out = [&](int t) {
      const float2 g = __fadd2_rn(p.gy[t], c);
      c = __fmul2_rn(p.da[t], g);
      store_pair<BF16>(px, __fmul2_rn(g, p.fx[t]));
      px -= yd;
      const float2 dr = __fmul2_rn(g, p.fr[t]);
      store_pair<BF16>(pg, dr);
      pg -= yd;
      pr = __fadd2_rn(pr, dr);
      pA = ffma2(g, p.fA[t], pA);
      if (IN) {
        const float2 di = __fmul2_rn(g, p.fi[t]);
        store_pair<BF16>(pp, di);
        pp -= yd;
        pi = __fadd2_rn(pi, di);
      }
    };
    if (np == kPiece) {
#pragma unroll
      for (int t = kPiece - 1; t >= 0; --t) out(t);
    } else {
#pragma unroll
      for (int t = kPiece - 1; t >= 0; --t)
        if (t < np) out(t);
    }
    sA = __fadd2_rn(sA, pA);
    sr = __fadd2_rn(sr, pr);
    si = __fadd2_rn(si, pi);
    return c;
  }
  // The CTA's sums over its warps, through red ([warps][32]), to part [3, D] (a thread's two channels of it).
  __device__ __forceinline__ void leave(float2* red, float* part, int D, int warps, bool in) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float2 own[3] = {sA, sr, si};
#pragma unroll
    for (int v = 0; v < 3; ++v) {
      __syncthreads();
      red[warp * 32 + lane] = own[v];
      __syncthreads();
      if (warp == v && in) {
        float2 t = red[lane];
        for (int w = 1; w < warps; ++w) t = __fadd2_rn(t, red[w * 32 + lane]);
        *reinterpret_cast<float2*>(part + (long long)v * D) = t;
      }
    }
  }
};

// sums: [n_seq, cluster, 3, D], the CTAs' parts of dA, dr_bias and di_bias.
template <bool BF16, bool IN, bool GATE, bool CLUSTER>
__global__ void __launch_bounds__(Tile<BF16>::threads, BF16 ? kResident : 2 * kResident)
palimpsa_gate_bwd_kernel(GateArgs a, int tiles, float* sums) {
  using G = Tile<BF16>;
  using S = BwdSmem<BF16, IN, GATE>;
  constexpr int ES = G::ES, RT = G::tokens, NP = G::pieces;
  constexpr int kI = 3, kZ = 3 + IN;  // places of the arrays x, r, dy, i, z
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t bars[2];
  __shared__ int told, held[32];  // see settle; the turns whose wait has held, for the first warp's threads
  float4* const agg = reinterpret_cast<float4*>(smem + S::agg);
  float2* const rates = reinterpret_cast<float2*>(smem + S::rates);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cs = CLUSTER ? a.cluster : 1;
  const int rank = CLUSTER ? (int)(blockIdx.x % cs) : 0;
  const long long rest = CLUSTER ? blockIdx.x / cs : blockIdx.x;
  const int ch0 = (int)(rest % tiles) * Tile<BF16>::CH, ch = ch0 + 2 * lane;
  const bool in = ch < a.D;
  const long long n = rest / tiles;
  const float2 zero = make_float2(0.f, 0.f);
  float* const part = sums + (n * cs + rank) * 3 * a.D + ch;
  long long row0;
  int len;
  if (!seq_rows(a.rows, n, &row0, &len)) {
    if (tid == 0) latch_status(a.status, kStatusDomain);
    if (warp < 3 && in) *reinterpret_cast<float2*>(part + (long long)warp * a.D) = zero;
    return;  // (the whole cluster)
  }
  const int step = cs * RT, rounds = (len + step - 1) / step;
  const float* const ckpt = a.ckpt_in + gate_ckpt_row0(a.rows, n, row0) * a.D + ch0;

  const int vec = tid % G::vecs, vrow = tid / G::vecs;
  const bool vin = ch0 * ES + vec * 16 < a.D * ES;
  auto stage = [&](int k) {  // copies of round k's tile, as one group
    const int t0 = k * step + rank * RT, nt = min(RT, len - t0);
    if (k >= 0) {
      unsigned char* const to = smem + (k & 1) * S::stage;
      const long long first = row0 + t0 + vrow, col = (long long)ch0 * ES + vec * 16;
      auto copy = [&](const void* from, long long ld, int slot) {
        const char* p = static_cast<const char*>(from) + first * ld * ES + col;
        unsigned char* const q = to + slot * G::bytes + tid * 16;
        const long long next = G::rows_at_once * ld * ES;
        if (nt == RT) {
#pragma unroll
          for (int j = 0; j < RT / G::rows_at_once; ++j, p += next) cp_async16(q + j * G::threads * 16, p);
        } else {
#pragma unroll
          for (int j = 0; j < RT / G::rows_at_once; ++j, p += next)
            if (j * G::rows_at_once + vrow < nt) cp_async16(q + j * G::threads * 16, p);
        }
      };
      if (vin) {
        copy(a.x, a.x_ld, 0);
        copy(a.r, a.r_ld, 1);
        copy(a.dy, a.dy_ld, 2);
        if (IN) copy(a.i, a.i_ld, kI);
        if (GATE) copy(a.z, a.z_ld, kZ);
      }
      // The states before the pieces: 16 vectors of 4 channels each.
      if (tid < NP * 16 && (tid >> 4) * kPiece < nt && ch0 + (tid & 15) * 4 < a.D)
        cp_async16(to + S::h + tid * 16, ckpt + (long long)(t0 / kPiece + (tid >> 4)) * a.D + (tid & 15) * 4);
    }
    cp_async_commit();
  };
  stage(rounds - 1);

  if (CLUSTER && tid == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    fence_mbar_init();
  }
  if (CLUSTER && warp == 0) held[lane] = rounds;
  const float2 A = pair_or(a.A, ch, in, 1.f);
  const float2 scale = make_float2(-kLog2e, -kLog2e);
  const float2 rb = __fmul2_rn(pair_or(a.r_bias, ch, in, 0.f), scale), ib = __fmul2_rn(pair_or(a.i_bias, ch, in, 0.f), scale);
  if (!pos_finite(A.x) || !pos_finite(A.y)) latch_status(a.status, kStatusDomain);
  // a g of the token behind this CTA's rounds, two places in turn.
  float2* const given = reinterpret_cast<float2*>(smem + S::given) + lane;
  if (rank == cs - 1 && warp == 0) given[0] = a.dh_T && in ? *reinterpret_cast<const float2*>(a.dh_T + n * a.D + ch) : zero;
  // The thread's sums over its rounds (in registers they would spill what the tokens keep).
  float2* const own = reinterpret_cast<float2*>(smem + S::own) + tid;
  own[0] = own[G::threads] = zero;
  if (IN) own[2 * G::threads] = zero;
  bool waits = true;
  const long long yd = (long long)a.D * ES;
  if (CLUSTER) cg::this_cluster().sync();  // every CTA has started, its barriers set: it may be written to
  if (CLUSTER && a.late && rank == cs - 1) pass_the_limit(a);

  for (int k = rounds - 1; k >= 0; --k) {
    const int tp = k * step + rank * RT + warp * kPiece;
    const int np = min(kPiece, len - tp);
    unsigned char* const raw = smem + (k & 1) * S::stage + warp * kPiece * G::row + lane * 2 * ES;
    cp_async_wait<0>();
    const int turn = rounds - 1 - k;
    const bool end = turn == 0 && rank == cs - 1;  // nothing comes from behind
    if (CLUSTER && tid == 0 && waits) mbar_arrive_expect_tx(&bars[turn & 1], end ? 0 : 256);
    __syncthreads();  // the round's inputs are here; the other stage and the summaries are free
    stage(k - 1);

    Piece<BF16, IN, GATE> p;
    const long long at = ((row0 + tp) * a.D + ch) * ES;  // bytes
    char* pz = static_cast<char*>(a.dz) + at;
    float2 h = np > 0 ? *reinterpret_cast<const float2*>(smem + (k & 1) * S::stage + S::h +
                                                         (warp * Tile<BF16>::CH + 2 * lane) * 4)
                      : zero;
    auto token = [&](int t) {
      auto load = [&](int array) { return load_pair<BF16>(raw + array * G::bytes + t * G::row); };
      const float2 dz = p.token(t, load(0), load(1), load(2), IN ? load(kI) : zero, GATE ? load(kZ) : zero, A, rb, ib, &h);
      if (GATE) {
        if (in) store_pair<BF16>(pz, dz);
        pz += yd;
      }
    };
    if (np == kPiece) {
#pragma unroll
      for (int t = 0; t < kPiece; ++t) token(t);
    } else {
#pragma unroll
      for (int t = 0; t < kPiece; ++t) {
        p.no_token(t);
        if (t < np) token(t);
      }
    }
    float2 P = make_float2(1.f, 1.f), C = zero;
#pragma unroll
    for (int t = kPiece - 1; t >= 0; --t) {
      C = __fmul2_rn(p.da[t], __fadd2_rn(p.gy[t], C));
      P = __fmul2_rn(P, p.da[t]);
    }
    agg[warp * 32 + lane] = make_float4(P.x, P.y, C.x, C.y);
    rates[warp * 32 + lane] = p.W;
    __syncthreads();

    // The first warp works out the CTA's summary, and hands on what goes back from the tile (as in the forward).
    float2 Cc = zero, Pc, Lc;
    if (warp == 0) {
      float2 Wc = zero, rest;
#pragma unroll
      for (int w = NP - 1; w >= 0; --w) {
        const float4 e = agg[w * 32 + lane];
        Cc = ffma2(make_float2(e.x, e.y), Cc, make_float2(e.z, e.w));
        Wc = __fadd2_rn(Wc, rates[w * 32 + lane]);
      }
      decay_of(Wc, &Pc, &rest, &Lc);
    }
    if (CLUSTER && waits && !cluster_wait(&bars[turn & 1], (turn >> 1) & 1, a.wait_timeout_ns)) {
      waits = false;
      if (warp == 0) held[lane] = turn;
      latch_status(a.status, kStatusTimeout);
    }
    float2 c = given[(turn & 1) * 32];
    if (warp == 0) {
      Cc = ffma2(Pc, c, with_left(Lc, c, Cc));
      const int next = rank == 0 ? turn + 1 : turn;  // the turn of the CTA before
      if (next >= rounds) {
        if (in && a.dh0) *reinterpret_cast<float2*>(a.dh0 + n * a.D + ch) = Cc;
      } else if (!CLUSTER) {
        given[(next & 1) * 32] = Cc;
      } else {
        const int to = rank == 0 ? cs - 1 : rank - 1;
        // (Where a wait has run out, nothing more is handed on: the others' waits run out too.)
        if (waits && !(a.withhold && end))
          st_async(cluster_addr(given + (next & 1) * 32, to), Cc, cluster_addr(&bars[next & 1], to));
      }
    }
    for (int w = NP - 1; w > warp; --w) {
      const float4 e = agg[w * 32 + lane];
      c = ffma2(make_float2(e.x, e.y), c, make_float2(e.z, e.w));
    }
    if (in && np > 0) {
      Results<BF16, IN, GATE> piece;
      piece.finish(a, p, np, at + (np - 1) * yd, yd, c);
      own[0] = __fadd2_rn(own[0], piece.sA);
      own[G::threads] = __fadd2_rn(own[G::threads], piece.sr);
      if (IN) own[2 * G::threads] = __fadd2_rn(own[2 * G::threads], piece.si);
    }
    __syncwarp();
  }
  if (rounds == 0 && rank == cs - 1 && warp == 0 && in && a.dh0) *reinterpret_cast<float2*>(a.dh0 + n * a.D + ch) = given[0];
  Results<BF16, IN, GATE> res;
  res.sA = own[0];
  res.sr = own[G::threads];
  if (IN) res.si = own[2 * G::threads];
  res.leave(reinterpret_cast<float2*>(agg), part, a.D, NP, in);
  if (CLUSTER) {
    // Nobody hands anything to a CTA that has left.
    if (warp == 0) {
      const int to = rank == 0 ? cs - 1 : rank - 1, on = rank == 0;
      const int mine = a.withhold && rank == cs - 1 ? 0 : held[lane], sent = __reduce_max_sync(~0u, mine);
      for (int k = mine + on; k < min(sent + on, rounds); ++k)
        st_async(cluster_addr(given + (k & 1) * 32, to), zero, cluster_addr(&bars[k & 1], to));
      if (lane == 0) *cg::this_cluster().map_shared_rank(&told, to) = min(sent + on, rounds);
    }
    cg::this_cluster().sync();
    if (tid == 0) settle(bars, held[0], told, 256);
  }
}

// Short sequences, many of them (see the forward's): a warp takes 64 channels of one sequence after
// another, piece by piece from the back, with nothing to exchange; its parameters' sums go over all
// its sequences. sums: [groups, 3, D]. (Read-only loads: behind stores that they might overlap, the
// next token's would wait: 308 us against 150 at 256 x 64 x 2048.)
constexpr int kShortWarps = 4, kShortCtas = 3;  // warps of a CTA, CTAs of an SM
template <bool BF16, bool IN, bool GATE>
__global__ void __launch_bounds__(32 * kShortWarps, kShortCtas) palimpsa_gate_short_bwd_kernel(GateArgs a, int tiles, float* sums) {
  constexpr int ES = BF16 ? 2 : 4;
  __shared__ float2 red[kShortWarps * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ch = (int)(blockIdx.x % tiles) * 64 + 2 * lane;
  const long long group = blockIdx.x / tiles, groups = gridDim.x / tiles;
  const bool in = ch < a.D;
  const float2 zero = make_float2(0.f, 0.f), scale = make_float2(-kLog2e, -kLog2e);
  const float2 A = pair_or(a.A, ch, in, 1.f);
  const float2 rb = __fmul2_rn(pair_or(a.r_bias, ch, in, 0.f), scale), ib = __fmul2_rn(pair_or(a.i_bias, ch, in, 0.f), scale);
  if (!pos_finite(A.x) || !pos_finite(A.y)) latch_status(a.status, kStatusDomain);
  const long long yd = (long long)a.D * ES;
  Results<BF16, IN, GATE> res;
  for (long long n = group * kShortWarps + warp; n < a.rows.n_seq; n += groups * kShortWarps) {
    long long row0;
    int len;
    if (!seq_rows(a.rows, n, &row0, &len)) {
      if (ch == 0) latch_status(a.status, kStatusDomain);
      continue;
    }
    if (!in) continue;
    const float* const ckpt = a.ckpt_in + gate_ckpt_row0(a.rows, n, row0) * a.D + ch;
    float2 c = a.dh_T ? *reinterpret_cast<const float2*>(a.dh_T + n * a.D + ch) : zero;
    for (int tp = (len - 1) / kPiece * kPiece; tp >= 0 && len > 0; tp -= kPiece) {
      const int np = min(kPiece, len - tp);
      const long long row = row0 + tp, at = (row * a.D + ch) * ES;
      auto start = [&](const void* p, long long ld) { return static_cast<const char*>(p) + (row * ld + ch) * ES; };
      const char *px = start(a.x, a.x_ld), *pr = start(a.r, a.r_ld), *py = start(a.dy, a.dy_ld), *pi = start(a.i, a.i_ld),
                 *pz = start(a.z, a.z_ld);
      Piece<BF16, IN, GATE> p;
      float2 h = *reinterpret_cast<const float2*>(ckpt + (long long)(tp / kPiece) * a.D);
      auto token = [&](int t) {
        auto load = [&](const char* q, long long ld) { return read_pair<BF16>(q + t * ld * ES); };
        const float2 dz = p.token(t, load(px, a.x_ld), load(pr, a.r_ld), load(py, a.dy_ld), IN ? load(pi, a.i_ld) : zero,
                                  GATE ? load(pz, a.z_ld) : zero, A, rb, ib, &h);
        if (GATE) store_pair<BF16>(static_cast<char*>(a.dz) + at + t * yd, dz);
      };
      if (np == kPiece) {
#pragma unroll
        for (int t = 0; t < kPiece; ++t) token(t);
      } else {
#pragma unroll
        for (int t = 0; t < kPiece; ++t) {
          p.no_token(t);
          if (t < np) token(t);
        }
      }
      // (What the piece's decays leave out of their product, for the gradient that goes on.)
      float2 P, q, left, Q = p.da[0];
      decay_of(p.W, &P, &q, &left);
#pragma unroll
      for (int t = 1; t < kPiece; ++t) Q = __fmul2_rn(Q, p.da[t]);
      left = __fadd2_rn(left, __fadd2_rn(P, make_float2(-Q.x, -Q.y)));
      c = with_left(left, c, res.finish(a, p, np, at + (np - 1) * yd, yd, c));
    }
    if (a.dh0) *reinterpret_cast<float2*>(a.dh0 + n * a.D + ch) = c;
  }
  res.leave(red, sums + group * 3 * a.D + ch, a.D, kShortWarps, in);
}

template <bool BF16, bool IN, bool GATE, bool CLUSTER>
cudaError_t run(const GateArgs& a, float* sums, cudaStream_t s) {
  using G = Tile<BF16>;
  const long long tiles = (a.D + G::CH - 1) / G::CH, blocks = tiles * a.rows.n_seq * a.cluster;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  constexpr int bytes = BwdSmem<BF16, IN, GATE>::bytes;
  const auto kernel = palimpsa_gate_bwd_kernel<BF16, IN, GATE, CLUSTER>;
  static SharedBytes allowed;
  cudaError_t e = allow_shared(kernel, bytes, &allowed, CLUSTER);
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
  return cudaLaunchKernelEx(&c, kernel, a, (int)tiles, sums);
}

template <bool BF16, bool IN, bool GATE>
cudaError_t backward(const GateArgs& a, float* sums, cudaStream_t s) {
  cudaError_t e;
  if (a.groups > 0) {
    const int tiles = (a.D + 63) / 64;
    palimpsa_gate_short_bwd_kernel<BF16, IN, GATE><<<(unsigned)(a.groups * tiles), 32 * kShortWarps, 0, s>>>(a, tiles, sums);
    e = cudaGetLastError();
  } else {
    e = a.cluster > 1 ? run<BF16, IN, GATE, true>(a, sums, s) : run<BF16, IN, GATE, false>(a, sums, s);
  }
  if (e != cudaSuccess) return e;
  float* const out[3] = {a.dA, a.dr_bias, a.di_bias};
  return launch_row_sums(sums, a.groups > 0 ? a.groups : (long long)a.rows.n_seq * a.cluster, 3, a.D, out, s);
}

}  // namespace

size_t plan_gate_backward(GateArgs* a) {
  // In fp32 an SM's shared memory holds 2 CTAs with both gates, 3 with one and 4 without.
  const int resident = a->bf16 ? kResident : 4 - (a->i != nullptr) - (a->z != nullptr);
  const int tokens = a->bf16 ? Tile<true>::tokens : Tile<false>::tokens;
  const GatePlan p = gate_plan(a->rows, a->D, tokens, resident, 64, {1.6, 1.4, 0.25, 0.04});
  a->cluster = p.cluster;
  a->groups = 0;
  long long rows = (long long)a->rows.n_seq * a->cluster;
  if (gate_short(a->rows, a->D, p, a->bf16 ? 225e3 : 150e3)) {
    // As many groups of warps as the GPU holds at once and the sequences fill.
    const long long tiles = (a->D + 63) / 64, held = (long long)kShortCtas * sms_of_device() / tiles;
    rows = a->groups = (int)std::max(1ll, std::min(held, (a->rows.n_seq + kShortWarps - 1ll) / kShortWarps));
  }
  return (size_t)rows * 3 * a->D;
}

cudaError_t launch_gate_backward(const GateArgs& a, float* scratch, cudaStream_t s) {
  PALIMPSA_GATE_DISPATCH(backward, a, scratch, s)
}

}  // namespace palimpsa
