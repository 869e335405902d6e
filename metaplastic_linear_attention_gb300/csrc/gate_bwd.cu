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
// of the second run, as in the forward: 1 % slower.) The rounds go from the back to the front, and in a cluster the gradient goes round the other way.
// The parameters' sums stay in registers over all rounds; they are added up over the CTA's
// pieces in shared memory and over CTAs by a second kernel, in a fixed order: no atomics, the
// same bits every time.
// Measured (GB300, bf16, both gates): 198 us at 8 x 4096 x 1536 (138 for its bytes at the rate of a
// copy), 40 at 4 x 2048 x 1024 (23); fp32 at 0.81 to 0.84 of that rate. What a token keeps
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
  static constexpr int agg = 2 * stage, given = agg + Tile<BF16>::pieces * 512;
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
  float4* const agg = reinterpret_cast<float4*>(smem + S::agg);
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
  const float2 A = pair_or(a.A, ch, in, 1.f);
  const float2 scale = make_float2(-kLog2e, -kLog2e);
  const float2 rb = __fmul2_rn(pair_or(a.r_bias, ch, in, 0.f), scale), ib = __fmul2_rn(pair_or(a.i_bias, ch, in, 0.f), scale);
  if (!pos_finite(A.x) || !pos_finite(A.y)) latch_status(a.status, kStatusDomain);
  float2 carry = zero;  // a g of the token behind the round (in a cluster, behind the sequence)
  if (a.dh_T && in) carry = *reinterpret_cast<const float2*>(a.dh_T + n * a.D + ch);
  float2 sA = zero, sr = zero, si = zero;
  bool waits = true;
  const long long yd = (long long)a.D * ES;
  if (CLUSTER) cg::this_cluster().sync();  // every CTA has started, its barriers set: it may be written to

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

    // The factors of g_t in dx, di, dr and dA, the decays, and dy silu(z).
    float2 da[kPiece], fx[kPiece], fi[IN ? kPiece : 1], fr[kPiece], fA[kPiece], gy[kPiece];
    const long long at = ((row0 + tp) * a.D + ch) * ES;  // bytes
    char* pz = static_cast<char*>(a.dz) + at;
    float2 h = np > 0 ? *reinterpret_cast<const float2*>(smem + (k & 1) * S::stage + S::h +
                                                         (warp * Tile<BF16>::CH + 2 * lane) * 4)
                      : zero;
    auto token = [&](int t) {
      const float2 x = load_pair<BF16>(raw + t * G::row);
      float2 closed;  // 1 - s
      const float2 s = sigmoid_of(ffma2(load_pair<BF16>(raw + G::bytes + t * G::row), scale, rb), &closed);
      gy[t] = load_pair<BF16>(raw + 2 * G::bytes + t * G::row);
      const float2 w = __fmul2_rn(A, s);
      float2 q;  // 1 - a^2
      decay_of(w, &da[t], &q);
      // (A rate of 0 has 1 / n of 5e18, and no gradient: the factor w of dr, or s of dA, is 0 too.)
      const float2 ni = make_float2(rsqrt_approx(q.x), rsqrt_approx(q.y));
      fx[t] = __fmul2_rn(q, ni);
      float2 u = x;
      if (IN) {
        float2 shut;  // 1 - p
        const float2 p = sigmoid_of(ffma2(load_pair<BF16>(raw + kI * G::bytes + t * G::row), scale, ib), &shut);
        fx[t] = __fmul2_rn(fx[t], p);
        fi[t] = __fmul2_rn(__fmul2_rn(fx[t], x), shut);
        u = __fmul2_rn(x, p);
      }
      const float2 old = __fmul2_rn(da[t], h);
      // dw / g = u a^2 / n - a h
      const float2 aa = __fmul2_rn(__fmul2_rn(da[t], da[t]), ni);
      const float2 dw = ffma2(u, aa, make_float2(-old.x, -old.y));
      fA[t] = __fmul2_rn(dw, s);
      fr[t] = __fmul2_rn(__fmul2_rn(dw, w), closed);
      h = ffma2(fx[t], x, old);
      if (GATE) {
        const float2 z = load_pair<BF16>(raw + kZ * G::bytes + t * G::row);
        float2 rest;
        const float2 c = sigmoid_of(__fmul2_rn(z, scale), &rest);
        const float2 m = ffma2(z, rest, make_float2(1.f, 1.f));  // silu' = c (1 + z (1 - c))
        const float2 dz = __fmul2_rn(__fmul2_rn(gy[t], h), __fmul2_rn(c, m));
        if (in) store_pair<BF16>(pz, dz);
        pz += yd;
        gy[t] = __fmul2_rn(gy[t], __fmul2_rn(z, c));
      }
    };
    if (np == kPiece) {
#pragma unroll
      for (int t = 0; t < kPiece; ++t) token(t);
    } else {
#pragma unroll
      for (int t = 0; t < kPiece; ++t) {
        da[t] = make_float2(1.f, 1.f);
        fx[t] = fr[t] = fA[t] = gy[t] = zero;
        if (IN) fi[t] = zero;
        if (t < np) token(t);
      }
    }
    float2 P = make_float2(1.f, 1.f), C = zero;
#pragma unroll
    for (int t = kPiece - 1; t >= 0; --t) {
      C = __fmul2_rn(da[t], __fadd2_rn(gy[t], C));
      P = __fmul2_rn(P, da[t]);
    }
    agg[warp * 32 + lane] = make_float4(P.x, P.y, C.x, C.y);
    __syncthreads();

    // The gradient that comes in from behind the piece, and the one that the round passes on.
    float2 c = carry;
    if (!CLUSTER) {
#pragma unroll
      for (int q = NP - 1; q >= 0; --q) {
        const float4 e = agg[q * 32 + lane];
        if (q == warp) c = carry;
        carry = ffma2(make_float2(e.x, e.y), carry, make_float2(e.z, e.w));
      }
    } else {
      // The first warp works out the CTA's summary, and hands on what goes back from the tile.
      float2 Pc = make_float2(1.f, 1.f), Cc = zero;
      if (warp == 0)
#pragma unroll
        for (int w = NP - 1; w >= 0; --w) {
          const float4 e = agg[w * 32 + lane];
          Cc = ffma2(make_float2(e.x, e.y), Cc, make_float2(e.z, e.w));
          Pc = __fmul2_rn(Pc, make_float2(e.x, e.y));
        }
      float2* const given = reinterpret_cast<float2*>(smem + S::given) + lane;
      waits = waits && cluster_wait(&bars[turn & 1], (turn >> 1) & 1, a.wait_timeout_ns);
      if (!waits) latch_status(a.status, kStatusTimeout);
      if (!end) c = given[(turn & 1) * 32];
      if (warp == 0) {
        Cc = ffma2(Pc, c, Cc);
        const int next = rank == 0 ? turn + 1 : turn;  // the turn of the CTA before
        if (next < rounds) {
          const int to = rank == 0 ? cs - 1 : rank - 1;
          // (Where a wait has run out, nothing more is handed on: the others' waits run out too.)
          if (waits && !(a.withhold && end))
            st_async(cluster_addr(given + (next & 1) * 32, to), Cc, cluster_addr(&bars[next & 1], to));
        } else if (in && a.dh0) {
          *reinterpret_cast<float2*>(a.dh0 + n * a.D + ch) = Cc;
        }
      }
      for (int w = NP - 1; w > warp; --w) {
        const float4 e = agg[w * 32 + lane];
        c = ffma2(make_float2(e.x, e.y), c, make_float2(e.z, e.w));
      }
    }
    if (in && np > 0) {
      float2 pA = zero, pr = zero, pi = zero;  // the piece's sums
      const long long last = at + (np - 1) * yd;
      char *px = static_cast<char*>(a.dx) + last, *pg = static_cast<char*>(a.dr) + last, *pp = static_cast<char*>(a.di) + last;
      auto out = [&](int t) {
        const float2 g = __fadd2_rn(gy[t], c);
        c = __fmul2_rn(da[t], g);
        store_pair<BF16>(px, __fmul2_rn(g, fx[t]));
        px -= yd;
        const float2 dr = __fmul2_rn(g, fr[t]);
        store_pair<BF16>(pg, dr);
        pg -= yd;
        pr = __fadd2_rn(pr, dr);
        pA = ffma2(g, fA[t], pA);
        if (IN) {
          const float2 di = __fmul2_rn(g, fi[t]);
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
    }
    __syncwarp();
  }
  if ((!CLUSTER || rounds == 0) && rank == 0 && warp == 0 && in && a.dh0)
    *reinterpret_cast<float2*>(a.dh0 + n * a.D + ch) = carry;
  // The CTA's sums over its pieces.
  float2* const red = reinterpret_cast<float2*>(agg);
  const float2 own[3] = {sA, sr, si};
#pragma unroll
  for (int v = 0; v < 3; ++v) {
    __syncthreads();
    red[warp * 32 + lane] = own[v];
    __syncthreads();
    if (warp == v && in) {
      float2 t = red[lane];
#pragma unroll
      for (int w = 1; w < NP; ++w) t = __fadd2_rn(t, red[w * 32 + lane]);
      *reinterpret_cast<float2*>(part + (long long)v * a.D) = t;
    }
  }
  if (CLUSTER) cg::this_cluster().sync();  // nobody hands anything to a CTA that has left
}

template <bool BF16, bool IN, bool GATE, bool CLUSTER>
cudaError_t run(const GateArgs& a, float* sums, cudaStream_t s) {
  using G = Tile<BF16>;
  const long long tiles = (a.D + G::CH - 1) / G::CH, blocks = tiles * a.rows.n_seq * a.cluster;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  constexpr int bytes = BwdSmem<BF16, IN, GATE>::given + (CLUSTER ? 512 : 0);
  const auto kernel = palimpsa_gate_bwd_kernel<BF16, IN, GATE, CLUSTER>;
  static SharedBytes allowed;
  cudaError_t e = allow_shared(kernel, bytes, &allowed);
  if (e == cudaSuccess && a.cluster > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
  e = cudaLaunchKernelEx(&c, kernel, a, (int)tiles, sums);
  if (e != cudaSuccess) return e;
  float* const out[3] = {a.dA, a.dr_bias, a.di_bias};
  return launch_row_sums(sums, (long long)a.rows.n_seq * a.cluster, 3, a.D, out, s);
}

template <bool BF16, bool IN, bool GATE>
cudaError_t backward(const GateArgs& a, float* sums, cudaStream_t s) {
  return a.cluster > 1 ? run<BF16, IN, GATE, true>(a, sums, s) : run<BF16, IN, GATE, false>(a, sums, s);
}

}  // namespace

size_t plan_gate_backward(GateArgs* a) {
  // In fp32 an SM's shared memory holds 2 CTAs with both gates, 3 with one and 4 without.
  const int resident = a->bf16 ? kResident : 4 - (a->i != nullptr) - (a->z != nullptr);
  const int tokens = a->bf16 ? Tile<true>::tokens : Tile<false>::tokens;
  a->cluster = gate_plan(a->rows, a->D, tokens, resident, 64).cluster;
  return (size_t)a->rows.n_seq * a->cluster * 3 * a->D;
}

cudaError_t launch_gate_backward(const GateArgs& a, float* scratch, cudaStream_t s) {
  PALIMPSA_GATE_DISPATCH(backward, a, scratch, s)
}

}  // namespace palimpsa
