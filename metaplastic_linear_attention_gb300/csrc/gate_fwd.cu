// Gated scan, forward and one token. Per channel d:
//   s_t = sigmoid(r_t + r_bias),  w_t = A s_t,  a_t = exp(-w_t),        A = A[d] > 0
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t + i_bias) x_t        (without i: its gate is 1)
//   y_t = h_t silu(z_t)                                                  (without z: h_t)
// The input's factor keeps the state's variance at the input's, whatever the decay.
//
// What bounds it: HBM. A channel-token moves 8 bytes in bf16 (10 with z), 0.37 clocks
// (0.47) of an SM's share of the measured 6.77 TB/s, against 3 2^x, 2 reciprocals and a
// root on the SFU (0.28 clocks; a 2^x and a reciprocal more with z) and about 30 FP32
// operations. So every input is read once: a thread takes 8 tokens of two channels (a piece),
// forms their decays and inputs a, b in registers, and runs them twice, first from 0 for
// the piece's summary (the product of its a and its end state), then, with the state
// before the piece known, for the states themselves. The summaries of a CTA's pieces (its
// warps, along time) pass through shared memory, and those of a cluster's CTAs through
// distributed shared memory; every thread folds the ones before its own. A CTA walks its
// sequence in rounds of such tiles, the next round's inputs coming by asynchronous
// copies meanwhile, and carries the state in registers.
//
// Rounding: gates, decays and states are fp32; y is rounded to the input type once.
#include <algorithm>

#include "gate.cuh"

namespace palimpsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kResident = 3;  // CTAs of an SM

// Shared memory: the ring of raw inputs, then the pieces' and the ranks' summaries.
template <bool BF16>
constexpr int fwd_smem(int arrays, bool cluster) {
  return 2 * arrays * GateTile<BF16>::bytes + GateTile<BF16>::warps * 32 * 16 +
         (cluster ? 2 * kGateCluster * 32 * 16 : 0);
}

template <bool BF16, bool IN, bool GATE, bool CLUSTER>
__global__ void __launch_bounds__(GateTile<BF16>::threads, kResident) palimpsa_gate_kernel(GateArgs a, int tiles) {
  using G = GateTile<BF16>;
  constexpr int ES = G::ES, NA = 2 + IN + GATE, RT = G::tokens;
  extern __shared__ __align__(128) unsigned char smem[];
  float4* const agg = reinterpret_cast<float4*>(smem + 2 * NA * G::bytes);
  float4* const xagg = agg + G::warps * 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cs = CLUSTER ? a.cluster : 1;
  const int rank = CLUSTER ? (int)(blockIdx.x % cs) : 0;
  const long long rest = CLUSTER ? blockIdx.x / cs : blockIdx.x;
  const int ch0 = (int)(rest % tiles) * kGateChannels, ch = ch0 + 2 * lane;
  const long long n = rest / tiles;
  long long row0;
  int len;
  if (!seq_rows(a.rows, n, &row0, &len)) {
    if (tid == 0) latch_status(a.status, kStatusDomain);
    return;  // (the whole cluster)
  }
  const int step = cs * RT, rounds = (len + step - 1) / step;

  // Copies of a round's tile, as one group: a thread takes the same vector of rows
  // rows_at_once apart. Rows past the end and channels past D are left as they are.
  const int vec = tid % G::vecs, vrow = tid / G::vecs;
  const bool vin = ch0 * ES + vec * 16 < a.D * ES;
  auto stage = [&](int k) {
    const int t0 = k * step + rank * RT, nt = min(RT, len - t0);
    if (k < rounds && vin) {
      unsigned char* const to = smem + (k & 1) * NA * G::bytes + tid * 16;
      const long long first = row0 + t0 + vrow, col = (long long)ch0 * ES + vec * 16;
      auto copy = [&](const void* from, long long ld, int slot) {
        const char* p = static_cast<const char*>(from) + first * ld * ES + col;
#pragma unroll
        for (int j = 0; j < RT / G::rows_at_once; ++j)
          if (j * G::rows_at_once + vrow < nt)
            cp_async16(to + slot * G::bytes + j * G::threads * 16, p + j * G::rows_at_once * ld * ES);
      };
      copy(a.x, a.x_ld, 0);
      copy(a.r, a.r_ld, 1);
      if (IN) copy(a.i, a.i_ld, 2);
      if (GATE) copy(a.z, a.z_ld, 2 + IN);
    }
    cp_async_commit();
  };
  stage(0);

  const bool in = ch < a.D;
  const float2 A = pair_or(a.A, ch, in, 1.f);
  const float2 rb = pair_or(a.r_bias, ch, in, 0.f), ib = pair_or(a.i_bias, ch, in, 0.f);
  if (!pos_finite(A.x) || !pos_finite(A.y)) latch_status(a.status, kStatusDomain);
  float2 carry = make_float2(0.f, 0.f);  // the state before the round
  if (a.h0 && in) carry = *reinterpret_cast<const float2*>(a.h0 + n * a.D + ch);
  if (CLUSTER) cg::this_cluster().sync();  // every CTA has started: its shared memory may be written

  for (int k = 0; k < rounds; ++k) {
    const int tp = k * step + rank * RT + warp * kPiece;  // the piece's first token
    const int np = min(kPiece, len - tp);                 // its tokens (0 or less: none)
    const unsigned char* const raw =
        smem + (k & 1) * NA * G::bytes + warp * kPiece * G::row + lane * 2 * ES;
    cp_async_wait<0>();
    __syncthreads();  // the round's inputs are here; the other stage and the summaries are free
    stage(k + 1);

    float2 da[kPiece], b[kPiece];
    float2 P = make_float2(1.f, 1.f), H = make_float2(0.f, 0.f);
#pragma unroll
    for (int t = 0; t < kPiece; ++t) {
      if (t < np) {
        const float2 x = load_pair<BF16>(raw + t * G::row);
        const Sigmoid s(__fadd2_rn(load_pair<BF16>(raw + G::bytes + t * G::row), rb));
        float2 rest2;
        decay_of(__fmul2_rn(A, s.p), &da[t], &rest2);
        b[t] = __fmul2_rn(make_float2(sqrt_approx(rest2.x), sqrt_approx(rest2.y)), x);
        if (IN) {
          const Sigmoid p(__fadd2_rn(load_pair<BF16>(raw + 2 * G::bytes + t * G::row), ib));
          b[t] = __fmul2_rn(b[t], p.p);
        }
      } else {
        da[t] = make_float2(1.f, 1.f);
        b[t] = make_float2(0.f, 0.f);
      }
      H = ffma2(da[t], H, b[t]);
      P = __fmul2_rn(P, da[t]);
    }
    agg[warp * 32 + lane] = make_float4(P.x, P.y, H.x, H.y);
    __syncthreads();

    // The state before the piece, and the one before the next round.
    float2 h = carry;
    if (!CLUSTER) {
#pragma unroll
      for (int q = 0; q < G::warps; ++q) {
        const float4 e = agg[q * 32 + lane];
        if (q == warp) h = carry;
        carry = ffma2(make_float2(e.x, e.y), carry, make_float2(e.z, e.w));
      }
    } else {
      // Warp q sends the CTA's summary to rank q. (Two sets of slots: a rank may be a round ahead.)
      float4* const slots = xagg + (k & 1) * kGateCluster * 32;
      cg::cluster_group cluster = cg::this_cluster();
      for (int q = warp; q < cs; q += G::warps) {
        float2 Pc = make_float2(1.f, 1.f), Hc = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < G::warps; ++w) {
          const float4 e = agg[w * 32 + lane];
          Hc = ffma2(make_float2(e.x, e.y), Hc, make_float2(e.z, e.w));
          Pc = __fmul2_rn(Pc, make_float2(e.x, e.y));
        }
        *cluster.map_shared_rank(slots + rank * 32 + lane, q) = make_float4(Pc.x, Pc.y, Hc.x, Hc.y);
      }
      cluster.sync();
      for (int q = 0; q < cs; ++q) {
        const float4 e = slots[q * 32 + lane];
        if (q == rank) h = carry;
        carry = ffma2(make_float2(e.x, e.y), carry, make_float2(e.z, e.w));
      }
      for (int w = 0; w < warp; ++w) {
        const float4 e = agg[w * 32 + lane];
        h = ffma2(make_float2(e.x, e.y), h, make_float2(e.z, e.w));
      }
    }
    if (in && np > 0) {
      if (a.ckpt)
        *reinterpret_cast<float2*>(a.ckpt + (gate_ckpt_row0(a.rows, n, row0) + tp / kPiece) * a.D + ch) = h;
      char* const py = static_cast<char*>(a.y) + ((row0 + tp) * a.D + ch) * ES;
#pragma unroll
      for (int t = 0; t < kPiece; ++t)
        if (t < np) {
          h = ffma2(da[t], h, b[t]);
          float2 y = h;
          if (GATE) y = __fmul2_rn(y, silu_fast(load_pair<BF16>(raw + (2 + IN) * G::bytes + t * G::row)));
          store_pair<BF16>(py + (long long)t * a.D * ES, y);
        }
    }
    __syncwarp();
  }
  if (rank == 0 && warp == 0 && in) *reinterpret_cast<float2*>(a.h_T + n * a.D + ch) = carry;
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
    const Sigmoid s(__fadd2_rn(r[j], pair_or(a.r_bias, ch + 2 * j, true, 0.f)));
    float2 da, rest;
    decay_of(__fmul2_rn(A, s.p), &da, &rest);
    float2 b = __fmul2_rn(make_float2(sqrt_approx(rest.x), sqrt_approx(rest.y)), x[j]);
    if (IN) b = __fmul2_rn(b, Sigmoid(__fadd2_rn(i[j], pair_or(a.i_bias, ch + 2 * j, true, 0.f))).p);
    h[j] = ffma2(da, h[j], b);
    y[j] = GATE ? __fmul2_rn(h[j], silu_fast(z[j])) : h[j];
  }
  *state = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
  *reinterpret_cast<typename Q::Raw*>(static_cast<char*>(a.y) + (n * a.D + ch) * ES) = Q::pack(y);
  if (bad) latch_status(a.status, kStatusDomain);
}

template <bool BF16, bool IN, bool GATE, bool CLUSTER>
cudaError_t run(const GateArgs& a, cudaStream_t s) {
  using G = GateTile<BF16>;
  const long long tiles = gate_tiles(a.D), blocks = tiles * a.rows.n_seq * a.cluster;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  constexpr int bytes = fwd_smem<BF16>(2 + IN + GATE, CLUSTER);
  const auto kernel = palimpsa_gate_kernel<BF16, IN, GATE, CLUSTER>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
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
  a.cluster = gate_cluster(a.rows, a.D, GateTile<BF16>::tokens, kResident);
  return a.cluster > 1 ? run<BF16, IN, GATE, true>(a, s) : run<BF16, IN, GATE, false>(a, s);
}

template <bool BF16, bool IN, bool GATE>
cudaError_t step(const GateArgs& a, cudaStream_t s) {
  const long long blocks = ((long long)(a.D / 4) * a.rows.n_seq + 127) / 128;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  palimpsa_gate_step_kernel<BF16, IN, GATE><<<(unsigned)blocks, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

// The cheapest of 1, 2, 4 and 8 CTAs a cluster. The GPU's rounds: every tile of every sequence
// takes its tokens in rounds of cluster x `tokens`, `resident` CTAs an SM at once; and no
// batch is faster than its longest sequence's rounds, one after the other, each with its
// exchange. (What is left of a round costs as much as a whole one.)
int gate_cluster(const SeqRows& r, int D, int tokens, long long resident) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 152;
  const long long slots = resident * sms, tiles = gate_tiles(D);
  int best = 1;
  long long least = 0;
  for (int cs = 1; cs <= kGateCluster; cs *= 2) {
    const long long per = (long long)cs * tokens, longest = (r.max_len + per - 1) / per;
    const long long all = r.cu ? cs * (r.T / per + r.n_seq) : cs * longest * r.n_seq;  // CTA rounds, a tile
    const long long cost = std::max((all * tiles + slots - 1) / slots, longest);
    if (cs == 1 || cost < least) {
      best = cs;
      least = cost;
    }
  }
  return best;
}

cudaError_t launch_gate_forward(const GateArgs& a, cudaStream_t s) { PALIMPSA_GATE_DISPATCH(forward, a, s) }
cudaError_t launch_gate_step(const GateArgs& a, cudaStream_t s) { PALIMPSA_GATE_DISPATCH(step, a, s) }

}  // namespace palimpsa
