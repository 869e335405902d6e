// Internal declarations of the state-space operators: the short causal
// convolution (conv.cu), the selective scan (scan_fwd.cu, scan_bwd.cu,
// scan_step.cu) and the gated scan (gate_fwd.cu, gate_bwd.cu), and of the
// layer norm between such layers (norm.cu). Their C ABI is ssm_api.cu.
//
// Layouts are token-major: a row of D channels per token, rows of one sequence
// following each other with a stride (`ld`, elements) that may exceed D, so
// that a slice of a wider projection goes in without a copy. A dense batch is
// n_seq sequences of T rows; a packed batch is n_seq sequences of rows
// [cu[n], cu[n+1]) among T rows in all.
#pragma once

#include <atomic>
#include <mutex>

#include "palimpsa_internal.cuh"

namespace palimpsa {

// Rows of sequence n: first row and length. Shared by both operators.
struct SeqRows {
  const int* cu = nullptr;  // null: dense
  int n_seq = 0;
  int T = 0;        // rows per sequence (dense) or in all (packed)
  int max_len = 0;  // longest sequence (= T when dense)
};

// Pieces of equal length (runs, segments, single rows) that a batch is cut into, one
// slot each: sequence n has slots n per_seq, ... With `starts`, of a packed batch, they
// lie close instead, and sequence n has slots starts[n] .. starts[n + 1] - 1.
struct Slots {
  const int* starts = nullptr;
  int per_seq = 1;      // of the longest sequence
  long long count = 0;  // slots in all; with `starts` their bound, ceil included
};
// Slots of pieces of `piece` tokens of every sequence, an empty one having one piece.
inline Slots slots_of(const SeqRows& r, long long piece) {
  Slots s;
  s.per_seq = r.max_len > piece ? (int)((r.max_len + piece - 1) / piece) : 1;
  s.count = (long long)r.n_seq * s.per_seq;
  return s;
}
inline long long close_slots(const SeqRows& r, long long piece) { return r.T / piece + r.n_seq; }
// Whether a packed batch's slots should lie close, when the usual ones come to `idle` CTAs
// without work. Those cost about 1.3 ns each (256 sequences, one of 32768 tokens and the
// rest of 100, D = 1536: convolution 518 us, where 53 go for its bytes); the kernel that
// lays the slots close and the searches for a slot's sequence cost 5 to 10 us.
inline bool close_pays(const SeqRows& r, long long idle) { return r.cu && idle > 16384; }
// starts[n_seq + 1] for pieces of `piece` tokens and, if not null, row_starts[n_seq + 1] for
// rows. A sequence that is skipped for its offsets has no slots; nor has one that would
// pass the bounds, which offsets in order never do.
cudaError_t launch_slot_starts(const SeqRows& r, int piece, int* starts, int* row_starts, unsigned* status,
                               cudaStream_t s);

struct ConvArgs {
  const void* x;
  const float* weight;  // [D, W]
  const float* bias;    // [D] or null
  const void* state0;   // [n_seq, W - 1, D] or null
  void* y;              // forward and step
  void* state_T;        // may be null; may be state0
  // backward
  const void* dy = nullptr;
  const void* dstate_T = nullptr;
  void* dx = nullptr;
  void* dstate0 = nullptr;
  float* dweight = nullptr;
  float* dbias = nullptr;
  long long x_ld, dy_ld = 0;
  SeqRows rows;
  Slots slots;  // runs, set by plan_conv
  int run = 0;  // tokens of a run
  int D, W;
  bool silu, bf16;
  unsigned int* status;
};
// Sets a->run and a->slots; returns the bytes of scratch that the launch takes.
size_t plan_conv(ConvArgs* a, bool backward);
cudaError_t launch_conv_forward(const ConvArgs& a, float* scratch, cudaStream_t s);
cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t s);
cudaError_t launch_conv_backward(const ConvArgs& a, float* scratch, cudaStream_t s);

// Zeros in what the kernels leave unwritten of a packed batch's outputs: rows that no
// sequence covers, and the rows and states of skipped sequences, of up to kZeroArrays dense
// arrays (widths in bytes, multiples of 16), the first row_arrays of them with a row per
// token, the others with an entry per sequence.
constexpr int kZeroArrays = 8;
struct ZeroArgs {
  void* p[kZeroArrays];
  long long width[kZeroArrays];
  int row_arrays;
  SeqRows rows;
};
cudaError_t launch_zero_outside(const ZeroArgs& a, int arrays, cudaStream_t s);

struct ScanArgs {
  const void* x;
  const void* dt;
  const float* A;        // [D, N]
  const void* B;         // rows of [G, N]
  const void* C;
  const float* skip;     // [D] or null
  const void* z;         // or null
  const float* dt_bias;  // [D] or null
  const float* h0;       // [n_seq, D, N] or null
  void* y;
  float* h_T;            // [n_seq, D, N]; the step's state, in place
  float* ckpt = nullptr;
  long long x_ld, dt_ld, B_ld, C_ld, z_ld;
  SeqRows rows;
  int D, G, N;
  bool softplus, bf16;
  unsigned int* status;
  // time split (set by the launcher)
  int nseg = 1, seg_len = 0;   // of the longest sequence
  Slots slots;                 // segments
  Slots row_slots;             // backward, if close: rows
  float* seg_state = nullptr;  // [slots, D, N]: summaries, then (if carried) start states
  bool carried = false;        // many segments: a kernel of its own folds the summaries
  float* seg_dt = nullptr;     // [slots, D]: sums of the step sizes
  // backward
  const float* ckpt_in = nullptr;
  const void* dy = nullptr;
  const float* dh_T = nullptr;
  void* dx = nullptr;
  void* ddt = nullptr;
  void* dz = nullptr;
  void* dB = nullptr;
  void* dC = nullptr;
  float* dA = nullptr;
  float* dskip = nullptr;
  float* ddt_bias = nullptr;
  float* dh0 = nullptr;
  long long dy_ld = 0;
};

constexpr int kScanChannels = 32;      // channels of a scan tile
constexpr int kScanCheckpoint = 16;    // tokens between training checkpoints

// Checkpoint rows of a batch, each [D, N]: sequence n's checkpoint c (the state
// before its token 16 c) is row scan_ckpt_row0(n) + c. A packed batch keeps
// T / 16 + n_seq rows, sequence n (from row s0) starting at s0 / 16 + n: the next
// sequence starts at least ceil(len / 16) rows later, so none are shared.
__host__ __device__ inline long long scan_ckpt_rows(const SeqRows& r) {
  if (r.cu) return (long long)r.T / kScanCheckpoint + r.n_seq;
  return (long long)r.n_seq * ((r.T + kScanCheckpoint - 1) / kScanCheckpoint);
}
__host__ __device__ inline long long scan_ckpt_row0(const SeqRows& r, long long n, long long s0) {
  if (r.cu) return s0 / kScanCheckpoint + n;
  return n * ((r.T + kScanCheckpoint - 1) / kScanCheckpoint);
}
inline long long scan_tiles(const ScanArgs& a) {
  const int dg = a.D / a.G;
  return (long long)a.G * ((dg + kScanChannels - 1) / kScanChannels);
}

// Plans a scan or its backward: sets a->nseg, a->seg_len (a multiple of kScanCheckpoint)
// and a->slots, and *close if the slots are to lie close.
cudaError_t plan_scan(ScanArgs* a, bool backward, bool* close);
// Scratch of a time split.
inline size_t scan_scratch_floats(const ScanArgs& a) {
  return a.nseg > 1 ? (size_t)a.slots.count * a.D * (a.N + 1) : 0;
}
cudaError_t launch_scan_forward(const ScanArgs& a, cudaStream_t s);
cudaError_t launch_scan_step(const ScanArgs& a, cudaStream_t s);
// Backward: scratch of scan_backward_scratch_floats() holds the per-tile sums of
// dB and dC and the per-segment sums of the parameters' gradients.
size_t scan_backward_scratch_floats(const ScanArgs& a);
cudaError_t launch_scan_backward(const ScanArgs& a, float* scratch, cudaStream_t s);
int scan_backward_resident(const ScanArgs& a);  // CTAs that an SM holds; 0 on failure
// Pass A of the backward's time split: each segment's gradient with respect to the
// state before it, from a zero gradient after it, and its sum of step sizes.
cudaError_t launch_scan_reverse_summary(const ScanArgs& a, cudaStream_t s);
// Above this many segments the folds get a kernel of their own: 11 us at 38 segments of 1
// x 32768 x 2048, where a fold in every CTA cost 22; 5 us less in all at 19 of 4 x 2048 x
// 1024, but 15 us more, mostly for its launch, at 17 of 2 x 777 x 520 (N = 8, training).
constexpr int kFoldSegments = 18;
// Turns the summaries into start states, in place: forward from h0, or in reverse from dh_T.
cudaError_t launch_scan_carry(const ScanArgs& a, bool reverse, cudaStream_t s);

// The current device's SMs (asked for once a device; 152 where that fails).
inline int sms_of_device() {
  static std::atomic<int> known[64] = {};
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (dev >= 0 && dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
  if (dev >= 0 && dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}
// Lets a kernel have `bytes` of dynamic shared memory (and, if wide, clusters of more than 8): calls of
// the runtime only when this device has not yet allowed it as many. `allowed` is the kernel's own.
struct SharedBytes {
  std::atomic<int> on[64] = {};
  std::mutex raising;  // two calls at once must not leave the smaller of their limits
};
template <class K>
cudaError_t allow_shared(K kernel, int bytes, SharedBytes* allowed, bool wide = false) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;  // (as the library's pools)
  std::atomic<int>& on = allowed->on[dev];
  if (on.load() >= bytes) return cudaSuccess;
  std::lock_guard<std::mutex> lock(allowed->raising);
  if (on.load() >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && wide) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) on.store(bytes);
  return e;
}
// What an SM of the current device holds of a kernel's CTAs, by their threads (a multiple of 32, up to 512; `bytes`
// of dynamic shared memory follow from them); asked for once a device. `known` is the kernel's own.
struct HeldCtas {
  std::atomic<int> ctas[64][17] = {};
};
template <class K>
cudaError_t held_ctas(K kernel, int threads, int bytes, HeldCtas* known, int* held) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::atomic<int>& ctas = known->ctas[dev][threads / 32];
  *held = ctas.load(std::memory_order_relaxed);
  if (*held > 0) return cudaSuccess;
  if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(held, kernel, threads, bytes)) != cudaSuccess) return e;
  if (*held < 1) return cudaErrorInvalidConfiguration;
  ctas.store(*held, std::memory_order_relaxed);
  return cudaSuccess;
}

// The gated scan: one state per channel, gates from the token (formulas in gate_fwd.cu).
struct GateArgs {
  const void* x;
  const void* r;
  const void* i;        // or null: the input gate is 1
  const void* z;        // or null
  const float* A;       // [D]
  const float* r_bias;  // [D] or null
  const float* i_bias;  // [D] or null
  const float* h0;      // [n_seq, D] or null
  void* y;
  float* h_T;           // [n_seq, D]; the step's state, in place
  float* ckpt = nullptr;
  long long x_ld, r_ld, i_ld, z_ld;
  SeqRows rows;
  int D;
  bool bf16;
  unsigned int* status;
  int cluster = 1;      // CTAs that share a sequence's time, set by the launcher
  unsigned long long wait_timeout_ns = 0;
  bool withhold = false, late = false;  // tests: the first CTA of a cluster hands nothing on in its first round, or late
  // backward
  const float* ckpt_in = nullptr;
  const void* dy = nullptr;
  const float* dh_T = nullptr;
  void* dx = nullptr;
  void* dr = nullptr;
  void* di = nullptr;
  void* dz = nullptr;
  float* dA = nullptr;
  float* dr_bias = nullptr;
  float* di_bias = nullptr;
  float* dh0 = nullptr;
  long long dy_ld = 0;
  int groups = 0;       // short sequences: groups of warps that walk them, set by plan_gate_backward
};

constexpr int kGateCheckpoint = 8;  // tokens between the gated scan's checkpoints

// Checkpoint rows, each [D]: as scan_ckpt_rows, with 8 tokens between two.
__host__ __device__ inline long long gate_ckpt_rows(const SeqRows& r) {
  if (r.cu) return (long long)r.T / kGateCheckpoint + r.n_seq;
  return (long long)r.n_seq * ((r.T + kGateCheckpoint - 1) / kGateCheckpoint);
}
__host__ __device__ inline long long gate_ckpt_row0(const SeqRows& r, long long n, long long s0) {
  if (r.cu) return s0 / kGateCheckpoint + n;
  return n * ((r.T + kGateCheckpoint - 1) / kGateCheckpoint);
}
cudaError_t launch_gate_forward(const GateArgs& a, cudaStream_t s);
cudaError_t launch_gate_step(const GateArgs& a, cudaStream_t s);
// Backward: sets a->cluster and a->groups; scratch of as many floats holds the parameters' sums of every CTA.
size_t plan_gate_backward(GateArgs* a);
cudaError_t launch_gate_backward(const GateArgs& a, float* scratch, cudaStream_t s);

// out[v][d] (null: not wanted) = sum over rows of parts[row, v, d]; V = 2 or 3 (row_sums.cu).
cudaError_t launch_row_sums(const float* parts, long long rows, int V, int D, float* const* out, cudaStream_t s);

// The layer norm of rows of D values, and the addition in front of it (norm.cu).
constexpr int kNormWidth = 8192;  // the widest row
struct NormArgs {
  const void* x;            // forward: the rows; backward: the rows that were normalised
  const void* residual;     // forward: or null
  const float* weight;      // [D] or null (1)
  const float* bias;        // [D] or null (0)
  void* y;
  void* sum = nullptr;      // x + residual, with residual
  float* stats;             // [rows, 2]: mean and 1 / deviation; forward: or null
  long long x_ld, residual_ld = 0;
  long long rows;
  int D;
  float eps;
  bool bf16;
  // backward
  const void* dy = nullptr;
  const void* ds = nullptr;  // or null
  void* dx = nullptr;
  float* dweight = nullptr;
  float* dbias = nullptr;
  long long dy_ld = 0, ds_ld = 0;
  int ctas = 0;
};
cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t s);
// Backward: sets a->ctas and the scratch that holds every CTA's sums of the parameters' gradients.
cudaError_t plan_norm_backward(NormArgs* a, size_t* floats);
cudaError_t launch_norm_backward(const NormArgs& a, float* scratch, cudaStream_t s);

#if defined(__CUDACC__)

// First row and length of sequence n; false (and nothing may be touched) when
// packed offsets are out of order, out of range or longer than max_len.
__device__ __forceinline__ bool seq_rows(const SeqRows& r, long long n, long long* row0, int* len) {
  if (!r.cu) {
    *row0 = n * r.T;
    *len = r.T;
    return true;
  }
  const int s0 = r.cu[n], s1 = r.cu[n + 1];
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= r.T && s1 - s0 <= r.max_len;
  *row0 = ok ? s0 : 0;
  *len = ok ? s1 - s0 : 0;
  return ok;
}

// The sequence n and the place k in it of a slot; false for a slot that no sequence has.
__device__ __forceinline__ bool slot_place(const SeqRows& r, const Slots& s, long long slot, int* n, int* k) {
  if (!s.starts) {
    *n = (int)(slot / s.per_seq);
    *k = (int)(slot % s.per_seq);
    return true;
  }
  if (slot >= s.starts[r.n_seq]) return false;
  int lo = 0, hi = r.n_seq;  // starts[lo] <= slot < starts[hi]
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (s.starts[mid] <= slot) lo = mid;
    else hi = mid;
  }
  *n = lo;
  *k = (int)(slot - s.starts[lo]);
  return true;
}
__device__ __forceinline__ long long first_slot(const Slots& s, int n) {
  return s.starts ? s.starts[n] : (long long)n * s.per_seq;
}

// A 16-byte vector of the input type as fp32 values: 8 bf16 or 4 fp32.
template <bool BF16>
struct Vec {
  static constexpr int n = BF16 ? 8 : 4;
  static constexpr int bytes = BF16 ? 2 : 4;  // of one value
  static __device__ __forceinline__ void unpack(const uint4& u, float* f) {
    if constexpr (BF16) {
      f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x); f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
      f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z); f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
    } else {
      f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
      f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
    }
  }
  // Rounds to the input type (to nearest even), once, at the store.
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint4 u;
    if constexpr (BF16) {
      u.x = two(f[0], f[1]); u.y = two(f[2], f[3]); u.z = two(f[4], f[5]); u.w = two(f[6], f[7]);
    } else {
      u.x = __float_as_uint(f[0]); u.y = __float_as_uint(f[1]);
      u.z = __float_as_uint(f[2]); u.w = __float_as_uint(f[3]);
    }
    return u;
  }
  static __device__ __forceinline__ uint32_t two(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
};

// 4 values of the input type: 8 bytes of bf16 or 16 of fp32, as two fp32 pairs.
template <bool BF16>
struct Quad {
  using Raw = uint4;
  static __device__ __forceinline__ void unpack(const Raw& u, float2* f) {
    f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ Raw pack(const float2* f) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
  }
  static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
};
template <>
struct Quad<true> {
  using Raw = uint2;
  static __device__ __forceinline__ void unpack(const Raw& u, float2* f) {
    f[0] = make_float2(bf16_lo(u.x), bf16_hi(u.x));
    f[1] = make_float2(bf16_lo(u.y), bf16_hi(u.y));
  }
  static __device__ __forceinline__ Raw pack(const float2* f) {
    return make_uint2(Vec<true>::two(f[0].x, f[0].y), Vec<true>::two(f[1].x, f[1].y));
  }
  static __device__ __forceinline__ Raw zero() { return make_uint2(0, 0); }
};

__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// The same, or 16 bytes of zeros where `in` is false (src is then not read).
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// NS = 2 or 4 floats: an asynchronous copy of them, and plain loads and stores.
template <int NS>
__device__ __forceinline__ void cp_async_states(void* dst, const float* src) {
  if constexpr (NS == 4) cp_async16(dst, src);
  else cp_async8(dst, src);
}
template <int NS>
__device__ __forceinline__ void load_own(float* f, const unsigned char* p) {
  if constexpr (NS == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(p);
    f[0] = v.x; f[1] = v.y;
  }
}
template <int NS>
__device__ __forceinline__ void store_own(unsigned char* p, const float* f) {
  if constexpr (NS == 4) *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  else *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
}
// A lane's states after `count` segments: h <- exp(-A dt) h + state, over the segments'
// summaries from `state` (its first channel; N apart per channel) and `dt` on, `step`
// segments apart (1 or -1). C channels, NS states. 4 segments' loads go out together.
template <int C, int NS>
__device__ __forceinline__ void fold_segments(float2 (*h)[NS], const float2 (*A2)[NS], const float* state,
                                              const float* dt, int count, int step, int D, int N) {
  const long long ss = (long long)step * D * N, sd = (long long)step * D;
  for (int k0 = 0; k0 < count; k0 += 4) {
    float q[4][C][NS], d[4][C];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k0 + k < count) {
        load_own<C>(d[k], reinterpret_cast<const unsigned char*>(dt + k * sd));
#pragma unroll
        for (int c = 0; c < C; ++c)
          load_own<NS>(q[k][c], reinterpret_cast<const unsigned char*>(state + k * ss + c * N));
      }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k0 + k < count)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            float& x = c & 1 ? h[c / 2][j].y : h[c / 2][j].x;
            x = fmaf(ex2_approx(d[k][c] * (c & 1 ? A2[c / 2][j].y : A2[c / 2][j].x)), x, q[k][c][j]);
          }
    state += 4 * ss;
    dt += 4 * sd;
  }
}
// A CTA of one warp needs no barrier.
template <int W>
__device__ __forceinline__ void cta_sync() {
  if constexpr (W == 1) __syncwarp();
  else __syncthreads();
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

constexpr float kLog2e = 1.4426950408889634f;

// Exponents A2 s of two decays 2^(A2 s). The SFU's 2^x comes out low, by 1.9e-8
// relative on average over [-0.1, -0.001] (measured; its largest error there is
// 1.2e-7), and a state of a long memory would gather that mean over every token it
// remembers: 2e-6 over 100 tokens. The addend takes the mean out; what is left is
// random and grows with the root of the tokens. The decay of a step of size 0 stays
// exactly 1 (2^2.7e-8 rounds to it).
constexpr float kDecayShift = 2.7e-8f;
__device__ __forceinline__ float2 decay_exponent(float2 s, float2 A2) {
  return __ffma2_rn(s, A2, make_float2(kDecayShift, kDecayShift));
}
// A as the decay exponents take it. (A above 2.3e38 would overflow, and a step of size 0
// would make a NaN of it.)
__device__ __forceinline__ float decay_rate(float A) { return fmaxf(-kLog2e * A, -3.0e38f); }
// The larger value, or NaN when one is (fmaxf drops it).
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// sigmoid(u) and u sigmoid(u) with the SFU's 2^x and reciprocal (a few ulp). Their
// flushes to zero do no harm: e^-u below 1e-38 next to 1, and 1 / (1 + e^-u) below it.
// e^-u overflows to infinity for very negative u, where the reciprocal is 0.
__device__ __forceinline__ float sigmoid_fast(float u) { return rcp_approx(1.f + ex2_approx(-kLog2e * u)); }
__device__ __forceinline__ float silu_fast(float u) { return u * sigmoid_fast(u); }
__device__ __forceinline__ float2 silu_fast(float2 u) {
  const float2 x = __fmul2_rn(u, make_float2(-kLog2e, -kLog2e));
  const float2 w = __fadd2_rn(make_float2(ex2_approx(x.x), ex2_approx(x.y)), make_float2(1.f, 1.f));
  return __fmul2_rn(u, make_float2(rcp_approx(w.x), rcp_approx(w.y)));
}

// softplus(u) = max(u, 0) + log(1 + e), e = e^-|u|. The step sizes of a trained scan
// are small (0.001 to 0.1, u from -7 to -2), where log(1 + e) has to be accurate
// relative to itself, which the SFU's logarithm near 1 is not. So
// log(1 + e) = 2 atanh(r), r = e / (2 + e) <= 1/3, by the series of atanh in r^2 up to
// r^13: what is left out is below 2e-8 of the sum (r^14 / 15 and on at r = 1/3). The
// SFU's 2^x flushes results below 1e-38 to zero, so e is the square of e^-(|u|/2), which
// costs nothing: halving is exact, and the exponent is rounded at its own size (with 64 added
// to it, to stay clear of the flush, it was rounded at 64's). s is off, relative, by 1.8e-7
// in root mean square and 6.3e-7 at most over u in [-10, -2] (7.6e-7 in the mean with the
// shift); at -80 by 4e-6, since e^u passes on u's rounding times u.
__device__ __forceinline__ float2 softplus_fast(float2 u) {
  const float2 x = __fmul2_rn(make_float2(fabsf(u.x), fabsf(u.y)), make_float2(-0.5f * kLog2e, -0.5f * kLog2e));
  const float2 q0 = make_float2(ex2_approx(x.x), ex2_approx(x.y)), e = __fmul2_rn(q0, q0);
  const float2 w = __fadd2_rn(e, make_float2(2.f, 2.f));
  const float2 r = __fmul2_rn(e, make_float2(rcp_approx(w.x), rcp_approx(w.y))), q = __fmul2_rn(r, r);
  float2 p = make_float2(1.f / 13.f, 1.f / 13.f);
  p = __ffma2_rn(p, q, make_float2(1.f / 11.f, 1.f / 11.f));
  p = __ffma2_rn(p, q, make_float2(1.f / 9.f, 1.f / 9.f));
  p = __ffma2_rn(p, q, make_float2(1.f / 7.f, 1.f / 7.f));
  p = __ffma2_rn(p, q, make_float2(1.f / 5.f, 1.f / 5.f));
  p = __ffma2_rn(p, q, make_float2(1.f / 3.f, 1.f / 3.f));
  p = __ffma2_rn(p, q, make_float2(1.f, 1.f));
  return __ffma2_rn(__fadd2_rn(r, r), p, make_float2(fmaxf(u.x, 0.f), fmaxf(u.y, 0.f)));
}
__device__ __forceinline__ float softplus_fast(float u) { return softplus_fast(make_float2(u, u)).x; }

#endif  // __CUDACC__

}  // namespace palimpsa
