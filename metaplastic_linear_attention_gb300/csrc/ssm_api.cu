// C ABI of the causal convolution and the selective scan: argument validation and
// dispatch to their launchers. Declared in palimpsa.h.
#include "palimpsa.h"
#include "ssm.cuh"

namespace palimpsa {

// api.cu: the device's status word, and scratch from the library's pool (freed with cudaFreeAsync).
palimpsa_status device_status_word(unsigned int** out);
cudaError_t acquire_scratch(size_t bytes, cudaStream_t s, float** p);

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool dtype_ok(palimpsa_dtype t) { return t == PALIMPSA_F32 || t == PALIMPSA_BF16; }

// Sizes of a batch: rows of D channels in n_seq sequences, dense or packed.
// (D up to 2^24 keeps a row's offsets in int, its groups' states among them.)
bool rows_ok(const SeqRows& r, int D) {
  // (T leaves room for the rounding up to whole runs and segments in int)
  if (r.n_seq < 1 || r.T < 0 || r.T > 0x7fff0000 || D < 1 || D > 1 << 24) return false;
  if (r.cu && (r.max_len < 0 || r.max_len > r.T)) return false;
  const long long rows = r.cu ? r.T : (long long)r.n_seq * r.T;
  const long long lim = 1LL << 40;
  return rows <= lim / D && (long long)r.n_seq <= lim / D / 256;
}

// A row stride: 0 means dense (`width`); otherwise at least width, and a whole number
// of 16-byte vectors. palimpsa_status of the refusal, or OK with *ld set.
palimpsa_status stride_of(long long given, long long width, palimpsa_dtype t, long long* ld) {
  if (given != 0 && (given < width || given > (1LL << 31))) return PALIMPSA_ERR_SHAPE;
  *ld = given ? given : width;
  return *ld * (t == PALIMPSA_BF16 ? 2 : 4) % 16 ? PALIMPSA_ERR_ALIGN : PALIMPSA_OK;
}

SeqRows rows_of(const int* cu, int n_seq, int T, int max_seqlen) {
  SeqRows r;
  r.cu = cu;
  r.n_seq = n_seq;
  r.T = T;
  r.max_len = cu ? max_seqlen : T;
  return r;
}

template <int NA, int NB>
palimpsa_status aligned_all(const void* const (&a16)[NA], const void* const (&a4)[NB]) {
  for (const void* p : a16)
    if (p && !aligned(p, 16)) return PALIMPSA_ERR_ALIGN;
  for (const void* p : a4)
    if (p && !aligned(p, 4)) return PALIMPSA_ERR_ALIGN;
  return PALIMPSA_OK;
}

palimpsa_status conv_checks(const ConvArgs& a, palimpsa_dtype t, unsigned int flags) {
  if (!dtype_ok(t)) return PALIMPSA_ERR_DTYPE;
  if (flags & ~(unsigned)PALIMPSA_CONV_SILU) return PALIMPSA_ERR_UNSUPPORTED;
  if (!rows_ok(a.rows, a.D)) return PALIMPSA_ERR_SHAPE;
  if (a.W < 2 || a.W > 4 || a.D % 8) return PALIMPSA_ERR_UNSUPPORTED;
  return aligned_all({a.x, a.state0, a.y, a.state_T, a.dy, a.dstate_T, a.dx, a.dstate0},
                     {a.weight, a.bias, a.rows.cu, a.dweight, a.dbias});
}

palimpsa_status scan_checks(const ScanArgs& a, palimpsa_dtype t, unsigned int flags) {
  if (!dtype_ok(t)) return PALIMPSA_ERR_DTYPE;
  if (flags & ~(unsigned)PALIMPSA_SCAN_SOFTPLUS) return PALIMPSA_ERR_UNSUPPORTED;
  if (!rows_ok(a.rows, a.D) || a.G < 1 || a.N < 1) return PALIMPSA_ERR_SHAPE;
  if (a.N != 8 && a.N != 16 && a.N != 32 && a.N != 64 && a.N != 128) return PALIMPSA_ERR_UNSUPPORTED;
  if (a.D % a.G || a.D / a.G % 8) return PALIMPSA_ERR_UNSUPPORTED;
  return aligned_all({a.x, a.dt, a.B, a.C, a.z, a.A, a.h0, a.y, a.h_T, a.ckpt, a.ckpt_in, a.dy, a.dh_T, a.dx, a.ddt, a.dz,
                      a.dB, a.dC, a.dh0},
                     {a.skip, a.dt_bias, a.rows.cu, a.dA, a.dskip, a.ddt_bias});
}

palimpsa_status scan_strides(ScanArgs* a, const palimpsa_scan_strides* st, palimpsa_dtype t) {
  const palimpsa_scan_strides dense = {};
  if (!st) st = &dense;
  const long long bc = (long long)a->G * a->N;
  palimpsa_status s = stride_of(st->x, a->D, t, &a->x_ld);
  if (!s) s = stride_of(st->dt, a->D, t, &a->dt_ld);
  if (!s) s = stride_of(st->B, bc, t, &a->B_ld);
  if (!s) s = stride_of(st->C, bc, t, &a->C_ld);
  if (!s) s = stride_of(st->z, a->D, t, &a->z_ld);
  if (!s) s = stride_of(st->dy, a->D, t, &a->dy_ld);
  return s;
}

ScanArgs scan_args(const void* x, const void* dt, const float* A, const void* B, const void* C, const float* skip,
                   const void* z, const float* dt_bias, const float* h0, int D, int G, int N, unsigned int flags,
                   palimpsa_dtype t) {
  ScanArgs a{};
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.B = B;
  a.C = C;
  a.skip = skip;
  a.z = z;
  a.dt_bias = dt_bias;
  a.h0 = h0;
  a.D = D;
  a.G = G;
  a.N = N;
  a.softplus = (flags & PALIMPSA_SCAN_SOFTPLUS) != 0;
  a.bf16 = t == PALIMPSA_BF16;
  return a;
}

// Scratch for a scan, `more` floats of it for the caller: the segments' states and step
// sums, and, if the slots are to lie close, the slots' starts, which are filled in here.
cudaError_t take_scratch(ScanArgs* a, size_t more, bool backward, bool close, cudaStream_t s, float** scratch) {
  *scratch = nullptr;
  const size_t split = (scan_scratch_floats(*a) + 3) / 4 * 4, n = a->rows.n_seq + 1ull;
  const size_t ints = close ? (backward ? 2 * n : n) : 0;
  if (split + more + ints == 0) return cudaSuccess;
  cudaError_t e = acquire_scratch((split + more + ints) * sizeof(float), s, scratch);
  if (e != cudaSuccess) {
    *scratch = nullptr;
    return e;
  }
  if (a->nseg > 1) {
    a->seg_state = *scratch + more;
    a->seg_dt = a->seg_state + (size_t)a->slots.count * a->D * a->N;
  }
  if (close) {
    int* const starts = reinterpret_cast<int*>(*scratch + more + split);
    int* const row_starts = backward ? starts + n : nullptr;
    a->slots.starts = starts;
    a->row_slots.starts = row_starts;
    a->row_slots.count = a->rows.T;
    return launch_slot_starts(a->rows, a->seg_len, starts, row_starts, a->status, s);
  }
  return cudaSuccess;
}

palimpsa_status release(cudaError_t e, float* scratch, cudaStream_t s) {
  const cudaError_t e2 = scratch ? cudaFreeAsync(scratch, s) : cudaSuccess;
  return e == cudaSuccess && e2 == cudaSuccess ? PALIMPSA_OK : PALIMPSA_ERR_CUDA;
}

}  // namespace
}  // namespace palimpsa

using namespace palimpsa;

extern "C" {

palimpsa_status palimpsa_causal_conv(const void* x, long long x_stride, const float* weight, const float* bias,
                                     const void* state0, void* y, void* state_T, const int* cu_seqlens, int B, int T,
                                     int max_seqlen, int D, int W, unsigned int flags, palimpsa_dtype in_dtype,
                                     void* cuda_stream) {
  if (!weight || (T != 0 && (!x || !y))) return PALIMPSA_ERR_NULL;
  ConvArgs a{};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.state0 = state0;
  a.y = y;
  a.state_T = state_T;
  a.rows = rows_of(cu_seqlens, B, T, max_seqlen);
  a.D = D;
  a.W = W;
  a.silu = (flags & PALIMPSA_CONV_SILU) != 0;
  a.bf16 = in_dtype == PALIMPSA_BF16;
  if (palimpsa_status s = conv_checks(a, in_dtype, flags)) return s;
  if (palimpsa_status s = stride_of(x_stride, D, in_dtype, &a.x_ld)) return s;
  if (palimpsa_status s = device_status_word(&a.status)) return s;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  float* scratch = nullptr;
  const size_t bytes = plan_conv(&a, false);
  if (bytes && acquire_scratch(bytes, s, &scratch) != cudaSuccess) return PALIMPSA_ERR_CUDA;
  return release(launch_conv_forward(a, scratch, s), scratch, s);
}

palimpsa_status palimpsa_zero_rows_outside(void* const* arrays, const long long* row_bytes, int n,
                                           const int* cu_seqlens, int B, int T, int max_seqlen, void* cuda_stream) {
  return palimpsa_zero_unwritten(arrays, row_bytes, n, nullptr, nullptr, 0, cu_seqlens, B, T, max_seqlen, cuda_stream);
}

palimpsa_status palimpsa_zero_unwritten(void* const* arrays, const long long* row_bytes, int n, void* const* states,
                                        const long long* state_bytes, int n_states, const int* cu_seqlens, int B, int T,
                                        int max_seqlen, void* cuda_stream) {
  if (!cu_seqlens || (n > 0 && (!arrays || !row_bytes)) || (n_states > 0 && (!states || !state_bytes)))
    return PALIMPSA_ERR_NULL;
  if (n < 0 || n_states < 0 || n > kZeroArrays || n_states > kZeroArrays - n) return PALIMPSA_ERR_SHAPE;
  if (B < 1 || T < 0 || max_seqlen < 0 || max_seqlen > T) return PALIMPSA_ERR_SHAPE;
  if (!aligned(cu_seqlens, 4)) return PALIMPSA_ERR_ALIGN;
  ZeroArgs a{};
  a.rows = rows_of(cu_seqlens, B, T, max_seqlen);
  a.row_arrays = T > 0 ? n : 0;
  int k = 0;
  auto add = [&](void* p, long long bytes, int entries) {
    if (!p && entries != 0) return PALIMPSA_ERR_NULL;
    if (bytes < 0 || bytes > (1LL << 40) / (entries > 0 ? entries : 1)) return PALIMPSA_ERR_SHAPE;
    if (!aligned(p, 16) || bytes % 16) return PALIMPSA_ERR_ALIGN;
    if (entries > 0) {
      a.p[k] = p;
      a.width[k++] = bytes;
    }
    return PALIMPSA_OK;
  };
  for (int i = 0; i < n; ++i)
    if (const palimpsa_status s = add(arrays[i], row_bytes[i], T)) return s;
  for (int i = 0; i < n_states; ++i)
    if (const palimpsa_status s = add(states[i], state_bytes[i], B)) return s;
  return launch_zero_outside(a, k, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? PALIMPSA_OK
                                                                                        : PALIMPSA_ERR_CUDA;
}

palimpsa_status palimpsa_causal_conv_step(const void* x, long long x_stride, const float* weight, const float* bias,
                                          void* state, void* y, int B, int D, int W, unsigned int flags,
                                          palimpsa_dtype in_dtype, void* cuda_stream) {
  if (!x || !weight || !state || !y) return PALIMPSA_ERR_NULL;
  ConvArgs a{};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.state_T = state;
  a.rows = rows_of(nullptr, B, 1, 1);
  a.D = D;
  a.W = W;
  a.silu = (flags & PALIMPSA_CONV_SILU) != 0;
  a.bf16 = in_dtype == PALIMPSA_BF16;
  if (palimpsa_status s = conv_checks(a, in_dtype, flags)) return s;
  if (palimpsa_status s = stride_of(x_stride, D, in_dtype, &a.x_ld)) return s;
  return launch_conv_step(a, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? PALIMPSA_OK
                                                                                  : PALIMPSA_ERR_CUDA;
}

palimpsa_status palimpsa_causal_conv_backward(const void* x, long long x_stride, const float* weight,
                                              const float* bias, const void* state0, const void* dy,
                                              long long dy_stride, const void* dstate_T, void* dx, float* dweight,
                                              float* dbias, void* dstate0, const int* cu_seqlens, int B, int T,
                                              int max_seqlen, int D, int W, unsigned int flags,
                                              palimpsa_dtype in_dtype, void* cuda_stream) {
  if (!weight || !dweight || (T != 0 && (!x || !dy || !dx))) return PALIMPSA_ERR_NULL;
  ConvArgs a{};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.state0 = state0;
  a.dy = dy;
  a.dstate_T = dstate_T;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.dstate0 = dstate0;
  a.rows = rows_of(cu_seqlens, B, T, max_seqlen);
  a.D = D;
  a.W = W;
  a.silu = (flags & PALIMPSA_CONV_SILU) != 0;
  a.bf16 = in_dtype == PALIMPSA_BF16;
  if (palimpsa_status s = conv_checks(a, in_dtype, flags)) return s;
  if (palimpsa_status s = stride_of(x_stride, D, in_dtype, &a.x_ld)) return s;
  if (palimpsa_status s = stride_of(dy_stride, D, in_dtype, &a.dy_ld)) return s;
  if (palimpsa_status s = device_status_word(&a.status)) return s;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  float* scratch = nullptr;
  if (acquire_scratch(plan_conv(&a, true), s, &scratch) != cudaSuccess) return PALIMPSA_ERR_CUDA;
  return release(launch_conv_backward(a, scratch, s), scratch, s);
}

size_t palimpsa_selective_scan_checkpoint_bytes(int B, int T, int packed, int D, int N) {
  if (B < 1 || T < 0 || D < 1 || N < 1) return 0;
  static const int some = 0;
  return (size_t)scan_ckpt_rows(rows_of(packed ? &some : nullptr, B, T, T)) * D * N * sizeof(float);
}

palimpsa_status palimpsa_selective_scan(const void* x, const void* dt, const float* A, const void* B_t,
                                        const void* C_t, const float* skip, const void* z, const float* dt_bias,
                                        const float* h0, void* y, float* h_T, float* ckpt,
                                        const palimpsa_scan_strides* strides, const int* cu_seqlens, int B, int T,
                                        int max_seqlen, int D, int G, int N, unsigned int flags,
                                        palimpsa_dtype in_dtype, void* cuda_stream) {
  if (!A || !h_T || (T != 0 && (!x || !dt || !B_t || !C_t || !y))) return PALIMPSA_ERR_NULL;
  ScanArgs a = scan_args(x, dt, A, B_t, C_t, skip, z, dt_bias, h0, D, G, N, flags, in_dtype);
  a.y = y;
  a.h_T = h_T;
  a.ckpt = ckpt;
  a.rows = rows_of(cu_seqlens, B, T, max_seqlen);
  if (palimpsa_status s = scan_checks(a, in_dtype, flags)) return s;
  if (palimpsa_status s = scan_strides(&a, strides, in_dtype)) return s;
  if (palimpsa_status s = device_status_word(&a.status)) return s;
  bool close;
  if (plan_scan(&a, false, &close) != cudaSuccess) return PALIMPSA_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  float* scratch = nullptr;
  cudaError_t e = take_scratch(&a, 0, false, close, s, &scratch);
  if (e == cudaSuccess) e = launch_scan_forward(a, s);
  return release(e, scratch, s);
}

palimpsa_status palimpsa_selective_scan_step(const void* x, const void* dt, const float* A, const void* B_t,
                                             const void* C_t, const float* skip, const void* z, const float* dt_bias,
                                             float* h, void* y, const palimpsa_scan_strides* strides, int B, int D,
                                             int G, int N, unsigned int flags, palimpsa_dtype in_dtype,
                                             void* cuda_stream) {
  if (!x || !dt || !A || !B_t || !C_t || !h || !y) return PALIMPSA_ERR_NULL;
  ScanArgs a = scan_args(x, dt, A, B_t, C_t, skip, z, dt_bias, nullptr, D, G, N, flags, in_dtype);
  a.y = y;
  a.h_T = h;
  a.rows = rows_of(nullptr, B, 1, 1);
  if (palimpsa_status s = scan_checks(a, in_dtype, flags)) return s;
  if (palimpsa_status s = scan_strides(&a, strides, in_dtype)) return s;
  if (palimpsa_status s = device_status_word(&a.status)) return s;
  return launch_scan_step(a, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? PALIMPSA_OK
                                                                                  : PALIMPSA_ERR_CUDA;
}

palimpsa_status palimpsa_selective_scan_backward(
    const void* x, const void* dt, const float* A, const void* B_t, const void* C_t, const float* skip, const void* z,
    const float* dt_bias, const float* ckpt, const void* dy, const float* dh_T, void* dx, void* ddt, float* dA, void* dB,
    void* dC, float* dskip, void* dz, float* ddt_bias, float* dh0, const palimpsa_scan_strides* strides,
    const int* cu_seqlens, int B, int T, int max_seqlen, int D, int G, int N, unsigned int flags,
    palimpsa_dtype in_dtype, void* cuda_stream) {
  if (!A || !dA || (T != 0 && (!x || !dt || !B_t || !C_t || !ckpt || !dy || !dx || !ddt || !dB || !dC)))
    return PALIMPSA_ERR_NULL;
  if (z && T != 0 && !dz) return PALIMPSA_ERR_NULL;
  ScanArgs a = scan_args(x, dt, A, B_t, C_t, skip, z, dt_bias, nullptr, D, G, N, flags, in_dtype);
  a.ckpt_in = ckpt;
  a.dy = dy;
  a.dh_T = dh_T;
  a.dx = dx;
  a.ddt = ddt;
  a.dz = dz;
  a.dB = dB;
  a.dC = dC;
  a.dA = dA;
  a.dskip = dskip;
  a.ddt_bias = ddt_bias;
  a.dh0 = dh0;
  a.rows = rows_of(cu_seqlens, B, T, max_seqlen);
  if (palimpsa_status s = scan_checks(a, in_dtype, flags)) return s;
  if (palimpsa_status s = scan_strides(&a, strides, in_dtype)) return s;
  if (palimpsa_status s = device_status_word(&a.status)) return s;
  bool close;
  if (plan_scan(&a, true, &close) != cudaSuccess) return PALIMPSA_ERR_CUDA;
  a.row_slots = slots_of(a.rows, 1);
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  float* scratch = nullptr;
  const size_t more = (scan_backward_scratch_floats(a) + 3) / 4 * 4;
  cudaError_t e = take_scratch(&a, more, true, close, s, &scratch);
  if (e == cudaSuccess) e = launch_scan_backward(a, scratch, s);
  return release(e, scratch, s);
}

}  // extern "C"
