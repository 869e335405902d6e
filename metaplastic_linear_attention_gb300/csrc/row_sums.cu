// Sums over the rows of [rows, V, D], the parts that a backward's CTAs leave of the gradients
// of its V parameter vectors: out[v][d] = sum over rows of parts[row, v, d].
//
// A thread takes 4 columns of one row in 64 (8 slices of a CTA, up to 8 CTAs of a cluster, which
// adds up through shared memory), always the same, so the bits are the same every time. It is a few
// MB at most: 760 rows of 2 x 1536 add 6 us to the layer norm's backward.
#include <algorithm>
#include <cooperative_groups.h>

#include "ssm.cuh"

namespace palimpsa {
namespace {

constexpr int kSlices = 8, kRanks = 8;

struct RowSums {
  const float* parts;
  float* out[3];
  long long rows;
  int V, D, ranks;
};

__global__ void __launch_bounds__(32 * kSlices) palimpsa_row_sums_kernel(RowSums a) {
  namespace cg = cooperative_groups;
  __shared__ float4 red[kSlices][32], ranks[kRanks][32];
  const int lane = threadIdx.x % 32, slice = threadIdx.x / 32, v = blockIdx.y;
  const int rank = blockIdx.x % a.ranks, col = (int)(blockIdx.x / a.ranks) * 128 + lane * 4;
  const cg::cluster_group cluster = cg::this_cluster();
  // Launched ahead of the end of the kernel that leaves the parts.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.ranks > 1) cluster.sync();  // every CTA has started: its shared memory may be written
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& e) {
    s.x += e.x; s.y += e.y; s.z += e.z; s.w += e.w;
  };
  if (col < a.D) {
    const float* p = a.parts + (size_t)v * a.D + col;
#pragma unroll 8
    for (long long r = rank * kSlices + slice; r < a.rows; r += a.ranks * kSlices)
      add(*reinterpret_cast<const float4*>(p + r * a.V * a.D));
  }
  red[slice][lane] = s;
  __syncthreads();
  if (slice == 0) {
    for (int k = 1; k < kSlices; ++k) add(red[k][lane]);
    if (a.ranks > 1) *cluster.map_shared_rank(&ranks[rank][lane], 0) = s;
  }
  if (a.ranks > 1) {
    cluster.sync();
    if (rank > 0 || slice > 0) return;
    s = ranks[0][lane];
    for (int k = 1; k < a.ranks; ++k) add(ranks[k][lane]);
  }
  float* const out = v == 0 ? a.out[0] : v == 1 ? a.out[1] : a.out[2];
  if (slice == 0 && col < a.D && out) {  // (aligned to 4 bytes)
    out[col] = s.x; out[col + 1] = s.y; out[col + 2] = s.z; out[col + 3] = s.w;
  }
}

}  // namespace

cudaError_t launch_row_sums(const float* parts, long long rows, int V, int D, float* const* out, cudaStream_t s) {
  RowSums a{parts, {out[0], out[1], V > 2 ? out[2] : nullptr}, rows, V, D, 1};
  while (a.ranks < kRanks && rows > 4ll * a.ranks * kSlices) a.ranks *= 2;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)((D + 127) / 128 * a.ranks), V);
  c.blockDim = dim3(32 * kSlices);
  c.stream = s;
  c.attrs = attr;
  c.numAttrs = a.ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&c, palimpsa_row_sums_kernel, a);
}

}  // namespace palimpsa
