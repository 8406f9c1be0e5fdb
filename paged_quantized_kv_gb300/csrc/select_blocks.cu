// select_blocks.cu -- the blocks of the context that each query row attends
// to: some always (the first ones, the last ones), then those of the best
// scores, sm_103a.
//
// A row that sees `seen` tokens has nb = ceil(seen / sel) blocks and takes k
// = min(top, nb) of them.  Scores become 32-bit keys in their order; the k-th
// largest key is found 8 bits at a time from a histogram of the keys that
// agree so far, and one pass in the order of the blocks writes those above it
// and the first ones equal to it, so that the list rises and ties go to the
// lowest index.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;

// Larger keys for larger scores; NaN as -inf, -0 as 0; ~0 for a block that is
// always taken.
__device__ __forceinline__ uint32_t key_of(float x, bool always) {
  if (always) return ~0u;
  x = x == x ? x + 0.0f : -INFINITY;
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) != 0u ? ~0u : 0x80000000u);
}

__global__ void __launch_bounds__(kThreads)
    select_kernel(const SelectParams p) {
  pdl_prologue();
  __shared__ int hist[256], scan[kThreads / 32], found[2];
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const dev::QueryRow r = dev::query_row(p.rows, row);
  if (row == 0) dev::check_rows(p.rows, tid, kThreads);
  if (r.seq < 0) return;
  const int nb = (r.seen + p.sel - 1) / p.sel;
  const int k = min(p.top, nb);
  const float* x = p.scores + row * p.scores_stride0;
  int32_t* out = p.selected + row * p.selected_stride0;
  for (int i = k + tid; i < p.top; i += kThreads) out[i] = -1;
  if (k == nb) {
    for (int i = tid; i < k; i += kThreads) out[i] = i;
    return;
  }
  auto key = [&](int j) {
    return key_of(x[j], j < p.first || j >= nb - p.last);
  };
  uint32_t prefix = 0;
  int need = k;  // of the keys that agree with prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    for (int j = tid; j < nb; j += kThreads) {
      const uint32_t u = key(j);
      if (shift == 24 || (u >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(u >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid < 32) {
      // lane l: bins 255 - 8 l down to 248 - 8 l
      int sum = 0;
      for (int i = 0; i < 8; ++i) sum += hist[255 - 8 * lane - i];
      int incl = sum;
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(~0u, incl, d);
        if (lane >= d) incl += y;
      }
      if (incl - sum < need && incl >= need) {
        int before = incl - sum, bin = 255 - 8 * lane;
        while (before + hist[bin] < need) before += hist[bin--];
        found[0] = bin;
        found[1] = need - before;
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(found[0]) << shift;
    need = found[1];
    __syncthreads();
  }
  // those above the k-th key, and the first `need` equal to it
  int written = 0, equal = 0;
  for (int j0 = 0; j0 < nb && written < k; j0 += kThreads) {
    const int j = j0 + tid;
    const uint32_t u = j < nb ? key(j) : 0u;
    const bool above = j < nb && u > prefix, same = j < nb && u == prefix;
    const uint32_t above_bits = __ballot_sync(~0u, above);
    const uint32_t same_bits = __ballot_sync(~0u, same);
    if (lane == 0)
      scan[tid >> 5] = __popc(above_bits) | __popc(same_bits) << 16;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < (tid >> 5)) before += scan[w];
      all += scan[w];
    }
    const uint32_t lower = (1u << lane) - 1u;
    const int above_at = (before & 0xFFFF) + __popc(above_bits & lower);
    const int same_at = equal + (before >> 16) + __popc(same_bits & lower);
    if (above || (same && same_at < need))
      out[written + above_at + min(same_at, need) - min(equal, need)] = j;
    written += (all & 0xFFFF) + min(equal + (all >> 16), need) -
               min(equal, need);
    equal += all >> 16;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_select_blocks(const SelectParams& p, cudaStream_t stream) {
  return launch_kernel(select_kernel, dim3(static_cast<unsigned>(p.rows.total)),
                       kThreads, 0, stream, p.pdl, p);
}

}  // namespace kvq
