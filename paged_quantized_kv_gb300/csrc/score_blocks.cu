// score_blocks.cu -- the indexer's score of every block of the context for
// every query row, over the paged e4m3 cache, sm_103a.
//
// For a query row and a token t that it sees, s_t = scale_t * sum over heads
// of w_h relu(q_h . k_t); a block's score is the largest of its tokens'.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 128;  // tokens of a thread block

__device__ __forceinline__ float2 widen(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
      : "=r"(h)
      : "h"(static_cast<uint16_t>(pair)));
  float2 f;
  asm("{ .reg .f16 a, b;\n"
      "  mov.b32 {a, b}, %2;\n"
      "  cvt.f32.f16 %0, a;\n"
      "  cvt.f32.f16 %1, b; }"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// One query row and 128 tokens, a thread for each.
__global__ void __launch_bounds__(kThreads)
    score_kernel(const ScoreParams p) {
  pdl_prologue();
  __shared__ float q[128], best[kThreads];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const dev::QueryRow r = dev::query_row(p.rows, static_cast<int>(row));
  if (row == 0 && blockIdx.y == 0) dev::check_rows(p.rows, tid, kThreads);
  if (r.seq < 0) return;
  const int t = blockIdx.y * kThreads + tid;
  const uint8_t* key = nullptr;
  float scale = 0.0f;
  if (t < r.seen) {
    const int page = t / p.B, off = t - page * p.B;
    const int32_t blk = __ldg(p.block_table + r.seq * p.bt_stride + page);
    if (blk < 0 || blk >= p.num_blocks) {
      if (p.rows.dev_error != nullptr)
        atomicOr(p.rows.dev_error, KVQ_DEVERR_BLOCK);
    } else {
      const uint8_t* base = p.cache + blk * p.block_stride;
      key = base + off * p.D;
      scale = *reinterpret_cast<const float*>(
          base + static_cast<int64_t>(p.B) * p.D + 4 * off);
    }
  }
  float sum = 0.0f;
  for (int h = 0; h < p.heads; ++h) {
    __syncthreads();
    if (tid < p.D / 2) {
      const uint16_t pair = *reinterpret_cast<const uint16_t*>(
          p.q + row * p.q_stride0 + h * p.D + 2 * tid);
      const float2 f = widen(pair);
      q[2 * tid] = f.x;
      q[2 * tid + 1] = f.y;
    }
    __syncthreads();
    if (key == nullptr) continue;
    float x = 0.0f;
    for (int d = 0; d < p.D; d += 4) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(key + d);
      const float2 a = widen(w & 0xFFFFu), b = widen(w >> 16);
      x += a.x * q[d] + a.y * q[d + 1] + b.x * q[d + 2] + b.y * q[d + 3];
    }
    x = x < 0.0f ? 0.0f : x;  // (NaN stays)
    sum += __ldg(p.weights + row * p.w_stride0 + h) * x;
  }
  sum *= scale;
  best[tid] = key != nullptr && sum == sum ? sum : -INFINITY;
  __syncthreads();
  if (tid < kThreads / p.sel) {
    float top = -INFINITY;
    for (int i = 0; i < p.sel; ++i) top = fmaxf(top, best[tid * p.sel + i]);
    const int column = blockIdx.y * (kThreads / p.sel) + tid;
    if (column < p.columns) p.scores[row * p.scores_stride0 + column] = top;
  }
}

}  // namespace

cudaError_t launch_score_blocks(const ScoreParams& p, cudaStream_t stream) {
  const unsigned tiles = static_cast<unsigned>(
      (static_cast<int64_t>(p.columns) * p.sel + kThreads - 1) / kThreads);
  return launch_kernel(score_kernel,
                       dim3(static_cast<unsigned>(p.rows.total), tiles), kThreads,
                       0, stream, p.pdl, p);
}

}  // namespace kvq
