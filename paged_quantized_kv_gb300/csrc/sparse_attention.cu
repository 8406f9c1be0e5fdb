// sparse_attention.cu -- attention of each query row over the blocks of its
// sequence's context that a list selects, over the NVFP4 pages, sm_103a.
//
// A list rises, so that only its last block can hold tokens behind the row:
// the tokens that a row sees are the first ones of the pages of its blocks,
// in order, and the row is a sequence of one query token over a block table
// of its own.  A first kernel writes that table and length for every row,
// the decode kernel does the rest.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kvq.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kPlanThreads = 128;  // a warp for each row
constexpr int kPart = 512;         // partition of the decode scratch
constexpr int kD = 128;

// The rows from p.row0 on: their tables and lengths (-1: not a row).
__global__ void __launch_bounds__(kPlanThreads)
    plan_rows_kernel(const SparseParams p) {
  pdl_prologue();
  const int i = blockIdx.x * (kPlanThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (p.row0 == 0 && blockIdx.x == 0)
    dev::check_rows(p.rows, threadIdx.x, kPlanThreads);
  if (i >= p.num_rows) return;
  const int64_t row = p.row0 + i;
  const dev::QueryRow r = dev::query_row(p.rows, static_cast<int>(row));
  if (r.seq < 0) {
    if (lane == 0) p.row_lens[i] = -1;
    return;
  }
  const ChunkParams& c = p.chunk;
  const int per = p.sel / c.B;  // pages of a block
  const int blocks = (r.seen + p.sel - 1) / p.sel;
  const int32_t* list = p.selected + row * p.selected_stride0;
  const int32_t* table = c.block_table + r.seq * c.bt_stride;
  int32_t* out = p.row_table + static_cast<int64_t>(i) * p.top * per;
  int taken = 0, last = -1;  // (the largest entry so far)
  bool bad = false;
  for (int j0 = 0; j0 < p.top; j0 += 32) {
    const int e = j0 + lane < p.top ? __ldg(list + j0 + lane) : -1;
    const bool in = e >= 0 && e < blocks;
    int most = in ? e : -1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(~0u, most, d);
      if (lane >= d) most = max(most, y);
    }
    int before = __shfl_up_sync(~0u, most, 1);
    before = max(last, lane > 0 ? before : -1);
    const bool take = in && e > before;
    bad |= e >= 0 && !take;
    const uint32_t bits = __ballot_sync(~0u, take);
    const int at = taken + __popc(bits & ((1u << lane) - 1u));
    if (take)
      for (int k = 0; k < per; ++k) {
        // (behind the context the table may have no entry)
        const int page = e * per + k;
        out[at * per + k] = page * c.B < r.seen ? __ldg(table + page) : -1;
      }
    taken += __popc(bits);
    last = max(last, __shfl_sync(~0u, most, 31));
  }
  if (__any_sync(~0u, bad) && lane == 0 && c.dev_error != nullptr)
    atomicOr(c.dev_error, KVQ_DEVERR_SEQ);
  if (lane == 0)
    p.row_lens[i] =
        taken == 0 ? 0
                   : (taken - 1) * p.sel + min(p.sel, r.seen - last * p.sel);
}

}  // namespace

// A round of rows of the decode kernel, and where its parts are in the
// workspace: its partial results (within what the tiles' kernel needs for
// its own, if that holds one row's), then lengths and tables.
struct Round {
  int64_t parts, rows, scratch;

  Round(int sms, int64_t total, int32_t Hq, int64_t tokens) {
    parts = (tokens + kPart - 1) / kPart;
    const int64_t row = parts > 1 ? Hq * parts * (kD + 2) * 4 : 4;
    const int64_t most = chunk_workspace_bytes(sms) / row;
    rows = std::max<int64_t>(
        1, std::min(total, std::min<int64_t>(most, 4096)));
    scratch = (std::max(chunk_workspace_bytes(sms), rows * row) + 31) / 32 *
              32;
  }
};

int64_t sparse_workspace_bytes(int sms, int64_t total, int32_t Hq,
                               int32_t top, int32_t sel, int32_t B) {
  const int64_t tokens = static_cast<int64_t>(top) * sel;
  const Round r(sms, total, Hq, tokens);
  return r.scratch + (r.rows * (tokens / B + 1) * 4 + 31) / 32 * 32;
}

cudaError_t launch_sparse_attention(const SparseParams& caller,
                                    cudaStream_t stream) {
  SparseParams p = caller;
  const ChunkParams& c = p.chunk;
  const int64_t tokens = static_cast<int64_t>(p.top) * p.sel;
  const Round round(sm_count(), c.total_q, c.Hq, tokens);
  const int64_t parts = round.parts, step = round.rows;
  p.row_lens = reinterpret_cast<int32_t*>(c.workspace + round.scratch);
  p.row_table = p.row_lens + step;
  AttnParams a{};
  a.q_stride0 = c.q_stride0;
  a.side[0] = c.side[0];
  a.side[1] = c.side[1];
  a.page_stride = c.page_stride;
  a.num_blocks = c.num_blocks;
  a.scale_off = c.scale_off;
  a.dhs = c.dhs;
  a.dts = c.dts;
  a.shs = c.shs;
  a.sts = c.sts;
  a.block_table = p.row_table;
  a.bt_stride = tokens / c.B;
  a.lens = p.row_lens;
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.scale = c.scale;
  a.out_stride0 = c.out_stride0;
  a.dev_error = c.dev_error;
  a.Hq = c.Hq;
  a.Hkv = c.Hkv;
  a.G = c.G;
  a.B = c.B;
  a.b_shift = c.b_shift;
  a.part = kPart;
  a.max_parts = static_cast<int32_t>(parts);
  a.len_cap = static_cast<int32_t>(
      std::min(tokens, static_cast<int64_t>(c.len_cap)));
  a.swizzle_k = c.swizzle_k;
  a.f16 = c.f16;
  a.pdl = true;
  a.cu = c.cu;
  a.listed = true;
  a.tmp_out = reinterpret_cast<float*>(c.workspace);
  for (p.row0 = 0; p.row0 < c.total_q; p.row0 += step) {
    p.num_rows = static_cast<int32_t>(std::min(step, c.total_q - p.row0));
    const unsigned ctas =
        (p.num_rows + kPlanThreads / 32 - 1) / (kPlanThreads / 32);
    cudaError_t err =
        launch_kernel(plan_rows_kernel, dim3(ctas), kPlanThreads, 0, stream,
                      c.pdl || p.row0 > 0, p);
    if (err != cudaSuccess) return err;
    a.q = c.q + p.row0 * c.q_stride0;
    a.out = c.out + p.row0 * c.out_stride0;
    a.num_seqs = p.num_rows;
    a.exp_sums = a.tmp_out + p.num_rows * c.Hq * parts * kD;
    a.max_logits = a.exp_sums + p.num_rows * c.Hq * parts;
    err = launch_paged_attention_mma(a, stream);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace kvq
