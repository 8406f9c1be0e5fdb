// sparse_attention.cu -- attention of each query row over the blocks of its
// sequence's context that a list selects, over the NVFP4 pages, sm_103a.
//
// Two ways, chosen for each item (256 / G tokens of a sequence, G query heads
// to a KV head) on the device:
//   * By rows.  A list rises, so that only its last block can hold tokens
//     behind the row: what a row sees are the first tokens of the pages of its
//     blocks, in order, and the row is a sequence of one query token over a
//     block table of its own, which the decode kernel runs.
//   * By tiles.  The blocks that any token of the item selects are laid one
//     after the other, and the chunks' kernel runs the item's rows over them,
//     each under a mask of a bit for each block.  Tokens that follow one
//     another select much the same blocks: a page is dequantised once for all
//     of them, and the products are those of 256 rows.
// A plan kernel unites the lists, counts and decides; another one writes the
// tables of the rows that are left.
//
// Measured, blocks of 64 tokens, 32 a row, 64 query and 8 KV heads: 64 single
// tokens (153 MB) 37 us, 4.1 TB/s, of which 5 us are the rows' tables and 4 the
// join of a row's two stretches (the decode kernel's own 32 us: 0.71 of the
// measured copy rate).  1024 rows over 32768 tokens 254 us: of the 69
// GFLOP that the rows ask for the tiles do 2.8 times as many, for the 90 blocks
// that 32 rows select together, at 853 TFLOP/s; by rows alone 422 us.  Items of
// 16 rows would select 78 blocks together for half the rows.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kvq.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kPlanThreads = 128;  // rows: a warp for each
constexpr int kPart = 512;         // partition of the decode scratch
constexpr int kD = 128;
constexpr int kUnionThreads = 1024;
constexpr int kUnionWarps = kUnionThreads / 32;
constexpr int kMaxUnion = 8192;    // blocks of a context that items can name
// An item goes by tiles if its rows' tokens add up to more than kTileCost for
// each of its tiles and kTileItem more: a tile of 128 tokens takes the SM as
// long as that many tokens of rows in the decode kernel (2.1 us at 4.2 ns).
constexpr int kTileCost = 500, kTileItem = 3;

// Tokens of all rows and KV heads from which on items are looked at (test
// builds: always).  Measured by rows and by tiles, 1 and 8 sequences, 1 to 8
// query heads to a KV head, 512 and 2048 tokens a row: at 2.5 million 66 to 75 us
// and 71 to 100, at 3.3 85 to 96 and 73 to 119, at 4.2 106 to 120 and 75 to 122,
// at 16.8 422 and 201 to 254.
#ifndef KVQ_SPARSE_ITEMS_FROM
#define KVQ_SPARSE_ITEMS_FROM 2500000
#endif
constexpr int64_t kItemsFrom = KVQ_SPARSE_ITEMS_FROM;

// The entries of a row's list that count: those that lie above all before
// them and hold something that the row sees.  fn(entry, their number so far),
// by the lane that holds it; every lane calls it.  Returns {how many, last};
// *bad: there were others.
template <typename Fn>
__device__ __forceinline__ int2 walk_list(const int32_t* list, int top,
                                          int blocks, bool* bad, Fn fn) {
  const int lane = threadIdx.x & 31;
  int taken = 0, last = -1;  // (the largest entry so far)
  for (int j0 = 0; j0 < top; j0 += 32) {
    const int e = j0 + lane < top ? __ldg(list + j0 + lane) : -1;
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
    *bad |= e >= 0 && !take;
    const uint32_t bits = __ballot_sync(~0u, take);
    if (take) fn(e, taken + __popc(bits & ((1u << lane) - 1u)));
    taken += __popc(bits);
    last = max(last, __shfl_sync(~0u, most, 31));
  }
  return {taken, last};
}
// Tokens of `taken` blocks, of which the last may go beyond what is seen.
__device__ __forceinline__ int tokens_of(int2 list, int sel, int seen) {
  return list.x == 0 ? 0
                     : (list.x - 1) * sel + min(sel, seen - list.y * sel);
}

// Item x of the plan: item i of sequence b has x = cu[b] / T + b + i, T tokens
// an item (all different, and at most total / T + num_seqs).
__global__ void __launch_bounds__(kUnionThreads)
    plan_items_kernel(const SparseParams p) {
  pdl_prologue();
  __shared__ uint32_t bits[kMaxUnion / 32], buffer[kUnionWarps][kMaxUnion / 32];
  __shared__ int rank[kMaxUnion / 32], scan[8], sum;
  const ChunkParams& c = p.chunk;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = c.item_tokens, x = blockIdx.x;
  if (x == 0) {
    dev::check_rows(p.rows, tid, kUnionThreads);
    for (int k = tid; k < p.rounds; k += kUnionThreads) p.live[k] = 0;
  }
  // the last sequence that begins at x or before
  int lo = 0, hi = c.num_seqs;
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5, at = lo + lane * step;
    const int n = __popc(__ballot_sync(
        ~0u, at < hi && max(__ldg(c.cu + at), 0) / T + at <= x));
    hi = min(hi, lo + n * step);
    if (n > 0) lo += (n - 1) * step + 1;
  }
  const int b = lo - 1, total = static_cast<int>(c.total_q);
  int q0 = 0, n = 0, i = 0;
  if (b >= 0) {
    q0 = min(max(__ldg(c.cu + b), 0), total);
    n = min(max(__ldg(c.cu + b + 1), q0), total) - q0;
    i = x - q0 / T - b;
  }
  const int tok0 = i * T, nt = min(T, n - tok0);
  int4* item = p.items + x;
  if (b < 0 || i < 0 || nt <= 0) {
    if (tid == 0) *item = make_int4(0, 0, 0, 0);
    return;
  }
  const int L = min(max(__ldg(c.lens + b), 0), c.len_cap);
  const int words = c.mask_words;
  for (int k = tid; k < words; k += kUnionThreads) bits[k] = 0;
  if (tid == 0) sum = 0;
  __syncthreads();
  bool bad = false;
  auto seen_of = [&](int j) { return max(L - n + tok0 + j + 1, 0); };
  auto list_of = [&](int j) {
    return p.selected + (q0 + tok0 + j) * p.selected_stride0;
  };
  auto blocks_of = [&](int j) { return (seen_of(j) + p.sel - 1) / p.sel; };
  for (int j = warp; j < nt; j += kUnionWarps) {
    const int2 list = walk_list(list_of(j), p.top, blocks_of(j), &bad,
                                [&](int e, int) {
                                  atomicOr(&bits[e >> 5], 1u << (e & 31));
                                });
    if (lane == 0) atomicAdd(&sum, tokens_of(list, p.sel, seen_of(j)));
  }
  if (__any_sync(~0u, bad) && lane == 0 && c.dev_error != nullptr)
    atomicOr(c.dev_error, KVQ_DEVERR_SEQ);
  __syncthreads();
  // (a word for each of the first threads)
  const uint32_t mine = tid < words ? bits[tid] : 0u;
  int incl = __popc(mine);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31 && warp < 8) scan[warp] = incl;
  __syncthreads();
  int U = 0;
  for (int w = 0; w < kMaxUnion / 1024; ++w) {
    if (w < warp) incl += scan[w];
    U += scan[w];
  }
  if (tid < kMaxUnion / 32) rank[tid] = incl - __popc(mine);
  const int W = static_cast<int>(
      (static_cast<int64_t>(U) * p.sel + 127) / 128);
  if (sum <= kTileCost * (kTileItem + W)) {  // (nothing is selected: by rows)
    if (tid == 0) *item = make_int4(0, 0, 0, 0);
    return;
  }
  // the pages of its blocks
  const int per = p.sel / c.B;
  const int32_t* table = c.block_table + b * c.bt_stride;
  int32_t* pages = p.item_pages + x * c.item_stride;
  int k = incl - __popc(mine);
  for (uint32_t m = mine; m != 0; m &= m - 1, ++k) {
    const int e = 32 * tid + __ffs(m) - 1;
    for (int j = 0; j < per; ++j) {
      // (behind the context the table may have no entry)
      const int page = e * per + j;
      pages[k * per + j] = page * c.B < L ? __ldg(table + page) : -1;
    }
    if (k == U - 1)
      *item = make_int4(W, b, i, k * p.sel + min(p.sel, L - e * p.sel));
  }
  __syncthreads();
  // each token's blocks among them
  for (int j = warp; j < nt; j += kUnionWarps) {
    uint32_t* own = buffer[warp];
    for (int w = lane; w < words; w += 32) own[w] = 0;
    __syncwarp();
    auto rank_of = [&](int e) {
      return rank[e >> 5] + __popc(bits[e >> 5] & ((1u << (e & 31)) - 1u));
    };
    const int2 list = walk_list(list_of(j), p.top, blocks_of(j), &bad,
                                [&](int e, int) {
                                  const int r = rank_of(e);
                                  atomicOr(&own[r >> 5], 1u << (r & 31));
                                });
    __syncwarp();
    const int64_t q = q0 + tok0 + j;
    for (int w = lane; w < words; w += 32) p.masks[q * words + w] = own[w];
    const bool edge = list.x > 0 && list.y == (seen_of(j) - 1) / p.sel;
    if (lane == 0)
      p.tokens[q] = make_int2(edge ? rank_of(list.y) : -1,
                              tokens_of(list, p.sel, seen_of(j)));
    __syncwarp();
  }
}

// The rows from p.row0 on: their tables and lengths (-1: not a row).  Where
// items are looked at, only those that no item has, in any order, with their
// numbers (a row's result does not depend on its place).
__global__ void __launch_bounds__(kPlanThreads)
    plan_rows_kernel(const SparseParams p) {
  pdl_prologue();
  int i = blockIdx.x * (kPlanThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (p.row0 == 0 && blockIdx.x == 0)
    dev::check_rows(p.rows, threadIdx.x, kPlanThreads);
  if (i >= p.num_rows) return;
  const int64_t row = p.row0 + i;
  const dev::QueryRow r = dev::query_row(p.rows, static_cast<int>(row));
  const ChunkParams& c = p.chunk;
  bool left = r.seq >= 0;
  if (left && p.items != nullptr) {
    const int T = c.item_tokens, q0 = static_cast<int>(row) - r.i;
    left = p.items[q0 / T + r.seq + r.i / T].x == 0;
  }
  if (!left) {
    if (lane == 0 && p.items == nullptr) p.row_lens[i] = -1;
    return;
  }
  if (p.items != nullptr) {
    const int id = i;
    if (lane == 0) {
      i = atomicAdd(p.live + p.round, 1);
      p.row_ids[i] = id;
    }
    i = __shfl_sync(~0u, i, 0);
  }
  const int per = p.sel / c.B;  // pages of a block
  const int32_t* table = c.block_table + r.seq * c.bt_stride;
  int32_t* out = p.row_table + static_cast<int64_t>(i) * p.top * per;
  bool bad = false;
  const int2 list = walk_list(
      p.selected + row * p.selected_stride0, p.top,
      (r.seen + p.sel - 1) / p.sel, &bad, [&](int e, int at) {
        for (int k = 0; k < per; ++k) {
          // (behind the context the table may have no entry)
          const int page = e * per + k;
          out[at * per + k] = page * c.B < r.seen ? __ldg(table + page) : -1;
        }
      });
  if (__any_sync(~0u, bad) && lane == 0 && c.dev_error != nullptr)
    atomicOr(c.dev_error, KVQ_DEVERR_SEQ);
  if (lane == 0) p.row_lens[i] = tokens_of(list, p.sel, r.seen);
}

// ---------------------------------------------------------------------------
// The workspace
// ---------------------------------------------------------------------------
// First the partial results, of the decode kernel's rows (a round of them) or
// of the tiles' kernel; then how many rows each round has, their numbers,
// lengths and tables; then the items, for contexts of up to `context` tokens.
struct Space {
  int64_t parts, rows, rounds, live, row_ids, row_lens, row_table;
  int64_t item_tokens, num_items, item_stride, words;  // (num_items 0: none)
  int64_t items, item_pages, masks, tokens, bytes;

  Space(int sms, int64_t total, int32_t num_seqs, int32_t Hq, int32_t Hkv,
        int32_t top, int32_t sel, int32_t B, int64_t context) {
    constexpr int64_t kScratch = int64_t{256} << 20, kItems = kScratch;
    const int64_t span = static_cast<int64_t>(top) * sel;
    auto up = [](int64_t x) { return (x + 31) / 32 * 32; };
    parts = (span + kPart - 1) / kPart;
    const int64_t row = parts > 1 ? Hq * parts * (kD + 2) * 4 : 4;
    rows = std::max<int64_t>(
        1, std::min(total, std::min<int64_t>(kScratch / row, 4096)));
    rounds = (total + rows - 1) / rows;
    live = up(std::max(chunk_workspace_bytes(sms), rows * row));
    row_ids = live + up(rounds * 4);
    row_lens = row_ids + up(rows * 4);
    row_table = row_lens + up(rows * 4);
    bytes = row_table + up(rows * (span / B) * 4);
    // items: blocks of 16, 32, 64 .. tokens, as the masks of a tile need them
    item_tokens = 256 / (Hq / Hkv);
    num_items = total / item_tokens + num_seqs;
    const int64_t blocks = (context + sel - 1) / sel;
    item_stride = std::min(blocks, item_tokens * top) * (sel / B);
    words = (blocks + 31) / 32;
    if (sel < 16 || (sel & (sel - 1)) != 0 || blocks > kMaxUnion ||
        total <= kFewRows) {
      num_items = 0;
      return;
    }
    items = bytes;
    if (num_items * (item_stride * 4 + 16) + total * (words * 4 + 8) >
        kItems) {
      // (what a call of fewer rows or sequences can need: a workspace for the
      // largest call is one for all)
      num_items = 0;
      bytes = items + kItems + 4 * 32;
      return;
    }
    item_pages = items + up(num_items * 16);
    tokens = item_pages + up(num_items * item_stride * 4);
    masks = tokens + up(total * 8);
    bytes = masks + up(total * words * 4);
  }
  // Chunks of up to this many tokens go by rows: even if they all select the
  // same t tokens, tiles would take 1500 + 3.9 t of the units of which the rows
  // take 4 t: more up to lists of 16000 tokens, and hardly less beyond.
  static constexpr int kFewRows = 4;
};

}  // namespace

int64_t sparse_workspace_bytes(int sms, int64_t total, int32_t num_seqs,
                               int32_t Hq, int32_t Hkv, int32_t top,
                               int32_t sel, int32_t B, int32_t max_blocks) {
  // (calls over longer contexts have no items: what those up to there need is
  // enough for them)
  const int64_t context =
      std::min(static_cast<int64_t>(max_blocks) * B,
               static_cast<int64_t>(kMaxUnion) * sel);
  return Space(sms, total, num_seqs, Hq, Hkv, top, sel, B, context).bytes;
}

cudaError_t launch_sparse_attention(const SparseParams& caller,
                                    cudaStream_t stream) {
  SparseParams p = caller;
  ChunkParams& c = p.chunk;
  const int64_t tokens = static_cast<int64_t>(p.top) * p.sel;
  const Space space(sm_count(), c.total_q, c.num_seqs, c.Hq, c.Hkv, p.top,
                    p.sel, c.B, c.len_cap);
  p.row_lens = reinterpret_cast<int32_t*>(c.workspace + space.row_lens);
  p.row_table = reinterpret_cast<int32_t*>(c.workspace + space.row_table);
  // (and where there is enough to do: else the decode kernel spreads its rows
  // over the SMs at once, 82 rows of 640 tokens of 8 KV heads in a call of 21 us,
  // by tiles of 50)
  const bool items = space.num_items > 0 && c.max_q_len > Space::kFewRows &&
                     c.total_q * c.Hkv * std::min<int64_t>(tokens, c.len_cap) >
                         kItemsFrom;
  bool pdl = c.pdl;
  if (items) {
    p.items = reinterpret_cast<int4*>(c.workspace + space.items);
    p.item_pages = reinterpret_cast<int32_t*>(c.workspace + space.item_pages);
    p.masks = reinterpret_cast<uint32_t*>(c.workspace + space.masks);
    p.tokens = reinterpret_cast<int2*>(c.workspace + space.tokens);
    p.live = reinterpret_cast<int32_t*>(c.workspace + space.live);
    p.row_ids = reinterpret_cast<int32_t*>(c.workspace + space.row_ids);
    p.rounds = static_cast<int32_t>(space.rounds);
    c.items = p.items;
    c.item_pages = p.item_pages;
    c.masks = p.masks;
    c.tokens = p.tokens;
    c.item_stride = space.item_stride;
    c.num_items = static_cast<int32_t>(space.num_items);
    c.item_tokens = static_cast<int32_t>(space.item_tokens);
    c.mask_words = static_cast<int32_t>(space.words);
    for (c.sel_shift = 4; 1 << c.sel_shift < p.sel;) ++c.sel_shift;
    const cudaError_t err = launch_kernel(
        plan_items_kernel, dim3(static_cast<unsigned>(c.num_items)),
        kUnionThreads, 0, stream, pdl, p);
    if (err != cudaSuccess) return err;
    pdl = true;
  }
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
  a.max_parts = static_cast<int32_t>(space.parts);
  a.len_cap = static_cast<int32_t>(
      std::min(tokens, static_cast<int64_t>(c.len_cap)));
  a.swizzle_k = c.swizzle_k;
  a.f16 = c.f16;
  a.pdl = true;
  a.cu = c.cu;
  a.listed = true;
  a.row_ids = p.row_ids;
  a.tmp_out = reinterpret_cast<float*>(c.workspace);
  for (; p.row0 < c.total_q; p.row0 += space.rows, ++p.round) {
    p.num_rows =
        static_cast<int32_t>(std::min(space.rows, c.total_q - p.row0));
    const unsigned ctas =
        (p.num_rows + kPlanThreads / 32 - 1) / (kPlanThreads / 32);
    cudaError_t err = launch_kernel(plan_rows_kernel, dim3(ctas),
                                    kPlanThreads, 0, stream, pdl, p);
    if (err != cudaSuccess) return err;
    pdl = true;
    a.q = c.q + p.row0 * c.q_stride0;
    a.out = c.out + p.row0 * c.out_stride0;
    a.num_seqs = p.num_rows;
    a.live = items ? p.live + p.round : nullptr;
    a.exp_sums = a.tmp_out + p.num_rows * c.Hq * space.parts * kD;
    a.max_logits = a.exp_sums + p.num_rows * c.Hq * space.parts;
    err = launch_paged_attention_mma(a, stream);
    if (err != cudaSuccess) return err;
  }
  if (!items) return cudaSuccess;
  c.pdl = true;
  return launch_listed_attention(c, stream);
}

}  // namespace kvq
