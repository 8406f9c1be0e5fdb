// select_blocks.cu -- the blocks of the context that each query row attends
// to: some always (the first ones, the last ones), then those of the best
// scores, sm_103a.
//
// A row that sees `seen` tokens has nb = ceil(seen / sel) blocks and takes k
// = min(top, nb) of them.  Scores become 32-bit keys in their order, and the
// k-th largest key is found from its top bit down: a bit is set if at least k
// keys are as large, and once there are exactly k the rest does not matter.
// The keys stay in the registers of a warp (up to 2048 of them) or of eight
// (up to 16384), the counts go over the lanes by one reduction.  A warp first
// finds a bound that few keys reach, and goes on with those.  Then a pass
// in the order of the blocks writes those above it and the first ones equal
// to it, so that the list rises and ties go to the lowest index.
// Longer rows are read again for every 8 bits of the key, counted in a
// histogram.
//
// 4096 rows of 1563 to 2048 blocks, 32 of each (32 MB): 34 us, 0.94 TB/s.
// Bound by a row's chain of latencies (its sequence, its scores, the counts) at
// 12 warps an SM, whose registers hold the keys; with the same keys searched
// whole, without the bound that leaves a few of them, 40 us.  Longer rows are
// far slower: 4096 of 2049 blocks 398 us, of 4096 and 8192 blocks 383.  Of their
// thread blocks (243 registers, 256 threads) an SM takes one at a time, and all
// of its keys are searched bit by bit, with a barrier each.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;

// Larger keys for larger scores; NaN as -inf, -0 as 0.  (All are above 0.)
__device__ __forceinline__ uint32_t key_of(float x) {
  x = x == x ? x + 0.0f : -INFINITY;
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) != 0u ? ~0u : 0x80000000u);
}

// The k largest of nb scores, 0 < k < nb: first + their places, rising, to
// out.  For kWarps warps, kKeys scores a lane; of one warp each, kRows rows a
// thread block.
template <int kWarps, int kKeys, int kRows>
__device__ __forceinline__ void select_best(const float* x, int nb, int k,
                                            int first, int32_t* out) {
  __shared__ int counts[2][kWarps];
  constexpr int kFew = 256;
  __shared__ uint2 few[kWarps == 1 ? kRows : 1][kFew];
  const int lane = threadIdx.x & 31;
  const int warp = kWarps > 1 ? threadIdx.x >> 5 : 0;
  // warp w: blocks w * 32 kKeys on, 32 at a time.  (0: none; no key is less)
  const int base = warp * 32 * kKeys + lane;
  uint32_t key[kKeys], all_or = 0, all_and = ~0u;
  // (all loads at once, those behind the row's end of its last score: one
  // behind the other the call took 75 us, not 43)
#pragma unroll
  for (int i = 0; i < kKeys; ++i)
    key[i] = __float_as_uint(__ldg(x + min(base + 32 * i, nb - 1)));
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const int j = base + 32 * i;
    const uint32_t u = key_of(__uint_as_float(key[i]));
    key[i] = j < nb ? u : 0u;
    all_or |= key[i];
    all_and &= j < nb ? u : ~0u;
  }
  const uint32_t lower = (1u << lane) - 1u;
  if constexpr (kWarps == 1) {
    // A bound: the keys cut into 32 c >= k groups, c a lane, the least of the
    // groups' largest; k keys are at least as large.  Mostly few more are (of
    // 2048 keys and k = 32 some 120), which go on alone, with their places.
    uint32_t most[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      most[g] = key[g * kKeys / 8];
#pragma unroll
      for (int i = 1; i < kKeys / 8; ++i)
        most[g] = max(most[g], key[g * kKeys / 8 + i]);
    }
#pragma unroll
    for (int c = 8; c > 1; c /= 2)
      if (k <= 16 * c) {
#pragma unroll
        for (int g = 0; g < c / 2; ++g) most[g] = max(most[g], most[g + c / 2]);
#pragma unroll
        for (int g = c / 2; g < c; ++g) most[g] = ~0u;
      }
#pragma unroll
    for (int g = 1; g < 8; ++g) most[0] = min(most[0], most[g]);
    const uint32_t bound = max(__reduce_min_sync(~0u, most[0]), 1u);
    uint2* own = few[threadIdx.x >> 5];
    int n = 0;
    if (k <= kFew && bound > 1u) {
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        const bool in = key[i] >= bound;
        const uint32_t bits = __ballot_sync(~0u, in);
        const int at = n + __popc(bits & lower);
        if (in && at < kFew) own[at] = make_uint2(key[i], base + 32 * i);
        n += __popc(bits);
      }
      __syncwarp();
    }
    if (n > 0 && n <= kFew) {
      uint2 left[kFew / 32];
      all_or = 0;
      all_and = ~0u;
#pragma unroll
      for (int i = 0; i < kFew / 32; ++i) {
        left[i] = make_uint2(0, 0);
        if (32 * i + lane >= n) continue;
        left[i] = own[32 * i + lane];
        all_or |= left[i].x;
        all_and &= left[i].x;
      }
      all_or = __reduce_or_sync(~0u, all_or);
      all_and = __reduce_and_sync(~0u, all_and);
      int bit = 31 - __clz(all_or ^ all_and), have = n;
      uint32_t limit = bit < 31 ? all_or >> (bit + 1) << (bit + 1) : 0u;
#pragma unroll 1
      for (; bit >= 0 && have != k; --bit) {
        const uint32_t next = limit | 1u << bit;
        int m = 0;
#pragma unroll
        for (int i = 0; i < kFew / 32; ++i) m += left[i].x >= next;
        m = __reduce_add_sync(~0u, m);
        if (m >= k) {
          limit = next;
          have = m;
        }
      }
      int spare = k;  // equal ones to take
      if (have != k) {
        int m = 0;
#pragma unroll
        for (int i = 0; i < kFew / 32; ++i) m += left[i].x > limit;
        spare = k - __reduce_add_sync(~0u, m);
      }
      int written = 0, equal = 0;
#pragma unroll
      for (int i = 0; i < kFew / 32; ++i) {
        const bool in = 32 * i + lane < n && left[i].x == limit;
        const uint32_t same = __ballot_sync(~0u, in);
        const bool mine = left[i].x > limit ||
                          (in && equal + __popc(same & lower) < spare);
        const uint32_t take = __ballot_sync(~0u, mine);
        if (mine) out[written + __popc(take & lower)] = first + left[i].y;
        written += __popc(take);
        equal += __popc(same);
      }
      return;
    }
  }
  int turn = 0;
  // the sum of n over the row's lanes
  auto total = [&](int n) {
    n = __reduce_add_sync(~0u, n);
    if constexpr (kWarps > 1) {
      if (lane == 0) counts[turn][warp] = n;
      __syncthreads();
      n = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) n += counts[turn][w];
      turn ^= 1;  // (the next sum's barrier is behind these reads)
    }
    return n;
  };
  // bits that all keys share are the threshold's too
  uint32_t limit = 0;
  int bit = 31, have = nb;  // keys that are at least `limit`
  if constexpr (kWarps == 1) {
    all_or = __reduce_or_sync(~0u, all_or);
    all_and = __reduce_and_sync(~0u, all_and);
    bit = 31 - __clz(all_or ^ all_and);
    limit = bit < 31 ? all_or >> (bit + 1) << (bit + 1) : 0u;
  }
  for (; bit >= 0 && have != k; --bit) {
    const uint32_t next = limit | 1u << bit;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kKeys; ++i) n += key[i] >= next;
    n = total(n);
    if (n >= k) {
      limit = next;
      have = n;
    }
  }
  // have == k: all that are as large; else those above and the first equal
  int equal = 0, spare = k;  // equal ones to take
  if (have != k) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kKeys; ++i) n += key[i] > limit;
    spare = k - total(n);
  }
  int written = 0;
  if constexpr (kWarps > 1) {
    // what the warps before this one write: their larger keys, and equal ones
    int above = 0, same = 0;
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      above += key[i] > limit;
      same += key[i] == limit;
    }
    above = __reduce_add_sync(~0u, above);
    same = __reduce_add_sync(~0u, same);
    __syncthreads();
    if (lane == 0) {
      counts[0][warp] = above;
      counts[1][warp] = same;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
      written += counts[0][w];
      equal += counts[1][w];
    }
    written += min(equal, spare);
  }
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const bool in = base + 32 * i < nb;
    const uint32_t above = __ballot_sync(~0u, in && key[i] > limit);
    const uint32_t same = __ballot_sync(~0u, in && key[i] == limit);
    if ((above | same) == 0u) continue;
    const int before = equal + __popc(same & lower);
    const bool mine = above >> lane & 1u ||
                      (same >> lane & 1u && before < spare);
    const uint32_t take = __ballot_sync(~0u, mine);
    if (mine) out[written + __popc(take & lower)] = first + base + 32 * i;
    written += __popc(take);
    equal += __popc(same);
  }
}

template <int kWarps, int kKeys, int kRows>
__global__ void __launch_bounds__(32 * kWarps * kRows, kWarps > 1 ? 1 : 3)
    select_few_kernel(const SelectParams p) {
  static_assert(kWarps == 1 || kRows == 1, "");
  pdl_prologue();
  const int lane = threadIdx.x & 31;
  const int warp = kWarps > 1 ? threadIdx.x >> 5 : 0;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows +
                      (kWarps > 1 ? 0 : threadIdx.x >> 5);
  if (blockIdx.x == 0)
    dev::check_rows(p.rows, threadIdx.x, 32 * kWarps * kRows);
  if (row >= p.rows.total) return;
  const dev::QueryRow r = dev::query_row(p.rows, static_cast<int>(row));
  if (r.seq < 0) return;
  const int nb = (r.seen + p.sel - 1) / p.sel;
  const int k = min(p.top, nb);
  int32_t* out = p.selected + row * p.selected_stride0;
  const int step = 32 * kWarps, me = 32 * warp + lane;
  for (int i = k + me; i < p.top; i += step) out[i] = -1;
  if (k == nb) {
    for (int i = me; i < k; i += step) out[i] = i;
    return;
  }
  // the blocks that are always taken; of those between them the best
  for (int i = me; i < p.first; i += step) out[i] = i;
  for (int i = me; i < p.last; i += step) out[k - p.last + i] = nb - p.last + i;
  if (k == p.first + p.last) return;
  select_best<kWarps, kKeys, kRows>(
      p.scores + row * p.scores_stride0 + p.first, nb - p.first - p.last,
      k - p.first - p.last, p.first, out + p.first);
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
  auto key = [&](int j) {  // (~0: always taken)
    return j < p.first || j >= nb - p.last ? ~0u : key_of(x[j]);
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
  auto run = [&](void (*kernel)(SelectParams), int rows, int threads) {
    const int64_t ctas = (p.rows.total + rows - 1) / rows;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(ctas)), threads, 0,
                         stream, p.pdl, p);
  };
  if (p.columns <= 512) return run(select_few_kernel<1, 16, 4>, 4, 128);
  if (p.columns <= 2048) return run(select_few_kernel<1, 64, 4>, 4, 128);
  if (p.columns <= 16384) return run(select_few_kernel<8, 64, 1>, 1, 256);
  return run(select_kernel, 1, kThreads);
}

}  // namespace kvq
