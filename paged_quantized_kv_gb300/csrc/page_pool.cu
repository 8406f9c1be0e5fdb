// page_pool.cu -- the device-side state of a paged cache, sm_103a: growing,
// forking, compacting and freeing sequences.
//
// State (the caller's): ref_count [num_blocks] (0 = free page), block_table
// rows (page of each block of the sequence, -1 = none) and seq_lens.  The
// rules are those of include/kvq.h; every result is the same from run to
// run: pages are handed out lowest index first, in the order of the lists,
// and the only atomics are integer counts.
//
// What bounds these kernels is latency: a call touches kilobytes.  So each
// list operation that hands out pages is ONE launch of one thread-block
// cluster: its CTAs count the free pages of their shares of ref_count in
// parallel, exchange the counts through distributed shared memory, and
// everything after the cluster barrier (pages to rows, slots, shared rows)
// is spread over the cluster's threads.  A grid with a scan between two
// launches would pay a second launch and a workspace; one CTA alone reads
// the counts of 65536 pages in eight times the rounds.
// Measured (back to back, with the calls that put the state back): extend of
// a few sequences with a free 12 us; 128 new sequences of 100 to 4000 tokens
// with a free 25 us; forks of a few rows with their page copies and a free
// 14 us; compaction of a few rows with its moves 28 us.  The counts are read
// by eight SMs, once for the sum and again up to the last page handed out:
// extend and free of four rows 11 us with 65536 pages, 17 with 2^20, 118 with
// 2^24 (13, 42 and 582 where only the last pages are free).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_internal.h"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;     // CTAs of a pool kernel (portable size)
constexpr int kThreads = 1024;
constexpr int kChunk = 4 * kThreads;  // counts of one scan round of a CTA
// Up to this many slots an extend writes itself (8192 threads, two each: a
// second launch takes longer); more are left to a second kernel.
constexpr int kClusterSlots = 16384;

__device__ __forceinline__ void flag(int32_t* err, int32_t bits) {
  if (err != nullptr) atomicOr(err, bits);
}

// Exclusive prefix of v over the CTA's threads in thread order; *total gets
// the sum.  s: 33 ints.  Every thread must call it.
__device__ __forceinline__ int block_scan(int v, int* s, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) s[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int n = blockDim.x >> 5;
    int w = lane < n ? s[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, w, d);
      if (lane >= d) w += y;
    }
    s[lane] = w;  // inclusive
  }
  __syncthreads();
  const int before = (warp > 0 ? s[warp - 1] : 0) + x - v;
  *total = s[31];
  __syncthreads();
  return before;
}

// Largest i in [0, n) with a[i] <= v (a[0] <= v), a non-decreasing.
__device__ __forceinline__ int last_at_most(const int* a, int n, int v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= v)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ bool page_ok(const PoolParams& p, int32_t page) {
  return page >= 0 && page < p.num_blocks;
}

// Bits of the rows that `ids` names more than once: every occurrence of
// such a row is refused (which one came first would depend on the order of
// the threads).
__device__ __forceinline__ void find_twice(const int32_t* ids, int n,
                                           int rows, uint32_t* seen,
                                           uint32_t* twice) {
  for (int w = threadIdx.x; w < (rows + 31) / 32; w += blockDim.x)
    seen[w] = twice[w] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int id = ids[i];
    if (id < 0 || id >= rows) continue;
    const uint32_t bit = 1u << (id & 31);
    if (atomicOr(&seen[id >> 5], bit) & bit) atomicOr(&twice[id >> 5], bit);
  }
  __syncthreads();
}

__device__ __forceinline__ bool is_twice(const uint32_t* twice, int id) {
  return (twice[id >> 5] >> (id & 31)) & 1u;
}

// Whether cu is a list of offsets: cu[0] == 0, non-decreasing, within total.
// Every thread must call it; the answer is the CTA's.
__device__ __forceinline__ bool offsets_ok(const int32_t* cu, int n,
                                           int64_t total) {
  int bad = 0;
  for (int i = threadIdx.x; i <= n; i += blockDim.x) {
    const int32_t c = cu[i];
    if (i == 0 ? c != 0 : c < cu[i - 1]) bad = 1;
    if (c > total) bad = 1;
  }
  return __syncthreads_or(bad) == 0;
}

// Hand out pages: needs are given as exclusive offsets off[0..n] in shared
// memory.  `give(i, j, page)` is called once for the j-th page of entry i,
// for every entry that is served (off[i + 1] <= free pages); returns the
// number of free pages.  Pages are taken lowest index first.  The CTAs'
// shares of ref_count are contiguous, in rank order.  `check()` runs between
// the cluster's two barriers, where every CTA has come as far and no count
// has changed yet; `settle()` behind them, before `off` is read.
template <typename Check, typename Settle, typename Give>
__device__ int hand_out(const PoolParams& p, const int* off, int* scan,
                        int* share, Check check, Settle settle, Give give) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int n = p.n;
  // shares in whole chunks, so that every share starts at a multiple of 4
  const int64_t chunks = (p.num_blocks + kChunk - 1) / kChunk;
  const int64_t per = (chunks + kCluster - 1) / kCluster * kChunk;
  const int64_t lo = min(p.num_blocks, per * rank);
  const int64_t hi = min(p.num_blocks, per * (rank + 1));
  const bool vec = (reinterpret_cast<uintptr_t>(p.ref) & 15) == 0;

  auto load = [&](int64_t at, int32_t (&r)[4]) {
    if (vec && at + 4 <= hi) {
      const int4 v = *reinterpret_cast<const int4*>(p.ref + at);
      r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = at + k < hi ? p.ref[at + k] : 1;
    }
  };

  int mine = 0;
  for (int64_t base = lo; base < hi; base += kChunk) {
    int32_t r[4];
    load(base + 4 * threadIdx.x, r);
#pragma unroll
    for (int k = 0; k < 4; ++k) mine += r[k] == 0;
  }
  int sum;
  block_scan(mine, scan, &sum);
  if (threadIdx.x == 0) *share = sum;
  cluster.sync();
  int before = 0, all = 0;
  for (int k = 0; k < kCluster; ++k) {
    const int c = *cluster.map_shared_rank(share, k);
    if (k < rank) before += c;
    all += c;
  }
  check();
  cluster.sync();  // nobody leaves, or writes a count, while one is read
  settle();
  const int want = off[n];
  for (int64_t base = lo; base < hi && before < want; base += kChunk) {
    const int64_t at = base + 4 * threadIdx.x;
    int32_t r[4];
    load(at, r);
    int c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) c += r[k] == 0;
    int got;
    int g = before + block_scan(c, scan, &got);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (r[k] != 0) continue;
      if (g < want) {
        const int i = last_at_most(off, n, g);
        if (off[i + 1] <= all) {
          p.ref[at + k] = 1;
          give(i, g - off[i], static_cast<int32_t>(at + k));
        }
      }
      ++g;
    }
    before += got;
  }
  return all;
}

// Shared memory of the cluster kernels: two bitmaps of the rows, then three
// int arrays of n + 1 entries.
struct PoolSmem {
  uint32_t *seen, *twice;
  int *a, *b, *c;
  __device__ PoolSmem(uint8_t* base, int rows, int n) {
    const int words = (rows + 31) / 32;
    seen = reinterpret_cast<uint32_t*>(base);
    twice = seen + words;
    a = reinterpret_cast<int*>(twice + words);
    b = a + (n + 1);
    c = b + (n + 1);
  }
};
size_t pool_smem(int rows, int n) {
  return 8 * static_cast<size_t>((rows + 31) / 32) +
         12 * static_cast<size_t>(n + 1);
}

// Exclusive offsets of value(i) over the list into out[0..n].
template <typename Value>
__device__ __forceinline__ void list_scan(int n, int* out, int* scan,
                                          Value value) {
  int carry = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + static_cast<int>(threadIdx.x);
    const int v = i < n ? value(i) : 0;
    int sum;
    const int e = block_scan(v, scan, &sum);
    if (i < n) out[i] = carry + e;
    carry += sum;
  }
  if (threadIdx.x == 0) out[n] = carry;
  __syncthreads();
}

// ---------------------------------------------------------------------------
// extend: pages and slots for new tokens
// ---------------------------------------------------------------------------
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    extend_kernel(const __grid_constant__ PoolParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int scan[33];
  __shared__ int share;
  pdl_prologue();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int n = p.n, B = p.B;
  const PoolSmem s(smem, p.rows, n);
  int* off = s.a;   // page offsets
  int* old = s.b;   // length before the call, -1: refused
  int* cus = s.c;   // offsets of the new tokens
  const bool ok = offsets_ok(p.cu, n, p.total);
  if (!ok && rank == 0 && threadIdx.x == 0) flag(p.err, KVQ_DEVERR_SEQ);
  for (int i = threadIdx.x; i <= n; i += kThreads) cus[i] = ok ? p.cu[i] : 0;
  find_twice(p.ids, n, p.rows, s.seen, s.twice);
  list_scan(n, off, scan, [&](int i) {
    old[i] = -1;
    const int id = p.ids[i];
    int32_t bad = 0;
    int need = 0;
    if (!ok || id < 0 || id >= p.rows || is_twice(s.twice, id)) {
      bad = KVQ_DEVERR_SEQ;
    } else {
      const int len = p.lens[id];
      const int64_t add = cus[i + 1] - cus[i];
      if (len < 0 || len + add > static_cast<int64_t>(p.width) * B) {
        bad = KVQ_DEVERR_SEQ;
      } else {
        // the new tokens that go into the last page must not be another
        // sequence's too
        if (add > 0 && len % B != 0) {
          const int32_t page = p.table[id * p.stride + len / B];
          if (!page_ok(p, page))
            bad = KVQ_DEVERR_BLOCK;
          else if (p.ref[page] != 1)
            bad = KVQ_DEVERR_REF;
        }
        if (bad == 0) {
          old[i] = len;
          need = static_cast<int>((len + add + B - 1) / B -
                                  (static_cast<int64_t>(len) + B - 1) / B);
        }
      }
    }
    if (bad != 0 && rank == 0) flag(p.err, bad);
    return need;
  });
  const int all = hand_out(
      p, off, scan, &share, [] {}, [] {}, [&](int i, int j, int page) {
        const int id = p.ids[i];
        p.table[id * p.stride + (old[i] + B - 1) / B + j] = page;
      });
  cluster.sync();
  const int tid = rank * kThreads + static_cast<int>(threadIdx.x);
  const int64_t covered = cus[n];
  if (p.total > kClusterSlots) {
    // the rest is slots_kernel's: each entry's first slot for it, or -1
    for (int i = tid; i < n; i += kCluster * kThreads) {
      if (cus[i + 1] == cus[i]) continue;
      int64_t slot = -1;
      if (old[i] >= 0 && off[i + 1] <= max(all, off[i]))
        slot = static_cast<int64_t>(
                   p.table[p.ids[i] * p.stride + old[i] / B]) * B +
               old[i] % B;
      p.slots[cus[i]] = slot;
    }
    if (!ok && tid == 0) p.slots[0] = -1;
  }
  for (int64_t t = tid; p.total <= kClusterSlots && t < p.total;
       t += kCluster * kThreads) {
    int64_t slot = -1;
    if (t < covered) {
      const int i = last_at_most(cus, n, static_cast<int>(t));
      if (old[i] >= 0 && off[i + 1] <= max(all, off[i])) {
        const int pos = old[i] + static_cast<int>(t) - cus[i];
        const int32_t page = p.table[p.ids[i] * p.stride + pos / B];
        slot = static_cast<int64_t>(page) * B + pos % B;
      }
    }
    p.slots[t] = slot;
  }
  // (every CTA has read seq_lens before the cluster barriers above)
  for (int i = tid; i < n; i += kCluster * kThreads) {
    if (old[i] < 0) continue;
    if (off[i + 1] <= max(all, off[i]))
      p.lens[p.ids[i]] = old[i] + (cus[i + 1] - cus[i]);
    else
      flag(p.err, KVQ_DEVERR_FULL);
  }
}

// The slots of many new tokens, by the whole GPU (241884 tokens, with a free
// before it: 47 us by the cluster's eight SMs, 25 us this way).  Reads the new state;
// an entry's first slot says whether it was served.
constexpr int kSlotThreads = 256;
__global__ void __launch_bounds__(kSlotThreads)
    slots_kernel(const __grid_constant__ PoolParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  int* cus = reinterpret_cast<int*>(smem);
  pdl_prologue();
  const int n = p.n, B = p.B;
  const bool ok = offsets_ok(p.cu, n, p.total);
  for (int i = threadIdx.x; i <= n; i += kSlotThreads)
    cus[i] = ok ? p.cu[i] : 0;
  __syncthreads();
  const int64_t covered = cus[n];
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kSlotThreads +
                   threadIdx.x;
       t < p.total; t += static_cast<int64_t>(gridDim.x) * kSlotThreads) {
    if (t >= covered) {
      p.slots[t] = -1;
      continue;
    }
    const int i = last_at_most(cus, n, static_cast<int>(t));
    if (t == cus[i]) continue;  // written
    int64_t slot = -1;
    if (p.slots[cus[i]] >= 0) {
      const int id = p.ids[i];
      const int pos = p.lens[id] - (cus[i + 1] - static_cast<int>(t));
      const int32_t page = p.table[id * p.stride + pos / B];
      slot = static_cast<int64_t>(page) * B + pos % B;
    }
    p.slots[t] = slot;
  }
}

// ---------------------------------------------------------------------------
// fork: a child shares its parent's full pages and gets a page of its own
// for the last, partly filled one
// ---------------------------------------------------------------------------
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    fork_kernel(const __grid_constant__ PoolParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int scan[33];
  __shared__ int share;
  pdl_prologue();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int n = p.n, B = p.B;
  const PoolSmem s(smem, p.rows, n);
  int* off = s.a;   // page offsets (one page or none per entry)
  int* len = s.b;   // the parent's length, -1: refused
  int* row = s.c;   // offsets of the shared pages (before check() refuses)
  find_twice(p.ids2, n, p.rows, s.seen, s.twice);
  list_scan(n, row, scan, [&](int i) {
    len[i] = -1;
    const int par = p.ids[i], chi = p.ids2[i];
    int32_t bad = 0;
    if (par < 0 || par >= p.rows || chi < 0 || chi >= p.rows ||
        is_twice(s.twice, chi) || p.lens[chi] != 0 ||
        (p.width > 0 && p.table[chi * p.stride] >= 0)) {
      bad = KVQ_DEVERR_SEQ;
    } else {
      const int L = p.lens[par];
      if (L < 0 || L > static_cast<int64_t>(p.width) * B) {
        bad = KVQ_DEVERR_SEQ;
      } else {
        if (L % B != 0) {
          const int32_t page = p.table[par * p.stride + L / B];
          if (!page_ok(p, page))
            bad = KVQ_DEVERR_BLOCK;
          else if (p.ref[page] <= 0)
            bad = KVQ_DEVERR_REF;
        }
        if (bad == 0) len[i] = L;
      }
    }
    if (bad != 0 && rank == 0) flag(p.err, bad);
    return len[i] < 0 ? 0 : len[i] / B;
  });
  const int tid = rank * kThreads + static_cast<int>(threadIdx.x);
  // A page that nobody holds may be handed out by this very call: a parent
  // with one is refused.  The cluster's threads share out the rows' entries
  // and tell every CTA what they find.  A thread keeps its first ones for the
  // end.  (64 rows forked four times, with a free and the copies: 48.0 us
  // without the check, 53.7 with each entry looked up for it and again at the
  // end, 50.8 this way; a few rows 13.3, 14.0, 13.8.)
  constexpr int kKept = 4, kStep = kCluster * kThreads;
  int owner[kKept];
  int32_t kept[kKept];
  auto look_up = [&](int e, int* i) {
    *i = last_at_most(row, n, e);
    return p.table[p.ids[*i] * p.stride + e - row[*i]];
  };
  auto refuse = [&](int i) {
    for (int k = 0; k < kCluster; ++k)
      *cluster.map_shared_rank(len + i, k) = -1;
    flag(p.err, KVQ_DEVERR_REF);
  };
  int32_t count[kKept];  // (loaded here, looked at behind the first barrier)
#pragma unroll
  for (int u = 0; u < kKept; ++u) {
    owner[u] = -1;
    if (tid + u * kStep < row[n]) kept[u] = look_up(tid + u * kStep, owner + u);
  }
#pragma unroll
  for (int u = 0; u < kKept; ++u)
    count[u] = owner[u] >= 0 && page_ok(p, kept[u]) ? p.ref[kept[u]] : 1;
  auto check = [&] {
#pragma unroll
    for (int u = 0; u < kKept; ++u)
      if (count[u] <= 0) refuse(owner[u]);
    for (int e = tid + kKept * kStep; e < row[n]; e += kStep) {
      int i;
      const int32_t page = look_up(e, &i);
      if (page_ok(p, page) && p.ref[page] <= 0) refuse(i);
    }
  };
  auto settle = [&] {
    list_scan(n, off, scan,
              [&](int i) { return len[i] >= 0 && len[i] % B != 0; });
  };
  const int all = hand_out(
      p, off, scan, &share, check, settle, [&](int i, int, int page) {
        p.table[p.ids2[i] * p.stride + len[i] / B] = page;
        p.src[i] = p.table[p.ids[i] * p.stride + len[i] / B];
        p.dst[i] = page;
      });
  auto served = [&](int i) {
    return len[i] >= 0 && off[i + 1] <= max(all, off[i]);
  };
  auto give_share = [&](int e, int i, int32_t page) {
    if (!served(i)) return;
    if (page_ok(p, page))
      atomicAdd(p.ref + page, 1);
    else
      flag(p.err, KVQ_DEVERR_BLOCK);
    p.table[p.ids2[i] * p.stride + e - row[i]] = page_ok(p, page) ? page : -1;
  };
#pragma unroll
  for (int u = 0; u < kKept; ++u)
    if (owner[u] >= 0) give_share(tid + u * kStep, owner[u], kept[u]);
  for (int e = tid + kKept * kStep; e < row[n]; e += kStep) {
    int i;
    const int32_t page = look_up(e, &i);
    give_share(e, i, page);
  }
  // (every CTA has read seq_lens before the barriers in hand_out)
  for (int i = tid; i < n; i += kCluster * kThreads) {
    if (!served(i) || off[i + 1] == off[i]) p.src[i] = p.dst[i] = -1;
    if (served(i))
      p.lens[p.ids2[i]] = len[i];
    else if (len[i] >= 0)
      flag(p.err, KVQ_DEVERR_FULL);
  }
}

// ---------------------------------------------------------------------------
// compact: the kept tokens of a sequence move to its front
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;

// Whether entry i of the list is a row, named once.  Every thread must call.
__device__ __forceinline__ bool row_once(const int32_t* ids, int n, int rows,
                                         int i) {
  const int id = ids[i];
  int bad = id < 0 || id >= rows;
  for (int k = threadIdx.x; k < n; k += blockDim.x)
    if (k != i && ids[k] == id) bad = 1;
  return __syncthreads_or(bad) == 0;
}

// First launch, reads the state only (one sequence's frees must not be seen
// by another's checks): checks entry blockIdx.x and writes its slots, or -1
// for every one of them when it is refused.
__global__ void __launch_bounds__(kRowThreads)
    compact_check_kernel(const __grid_constant__ PoolParams p) {
  pdl_prologue();
  const int i = blockIdx.x, n = p.n, B = p.B;
  if (!offsets_ok(p.cu, n, p.total)) {
    if (i == 0) {
      if (threadIdx.x == 0) flag(p.err, KVQ_DEVERR_SEQ);
      for (int64_t t = threadIdx.x; t < p.total; t += kRowThreads)
        p.slots[t] = p.slots2[t] = -1;
    }
    return;
  }
  if (i == 0)  // behind the last list
    for (int64_t t = p.cu[n] + threadIdx.x; t < p.total; t += kRowThreads)
      p.slots[t] = p.slots2[t] = -1;
  const int at = p.cu[i], kept = p.cu[i + 1] - at;
  const int32_t* keep = p.keep + at;
  int32_t bad = 0;
  const bool once = row_once(p.ids, n, p.rows, i);
  const int id = p.ids[i];
  const int32_t* table = p.table + (once ? id * p.stride : 0);
  if (!once) {
    bad = KVQ_DEVERR_SEQ;
  } else {
    const int len = p.lens[id];
    if (len < 0 || len > static_cast<int64_t>(p.width) * B)
      bad = KVQ_DEVERR_SEQ;
    else
      for (int j = threadIdx.x; j < kept; j += kRowThreads) {
        const int k = keep[j];
        if (k < 0 || k >= len || (j > 0 && k <= keep[j - 1])) {
          bad |= KVQ_DEVERR_SEQ;
          continue;
        }
        const int32_t from = table[k / B];
        if (!page_ok(p, from)) bad |= KVQ_DEVERR_BLOCK;
        if (k == j) continue;  // stays where it is
        // (j < k < len: inside the row)
        const int32_t to = table[j / B];
        if (!page_ok(p, to))
          bad |= KVQ_DEVERR_BLOCK;
        else if (p.ref[to] != 1)
          bad |= KVQ_DEVERR_REF;
      }
  }
  if (bad != 0) flag(p.err, bad);
  const bool refused = __syncthreads_or(bad) != 0;
  for (int j = threadIdx.x; j < kept; j += kRowThreads) {
    int64_t from = -1, to = -1;
    if (!refused) {
      const int k = keep[j];
      from = static_cast<int64_t>(table[k / B]) * B + k % B;
      to = static_cast<int64_t>(table[j / B]) * B + j % B;
    }
    p.slots[at + j] = from;
    p.slots2[at + j] = to;
  }
}

__device__ __forceinline__ void drop_page(const PoolParams& p, int32_t page) {
  if (!page_ok(p, page)) {
    flag(p.err, KVQ_DEVERR_BLOCK);
    return;
  }
  if (atomicSub(p.ref + page, 1) <= 0) {
    atomicAdd(p.ref + page, 1);
    flag(p.err, KVQ_DEVERR_REF);
  }
}

// Second launch: the lengths, and the pages behind the kept tokens.
__global__ void __launch_bounds__(kRowThreads)
    compact_commit_kernel(const __grid_constant__ PoolParams p) {
  pdl_prologue();
  const int i = blockIdx.x, n = p.n, B = p.B;
  if (!offsets_ok(p.cu, n, p.total)) return;
  if (!row_once(p.ids, n, p.rows, i)) return;
  const int at = p.cu[i], kept = p.cu[i + 1] - at;
  const int id = p.ids[i];
  if (kept > 0 && p.slots2[at] < 0) return;  // refused
  const int len = p.lens[id];
  if (len < 0 || len > static_cast<int64_t>(p.width) * B) return;
  __syncthreads();
  if (threadIdx.x == 0) p.lens[id] = kept;
  int32_t* table = p.table + id * p.stride;
  for (int j = (kept + B - 1) / B + static_cast<int>(threadIdx.x);
       j < p.width; j += kRowThreads) {
    const int32_t page = table[j];
    if (page < 0) continue;
    table[j] = -1;
    drop_page(p, page);
  }
}

// ---------------------------------------------------------------------------
// free
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kRowThreads)
    free_kernel(const __grid_constant__ PoolParams p) {
  pdl_prologue();
  const int id = p.ids[blockIdx.x];
  if (id < 0 || id >= p.rows) {
    if (threadIdx.x == 0) flag(p.err, KVQ_DEVERR_SEQ);
    return;
  }
  int32_t* table = p.table + id * p.stride;
  for (int j = threadIdx.x; j < p.width; j += kRowThreads) {
    if (table[j] < 0) continue;
    // the exchange lets only one of two entries that name the row drop it
    const int32_t page = atomicExch(table + j, -1);
    if (page >= 0) drop_page(p, page);
  }
  if (threadIdx.x == 0) p.lens[id] = 0;
}

template <typename K>
cudaError_t launch_cluster(K kernel, const PoolParams& p,
                           cudaStream_t stream) {
  const size_t smem = pool_smem(p.rows, p.n);
  if (smem > 40 * 1024) {
    // the most that any call can need: the attribute is the kernel's, and a
    // size of this call's own could be put back by another host thread
    // before the launch
    const cudaError_t err = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        static_cast<int>(pool_smem(kPoolMaxRows, kPoolMaxList)));
    if (err != cudaSuccess) return err;
  }
  return launch_kernel(kernel, dim3(kCluster), kThreads, smem, stream, p.pdl,
                       p);
}

}  // namespace

cudaError_t launch_extend(const PoolParams& p, cudaStream_t stream) {
  const cudaError_t err = launch_cluster(extend_kernel, p, stream);
  if (err != cudaSuccess || p.total <= kClusterSlots) return err;
  const int64_t ctas = (p.total + kSlotThreads - 1) / kSlotThreads;
  return launch_kernel(slots_kernel,
                       dim3(static_cast<unsigned>(
                           ctas < 8 * sm_count() ? ctas : 8 * sm_count())),
                       kSlotThreads, 4 * static_cast<size_t>(p.n + 1), stream,
                       true, p);
}

cudaError_t launch_fork(const PoolParams& p, cudaStream_t stream) {
  return launch_cluster(fork_kernel, p, stream);
}

cudaError_t launch_compact(const PoolParams& p, cudaStream_t stream) {
  const cudaError_t err =
      launch_kernel(compact_check_kernel, dim3(p.n), kRowThreads, 0, stream,
                    p.pdl, p);
  if (err != cudaSuccess) return err;
  return launch_kernel(compact_commit_kernel, dim3(p.n), kRowThreads, 0,
                       stream, true, p);
}

cudaError_t launch_free(const PoolParams& p, cudaStream_t stream) {
  return launch_kernel(free_kernel, dim3(p.n), kRowThreads, 0, stream, p.pdl,
                       p);
}

}  // namespace kvq
