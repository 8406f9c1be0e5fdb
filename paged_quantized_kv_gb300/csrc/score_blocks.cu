// score_blocks.cu -- the indexer's score of every block of the context for
// every query row, over the paged e4m3 cache, sm_103a.
//
// For a query row and a token t that it sees, s_t = c_t * sum over heads of
// w_h max(0, q_h . k_t); a block's score is the largest of its tokens'.
//
// The dot products of a tile of 128 tokens with the heads of some rows are
// one tcgen05 product X = K Q^T (e4m3, M = 128 tokens, N = rows x heads): a
// token is a lane of tensor memory, so that the sum over the heads stays in a
// thread, and the token's scale is multiplied once.  One CTA per SM:
//   * One warp has the pages' rows and scales copied by TMA and bulk copies, a
//     few tiles ahead, in boxes of as many rows as divide both a page and a
//     tile (whole pages of up to 128 tokens, mostly).
//   * Two warps take turns to issue the products (what one spends between
//     two, 470 cycles of waits and commits, is hidden by the other's).
//   * Four warpgroups read the accumulators, one token per thread, add up w_h
//     max(0, x_h) for each row in packed fp32, and take the largest token over
//     the lanes.
//   * One warp has the queries and weights of the next row tile copied, joins
//     the warps' largest tokens of each block, and writes the scores.
// Rows of one sequence share a tile: up to 512 columns for longer chunks, so
// that a tile is read once for 8 rows of 64 heads.
//
// Measured: 1024 rows of 64 heads over 24576 tokens (404 GFLOP) 284 us, 1.42
// PFLOP/s; 77 rows of 48 sequences over 9001 to 33333 tokens (130 MB) 35 us,
// 3.7 TB/s, 55 % of the measured copy rate.  In copies with wrong results the
// first took 114 us without the sums over the heads and 84 without the products
// as well: the sums bound it.  No unit of theirs is full (57 % of the ALU's
// cycles, 20 % of the FMA's, 68 % of the issue slots): it took 248 us without
// the maximum with 0 and 269 without the weights' loads, and the rest is what a
// warp waits for from one load of 32 columns to the next, which the three others
// of its quarter cover in part.  The second took 29 us without the sums and 28
// without the products too, and takes 8 over contexts of two tokens: 7 us to
// start and to end, 21 for the copies (6.2 TB/s), 7 for sums that the copies do
// not cover.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <numeric>

#include "kvq.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

using namespace dev;

constexpr int kTokens = 128;            // of a tile
constexpr int kTile = kTokens * 128;    // bytes of its rows, 128 apart
constexpr int kGroups = 4;              // warpgroups that read accumulators
constexpr int kEpiWarps = 4 * kGroups;
constexpr int kRowWarp = kEpiWarps, kIssueWarp = kRowWarp + 1;
constexpr int kIssueWarps = 3;          // of copies and of products
// (20 warps: 96 registers each)
constexpr int kThreads = 32 * (kIssueWarp + kIssueWarps);

// Test builds only: in every other thread block a warp of each warpgroup gives
// up at its first or second product as if its wait there had run out (0 in
// the library).
#ifndef KVQ_TEST_SCORE_GIVE_UP
#define KVQ_TEST_SCORE_GIVE_UP 0
#endif

// The rows that share a tile of tokens are cut into kTiles parts of equal
// rows, one for a warpgroup each: kShare of them, side by side, are a product
// and an accumulator, kJobs products a tile.
//   1: single tokens and few heads; four accumulators of 128 columns.  Bound
//      by the copies: two warps issue them.
//   2, 4: two accumulators, half of each a warpgroup's.
//   8: of heads up to 64; all four warpgroups read one accumulator while the
//      other is written (1024 rows over 24576 tokens 291 us against 311 by 4).
// More rows need as many times the queries in shared memory.
template <int kTiles>
struct Smem {
  static constexpr int kShare = kTiles == 8 ? 4 : kTiles == 1 ? 1 : 2;
  static constexpr int kAccs = kTiles == 1 ? 4 : 2;
  static constexpr int kJobs = kTiles / kShare;
  static constexpr int kTmaWarps = kTiles == 1 ? 2 : 1;
  static constexpr int kMmaWarps = kIssueWarps - kTmaWarps;
  static constexpr int kMmaWarp = kIssueWarp + kTmaWarps;
  static constexpr int kColumns = kTiles == 8 ? 64 : 128;  // of a part
  static constexpr int kMaxRows = kColumns / 16;
  static constexpr int kStages = kTiles >= 4 ? 5 : 8;
  static constexpr int kQueries = kTiles * kColumns * 128;
  static constexpr int kQ = 0;  // two row tiles, in turn
  static constexpr int kK = kQ + 2 * kQueries;
  static constexpr int kWeights = kK + kStages * kTile;
  static constexpr int kScales = kWeights + 2 * kTiles * kColumns * 4;
  static constexpr int kBest = kScales + kStages * kTokens * 4;
  // (of a stage's tile: [part][half of the lanes][warp][row])
  static constexpr int kBestTile = kTiles * 2 * 4 * kMaxRows;
  static constexpr int kBar = kBest + kStages * kBestTile * 4;
  // [stage] filled, [stage] its tile's maxima are there, [stage] empty,
  // [accumulator] written, [accumulator] read, [row tile & 1] its queries are
  // there, [row tile & 1] read, the last ones
  static constexpr int kFull = 0, kScored = kStages, kEmpty = 2 * kStages,
                       kDone = 3 * kStages,
                       kFree = kDone + kAccs, kQuery = kFree + kAccs,
                       kRead = kQuery + 2, kLast = kRead + 2;
  static constexpr int kMisc = kBar + (kLast + 1) * 8;  // abort, tmem address
  static constexpr int kScan = (kMisc + 16 + 7) / 8 * 8;
  static constexpr int kStart = kScan + 32 * 8;  // total, place, sequence
  static constexpr int kBytes = kStart + 32 + 1024;
  static_assert(kBytes <= 227 * 1024, "");
  // (a stage is always filled by the same warp)
  static_assert(kStages % kTmaWarps == 0, "");
};

// kind::f8f6f4, e4m3 operands, fp32 accumulator, M = 128, K-major; N to add.
constexpr uint32_t kIdesc = (1u << 4) | ((128u >> 4) << 24);
// Shared-memory matrix descriptors, high word: rows of D bytes swizzled over
// D bytes, 8 D from one group of 8 rows to the next.
__device__ __forceinline__ uint32_t desc_hi(int D) {
  const uint32_t swizzle = D == 128 ? 2u : D == 64 ? 4u : 6u;
  return (8u * D >> 4) | (1u << 14) | (swizzle << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) {
  return ((addr >> 4) & 0x3FFFu) | (1u << 16);
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint32_t a, uint32_t b,
                                       uint32_t hi, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{ .reg .pred p;\n"
      "  .reg .b64 da, db;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  mov.b64 da, {%1, %5};\n"
      "  mov.b64 db, {%2, %5};\n"
      "  tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p; }" ::"r"(
          d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(hi)
      : "memory");
}

// ---------------------------------------------------------------------------
// The schedule
// ---------------------------------------------------------------------------
// An item is a row tile (R consecutive rows) of a sequence, and spans the
// tiles of tokens that its last row sees (one at least, so that rows that see
// nothing are written).  Its length is measured in tokens: kItem for its own,
// and as many as its last row sees, were the row tile full.  Item i of a
// sequence of n rows and L tokens so begins at i (kItem + max(L - n, 0)) + R
// i (i + 1) / 2: sums in closed form.  The lengths of all items one after the
// other are cut into equal shares, and a tile belongs to the share in which
// its first token falls.  (Blocks of scores lie within a tile: nothing is to
// be joined.)
constexpr int kItem = 256;

struct Seq {
  int q0, n, L;
};
__device__ __forceinline__ Seq seq_of(const ScoreParams& p, int b) {
  const int total = static_cast<int>(p.rows.total);
  Seq s;
  s.q0 = min(max(__ldg(p.rows.cu + b), 0), total);
  s.n = min(max(__ldg(p.rows.cu + b + 1), s.q0), total) - s.q0;
  s.L = min(max(__ldg(p.rows.lens + b), 0), p.rows.len_cap);
  return s;
}
__device__ __forceinline__ int64_t begin_of(const Seq& s, int R, int64_t i) {
  return i * (kItem + max(s.L - s.n, 0)) + R * (i * (i + 1) / 2);
}
__device__ __forceinline__ int items_of(const Seq& s, int R) {
  return (s.n + R - 1) / R;
}

// A warp's place in its share: the tiles t0 .. t1 - 1 of item i of sequence
// b; `at`: where the item begins.
struct Walk {
  int64_t at, u0, u1;
  Seq s;
  int b, i, items, W, t0, t1;

  __device__ __forceinline__ void enter(int R) {
    const int last = min((i + 1) * R, s.n);
    W = max((s.L - s.n + last + kTokens - 1) / kTokens, 1);
    const int64_t x0 = u0 - at - kItem, x1 = u1 - at - kItem;
    t0 = x0 <= 0 ? 0
                 : static_cast<int>(min((x0 + kTokens - 1) / kTokens,
                                        static_cast<int64_t>(W)));
    t1 = x1 <= 0 ? 0
                 : static_cast<int>(min((x1 + kTokens - 1) / kTokens,
                                        static_cast<int64_t>(W)));
  }
  // To the next item with a tile in the share (the first time: this one).
  __device__ __forceinline__ bool next(const ScoreParams& p, int R,
                                       bool first) {
    do {
      if (!first) {
        at += kItem + max(s.L - s.n, 0) + static_cast<int64_t>(R) * (i + 1);
        if (at >= u1) return false;
        if (++i == items) {
          do {
            if (++b >= p.rows.num_seqs) return false;
            s = seq_of(p, b);
          } while (s.n == 0);
          i = 0;
          items = items_of(s, R);
        }
      }
      first = false;
      enter(R);
    } while (t0 >= t1);
    return true;
  }
};

// max(0, x); NaN stays NaN.
__device__ __forceinline__ float relu(uint32_t x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(__uint_as_float(x)));
  return y;
}

// kWide columns of the accumulator at `acc`, and w max(0, x) of them added to
// `sum`, two at a time; w in shared memory.  (The weights are loaded while
// the columns are on their way: one after the other the two cost 10 %.)
template <int kWide>
__device__ __forceinline__ void add_columns(uint32_t acc, uint32_t weights,
                                            uint64_t (&sum)[4]) {
  uint32_t x[kWide];
  uint64_t w[kWide / 2];
  if constexpr (kWide == 32)
    tmem_ld32(acc, x);
  else
    tmem_ld16(acc, x);
#pragma unroll
  for (int k = 0; k < kWide / 2; k += 2)
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];"
                 : "=l"(w[k]), "=l"(w[k + 1])
                 : "r"(weights + 8 * k));
  tmem_wait_ld16(x);
  if constexpr (kWide == 32) tmem_wait_ld16(x + 16);
#pragma unroll
  for (int k = 0; k < kWide / 2; ++k)
    sum[k & 3] =
        fma2(pack2(relu(x[2 * k]), relu(x[2 * k + 1])), w[k], sum[k & 3]);
}

// The largest value over the warp's lanes (over each half's, for blocks of 16
// tokens).  No value is NaN.
__device__ __forceinline__ float largest(float s, bool halves) {
  if (!halves) {
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(s));
    return m;
  }
#pragma unroll
  for (int d = 8; d > 0; d >>= 1)
    s = fmaxf(s, __shfl_xor_sync(0xFFFFFFFFu, s, d));
  return s;
}

// One accumulator: the score of this lane's token for each of `rows` rows of
// Hp columns, and the largest over the lanes, lane r (and 16 + r) keeping row
// r's.  seen: this lane's token is seen by rows r > -seen.
template <int kWide>
__device__ __forceinline__ float score_rows(uint32_t acc, uint32_t weights,
                                            int rows, int Hp, float scale,
                                            int seen, bool halves) {
  const int lane = threadIdx.x & 31, key = halves ? lane & 15 : lane;
  float mine = -INFINITY;
#pragma unroll 1
  for (int r = 0; r < rows; ++r) {
    uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll 1
    for (int c = 0; c < Hp; c += kWide) {
      add_columns<kWide>(acc, weights, sum);
      acc += kWide;
      weights += 4 * kWide;
    }
    float a, b;
    unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
    const float s = (a + b) * scale;
    const float m = largest(seen + r > 0 && s == s ? s : -INFINITY, halves);
    if (key == r) mine = m;
  }
  return mine;
}

template <int kTiles>
__global__ void __launch_bounds__(kThreads, 1)
    score_kernel(const __grid_constant__ ScoreParams p,
                 const __grid_constant__ CUtensorMap pages,
                 const __grid_constant__ CUtensorMap queries, int R, int Hp,
                 int box_shift) {
  using S = Smem<kTiles>;
  extern __shared__ __align__(16) uint8_t raw_smem[];
  uint8_t* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* misc = reinterpret_cast<volatile int*>(smem + S::kMisc);
  volatile int* abort = misc;
  auto bar = [&](int i) { return base + S::kBar + 8 * i; };
  const int per = R / kTiles;  // rows of a part

  if (warp == 0) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
        ::"r"(base + S::kMisc + 4)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 32) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(bar(S::kFull + s), 1);
      mbar_init(bar(S::kScored + s), 4 * kTiles);
      mbar_init(bar(S::kEmpty + s), 1);
    }
    for (int a = 0; a < S::kAccs; ++a) {
      mbar_init(bar(S::kDone + a), 1);
      mbar_init(bar(S::kFree + a), 4 * S::kShare);
    }
    for (int i = 0; i < 2; ++i) {
      // (the weights' copies by each lane, and the queries' bytes)
      mbar_init(bar(S::kQuery + i), 33);
      mbar_init(bar(S::kRead + i), kEpiWarps + S::kMmaWarps);
    }
    mbar_init(bar(S::kLast), S::kMmaWarps);
    misc[0] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) check_rows(p.rows, tid, kThreads);

  // --- this CTA's share -----------------------------------------------------
  // (twice over the sequences: the total, then where the share begins)
  Walk walk;
  walk.u0 = walk.u1 = 0;
  {
    int64_t* scan = reinterpret_cast<int64_t*>(smem + S::kScan);
    volatile int64_t* start =
        reinterpret_cast<volatile int64_t*>(smem + S::kStart);
    const int rounds = (p.rows.num_seqs + kThreads - 1) / kThreads;
    int64_t U = 0, length = 0, incl = 0;
    if (tid == 0) start[1] = -1;
#pragma unroll 1
    for (int r = 0; r < (rounds > 1 ? 2 * rounds : 1); ++r) {
      if (r == rounds) U = 0;
      const int b = r % rounds * kThreads + tid;
      length = 0;
      if (b < p.rows.num_seqs) {
        const Seq s = seq_of(p, b);
        length = begin_of(s, R, items_of(s, R));
      }
      int64_t x = length;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
        if (lane >= d) x += y;
      }
      __syncthreads();
      if (lane == 31) scan[warp] = x;
      __syncthreads();
      incl = U + x;
#pragma unroll 1
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) incl += scan[w];
        U += scan[w];
      }
      if (r == rounds - 1) {
        // shares of a tile and a half at least
        const int64_t n = max(
            min(static_cast<int64_t>(gridDim.x), U / (kTokens + kTokens / 2)),
            int64_t{1});
        const int64_t cta = min(static_cast<int64_t>(blockIdx.x), n);
        walk.u0 = U / n * cta + min(cta, U % n);
        walk.u1 = min(cta + 1, n);
        walk.u1 = U / n * walk.u1 + min(walk.u1, U % n);
      }
      if ((rounds > 1 && r < rounds) || length == 0) continue;
      if (walk.u0 >= incl - length && walk.u0 < incl) {
        start[0] = incl - length;
        start[1] = b;
      }
    }
    __syncthreads();
    walk.b = static_cast<int>(start[1]);
    walk.at = start[0];
  }
  bool any = walk.u0 < walk.u1 && walk.b >= 0;
  if (any) {
    walk.s = seq_of(p, walk.b);
    walk.items = items_of(walk.s, R);
    // the item in which the share begins: the largest i whose begin is not
    // behind it
    const int64_t off = walk.u0 - walk.at;
    // (in fp32: fp64 arithmetic of all threads took 10 us here)
    const float half = 0.5f * R, x = static_cast<float>(off);
    const float lin = kItem + max(walk.s.L - walk.s.n, 0) + half;
    int64_t i = static_cast<int64_t>(
        2.0f * x / (lin + sqrtf(lin * lin + 4.0f * half * x)));
    i = min(max(i, int64_t{0}), static_cast<int64_t>(walk.items - 1));
    while (i > 0 && begin_of(walk.s, R, i) > off) --i;
    while (i + 1 < walk.items && begin_of(walk.s, R, i + 1) <= off) ++i;
    walk.i = static_cast<int>(i);
    walk.at += begin_of(walk.s, R, i);
    any = walk.next(p, R, true);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[1]);
  const int N = per * Hp;  // columns of a part
  uint32_t issued = 0, loads = 0;  // (the TMA warp's tiles; queries)

  if (any && warp < kEpiWarps) {
    // --- scores ---------------------------------------------------------------
    const int g = warp >> 2, part = warp & 3;
    const int h = g % S::kShare;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(part * 32) << 16) +
                           h * N;
    float* best = reinterpret_cast<float*>(smem + S::kBest) +
                  ((lane >> 4) * 4 + part) * S::kMaxRows + (lane & 15);
    const bool keeps = (lane & 15) < S::kMaxRows &&
                       (lane < 16 || p.sel == 16);
    uint32_t cnt = 0;  // tiles
    [[maybe_unused]] uint32_t test = 0;  // (of test builds: jobs)
    for (uint32_t seg = 0;; ++seg) {
      // (The queries of row tile seg come only once every warp that waits
      // for them, whether it has a tile in seg - 2 or not, has said that it is
      // through with that one: none runs ahead, and none misses a phase.)
      if (!warp_wait(bar(S::kQuery + (seg & 1)), (seg >> 1) & 1, abort))
        goto done;
      const uint32_t weights = base + S::kWeights +
                               (seg & 1) * kTiles * S::kColumns * 4;
      for (int t = walk.t0; t < walk.t1; ++t, ++cnt) {
        const int stage = cnt % S::kStages;
#pragma unroll
        for (int j = 0; j < S::kJobs; ++j) {
          const uint32_t job = cnt * S::kJobs + j;
          const int a = job % S::kAccs;
          if (S::kShare < kGroups && a != g / S::kShare) continue;
          if (!warp_wait(bar(S::kDone + a), job / S::kAccs & 1, abort))
            goto done;
          // (over as well: what orders the scales' copies before their reads)
          if (!warp_wait(bar(S::kFull + stage), cnt / S::kStages & 1, abort))
            goto done;
          fence_after();
          if (KVQ_TEST_SCORE_GIVE_UP != 0 && blockIdx.x % 2 == 1 &&
              test++ == blockIdx.x / 2 % 2 && part == 1) {
            *abort = 1;
            goto done;
          }
          const float scale = *reinterpret_cast<const float*>(
              smem + S::kScales + (stage * kTokens + part * 32 + lane) * 4);
          const int m = j * S::kShare + h;
          const int row0 = walk.i * R + m * per;
          const int rows = min(per, walk.s.n - row0);  // (may be 0 or less)
          // this lane's token is seen by rows from -seen on, counted from 1
          const int seen = walk.s.L - walk.s.n + row0 + 1 - t * kTokens -
                           part * 32 - lane;
          const uint32_t acc = lanes + a * (512 / S::kAccs);
          __syncwarp();
          const float mine =
              Hp % 32 == 0
                  ? score_rows<32>(acc, weights + m * N * 4, rows, Hp, scale,
                                   seen, p.sel == 16)
                  : score_rows<16>(acc, weights + m * N * 4, rows, Hp, scale,
                                   seen, p.sel == 16);
          if (keeps)
            best[stage * S::kBestTile + m * 8 * S::kMaxRows] = mine;
          fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(S::kFree + a));
            mbar_arrive(bar(S::kScored + stage));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(S::kRead + (seg & 1)));
      if (!walk.next(p, R, false)) break;
    }
  } else if (any && warp == kRowWarp) {
    // --- queries, weights, scores -----------------------------------------------
    Walk ahead = walk;  // the row tile whose queries come next
    bool more = true;
    auto load = [&](uint32_t seg) {
      const int buf = seg & 1;
      if (seg >= 2 &&
          !warp_wait(bar(S::kRead + buf), ((seg >> 1) - 1) & 1, abort))
        return false;
      const int row0 = ahead.i * R, rows = min(R, ahead.s.n - row0);
      const uint32_t q_to = base + S::kQ + buf * S::kQueries;
      const uint32_t w_to = base + S::kWeights + buf * kTiles * S::kColumns * 4;
      // (heads behind the last one are zeros, and so are their weights; rows
      // behind the sequence's last are not used)
      if (lane == 0)
        asm volatile(
            "mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], "
            "%1;" ::"r"(bar(S::kQuery + buf)),
            "r"(rows * Hp * p.D)
            : "memory");
      __syncwarp();
      if (lane < rows)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::"
            "complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                q_to + lane * Hp * p.D),
            "l"(&queries), "r"(0), "r"(0), "r"(ahead.s.q0 + row0 + lane),
            "r"(bar(S::kQuery + buf))
            : "memory");
      __syncwarp();
#pragma unroll 1
      for (int r = 0; r < rows; ++r) {
        const float* w = p.weights + (ahead.s.q0 + row0 + r) * p.w_stride0;
        for (int h = lane; h < Hp; h += 32) {
          const bool in = h < p.heads;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                           w_to + 4 * (r * Hp + h)),
                       "l"(in ? w + h : p.weights), "r"(in ? 4 : 0)
                       : "memory");
        }
      }
      // (the barrier counts this thread's copies when they land)
      asm volatile(
          "cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
              bar(S::kQuery + buf))
          : "memory");
      loads = seg + 1;
      more = ahead.next(p, R, false);
      return true;
    };
    if (!load(0)) goto done;
    const int in_tile = kTokens / p.sel;
    const int shift = 31 - __clz(in_tile);
    uint32_t cnt = 0;
    for (uint32_t seg = 0;; ++seg) {
      if (more && !load(seg + 1)) goto done;
      const int row0 = walk.i * R, rows = min(R, walk.s.n - row0);
      float* out = p.scores + (walk.s.q0 + row0) * p.scores_stride0;
      if (walk.t0 == 0) {  // columns behind the last tile
        const int from = min(walk.W * in_tile, p.columns);
        for (int r = 0; r < rows; ++r)
          for (int c = from + lane; c < p.columns; c += 32)
            out[r * p.scores_stride0 + c] = -INFINITY;
      }
      for (int t = walk.t0; t < walk.t1; ++t, ++cnt) {
        const int stage = cnt % S::kStages;
        const float* best = reinterpret_cast<const float*>(smem + S::kBest) +
                            stage * S::kBestTile;
        if (!warp_wait(bar(S::kScored + stage), cnt / S::kStages & 1, abort))
          goto done;
        // a block of a row for each lane
        for (int i = lane; i < rows << shift; i += 32) {
          const int row = i >> shift, c = i & (in_tile - 1), m = row / per;
          const float* from = best + m * 8 * S::kMaxRows + row - m * per;
          float s;
          if (p.sel == 16) {  // half c % 2 of warp c / 2
            s = from[((c & 1) * 4 + (c >> 1)) * S::kMaxRows];
          } else {
            from += c * (p.sel >> 5) * S::kMaxRows;
            s = from[0];
            if (p.sel >= 64) s = fmaxf(s, from[S::kMaxRows]);
            if (p.sel >= 128)
              s = fmaxf(s, fmaxf(from[2 * S::kMaxRows], from[3 * S::kMaxRows]));
          }
          if (t * in_tile + c < p.columns)
            out[row * p.scores_stride0 + t * in_tile + c] = s;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::kEmpty + stage));
      }
      if (!walk.next(p, R, false)) break;
    }
  } else if (any && warp < S::kMmaWarp) {
    // --- the pages' rows and scales ---------------------------------------------
    // A box of 2^box_shift rows for each lane; the pages of as many tiles as
    // there are lanes for are looked up at once.  Tokens whose page is not a
    // page get NaN for their scale: they are left out.
    // (Two such warps take turns: a tile's copies take one 1300 cycles to
    // issue.)
    const uint32_t who = warp - kIssueWarp;
    const bool bulk = box_shift >= 0;
    const int bits = bulk ? 7 - box_shift : 5;  // log2 of a tile's boxes
    const int batch = 32 >> bits;               // tiles of a look-up
    do {
      const int32_t* table = p.block_table + walk.b * p.bt_stride;
      // this lane's box of the batch: its page, place in it, its scales
      int32_t blk = -1;
      int off = 0;
      const uint8_t* scales = nullptr;
      uint32_t oks = 0, bads = 0;  // boxes that are pages, or should be
#pragma unroll 1
      for (int t = walk.t0; t < walk.t1; ++t, ++issued) {
        const int stage = issued % S::kStages;
        const uint32_t to = base + S::kK + stage * kTile;
        const uint32_t s_to = base + S::kScales + stage * kTokens * 4;
        const uint32_t full = bar(S::kFull + stage);
        const int turn = (t - walk.t0) & (batch - 1);
        if (!bulk && issued % S::kTmaWarps != who) continue;
        if (bulk && turn == 0) {
          const int64_t pos = static_cast<int64_t>(t) * kTokens +
                              (lane << box_shift);
          const bool seen = pos < min(walk.s.L, walk.t1 * kTokens);
          blk = -1;
          if (seen) {
            const int at = static_cast<int>(pos);
            const int page = p.b_shift >= 0 ? at >> p.b_shift : at / p.B;
            off = at - page * p.B;
            blk = __ldg(table + page);
          }
          const bool ok = blk >= 0 && blk < p.num_blocks;
          if (ok)
            scales = p.cache + blk * p.block_stride +
                     static_cast<int64_t>(p.B) * p.D + 4 * off;
          oks = __ballot_sync(0xFFFFFFFFu, ok);
          bads = __ballot_sync(0xFFFFFFFFu, seen && !ok);
          if (bads != 0 && lane == 0 && who == 0)
            flag(p.rows.dev_error, KVQ_DEVERR_BLOCK);
        }
        if (issued % S::kTmaWarps != who) continue;
        if (issued >= S::kStages &&
            !warp_wait(bar(S::kEmpty + stage),
                       (issued / S::kStages - 1) & 1, abort))
          goto done;
        if (bulk) {
          const uint32_t its =
              (bits == 5 ? ~0u : (1u << (1 << bits)) - 1u) << (turn << bits);
          const int i = lane - (turn << bits);  // the box in the tile
          if ((bads & its) != 0) {
            if (bads & its & 1u << lane)
              for (int k = 0; k < 1 << box_shift; ++k)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(
                                 s_to + 4 * ((i << box_shift) + k)),
                             "r"(0x7FFFFFFF)
                             : "memory");
            __syncwarp();
          }
          if (lane == 0)
            asm volatile(
                "mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, "
                "[%0], %1;" ::"r"(full),
                "r"((__popc(oks & its) << box_shift) * (p.D + 4))
                : "memory");
          __syncwarp();
          if (oks & its & 1u << lane) {
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::"
                "complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                    to + (i << box_shift) * p.D),
                "l"(&pages), "r"(0), "r"(off), "r"(blk), "r"(full)
                : "memory");
            asm volatile(
                "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::"
                "bytes [%0], [%1], %2, [%3];" ::"r"(
                    s_to + 4 * (i << box_shift)),
                "l"(scales), "r"(4 << box_shift), "r"(full)
                : "memory");
          }
          __syncwarp();
          continue;
        }
        // Boxes that the bulk copies cannot place: row by row, a tile at a
        // time.
        for (int i = lane; i < kTokens; i += 32) {
          const int pos = t * kTokens + i;
          if (pos >= walk.s.L) break;
          blk = __ldg(table + pos / p.B);
          const uint32_t s_at = s_to + 4 * i;
          if (blk < 0 || blk >= p.num_blocks) {
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(s_at),
                         "r"(0x7FFFFFFF)
                         : "memory");
            flag(p.rows.dev_error, KVQ_DEVERR_BLOCK);
            continue;
          }
          const uint8_t* page = p.cache + blk * p.block_stride;
          const int off = pos % p.B;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s_at),
                       "l"(page + static_cast<int64_t>(p.B) * p.D + 4 * off)
                       : "memory");
          for (int c = 0; c < p.D; c += 16) {
            const int at = i * p.D + c;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             to + (at ^ (at >> 3 & (p.D - 16)))),
                         "l"(page + off * p.D + c)
                         : "memory");
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
      }
    } while (walk.next(p, R, false));
  } else if (any) {
    // --- products ---------------------------------------------------------------
    const uint32_t hi = desc_hi(p.D);
    const uint32_t idesc =
        kIdesc | (static_cast<uint32_t>(S::kShare * N >> 3) << 17);
    const uint32_t mine = warp - S::kMmaWarp;
    uint32_t cnt = 0, job = 0;
    for (uint32_t seg = 0;; ++seg) {
      const uint32_t q = base + S::kQ + (seg & 1) * S::kQueries;
      if (!warp_wait(bar(S::kQuery + (seg & 1)), (seg >> 1) & 1, abort))
        goto done;
      for (int t = walk.t0; t < walk.t1; ++t, ++cnt) {
        const int stage = cnt % S::kStages;
#pragma unroll 1
        for (int j = 0; j < S::kJobs; ++j, ++job) {
          if (job % S::kMmaWarps != mine) continue;
          // (a tile's stage is not filled again before its products are read:
          // of the tiles that are not its own a warp need not see the phases)
          if (!warp_wait(bar(S::kFull + stage), (cnt / S::kStages) & 1, abort))
            goto done;
          const int a = job % S::kAccs;
          if (job >= S::kAccs &&
              !warp_wait(bar(S::kFree + a), (job / S::kAccs - 1) & 1, abort))
            goto done;
          fence_after();
          if (elect()) {
            const uint32_t k = desc_lo(base + S::kK + stage * kTile);
            const uint32_t qd = desc_lo(q + j * S::kShare * N * p.D);
            for (int x = 0; x < p.D / 32; ++x)
              mma_f8(tmem + a * (512 / S::kAccs), k + 2 * x, qd + 2 * x, hi,
                     idesc, x > 0);
            mma_commit(bar(S::kDone + a));
          }
          __syncwarp();
        }
      }
      if (lane == 0) mbar_arrive(bar(S::kRead + (seg & 1)));
      __syncwarp();
      if (!walk.next(p, R, false)) break;
    }
  }
done:
  __syncwarp();
  asm volatile("cp.async.wait_all;" ::: "memory");
  fence_before();
  __syncthreads();
  fence_after();
  if (*abort != 0) {  // (the same in every thread: all waits are over)
    // copies and products in flight end by themselves; wait for them before
    // the shared and the tensor memory go
    if (warp == kRowWarp)
      for (uint32_t k = loads > 2 ? loads - 2 : 0; k < loads; ++k)
        mbar_wait(bar(S::kQuery + (k & 1)), k >> 1 & 1);
    // (its own copies: what the other such warp has not begun never lands)
    if (warp >= kIssueWarp && warp < S::kMmaWarp && box_shift >= 0)
      for (uint32_t k = issued > S::kStages ? issued - S::kStages : 0;
           k < issued; ++k)
        if (k % S::kTmaWarps == static_cast<uint32_t>(warp - kIssueWarp))
          mbar_wait(bar(S::kFull + k % S::kStages), k / S::kStages & 1);
    if (warp >= S::kMmaWarp) {
      if (elect()) {
        mma_commit(bar(S::kLast));
        const uint64_t since = global_ns();
        while (!mbar_try(bar(S::kLast), 0) &&
               global_ns() - since < KVQ_WAIT_LIMIT_NS) {
        }
      }
      __syncwarp();
    }
    if (tid == 0) flag(p.rows.dev_error, KVQ_DEVERR_TIMEOUT);
    fence_before();
    __syncthreads();
    fence_after();
  }
  if (warp == 0)
    asm volatile(
        "tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// A tensor [outer, rows, D] of bytes, rows D and the outer ones `stride` apart,
// copied in boxes of `box` rows; what lies outside is zeros.
using EncodeTiled = decltype(&cuTensorMapEncodeTiled);
cudaError_t tensor_of(const uint8_t* at, int D, int64_t rows, int64_t outer,
                      int64_t stride, int box, CUtensorMap* map) {
  static const EncodeTiled encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                         cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t sizes[3] = {
      static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows),
      static_cast<cuuint64_t>(std::max<int64_t>(
          std::min<int64_t>(outer, INT32_MAX), 1))};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D),
                                 static_cast<cuuint64_t>(stride)};
  const cuuint32_t boxes[3] = {static_cast<cuuint32_t>(D),
                               static_cast<cuuint32_t>(box), 1};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult got = encode(
      map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(at), sizes,
      strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
      D == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
      : D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                : CU_TENSOR_MAP_SWIZZLE_32B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return got == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int kTiles>
cudaError_t launch(const ScoreParams& p, int R, int Hp, cudaStream_t stream) {
  auto kernel = score_kernel<kTiles>;
  static bool configured[64] = {false};  // per instantiation and device
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (!configured[dev & 63]) {
    err = cudaFuncSetAttribute(kernel,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Smem<kTiles>::kBytes);
    if (err != cudaSuccess) return err;
    configured[dev & 63] = true;
  }
  // (a power of two; the copies' places and sizes are multiples of 128 and 16
  // bytes)
  const int box = std::gcd(p.B, kTokens);
  int box_shift = -1;
  CUtensorMap pages{}, queries;
  err = tensor_of(p.q, p.D, p.heads, p.rows.total, p.q_stride0, Hp, &queries);
  if (err != cudaSuccess) return err;
  if (box >= 4 && box * p.D % 128 == 0) {
    for (box_shift = 2; 1 << box_shift < box;) ++box_shift;
    err = tensor_of(p.cache, p.D, p.B, p.num_blocks, p.block_stride, box,
                    &pages);
    if (err != cudaSuccess) return err;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sm_count()));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem<kTiles>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p, pages, queries, R, Hp, box_shift);
}

}  // namespace

cudaError_t launch_score_blocks(const ScoreParams& p, cudaStream_t stream) {
  const int Hp = (p.heads + 15) / 16 * 16;
  const int most = 128 / Hp, q = std::max(p.max_q_len, 1);
  if (q <= most) return launch<1>(p, q, Hp, stream);
  if (q <= 2 * most) return launch<2>(p, 2 * most, Hp, stream);
  if (Hp <= 64) return launch<8>(p, 8 * (64 / Hp), Hp, stream);
  return launch<4>(p, 4 * most, Hp, stream);
}

}  // namespace kvq
