// score_blocks.cu -- the indexer's score of every block of the context for
// every query row, over the paged e4m3 cache, sm_103a.
//
// For a query row and a token t that it sees, s_t = c_t * sum over heads of
// w_h max(0, q_h . k_t); a block's score is the largest of its tokens'.
//
// The dot products of a tile of 128 tokens with the heads of some rows are
// one tcgen05 product X = K Q^T (e4m3, M = 128 tokens, N = rows x heads, up
// to 128): a token is a lane of tensor memory, so that the sum over the heads
// stays in a thread, and the token's scale is multiplied once.  One CTA per
// SM:
//   * One warp has the pages' rows copied by TMA, a few tiles ahead, in boxes
//     of as many rows as divide both a page and a tile (whole pages of up to
//     128 tokens, mostly); two warps copy the scales, and the queries and
//     weights of a new row tile.
//   * One warp issues the products, into four accumulators of 128 columns in
//     turn.
//   * A warpgroup for each accumulator reads it, one token per thread, adds
//     up w_h max(0, x_h) for each row in packed fp32, and takes the largest
//     token of each block over the lanes.
// Rows of one sequence share a tile: up to 512 columns for longer chunks, so
// that a tile is read once for 8 rows of 64 heads.
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
constexpr int kColumns = 128;           // of an accumulator
constexpr int kAccs = 4;
constexpr int kEpiWarps = 4 * kAccs;    // a warpgroup for each accumulator
constexpr int kScaleWarps = 2;          // scales, queries, weights
constexpr int kTmaWarp = kEpiWarps + kScaleWarps, kMmaWarp = kTmaWarp + 1;
// (20 warps: 96 registers each)
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kMaxRows = kColumns / 16;  // of an accumulator

// Test builds only: in every other thread block an epilogue warp gives up at
// its third tile as if its wait there had run out (0 in the library).
#ifndef KVQ_TEST_SCORE_GIVE_UP
#define KVQ_TEST_SCORE_GIVE_UP 0
#endif

// kTiles: accumulators that share a tile of tokens (1, or 2 or 4 for longer
// chunks, with queries of as many times the size in shared memory).
template <int kTiles>
struct Smem {
  static constexpr int kStages = kTiles == 4 ? 5 : 8;
  static constexpr int kQueries = kTiles * kColumns * 128;
  static constexpr int kQ = 0;  // two row tiles, in turn
  static constexpr int kK = kQ + 2 * kQueries;
  static constexpr int kWeights = kK + kStages * kTile;
  static constexpr int kScales = kWeights + 2 * kTiles * kColumns * 4;
  static constexpr int kBest = kScales + kStages * kTokens * 4;
  static constexpr int kBar = kBest + kAccs * 2 * 4 * kMaxRows * 4;
  // [stage] its rows are there, [stage] its scales (and what came with them),
  // [stage] read, [accumulator] written, [accumulator] read,
  // [accumulator] its warps' maxima are there, [row tile & 1] begun, [row tile
  // & 1] read, the last
  static constexpr int kFull = 0, kScaled = kStages, kEmpty = 2 * kStages,
                       kDone = 3 * kStages,
                       kFree = kDone + kAccs, kJoined = kFree + kAccs,
                       kBegun = kJoined + kAccs, kRead = kBegun + 2,
                       kLast = kRead + 2;
  static constexpr int kMisc = kBar + (kLast + 1) * 8;  // abort, tmem address
  static constexpr int kScan = (kMisc + 16 + 7) / 8 * 8;
  static constexpr int kStart = kScan + 32 * 8;  // total, place, sequence
  static constexpr int kBytes = kStart + 32 + 1024;
  static_assert(kBytes <= 227 * 1024, "");
};

// kind::f8f6f4, e4m3 operands, fp32 accumulator, M = 128, K-major; N to add.
constexpr uint32_t kIdesc = (1u << 4) | ((128u >> 4) << 24);
// Shared-memory matrix descriptors, high word: rows of D bytes swizzled over
// D bytes, 8 D from one group of 8 rows to the next.  (The tokens' rows; the
// queries' are 128 bytes apart whatever D is.)
__device__ __forceinline__ uint32_t desc_hi(int D) {
  const uint32_t swizzle = D == 128 ? 2u : D == 64 ? 4u : 6u;
  return (8u * D >> 4) | (1u << 14) | (swizzle << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) {
  return ((addr >> 4) & 0x3FFFu) | (1u << 16);
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint32_t a, uint32_t a_hi,
                                       uint32_t b, uint32_t b_hi,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p;\n"
      "  .reg .b64 da, db;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  mov.b64 da, {%1, %5};\n"
      "  mov.b64 db, {%2, %6};\n"
      "  tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p; }" ::"r"(
          d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(a_hi), "r"(b_hi)
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
                 const __grid_constant__ CUtensorMap pages, int R, int Hp,
                 int box) {
  using S = Smem<kTiles>;
  extern __shared__ __align__(16) uint8_t raw_smem[];
  uint8_t* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* misc = reinterpret_cast<volatile int*>(smem + S::kMisc);
  volatile int* abort = misc;
  auto bar = [&](int i) { return base + S::kBar + 8 * i; };
  const int per = R / kTiles;  // rows of an accumulator

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
      // (each thread's copies, and each warp's ordinary stores)
      mbar_init(bar(S::kScaled + s), 33 * kScaleWarps);
      mbar_init(bar(S::kEmpty + s), 4 * kTiles);
    }
    for (int a = 0; a < kAccs; ++a) {
      mbar_init(bar(S::kDone + a), 2);
      mbar_init(bar(S::kFree + a), 4);
      mbar_init(bar(S::kJoined + a), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(S::kBegun + i), kScaleWarps);
      mbar_init(bar(S::kRead + i), kEpiWarps);
    }
    mbar_init(bar(S::kLast), 1);
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
    const double half = 0.5 * R, lin = kItem + max(walk.s.L - walk.s.n, 0) +
                                       half;
    int64_t i = static_cast<int64_t>(
        (sqrt(lin * lin + 4.0 * half * static_cast<double>(off)) - lin) /
        (2.0 * half));
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
  const int N = per * Hp;  // columns of an accumulator
  uint32_t issued = 0;     // (the TMA warp: tiles)

  if (any && warp < kEpiWarps) {
    // --- scores ---------------------------------------------------------------
    // accumulator g: columns m of the tiles `turn`, turn + kAccs / kTiles, ..
    const int g = warp >> 2, part = warp & 3;
    const int m = g % kTiles, turn = g / kTiles;
    const uint32_t acc = tmem + (static_cast<uint32_t>(part * 32) << 16) +
                         g * kColumns;
    float* best = reinterpret_cast<float*>(smem + S::kBest) +
                  g * 2 * 4 * kMaxRows;
    const int in_tile = kTokens / p.sel;
    const float none = -INFINITY;
    uint32_t cnt = 0, job = 0;  // tiles; jobs of this warpgroup
    for (uint32_t seg = 0;; ++seg) {
      // A warp that has no tile in a row tile would run ahead, and arrive
      // twice for another's part in kRead: the copies begin row tile seg
      // only once all have read seg - 2.
      if (!warp_wait(bar(S::kBegun + (seg & 1)), (seg >> 1) & 1, abort))
        goto done;
      const uint32_t weights = base + S::kWeights +
                               (seg & 1) * kTiles * kColumns * 4 + m * N * 4;
      const int row0 = walk.i * R + m * per;
      const int rows = min(per, walk.s.n - row0);  // (may be 0 or less)
      float* out = p.scores + (walk.s.q0 + row0) * p.scores_stride0;
      if (walk.t0 == 0) {  // columns behind the last tile
        const int from = min(walk.W * in_tile, p.columns);
        const int wide = p.columns - from;
        if (turn == 0)
          for (int r = part; r < rows; r += 4)
            for (int c = lane; c < wide; c += 32)
              out[r * p.scores_stride0 + from + c] = none;
      }
      for (int t = walk.t0; t < walk.t1; ++t, ++cnt) {
        if (cnt % (kAccs / kTiles) != static_cast<uint32_t>(turn)) continue;
        if (!warp_wait(bar(S::kDone + g), job & 1, abort)) goto done;
        fence_after();
        if (KVQ_TEST_SCORE_GIVE_UP != 0 && blockIdx.x % 2 == 1 && job == 2 &&
            part == 1) {
          *abort = 1;
          goto done;
        }
        const int stage = cnt % S::kStages;
        const float scale = *reinterpret_cast<const float*>(
            smem + S::kScales + (stage * kTokens + part * 32 + lane) * 4);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::kEmpty + stage));
        // tokens of the tile that row 0 sees (one more for each row)
        const int seen = walk.s.L - walk.s.n + row0 + 1 - t * kTokens;
        __syncwarp();
        const float mine =
            Hp % 32 == 0
                ? score_rows<32>(acc, weights, rows, Hp, scale,
                                 seen - part * 32 - lane, p.sel == 16)
                : score_rows<16>(acc, weights, rows, Hp, scale,
                                 seen - part * 32 - lane, p.sel == 16);
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::kFree + g));
        const int first = t * in_tile;
        if (p.sel <= 32) {
          const int r = lane & 15;
          const int c = first + (p.sel == 16 ? 2 * part + (lane >> 4) : part);
          if (r < rows && c < p.columns && (p.sel == 16 || lane < 16))
            out[r * p.scores_stride0 + c] = mine;
        } else {
          // (a warp is at most one job ahead of another: two places in turn)
          float* x_best = best + (job & 1) * 4 * kMaxRows;
          if (lane < kMaxRows) x_best[part * kMaxRows + lane] = mine;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(S::kJoined + g));
          if (!warp_wait(bar(S::kJoined + g), job & 1, abort)) goto done;
          const int at = tid & 127, r = at & 15, c = at >> 4;
          if (r < rows && c < in_tile && first + c < p.columns) {
            const int n = 4 / in_tile;  // warps of a block
            float s = none;
            for (int w = 0; w < n; ++w)
              s = fmaxf(s, x_best[(c * n + w) * kMaxRows + r]);
            out[r * p.scores_stride0 + first + c] = s;
          }
        }
        ++job;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(S::kRead + (seg & 1)));
      if (!walk.next(p, R, false)) break;
    }
  } else if (any && warp < kTmaWarp) {
    // --- scales, queries, weights ---------------------------------------------
    constexpr int kPer = kTokens / (32 * kScaleWarps);  // tokens of a thread
    const int here = tid - 32 * kEpiWarps;
    uint32_t cnt = 0;
    for (uint32_t seg = 0;; ++seg) {
      const int buf = seg & 1;
      if (seg >= 2 &&
          !warp_wait(bar(S::kRead + buf), ((seg >> 1) - 1) & 1, abort))
        goto done;
      if (lane == 0) mbar_arrive(bar(S::kBegun + buf));
      __syncwarp();
      // the row tile's queries (heads behind the last one and rows behind the
      // last are zeros) and weights
      const int row0 = walk.i * R, rows = min(R, walk.s.n - row0);
      const uint32_t q_to = base + S::kQ + buf * S::kQueries;
      const uint32_t w_to = base + S::kWeights + buf * kTiles * kColumns * 4;
      for (int c = here; c < R * Hp * 8; c += 32 * kScaleWarps) {
        const int line = c >> 3, r = line / Hp, h = line - r * Hp;
        if ((c & 7) >= p.D / 16) continue;
        const bool in = r < rows && h < p.heads;
        const uint8_t* from =
            in ? p.q + (walk.s.q0 + row0 + r) * p.q_stride0 + h * p.D +
                     16 * (c & 7)
               : p.q;
        asm volatile(
            "cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                q_to + line * 128 + (((c & 7) ^ (line & 7)) << 4)),
            "l"(from), "r"(in ? 16 : 0)
            : "memory");
      }
      for (int c = here; c < R * Hp; c += 32 * kScaleWarps) {
        const int r = c / Hp, h = c - r * Hp;
        const bool in = r < rows && h < p.heads;
        const float* from =
            in ? p.weights + (walk.s.q0 + row0 + r) * p.w_stride0 + h
               : p.weights;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                         w_to + 4 * c),
                     "l"(from), "r"(in ? 4 : 0)
                     : "memory");
      }
      const int32_t* table = p.block_table + walk.b * p.bt_stride;
      // the pages of this thread's tokens of tile t
      int32_t blk[kPer];
      auto look_up = [&](int t) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int pos = t * kTokens + i * 32 * kScaleWarps + here;
          blk[i] = -1;
          if (t < walk.t1 && pos < walk.s.L)
            blk[i] = __ldg(table +
                           (p.b_shift >= 0 ? pos >> p.b_shift : pos / p.B));
        }
      };
      look_up(walk.t0);
      for (int t = walk.t0; t < walk.t1; ++t, ++cnt) {
        const int stage = cnt % S::kStages;
        if (cnt >= S::kStages &&
            !warp_wait(bar(S::kEmpty + stage), (cnt / S::kStages - 1) & 1,
                       abort))
          goto done;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int r = i * 32 * kScaleWarps + here, pos = t * kTokens + r;
          const uint32_t to = base + S::kScales + (stage * kTokens + r) * 4;
          if (blk[i] >= 0 && blk[i] < p.num_blocks) {
            const int off = p.b_shift >= 0 ? pos & (p.B - 1) : pos % p.B;
            const uint8_t* from = p.cache + blk[i] * p.block_stride +
                                  static_cast<int64_t>(p.B) * p.D + 4 * off;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to),
                         "l"(from)
                         : "memory");
          } else {  // (left out: NaN is)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(0x7FFFFFFF)
                         : "memory");
            if (pos < walk.s.L) flag(p.rows.dev_error, KVQ_DEVERR_BLOCK);
          }
        }
        look_up(t + 1);
        // (the barrier counts this thread's copies when they land)
        asm volatile(
            "cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                bar(S::kScaled + stage))
            : "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::kScaled + stage));
      }
      if (!walk.next(p, R, false)) break;
    }
  } else if (any && warp == kTmaWarp) {
    // --- the pages' rows --------------------------------------------------------
    // A box for each lane (boxes of fewer than 4 rows: several, in turn); one
    // whose page is not a page lies outside the tensor and becomes zeros.
    // Boxes of fewer than 128 bytes (box == 0), which TMA cannot place, go by
    // rows of 16-byte copies, a tile at a time.
    const bool rows = box == 0;
    if (rows) box = 1;
    const int boxes = kTokens / box;
    uint32_t& cnt = issued;
    do {
      const int32_t* table = p.block_table + walk.b * p.bt_stride;
      auto look_up = [&](int t, int i) -> int32_t {
        const int pos = t * kTokens + i * box;
        return i < boxes && t < walk.t1 && pos < walk.s.L
                   ? __ldg(table +
                           (p.b_shift >= 0 ? pos >> p.b_shift : pos / p.B))
                   : -1;
      };
      int32_t blk = look_up(walk.t0, lane);
      for (int t = walk.t0; t < walk.t1; ++t, ++cnt) {
        const int stage = cnt % S::kStages;
        if (cnt >= S::kStages &&
            !warp_wait(bar(S::kEmpty + stage), (cnt / S::kStages - 1) & 1,
                       abort))
          goto done;
        const uint32_t to = base + S::kK + stage * kTile;
        const uint32_t full = bar(S::kFull + stage);
        // (rows behind the context stay as they are: nobody sees them)
        const int n = min(boxes, (max(walk.s.L - t * kTokens, 0) + box - 1) /
                                     box);
        if (rows) {
          for (int i = lane; i < n; i += 32) {
            if (i >= 32) blk = look_up(t, i);
            const bool ok = blk >= 0 && blk < p.num_blocks;
            const uint8_t* from = p.q;
            if (ok)
              from = p.cache + blk * p.block_stride +
                     (t * kTokens + i) % p.B * p.D;
            for (int c = 0; c < p.D; c += 16) {
              const int at = i * p.D + c;
              asm volatile(
                  "cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                      to + (at ^ (at >> 3 & (p.D - 16)))),
                  "l"(ok ? from + c : from), "r"(ok ? 16 : 0)
                  : "memory");
            }
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full);
          blk = look_up(t + 1, lane);
          continue;
        }
        if (lane == 0)
          asm volatile(
              "mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0],"
              " %1;" ::"r"(full),
              "r"(n * box * p.D)
              : "memory");
        __syncwarp();
        for (int i = lane; i < n; i += 32) {
          if (i >= 32) blk = look_up(t, i);
          const int pos = t * kTokens + i * box;
          const int off = p.b_shift >= 0 ? pos & (p.B - 1) : pos % p.B;
          asm volatile(
              "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::"
              "complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                  to + i * box * p.D),
              "l"(&pages), "r"(0), "r"(off),
              "r"(blk >= 0 && blk < p.num_blocks ? blk : -1), "r"(full)
              : "memory");
        }
        blk = look_up(t + 1, lane);
      }
    } while (walk.next(p, R, false));
  } else if (any) {
    // --- products ---------------------------------------------------------------
    const uint32_t k_hi = desc_hi(p.D), q_hi = desc_hi(128);
    const uint32_t idesc = kIdesc | (static_cast<uint32_t>(N >> 3) << 17);
    uint32_t cnt = 0, job = 0;
    for (uint32_t seg = 0;; ++seg) {
      const uint32_t q = base + S::kQ + (seg & 1) * S::kQueries;
      for (int t = walk.t0; t < walk.t1; ++t, ++cnt) {
        const int stage = cnt % S::kStages;
        if (!warp_wait(bar(S::kFull + stage), (cnt / S::kStages) & 1, abort) ||
            !warp_wait(bar(S::kScaled + stage), (cnt / S::kStages) & 1,
                       abort))
          goto done;
        fence_async_smem();  // (the queries' copies are ordinary writes)
        for (int m = 0; m < kTiles; ++m, ++job) {
          const int a = job % kAccs;
          if (job >= kAccs &&
              !warp_wait(bar(S::kFree + a), (job / kAccs - 1) & 1, abort))
            goto done;
          fence_after();
          if (elect()) {
            const uint32_t k = desc_lo(base + S::kK + stage * kTile);
            const uint32_t qd = desc_lo(q + m * N * 128);
            for (int x = 0; x < p.D / 32; ++x)
              mma_f8(tmem + a * kColumns, k + 2 * x, k_hi, qd + 2 * x, q_hi,
                     idesc, x > 0);
            mma_commit(bar(S::kDone + a));
            // (for what the loaders wrote by ordinary stores, too)
            mbar_arrive(bar(S::kDone + a));
          }
          __syncwarp();
        }
      }
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
    if (warp == kTmaWarp && box > 0)
      for (uint32_t k = issued > S::kStages ? issued - S::kStages : 0;
           k < issued; ++k)
        mbar_wait(bar(S::kFull + k % S::kStages), k / S::kStages & 1);
    if (warp == kMmaWarp) {
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

// The pages as a tensor [num_blocks, B, D] of bytes, copied in boxes of `box`
// rows of a page.
using EncodeTiled = decltype(&cuTensorMapEncodeTiled);
cudaError_t tensor_of_pages(const ScoreParams& p, int box, CUtensorMap* map) {
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
  const cuuint64_t sizes[3] = {static_cast<cuuint64_t>(p.D),
                               static_cast<cuuint64_t>(p.B),
                               static_cast<cuuint64_t>(std::max<int64_t>(
                                   std::min<int64_t>(p.num_blocks, INT32_MAX),
                                   1))};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.D),
                                 static_cast<cuuint64_t>(p.block_stride)};
  const cuuint32_t boxes[3] = {static_cast<cuuint32_t>(p.D),
                               static_cast<cuuint32_t>(box), 1};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult got = encode(
      map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(p.cache),
      sizes, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
      p.D == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
      : p.D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                  : CU_TENSOR_MAP_SWIZZLE_32B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return got == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int kTiles>
cudaError_t launch(const ScoreParams& p, int R, int Hp, cudaStream_t stream) {
  auto kernel = score_kernel<kTiles>;
  cudaError_t err = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
      Smem<kTiles>::kBytes);
  if (err != cudaSuccess) return err;
  int box = std::gcd(p.B, kTokens);
  CUtensorMap pages{};
  if (box * p.D % 128 != 0)
    box = 0;
  else
    err = tensor_of_pages(p, box, &pages);
  if (err != cudaSuccess) return err;
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
  return cudaLaunchKernelEx(&cfg, kernel, p, pages, R, Hp, box);
}

}  // namespace

cudaError_t launch_score_blocks(const ScoreParams& p, cudaStream_t stream) {
  const int Hp = (p.heads + 15) / 16 * 16;
  const int most = kColumns / Hp, q = std::max(p.max_q_len, 1);
  if (q <= most) return launch<1>(p, q, Hp, stream);
  if (q <= 2 * most) return launch<2>(p, 2 * most, Hp, stream);
  return launch<4>(p, 4 * most, Hp, stream);
}

}  // namespace kvq
