// chunk_attention.cu -- attention of a chunk of new tokens over the NVFP4
// pages, sm_103a: tcgen05 products with everything between them on chip.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

using dev::mbar_try;
using dev::smem_addr;

constexpr int kD = 128;                    // head_size
constexpr int kKeys = 128;                 // tokens of a KV tile
constexpr int kHalf = 128 * 128;           // bytes of half a tile (64 dims)
constexpr int kTile = 2 * kHalf;           // a [128 x 128] fp16 tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLag = 8.0f;               // see the softmax

// ---------------------------------------------------------------------------
// tcgen05 helpers
// ---------------------------------------------------------------------------
// Shared-memory matrix descriptors of a tile whose rows are 128 bytes (64
// fp16) with their 16-byte chunks XOR-swizzled by the row's low three bits
// (the hardware's 128-byte swizzle): `lbo` from one 64-element half to the
// next (used by the MN-major operand), 1024 bytes from one group of 8 rows
// to the next.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (uint64_t{1} << 46) |
         (uint64_t{2} << 61);
}

// kind::f16, fp16 operands, fp32 accumulator, M = N = 128.
constexpr uint32_t kIdesc =
    (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescBmn = kIdesc | (1u << 16);  // B is MN-major

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64"
      " [%0];" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

#define KVQ_R8(r, i) \
  "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), \
      "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define KVQ_I8(r, i) \
  "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
      "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of this warp's 32 TMEM lanes, one lane per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31}, [%32];"
      : KVQ_R8(r, 0), KVQ_R8(r, 8), KVQ_R8(r, 16), KVQ_R8(r, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31};" ::KVQ_I8(r, 0),
      KVQ_I8(r, 8), KVQ_I8(r, 16), KVQ_I8(r, 24), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------------------
// small helpers
// ---------------------------------------------------------------------------
__device__ __forceinline__ void flag(int32_t* err, int32_t bits) {
  if (err != nullptr) atomicOr(err, bits);
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar),
               "r"(count)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(
                   bar)
               : "memory");
}

// Wait for phase `parity`, for at most KVQ_WAIT_LIMIT_NS (and 2^24 polls),
// or until another thread of the CTA has given up.  False: give up.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity,
                                     volatile int* abort) {
  if (mbar_try(bar, parity)) return true;
  const uint64_t start = dev::global_ns();
  for (uint32_t polls = 0; polls < (1u << 24); ++polls) {
    if (mbar_try(bar, parity)) return true;
    if (*abort != 0) return false;
    if (dev::global_ns() - start > KVQ_WAIT_LIMIT_NS) break;
  }
  *abort = 1;
  return false;
}

// The same for a whole warp: true in every lane or in none.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity,
                                          volatile int* abort) {
  return __all_sync(0xFFFFFFFFu, wait(bar, parity, abort));
}

__device__ __forceinline__ void sts128(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

__device__ __forceinline__ uint4 ldg128(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg64(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b,
                                         uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t h;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  return pack_f16x2(__uint_as_float(w << 16),
                    __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
      : "=r"(h)
      : "h"(static_cast<uint16_t>(pair)));
  return h;
}

// Four bytes of e2m1 pairs times the f16x2 scale -> 8 fp16 (exact: the
// products have at most 6 significant bits).
__device__ __forceinline__ void dequant_word(uint32_t w, uint32_t sf2,
                                             uint32_t (&o)[4]) {
  asm("{ .reg .b8 q0, q1, q2, q3;\n"
      "  .reg .b32 h0, h1, h2, h3;\n"
      "  mov.b32 {q0, q1, q2, q3}, %4;\n"
      "  cvt.rn.f16x2.e2m1x2 h0, q0;  cvt.rn.f16x2.e2m1x2 h1, q1;\n"
      "  cvt.rn.f16x2.e2m1x2 h2, q2;  cvt.rn.f16x2.e2m1x2 h3, q3;\n"
      "  mul.rn.f16x2 %0, h0, %5;  mul.rn.f16x2 %1, h1, %5;\n"
      "  mul.rn.f16x2 %2, h2, %5;  mul.rn.f16x2 %3, h3, %5; }"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w), "r"(sf2));
}

// Whether one of a word's four e4m3 codes is NaN (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// ---------------------------------------------------------------------------
// The schedule
// ---------------------------------------------------------------------------
// Work is counted in units of one KV tile of one item; an item is a block of
// kRows rows (token, head of the KV head) of one sequence and KV head and
// spans the tiles up to its last row's position (one at least, so that rows
// that see nothing are written too).  The units of all items, in the order
// sequence, block, KV head, tile, are cut into equal shares, one per CTA; an
// item that is cut leaves partial results, which the merge kernel joins.
struct Seq {
  int q0, n, L;
};

__device__ __forceinline__ Seq seq_of(const ChunkParams& p, int b) {
  const int total = static_cast<int>(p.total_q);
  Seq s;
  s.q0 = min(max(__ldg(p.cu + b), 0), total);
  s.n = min(max(__ldg(p.cu + b + 1), s.q0), total) - s.q0;
  s.L = min(max(__ldg(p.lens + b), 0), p.len_cap);
  return s;
}

template <int kRows>
struct Schedule {
  // tiles of block i of a sequence
  static __device__ __forceinline__ int width(const ChunkParams& p,
                                              const Seq& s, int i) {
    const int last = min((i + 1) * kRows, s.n * p.G) - 1;  // last row
    const int seen = s.L - s.n + last / p.G + 1;
    return seen <= 0 ? 1 : (seen + kKeys - 1) / kKeys;
  }
  static __device__ __forceinline__ int blocks(const ChunkParams& p,
                                               const Seq& s) {
    return (s.n * p.G + kRows - 1) / kRows;
  }
  static __device__ __forceinline__ int64_t units(const ChunkParams& p,
                                                  const Seq& s) {
    int64_t u = 0;
    for (int i = 0, n = blocks(p, s); i < n; ++i) u += width(p, s, i);
    return u * p.Hkv;
  }
};

// A share's position: the next segment (one item's tiles kv0 .. kv1).
template <int kRows>
struct Walk {
  int b, block, h, kv0;
  int64_t left;  // units of the share from here on
  Seq s;
  int W, kv1;    // tiles of the item; end of this segment
  int row0, rows;

  __device__ __forceinline__ void load(const ChunkParams& p) {
    s = seq_of(p, b);
    enter(p);
  }
  __device__ __forceinline__ void enter(const ChunkParams& p) {
    W = Schedule<kRows>::width(p, s, block);
    kv1 = static_cast<int>(min(static_cast<int64_t>(W), kv0 + left));
    row0 = block * kRows;
    rows = min(kRows, s.n * p.G - row0);
  }
  // To the next segment; false at the end of the share.
  __device__ __forceinline__ bool next(const ChunkParams& p) {
    left -= kv1 - kv0;
    if (left <= 0) return false;
    kv0 = 0;
    if (++h == p.Hkv) {
      h = 0;
      if (++block == Schedule<kRows>::blocks(p, s)) {
        block = 0;
        do {
          if (++b >= p.num_seqs) return false;
          s = seq_of(p, b);
        } while (s.n == 0);
      }
    }
    enter(p);
    return true;
  }
};

// What the merge kernel needs of an item that begins in a CTA's share and
// goes on in the next ones': partial results in this CTA's slot `slot` and
// in slot 0 of the `more` CTAs behind it.
struct Cut {
  int32_t b, block, h, slot, more, pad[3];
};
constexpr int kMaxCtas = 512;
constexpr int64_t kCutBytes = kMaxCtas * sizeof(Cut);
constexpr int kSlotRows = 256;
constexpr int64_t kSlotFloats = kSlotRows * (kD + 2);

__device__ __forceinline__ float* slot_of(const ChunkParams& p, int cta,
                                          int slot) {
  return reinterpret_cast<float*>(p.workspace + kCutBytes) +
         (2 * static_cast<int64_t>(cta) + slot) * kSlotFloats;
}

// ---------------------------------------------------------------------------
// Shared memory
// ---------------------------------------------------------------------------
constexpr int kStages = 2;

template <int kTiles>
struct Smem {
  static constexpr int kQ = 0;                              // kTiles tiles
  static constexpr int kK = kQ + kTiles * kTile;            // kStages tiles
  static constexpr int kV = kK + kStages * kTile;           // kStages tiles
  static constexpr int kBar = kV + kStages * kTile;
  static constexpr int kBars = 4 * kStages + 4 * kTiles;
  static constexpr int kValid = kBar + 8 * 18;  // [4][4] words
  static constexpr int kNan = kValid + 64;      // [4][8][4] ints
  static constexpr int kMisc = kNan + 512;      // 16 ints
  static constexpr int kScan = kMisc + 64;      // 32 int64
  static constexpr int kBytes = kScan + 256 + 1024;  // 1024: alignment
  static_assert(kBars < 18 && kValid % 16 == 0, "");
};

// Roles of the warps: kTiles softmax warpgroups (one query tile each, one
// row per thread), one dequantising warpgroup (one token per thread), one
// warpgroup of which one thread issues the products.
template <int kTiles>
constexpr int kThreadsOf = 128 * (kTiles + 2);

template <int kTiles, bool kF16>
__global__ void __launch_bounds__(kThreadsOf<kTiles>, 1)
    chunk_kernel(const __grid_constant__ ChunkParams p) {
  using L = Smem<kTiles>;
  constexpr int kRows = 128 * kTiles;
  constexpr int kThreads = kThreadsOf<kTiles>;
  extern __shared__ __align__(16) uint8_t raw_smem[];
  uint8_t* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wg = warp >> 2;
  volatile int* misc = reinterpret_cast<volatile int*>(smem + L::kMisc);
  volatile int* abort = misc;                    // a wait gave up
  int* nan_at = reinterpret_cast<int*>(smem + L::kNan);
  int64_t* scan = reinterpret_cast<int64_t*>(smem + L::kScan);

  auto bar = [&](int i) { return base + L::kBar + 8 * i; };
  auto k_full = [&](int s) { return bar(s); };
  auto k_empty = [&](int s) { return bar(kStages + s); };
  auto v_full = [&](int s) { return bar(2 * kStages + s); };
  auto v_empty = [&](int s) { return bar(3 * kStages + s); };
  auto q_full = [&](int m) { return bar(4 * kStages + m); };
  auto s_full = [&](int m) { return bar(4 * kStages + kTiles + m); };
  auto p_full = [&](int m) { return bar(4 * kStages + 2 * kTiles + m); };
  auto o_done = [&](int m) { return bar(4 * kStages + 3 * kTiles + m); };

  if (warp == 0) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::
            "r"(base + L::kMisc + 4),
        "r"(256u * kTiles)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 32) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(k_full(s), 4);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), 4);
      mbar_init(v_empty(s), 1);
    }
    for (int m = 0; m < kTiles; ++m) {
      mbar_init(q_full(m), 4);
      mbar_init(s_full(m), 1);
      mbar_init(p_full(m), 4);
      mbar_init(o_done(m), 1);
    }
    misc[0] = 0;
    misc[2] = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < 128) nan_at[tid] = INT32_MAX;
  if (tid == 0)  // nothing to join, unless the end of this CTA says so
    (reinterpret_cast<Cut*>(p.workspace) + blockIdx.x)->more = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // --- this CTA's share -----------------------------------------------------
  // inclusive scan of the sequences' units, kThreads of them at a time; with
  // no more sequences than threads each is looked at once
  const int rounds = (p.num_seqs + kThreads - 1) / kThreads;
  int64_t units = 0, incl = 0, total = 0;
  auto scan_round = [&](int r, bool check) {
    const int b = r * kThreads + tid;
    units = 0;
    if (b < p.num_seqs) {
      const Seq s = seq_of(p, b);
      units = Schedule<kRows>::units(p, s);
      if (check && blockIdx.x == 0 &&
          (s.q0 != __ldg(p.cu + b) || s.q0 + s.n != __ldg(p.cu + b + 1) ||
           __ldg(p.lens + b) > s.L))
        flag(p.dev_error, KVQ_DEVERR_SEQ);
    }
    int64_t x = units;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
      if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += scan[w];
      all += scan[w];
    }
    incl = total + before + x;
    total += all;
  };
  for (int r = 0; r < rounds; ++r) scan_round(r, true);
  const int64_t U = total;
  const int ctas = static_cast<int>(
      min(static_cast<int64_t>(gridDim.x), max(U, int64_t{1})));
  const int cta = blockIdx.x;
  const int64_t u0 = cta < ctas ? U * cta / ctas : U;
  const int64_t u1 = cta < ctas ? U * (cta + 1) / ctas : U;
  if (rounds > 1) total = 0;
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) scan_round(r, false);
    if (units > 0 && u0 < u1 && incl - units <= u0 && u0 < incl) {
      const int b = r * kThreads + tid;
      const Seq s = seq_of(p, b);
      int64_t rem = u0 - (incl - units);
      int i = 0, w = Schedule<kRows>::width(p, s, 0);
      while (rem >= static_cast<int64_t>(w) * p.Hkv) {
        rem -= static_cast<int64_t>(w) * p.Hkv;
        w = Schedule<kRows>::width(p, s, ++i);
      }
      misc[2] = b;
      misc[3] = i;
      misc[4] = static_cast<int>(rem / w);
      misc[5] = static_cast<int>(rem % w);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[1]);
  Walk<kRows> walk;
  walk.b = misc[2];
  walk.block = misc[3];
  walk.h = misc[4];
  walk.kv0 = misc[5];
  walk.left = u1 - u0;
  const bool any = walk.b >= 0;
  if (any) walk.load(p);

  const float c0 = p.scale * __ldg(p.k_scale);

  if (wg < kTiles) {
    // --- softmax: tile m, one row per thread --------------------------------
    if constexpr (kTiles == 2)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int m = wg, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + 128 * m;
    const uint32_t o_col = tmem + lanes + 128 * kTiles + 128 * m;
    // (c0 == 0: a query of zeros, and any c > 0)
    const float c = c0 != 0.0f ? fabsf(c0) * kLog2e : 1.0f;
    const uint32_t flip = c0 < 0.0f ? 0x80008000u : 0u;
    const float v_scale = __ldg(p.v_scale);
    Cut cut = {0, 0, 0, 0, 0, {0, 0, 0}};
    uint32_t cnt = 0;    // tiles of this warpgroup so far
    uint32_t tiles = 0;  // tiles of the CTA so far
    int seg = 0;
    int64_t u = u0;
    bool go = any;
    while (go) {
      const int n_rows = walk.rows - 128 * m;  // rows of this tile
      if (n_rows > 0) {
        const int r = walk.row0 + 128 * m + row;   // row of the sequence
        const int tok = r / p.G;
        const bool live = row < n_rows;
        const int64_t q_row = walk.s.q0 + tok;
        const int head = walk.h * p.G + (r - tok * p.G);
        const int pos = live ? walk.s.L - walk.s.n + tok : -1;
        // the query row, rounded to fp16, its sign folded with the scale's
        {
          const uint16_t* src = p.q + q_row * p.q_stride0 + head * kD;
          const uint32_t dst = base + L::kQ + m * kTile + row * 128;
#pragma unroll
          for (int g = 0; g < 16; ++g) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (live && c0 != 0.0f) v = ldg128(src + 8 * g);
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = (kF16 ? w[k] : bf16x2_to_f16x2(w[k])) ^ flip;
            sts128(dst + (g >> 3) * kHalf + (((g & 7) ^ (row & 7)) << 4), w);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full(m));
        }
        float ref = -INFINITY, sum = 0.0f;
        for (int kt = walk.kv0; kt < walk.kv1; ++kt) {
          if (!warp_wait(s_full(m), cnt & 1, abort)) goto done;
          fence_after();
          uint32_t s[128];
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld32(s_col + 32 * k, s + 32 * k);
          const uint32_t* valid = reinterpret_cast<const uint32_t*>(
              smem + L::kValid + ((tiles + kt - walk.kv0) & 3) * 16);
          const uint32_t v0 = valid[0], v1 = valid[1], v2 = valid[2],
                         v3 = valid[3];
          tmem_wait_ld();
          const int lim = pos - kt * kKeys;  // columns 0 .. lim are seen
          const bool all = lim >= kKeys - 1 && (v0 & v1 & v2 & v3) == ~0u;
          if (!__all_sync(0xFFFFFFFFu, all)) {
            const uint32_t vs[4] = {v0, v1, v2, v3};
#pragma unroll
            for (int k = 0; k < 128; ++k)
              if (k > lim || !((vs[k >> 5] >> (k & 31)) & 1u))
                s[k] = 0xFF800000u;  // -inf
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 128; ++k)
            mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(s[k]));
          const float top =
              fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
          // The reference follows the maximum only when it lags by more
          // than kLag, so weights stay below 2^kLag and few tiles rescale.
          const bool move = top > ref + kLag;
          if (__any_sync(0xFFFFFFFFu, move)) {
            const float f = move ? ex2(ref - top) : 1.0f;
            if (move) {
              ref = top;
              sum *= f;
            }
            if (kt > walk.kv0) {
              if (!warp_wait(o_done(m), (cnt - 1) & 1, abort)) goto done;
              fence_after();
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t o[32];
                tmem_ld32(o_col + 32 * k, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tmem_st32(o_col + 32 * k, o);
              }
            }
          }
          const float low = ref == -INFINITY ? 0.0f : ref;
          float add[4] = {0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < 128; k += 2) {
            const float a = ex2(fmaf(__uint_as_float(s[k]), c, -low));
            const float b = ex2(fmaf(__uint_as_float(s[k + 1]), c, -low));
            add[k & 3] += a;
            add[(k & 3) + 1] += b;
            s[k >> 1] = pack_f16x2(a, b);
          }
          sum += (add[0] + add[1]) + (add[2] + add[3]);
          tmem_st32(s_col, s);
          tmem_st32(s_col + 32, s + 32);
          tmem_wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(m));
          ++cnt;
        }
        // --- epilogue -------------------------------------------------------
        if (!warp_wait(o_done(m), (cnt - 1) & 1, abort)) goto done;
        fence_after();
        const int4* nan_row =
            reinterpret_cast<const int4*>(nan_at + (seg & 3) * 32);
        const bool whole = walk.kv0 == 0 && walk.kv1 == walk.W;
        const float inv =
            sum > 0.0f ? v_scale / sum : (sum == 0.0f ? 0.0f : sum);
        float* slot = slot_of(p, cta, seg > 0);
        uint16_t* dst = p.out + q_row * p.out_stride0 + head * kD;
        float* part = slot + (128 * m + row) * kD;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(o_col + 32 * k, o);
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int4 at = nan_row[2 * k + g];
            if (min(min(at.x, at.y), min(at.z, at.w)) <= pos) {
#pragma unroll
              for (int j = 0; j < 16; ++j) o[16 * g + j] = 0x7FFFFFFFu;
            }
          }
          if (live && whole) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float x = __uint_as_float(o[8 * g + 2 * j]) * inv;
                const float y = __uint_as_float(o[8 * g + 2 * j + 1]) * inv;
                w[j] = kF16 ? pack_f16x2(x, y) : pack_bf16x2(x, y);
              }
              *reinterpret_cast<uint4*>(dst + 32 * k + 8 * g) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (live) {
#pragma unroll
            for (int g = 0; g < 8; ++g)
              *reinterpret_cast<uint4*>(part + 32 * k + 4 * g) =
                  make_uint4(o[4 * g], o[4 * g + 1], o[4 * g + 2],
                             o[4 * g + 3]);
          }
        }
        __syncwarp();
        if (!whole && live) {
          slot[kSlotRows * kD + 128 * m + row] = ref;
          slot[kSlotRows * (kD + 1) + 128 * m + row] = sum;
        }
        fence_before();
      }
      u += walk.kv1 - walk.kv0;
      tiles += walk.kv1 - walk.kv0;
      if (walk.kv0 == 0 && walk.kv1 < walk.W) {
        // goes on in the next CTAs' shares
        const int64_t end = u + (walk.W - walk.kv1);
        int more = 1;
        while (cta + more + 1 < ctas && U * (cta + more + 1) / ctas < end)
          ++more;
        cut = {walk.b, walk.block, walk.h, seg > 0, more, {0, 0, 0}};
      }
      ++seg;
      go = walk.next(p);
    }
    if (tid == 0)
      *(reinterpret_cast<Cut*>(p.workspace) + cta) = cut;
  } else if (wg == kTiles) {
    // --- dequantise: one token of a tile per thread --------------------------
    if constexpr (kTiles == 2)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    const int t = tid & 127;
    const uint32_t row_at = t * 128, sw = t & 7;
    // the tile ahead: coordinates, then raw bytes
    int kt = walk.kv0, seg = 0;
    bool have = any;
    uint4 kd[4], vd[4];
    uint2 ksc, vsc;
    bool k_ok = false, v_ok = false;  // token to be read
    uint32_t mask = 0;                // ballot: not to be left out
    const uint8_t *k_page = nullptr, *v_page = nullptr;
    int off = 0;
    // page of this thread's token of tile (walk, kt)
    auto locate = [&]() {
      const int pos = kt * kKeys + t;
      const bool in = pos < walk.s.L;
      const bool quad = (pos & ~3) < walk.s.L;  // (a quad is in one page)
      bool bad = false;
      k_ok = false;
      if (quad) {
        const int j = p.b_shift >= 0 ? pos >> p.b_shift : pos / p.B;
        off = pos - j * p.B;
        const int32_t blk = __ldg(p.block_table + walk.b * p.bt_stride + j);
        bad = blk < 0 || blk >= p.num_blocks;
        if (!bad) {
          k_ok = true;
          k_page = p.side[0] + blk * p.page_stride;
          v_page = p.side[1] + blk * p.page_stride;
        } else if (in) {
          flag(p.dev_error, KVQ_DEVERR_BLOCK);
        }
      }
      mask = __ballot_sync(0xFFFFFFFFu, !bad);
    };
    auto load_side = [&](const uint8_t* page, bool ok, bool in, bool swz,
                         uint4 (&d)[4], uint2& sc) {
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = make_uint4(0, 0, 0, 0);
      sc = make_uint2(0, 0);
      if (!ok) return;
      if (in) {
        const uint8_t* src = page + walk.h * p.dhs + off * p.dts;
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = ldg128(src + 16 * i);
      }
      // swizzled: row off % 4 of the 4-token band (other lanes' scales too)
      if (in || swz)
        sc = ldg64(page + p.scale_off + walk.h * p.shs + off * p.sts);
    };
    // dequantise a row into a tile; scale words in group order
    auto put = [&](const uint4 (&d)[4], uint32_t lo, uint32_t hi,
                   bool linear, uint32_t dst) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {  // groups 2g, 2g + 1
        const uint32_t pair =
            linear ? (g < 2 ? lo : hi) >> (16 * (g & 1))
                   : prmt(lo, hi, g | ((g + 4) << 4));
        const uint32_t sf = e4m3x2_to_f16x2(pair & 0xFFFFu);
        const uint32_t se = prmt(sf, sf, 0x1010u), so = prmt(sf, sf, 0x3232u);
        const uint32_t w[4] = {d[g].x, d[g].y, d[g].z, d[g].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
          dequant_word(w[i], i < 2 ? se : so, o);
          const int ch = 4 * g + i;  // 16-byte chunk of the row
          sts128(dst + (ch >> 3) * kHalf + row_at + (((ch & 7) ^ sw) << 4),
                 o);
        }
      }
    };
    // swizzled scales: 4 x 4 byte transposition over the quad's lanes, to
    // words of the even and the odd groups of this thread's token
    auto untwist = [&](uint32_t w) {
      const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
      const uint32_t z = prmt(w, y, (lane & 1) ? 0x3715u : 0x6240u);
      const uint32_t x = __shfl_xor_sync(0xFFFFFFFFu, z, 2);
      return prmt(z, x, (lane & 2) ? 0x3276u : 0x5410u);
    };

    uint32_t cnt = 0;
    bool in = false, in_v = false;
    if (have) {
      locate();
      in = k_ok && kt * kKeys + t < walk.s.L;
      load_side(k_page, k_ok, in, p.swizzle_k, kd, ksc);
      load_side(v_page, k_ok, in, true, vd, vsc);
      v_ok = k_ok;
      in_v = in;
    }
    while (have) {
      const int stage = cnt & 1;
      const uint32_t phase = (cnt >> 1) & 1;
      const int cur_kt = kt, cur_seg = seg;
      const bool first = kt == walk.kv0;
      const uint32_t cur_mask = mask;
      // K
      if (!warp_wait(k_empty(stage), phase ^ 1, abort)) goto done;
      {
        uint32_t lo = ksc.x, hi = ksc.y;
        if (p.swizzle_k) {
          lo = untwist(lo);
          hi = untwist(hi);
          if (!in) lo = hi = 0;
        }
        put(kd, lo, hi, !p.swizzle_k, base + L::kK + stage * kTile);
        if (lane == 0)
          reinterpret_cast<volatile uint32_t*>(
              smem + L::kValid)[(cnt & 3) * 4 + (warp & 3)] = cur_mask;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full(stage));
      }
      const bool in_now = in_v;
      // the next tile's K (its latency passes while V is converted)
      if (++kt == walk.kv1) {
        have = walk.next(p);
        kt = walk.kv0;
        ++seg;
      }
      if (have) {
        locate();
        in = k_ok && kt * kKeys + t < walk.s.L;
        load_side(k_page, k_ok, in, p.swizzle_k, kd, ksc);
      }
      // V
      if (!warp_wait(v_empty(stage), phase ^ 1, abort)) goto done;
      {
        // this warp's list of the segment's NaN places (last used four
        // segments ago)
        int* nan_row = nan_at + (cur_seg & 3) * 32 + (warp & 3);
        if (first) {
          if (lane < 8) nan_row[4 * lane] = INT32_MAX;
          __syncwarp();
        }
        uint32_t lo = untwist(vsc.x), hi = untwist(vsc.y);
        if (!in_now) lo = hi = 0;
        if ((nan_bytes(lo) | nan_bytes(hi)) != 0u) {
          // 0 * NaN would reach rows that do not see the token: its place
          // goes on the list, zeros into the tile
          uint32_t w[2] = {lo, hi};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int sh = 8 * (j >> 1);
            if (((w[j & 1] >> sh) & 0x7Fu) == 0x7Fu) {
              atomicMin(nan_row + 4 * j, cur_kt * kKeys + t);
              w[j & 1] &= ~(0xFFu << sh);
            }
          }
          lo = w[0];
          hi = w[1];
        }
        put(vd, lo, hi, false, base + L::kV + stage * kTile);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full(stage));
      }
      if (have) {
        load_side(v_page, k_ok, in, true, vd, vsc);
        in_v = in;
      }
      ++cnt;
    }
  } else {
    if constexpr (kTiles == 2)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (tid == (kTiles + 1) * 128 && any) {
      // --- products -----------------------------------------------------------
      uint32_t cnt = 0;  // KV tiles
      uint32_t q_phase[kTiles] = {}, done[kTiles] = {};
      auto qk = [&](int m, uint32_t n) {
        const uint32_t q = base + L::kQ + m * kTile;
        const uint32_t k = base + L::kK + (n & 1) * kTile;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t at = (i >> 2) * kHalf + (i & 3) * 32;
          mma_ss(tmem + 128 * m, smem_desc(q + at, 16),
                 smem_desc(k + at, 16), kIdesc, i > 0);
        }
        mma_commit(s_full(m));
      };
      bool go = true;
      while (go) {
        const int T = kTiles == 2 && walk.rows > 128 ? 2 : 1;
        const int n = walk.kv1 - walk.kv0;
        if (!wait(k_full(cnt & 1), (cnt >> 1) & 1, abort)) goto done;
        for (int m = 0; m < T; ++m) {
          if (!wait(q_full(m), q_phase[m] & 1, abort)) goto done;
          ++q_phase[m];
          fence_after();
          qk(m, cnt);
        }
        mma_commit(k_empty(cnt & 1));
        for (int j = 0; j < n; ++j, ++cnt) {
          for (int m = 0; m < T; ++m) {
            if (m == 0 &&
                !wait(v_full(cnt & 1), (cnt >> 1) & 1, abort))
              goto done;
            if (!wait(p_full(m), done[m] & 1, abort)) goto done;
            ++done[m];
            fence_after();
            const uint32_t v = base + L::kV + (cnt & 1) * kTile;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              mma_ts(tmem + 128 * kTiles + 128 * m, tmem + 128 * m + 8 * i,
                     smem_desc(v + i * 2048, kHalf), kIdescBmn,
                     j > 0 || i > 0);
            mma_commit(o_done(m));
            if (m == T - 1) mma_commit(v_empty(cnt & 1));
            if (j + 1 < n) {
              if (m == 0 && !wait(k_full((cnt + 1) & 1),
                                  ((cnt + 1) >> 1) & 1, abort))
                goto done;
              qk(m, cnt + 1);
              if (m == T - 1) mma_commit(k_empty((cnt + 1) & 1));
            }
          }
        }
        go = walk.next(p);
      }
    }
  }
done:
  __syncwarp();
  if (*abort != 0) {
    // products in flight end by themselves; wait for them before the tensor
    // memory goes
    if (tid == (kTiles + 1) * 128) {
      mbar_init(bar(L::kBars), 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      mma_commit(bar(L::kBars));
      for (int i = 0; i < 1 << 20 && !mbar_try(bar(L::kBars), 0); ++i) {
      }
      flag(p.dev_error, KVQ_DEVERR_TIMEOUT);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(
                     tmem),
                 "r"(256u * kTiles));
}

// ---------------------------------------------------------------------------
// The items that were cut: their parts joined
// ---------------------------------------------------------------------------
constexpr int kMergeRows = 32;  // rows of a CTA, four to a warp

template <int kTiles, bool kF16>
__global__ void __launch_bounds__(256)
    chunk_merge_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int kRows = 128 * kTiles;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int cta = blockIdx.x;
  const Cut cut = *(reinterpret_cast<const Cut*>(p.workspace) + cta);
  if (cut.more == 0) return;
  const Seq s = seq_of(p, cut.b);
  const int row0 = cut.block * kRows;
  const int rows = min(kRows, s.n * p.G - row0);
  const int lane = threadIdx.x & 31;
  const float vs = __ldg(p.v_scale);
  for (int i = 0; i < kMergeRows / 8; ++i) {
    const int row = blockIdx.y * kMergeRows + 8 * i + (threadIdx.x >> 5);
    if (row >= rows) return;
    float top = -INFINITY;
    for (int k = 0; k <= cut.more; ++k)
      top = fmaxf(top, slot_of(p, cta + k,
                               k == 0 ? cut.slot : 0)[kSlotRows * kD + row]);
    float sum = 0.0f;
    float4 o = make_float4(0, 0, 0, 0);
    for (int k = 0; k <= cut.more; ++k) {
      const float* slot = slot_of(p, cta + k, k == 0 ? cut.slot : 0);
      const float ref = slot[kSlotRows * kD + row];
      const float w = ref == top ? 1.0f : ex2(ref - top);
      sum += slot[kSlotRows * (kD + 1) + row] * w;
      const float4 x =
          *reinterpret_cast<const float4*>(slot + row * kD + 4 * lane);
      o.x += x.x * w;
      o.y += x.y * w;
      o.z += x.z * w;
      o.w += x.w * w;
    }
    const float inv = sum > 0.0f ? vs / sum : (sum == 0.0f ? 0.0f : sum);
    const int tok = (row0 + row) / p.G;
    const int head = cut.h * p.G + (row0 + row - tok * p.G);
    uint16_t* dst = p.out + (s.q0 + tok) * p.out_stride0 + head * kD +
                    4 * lane;
    uint2 w;
    w.x = kF16 ? pack_f16x2(o.x * inv, o.y * inv)
               : pack_bf16x2(o.x * inv, o.y * inv);
    w.y = kF16 ? pack_f16x2(o.z * inv, o.w * inv)
               : pack_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(dst) = w;
  }
}

template <int kTiles, bool kF16>
cudaError_t launch(const ChunkParams& p, cudaStream_t stream) {
  constexpr int kSmem = Smem<kTiles>::kBytes;
  const cudaError_t set = cudaFuncSetAttribute(
      chunk_kernel<kTiles, kF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
      kSmem);
  if (set != cudaSuccess) return set;
  const unsigned ctas = static_cast<unsigned>(sm_count());
  if (ctas > kMaxCtas) return cudaErrorInvalidConfiguration;
  const cudaError_t err =
      launch_kernel(chunk_kernel<kTiles, kF16>, dim3(ctas),
                    kThreadsOf<kTiles>, kSmem, stream, p.pdl, p);
  if (err != cudaSuccess) return err;
  return launch_kernel(chunk_merge_kernel<kTiles, kF16>,
                       dim3(ctas, 128 * kTiles / kMergeRows), 256, 0, stream,
                       true, p);
}

}  // namespace

int64_t chunk_workspace_bytes(int sms) {
  return kCutBytes + static_cast<int64_t>(sms) * 2 * kSlotFloats * 4;
}

cudaError_t launch_chunk_attention(const ChunkParams& p,
                                   cudaStream_t stream) {
  return p.f16 ? launch<2, true>(p, stream) : launch<2, false>(p, stream);
}

}  // namespace kvq
