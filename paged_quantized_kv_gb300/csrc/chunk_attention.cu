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
// (the hardware's 128-byte swizzle): `kLbo` bytes from one 64-element half to
// the next (used by the MN-major operand), 1024 bytes from one group of 8
// rows to the next.  The low word holds the address and kLbo, the high word
// is a constant.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
template <uint32_t kLbo>
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) {
  return ((addr >> 4) & 0x3FFFu) | ((kLbo >> 4) << 16);
}

// kind::f16, fp16 operands, fp32 accumulator, M = N = 128.
constexpr uint32_t kIdesc =
    (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescBmn = kIdesc | (1u << 16);  // B is MN-major

// D[tmem] (+)= A[smem] B[smem]; a, b: low descriptor words.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p;\n"
      "  .reg .b64 da, db;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  mov.b64 da, {%1, %5};\n"
      "  mov.b64 db, {%2, %5};\n"
      "  tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p; }" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHi)
      : "memory");
}

// D[tmem] (+)= A[tmem] B[smem].
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p;\n"
      "  .reg .b64 db;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  mov.b64 db, {%2, %5};\n"
      "  tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p; }" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHi)
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
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : KVQ_R8(r, 0), KVQ_R8(r, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::KVQ_I8(r, 0),
      KVQ_I8(r, 8), "r"(addr)
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
// One lane of the (converged) warp: the same one every time.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p;\n"
      "  elect.sync _|p, 0xFFFFFFFF;\n"
      "  selp.u32 %0, 1, 0, p; }"
      : "=r"(r));
  return r != 0;
}

// A value that every lane holds, told to the compiler as such.
__device__ __forceinline__ int uniform(int x) {
  return __shfl_sync(0xFFFFFFFFu, x, 0);
}

// Two fp32 at once: a * b + c, a + b.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b,
                                         uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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

// CTAs that get a share of U units.
__device__ __forceinline__ int ctas_of(int64_t U) {
  return static_cast<int>(
      min(static_cast<int64_t>(gridDim.x), max(U, int64_t{1})));
}

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
constexpr int kWalkBytes = 80;

template <int kTiles>
struct Smem {
  static constexpr int kQ = 0;                              // kTiles tiles
  static constexpr int kK = kQ + kTiles * kTile;            // kStages tiles
  static constexpr int kV = kK + kStages * kTile;           // kStages tiles
  static constexpr int kBar = kV + kStages * kTile;
  static constexpr int kBars = 4 * kStages + 4 * kTiles;
  // Per tile and quarter: the tokens that are not left out.  A filler is at
  // most a few tiles ahead of the softmax: K of tile k + 3 waits for the
  // products of tile k + 1, which wait for the weights of tile k.
  static constexpr int kValid = kBar + 8 * 18;  // [8][4] words
  // Per segment, group and quarter: the first token whose V scale is NaN.
  // V of tile k waits for the products of tile k - 2, so when segment s is
  // filled the epilogues of the segments up to s - 3 are over.
  static constexpr int kNan = kValid + 128;     // [8][8][4] ints
  static constexpr int kMisc = kNan + 1024;     // 16 ints
  static constexpr int kScan = kMisc + 64;      // 36 int64
  // The softmax warps' positions, kept out of their registers.
  static constexpr int kWalk = kScan + 288;
  static constexpr int kBytes =
      kWalk + 4 * kTiles * kWalkBytes + 1024;   // 1024: alignment
  static_assert(kBars < 18 && kValid % 16 == 0, "");
};

// Roles of the warps: kTiles softmax warpgroups (one query tile each, one
// row per thread), then one warp that issues the products and seven that
// dequantise (one token's K or V row per thread).  An SM quarter holds the
// registers of four warps of 128, so a 17th warp would cost every warp a
// quarter of its registers.
template <int kTiles>
constexpr int kThreadsOf = 128 * (kTiles + 2);
constexpr int kFillers = 7;

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
  if (tid < 256) nan_at[tid] = INT32_MAX;
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
  const int cta = blockIdx.x, ctas = ctas_of(U);
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
  if (tid == 0) {
    scan[32] = U;
    scan[33] = u0;
    scan[34] = u1;
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[1]);
  volatile int64_t* kept_units = scan + 32;  // U, u0, u1
  Walk<kRows> walk;
  walk.b = misc[2];
  walk.block = misc[3];
  walk.h = misc[4];
  walk.kv0 = misc[5];
  walk.left = kept_units[2] - kept_units[1];
  const bool any = walk.b >= 0;
  if (any) walk.load(p);

  if (wg < kTiles) {
    // --- softmax: tile m, one row per thread --------------------------------
    if constexpr (kTiles == 2)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    const int m = wg, row = tid & 127;
    const float c0 = p.scale * __ldg(p.k_scale);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + 128 * m;
    const uint32_t o_col = tmem + lanes + 128 * kTiles + 128 * m;
    // (c0 == 0: a query of zeros, and any c > 0)
    const float c = c0 != 0.0f ? fabsf(c0) * kLog2e : 1.0f;
    // A tile's logits take 128 registers.  The warp's position waits in
    // shared memory meanwhile.
    struct Kept {
      Walk<kRows> walk;
      int seg;
    };
    static_assert(sizeof(Kept) <= kWalkBytes, "");
    Kept* kept = reinterpret_cast<Kept*>(smem + L::kWalk + warp * kWalkBytes);
    if (lane == 0) *kept = {walk, 0};
    __syncwarp();
    uint32_t cnt = 0;  // tiles of this warpgroup so far
    bool go = any;
    while (go) {
      int kv0, kv1, pos, tiles, rows;
      {
        const Walk<kRows> w = kept->walk;
        kv0 = w.kv0;
        kv1 = w.kv1;
        rows = w.rows - 128 * m;  // rows of this tile
        // (tile kt of this segment is the CTA's (tiles + kt)-th)
        tiles = static_cast<int>(kept_units[2] - kept_units[1] - w.left) - kv0;
        const int r = w.row0 + 128 * m + row;  // row of the sequence
        const int tok = r / p.G;
        const bool live = row < rows;
        pos = live ? w.s.L - w.s.n + tok : -1;
        if (rows > 0) {
          // the query row, rounded to fp16, its sign folded with the scale's
          const uint16_t* src = p.q + (w.s.q0 + tok) * p.q_stride0 +
                                (w.h * p.G + (r - tok * p.G)) * kD;
          const uint32_t dst = base + L::kQ + m * kTile + row * 128;
          const uint32_t flip = c0 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
          for (int g = 0; g < 16; ++g) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (live && c0 != 0.0f) v = ldg128(src + 8 * g);
            uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[k] = (kF16 ? x[k] : bf16x2_to_f16x2(x[k])) ^ flip;
            sts128(dst + (g >> 3) * kHalf + (((g & 7) ^ (row & 7)) << 4), x);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full(m));
        }
      }
      if (rows > 0) {
        float ref = -INFINITY, sum = 0.0f;
        for (int kt = kv0; kt < kv1; ++kt) {
          if (!warp_wait(s_full(m), cnt & 1, abort)) goto done;
          fence_after();
          uint32_t s[128];
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld32(s_col + 32 * k, s + 32 * k);
          const uint32_t* valid = reinterpret_cast<const uint32_t*>(
              smem + L::kValid + ((tiles + kt) & 7) * 16);
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
          for (int k = 0; k < 128; k += 2)
            mx[(k >> 1) & 3] =
                max3(mx[(k >> 1) & 3], __uint_as_float(s[k]),
                     __uint_as_float(s[k + 1]));
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
            if (kt > kv0) {
              if (!warp_wait(o_done(m), (cnt - 1) & 1, abort)) goto done;
              fence_after();
#pragma unroll 1
              for (int k = 0; k < 8; ++k) {
                uint32_t o[16];
                tmem_ld16(o_col + 16 * k, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tmem_st16(o_col + 16 * k, o);
              }
            }
          }
          const float low = ref == -INFINITY ? 0.0f : ref;
          const uint64_t cc = pack2(c, c), ll = pack2(-low, -low);
          uint64_t add[2] = {0, 0};
#pragma unroll
          for (int k = 0; k < 128; k += 2) {
            float a, b;
            unpack2(fma2(pack2(__uint_as_float(s[k]),
                               __uint_as_float(s[k + 1])), cc, ll), a, b);
            a = ex2(a);
            b = ex2(b);
            add[(k >> 1) & 1] = add2(add[(k >> 1) & 1], pack2(a, b));
            s[k >> 1] = pack_f16x2(a, b);
          }
          float e, o;
          unpack2(add2(add[0], add[1]), e, o);
          sum += e + o;
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
        const Walk<kRows> w = kept->walk;
        const int seg = kept->seg;
        const int4* nan_row =
            reinterpret_cast<const int4*>(nan_at + (seg & 7) * 32);
        const bool live = row < rows;
        const bool whole = kv0 == 0 && kv1 == w.W;
        const float inv = sum > 0.0f ? __ldg(p.v_scale) / sum
                                     : (sum == 0.0f ? 0.0f : sum);
        float* slot = slot_of(p, blockIdx.x, seg > 0);
        const int r = w.row0 + 128 * m + row, tok = r / p.G;
        uint16_t* dst = p.out + (w.s.q0 + tok) * p.out_stride0 +
                        (w.h * p.G + (r - tok * p.G)) * kD;
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
      Walk<kRows> w = kept->walk;
      const int seg = kept->seg;
      if (tid == 0 && kv0 == 0 && kv1 < w.W) {
        // goes on in the next CTAs' shares
        const int64_t all = kept_units[0];
        const int64_t end = kept_units[2] - w.left + w.W;
        const int cta = blockIdx.x, ctas = ctas_of(all);
        int more = 1;
        while (cta + more + 1 < ctas && all * (cta + more + 1) / ctas < end)
          ++more;
        *(reinterpret_cast<Cut*>(p.workspace) + cta) = {
            w.b, w.block, w.h, seg > 0, more, {0, 0, 0}};
      }
      go = w.next(p);
      __syncwarp();
      if (lane == 0) *kept = {w, seg + 1};
      __syncwarp();
    }
  } else {
    if constexpr (kTiles == 2)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  }
  if (wg >= kTiles && warp != 4 * kTiles) {
    // --- dequantise: a quarter (32 tokens) of a tile's K or V at a time ------
    // The quarters K 0..3, V 0..3 of the share's tiles, in order, are dealt
    // round-robin to the warps.  A warp has three in hand: the one whose raw
    // bytes are in registers, the next one, whose page is known, and the one
    // behind it, whose block id is on its way (`job`, `kt` and `walk` are at
    // that one).
    int job = warp - 4 * kTiles - 1;  // 0..3: K quarters, 4..7: V quarters
    int kt = walk.kv0, seg = 0;
    uint32_t cnt = 0;      // tile of the share
    bool more = any;       // there is a tile at (walk, kt)
    int32_t blk = -1;      // the block id of this thread's token
    int pos = 0, off = 0;  // the token, and its place in the page
    bool quad = false;     // its 4-token band is inside the context
    auto look_up = [&]() {
      pos = kt * kKeys + 32 * (job & 3) + lane;
      quad = more && (pos & ~3) < walk.s.L;  // (a band is in one page)
      if (quad) {
        const int j = p.b_shift >= 0 ? pos >> p.b_shift : pos / p.B;
        off = pos - j * p.B;
        blk = __ldg(p.block_table + walk.b * p.bt_stride + j);
      }
    };
    // The next job.  Tokens that are not to be read load the query's first
    // bytes instead, and scale them by 0: loads without a branch need no
    // moves at the end of the loop, where they would wait for the data.
    const uint8_t *data = nullptr, *scales = nullptr;
    bool next_some = false, next_first = false, next_in = false;
    int next_pos = 0, next_job = 0;
    uint32_t next_mask = 0, next_cnt = 0, next_seg = 0;
    auto step = [&]() {
      bool bad = false;
      data = scales = reinterpret_cast<const uint8_t*>(p.q);
      next_in = false;
      next_some = more;
      next_pos = pos;
      next_job = job;
      next_cnt = cnt;
      next_seg = seg;
      next_first = kt == walk.kv0;
      const bool v = job >= 4;
      if (quad) {
        bad = blk < 0 || blk >= p.num_blocks;
        const bool in = pos < walk.s.L;
        if (!bad) {
          const uint8_t* page =
              (v ? p.side[1] : p.side[0]) + blk * p.page_stride;
          data = page + walk.h * p.dhs + off * p.dts;
          // swizzled: row off % 4 of the band, other lanes' scales too
          scales = page + p.scale_off + walk.h * p.shs + off * p.sts;
          next_in = in;
        } else if (in && !v) {
          flag(p.dev_error, KVQ_DEVERR_BLOCK);
        }
      }
      next_mask = __ballot_sync(0xFFFFFFFFu, !bad);
      if (more) {
        job += kFillers;
        if (job >= 8) {
          job -= 8;
          ++cnt;
          if (++kt == walk.kv1) {
            more = walk.next(p);
            kt = walk.kv0;
            ++seg;
          }
        }
        look_up();
      }
    };
    uint4 d[4];
    uint2 sc;
    auto load = [&](int i) {
      asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(d[i].x), "=r"(d[i].y), "=r"(d[i].z), "=r"(d[i].w)
                   : "l"(data + 16 * i));
    };
    auto load_scales = [&]() {
      asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];"
                   : "=r"(sc.x), "=r"(sc.y)
                   : "l"(scales));
    };
    // swizzled scales: 4 x 4 byte transposition over the band's lanes, to
    // words of the even and the odd groups of this thread's token
    auto untwist = [&](uint32_t w) {
      const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
      const uint32_t z = prmt(w, y, (lane & 1) ? 0x3715u : 0x6240u);
      const uint32_t x = __shfl_xor_sync(0xFFFFFFFFu, z, 2);
      return prmt(z, x, (lane & 2) ? 0x3276u : 0x5410u);
    };

    look_up();
    step();
#pragma unroll
    for (int i = 0; i < 4; ++i) load(i);
    load_scales();
    while (next_some) {
      const int stage = next_cnt & 1;
      const uint32_t phase = (next_cnt >> 1) & 1;
      const bool is_v = next_job >= 4, in = next_in;
      const int quarter = next_job & 3, cur_pos = next_pos;
      const bool swz = is_v || p.swizzle_k;
      const uint32_t mask = next_mask, cur = next_cnt, cur_seg = next_seg;
      const bool first = next_first;
      step();
      if (!warp_wait(is_v ? v_empty(stage) : k_empty(stage), phase ^ 1,
                     abort))
        goto done;
      if (!is_v && lane == 0)
        reinterpret_cast<volatile uint32_t*>(
            smem + L::kValid)[(cur & 7) * 4 + quarter] = mask;
      // this quarter's list of NaN places for the segment four ahead (its
      // last user, four back, is done: see kNan)
      if (is_v && first && lane < 8)
        nan_at[((cur_seg + 4) & 7) * 32 + 4 * lane + quarter] = INT32_MAX;
      uint32_t lo = sc.x, hi = sc.y;
      if (swz) {
        lo = untwist(lo);
        hi = untwist(hi);
      }
      if (!in) lo = hi = 0;
      if (is_v && (nan_bytes(lo) | nan_bytes(hi)) != 0u) {
        // 0 * NaN would reach rows that do not see the token: its place goes
        // on the list, zeros into the tile
        uint32_t w[2] = {lo, hi};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int sh = 8 * (j >> 1);
          if (((w[j & 1] >> sh) & 0x7Fu) == 0x7Fu) {
            atomicMin(nan_at + (cur_seg & 7) * 32 + 4 * j + quarter, cur_pos);
            w[j & 1] &= ~(0xFFu << sh);
          }
        }
        lo = w[0];
        hi = w[1];
      }
      const uint32_t dst = base + (is_v ? L::kV : L::kK) + stage * kTile +
                           (32 * quarter + lane) * 128;
      const uint32_t sw = lane & 7;
      load_scales();
#pragma unroll
      for (int g = 0; g < 4; ++g) {  // groups 2g, 2g + 1
        const uint32_t pair = swz ? prmt(lo, hi, g | ((g + 4) << 4))
                                  : (g < 2 ? lo : hi) >> (16 * (g & 1));
        const uint32_t sf = e4m3x2_to_f16x2(pair & 0xFFFFu);
        const uint32_t se = prmt(sf, sf, 0x1010u), so = prmt(sf, sf, 0x3232u);
        const uint32_t w[4] = {d[g].x, d[g].y, d[g].z, d[g].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
          dequant_word(w[i], i < 2 ? se : so, o);
          const int ch = 4 * g + i;  // 16-byte chunk of the row
          sts128(dst + (ch >> 3) * kHalf + (((ch & 7) ^ sw) << 4), o);
        }
        load(g);  // the next job's bytes into the registers just used
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(is_v ? v_full(stage) : k_full(stage));
    }
  } else if (warp == 4 * kTiles && any) {
    // --- products: the warp waits, one lane issues ---------------------------
    uint32_t cnt = 0;  // KV tiles
    uint32_t q_phase[kTiles] = {}, p_phase[kTiles] = {};
    auto qk = [&](int m, uint32_t n, bool last) {
      const uint32_t q = desc_lo<16>(base + L::kQ + m * kTile);
      const uint32_t k = desc_lo<16>(base + L::kK + (n & 1) * kTile);
      if (elect()) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t at = ((i >> 2) * kHalf + (i & 3) * 32) >> 4;
          mma_ss(tmem + 128 * m, q + at, k + at, kIdesc, i > 0);
        }
        mma_commit(s_full(m));
        if (last) mma_commit(k_empty(n & 1));
      }
      __syncwarp();
    };
    bool go = true;
    while (go) {
      const int T = kTiles == 2 && uniform(walk.rows) > 128 ? 2 : 1;
      const int n = uniform(walk.kv1 - walk.kv0);
      if (!warp_wait(k_full(cnt & 1), (cnt >> 1) & 1, abort)) goto done;
      for (int m = 0; m < T; ++m) {
        if (!warp_wait(q_full(m), q_phase[m] & 1, abort)) goto done;
        ++q_phase[m];
        fence_after();
        qk(m, cnt, m == T - 1);
      }
      for (int j = 0; j < n; ++j, ++cnt) {
        for (int m = 0; m < T; ++m) {
          if (m == 0 && !warp_wait(v_full(cnt & 1), (cnt >> 1) & 1, abort))
            goto done;
          if (!warp_wait(p_full(m), p_phase[m] & 1, abort)) goto done;
          ++p_phase[m];
          fence_after();
          const uint32_t v =
              desc_lo<kHalf>(base + L::kV + (cnt & 1) * kTile);
          if (elect()) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              mma_ts(tmem + 128 * kTiles + 128 * m, tmem + 128 * m + 8 * i,
                     v + i * (2048 >> 4), kIdescBmn, j > 0 || i > 0);
            mma_commit(o_done(m));
            if (m == T - 1) mma_commit(v_empty(cnt & 1));
          }
          __syncwarp();
          if (j + 1 < n) {
            if (m == 0 && !warp_wait(k_full((cnt + 1) & 1),
                                     ((cnt + 1) >> 1) & 1, abort))
              goto done;
            fence_after();
            qk(m, cnt + 1, m == T - 1);
          }
        }
      }
      go = walk.next(p);
    }
  }
done:
  __syncwarp();
  if (*abort != 0) {
    // products in flight end by themselves; wait for them before the tensor
    // memory goes
    if (warp == 4 * kTiles && elect()) {
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
