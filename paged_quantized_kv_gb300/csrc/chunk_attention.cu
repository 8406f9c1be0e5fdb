// chunk_attention.cu -- attention of a chunk of new tokens over the NVFP4
// pages, sm_103a: tcgen05 products with everything between them on chip.
//
// For the rows (new token, head of a KV head) of a sequence, with positions
// P: S = Q K^T, W = exp2(c S - reference) for the tokens t <= P, O = W V,
// out = O v_scale / sum W, where K = e2m1 * e4m3 in fp16 (exact: 6 bits) and
// c = scale * k_scale * log2 e.
//
// One CTA per SM.  Its unit of work is a KV tile of 128 tokens for up to two
// query tiles of 128 rows ("slots"):
//   * Fillers copy the tile's raw NVFP4 rows to shared memory two jobs ahead
//     and dequantise them into the operands' swizzled layouts, K (rows x
//     dims) and V (the same bytes, read MN-major): the cache is read as
//     NVFP4, once per 256 rows, and nothing dequantised leaves the SM.
//   * Product warps issue S (both operands in shared memory) and O += W V (W
//     in tensor memory): 16 tcgen05.mma of 128 x 128 x 16 per slot and tile,
//     512 cycles for each product (measured, the unit's full rate).
//   * Softmax warps hold a row per thread: logits from tensor memory, weights
//     back over them, no exchange between threads.  The reference comes from
//     the maximum of the first half tile; later ones go without theirs (see
//     kMost).
// Chunks of up to 128 rows have one query tile; its KV tiles alternate
// between the slots, whose two results the epilogue joins.
// Work is cut over the context into equal shares (the schedule below), so
// few rows over a long context use every SM; a second kernel joins the parts.
//
// Measured: 2048 tokens over 8192 with 64 query and 8 KV heads (481 GFLOP)
// 0.40 ms, 1202 TFLOP/s, 61 % of the measured bf16 rate; 500 over 131000 1.54
// ms, 1393 TFLOP/s, 71 %.  No pipe is saturated (on the first, by the
// counters: tensor cores 53 %, issue 49 %, exponentials and conversions 27 %).
// What bounds it is a slot's round, a chain of logits, softmax, weights and
// product through units that hand over to one another, with two slots in all:
// more do not fit tensor memory.  The softmax is the chain's longest link:
// with half of its exponentials left out (wrong results, a copy of an earlier
// step) the second case took 1.34 ms where that step took 1.60, without the
// dequantisation's conversions 1.60.  Alone, a softmax step of 128 x 128
// takes 1200 cycles with one slot's warps running and 1650 with both (the
// exponentials' unit takes one warp's in 4 cycles), and each hand-over some
// 340 for both ways.
// Sixteen softmax warps of half a row each were slower, 2.02 ms against 1.65.
// 16 tokens of 32 sequences over 2000 to 4000: 0.117 to 0.124 ms for 0.13 GB.  Chunks
// of a few tokens go through the decode kernel instead (short_chunk).
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
constexpr float kMost = 65504.0f;          // see the softmax
constexpr float kBelow = 8.0f;

// Test builds only: in three of four thread blocks one softmax warp, another
// from block to block, gives up at the end of the first or second segment as
// if its wait there had run out (0 in the library).
#ifndef KVQ_TEST_GIVE_UP
#define KVQ_TEST_GIVE_UP 0
#endif
__device__ __forceinline__ bool test_gives_up(int warp, uint32_t seg) {
  return KVQ_TEST_GIVE_UP != 0 && blockIdx.x % 4 != 3 &&
         warp == static_cast<int>(blockIdx.x * 3 % 8) &&
         seg == blockIdx.x / 8 % 2;
}

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
// or until another thread of the CTA has given up.  False: give up.  The
// timer is looked at only every 64th poll: reading it takes
// longer than most of these waits.
__device__ __forceinline__ bool keep_waiting(uint32_t polls, uint64_t* start,
                                          volatile int* abort) {
  if (*abort != 0) return false;
  const uint64_t now = dev::global_ns();
  if (*start == 0) *start = now;
  if (now - *start <= KVQ_WAIT_LIMIT_NS && polls < (1u << 24)) return true;
  *abort = 1;
  return false;
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity,
                                     volatile int* abort) {
  if (mbar_try(bar, parity)) return true;
  uint64_t start = 0;
#pragma unroll 1
  for (uint32_t polls = 1;; ++polls) {
    if (mbar_try(bar, parity)) return true;
    if (polls % 64 == 0 && !keep_waiting(polls, &start, abort)) return false;
  }
}

// The same for a whole warp: true in every lane or in none.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity,
                                          volatile int* abort) {
  return __all_sync(0xFFFFFFFFu, wait(bar, parity, abort));
}

// The same with every register of a tile live: no call, bounded by the count
// alone (of polls that do not suspend the warp).
__device__ __forceinline__ bool warp_spin(uint32_t bar, uint32_t parity,
                                          volatile int* abort) {
  uint32_t done = 0;
#pragma unroll 1
  for (uint32_t polls = 0; polls < (1u << 24) && !done; ++polls) {
    asm volatile(
        "{ .reg .pred p;\n"
        "  mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "  selp.u32 %0, 1, 0, p; }"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (polls % 256 == 255 && *abort != 0) break;
  }
  if (!done) *abort = 1;
  return __all_sync(0xFFFFFFFFu, done);
}

__device__ __forceinline__ void sts128(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

// Named barriers of warps that share TMEM lanes.
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(a));
  return v;
}
__device__ __forceinline__ void stg256(void* p, const uint32_t* v) {
  asm volatile(
      "st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
      "r"(v[6]), "r"(v[7])
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

// Four scales of every other group: zeros for those that are NaN, their
// token on the groups' lists (8 apart).
__device__ __noinline__ uint32_t drop_nan(uint32_t w, int* at, int pos) {
  for (int j = 0; j < 4; ++j)
    if (((w >> (8 * j)) & 0x7Fu) == 0x7Fu) {
      atomicMin(at + 8 * j, pos);
      w &= ~(0xFFu << (8 * j));
    }
  return w;
}

// -inf for the logits whose bit is not set.
__device__ __forceinline__ void mask32(uint32_t* s, uint32_t bits) {
#pragma unroll
  for (int k = 0; k < 32; ++k)
    if ((bits & (1u << k)) == 0u) s[k] = 0xFF800000u;
}
// The first lim + 1 of 32 bits.
__device__ __forceinline__ uint32_t first_bits(int lim) {
  return lim >= 31 ? ~0u : lim < 0 ? 0u : (2u << lim) - 1u;
}

__device__ __forceinline__ float max64(const uint32_t* s) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int k = 0; k < 64; k += 2)
    mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], __uint_as_float(s[k]),
                            __uint_as_float(s[k + 1]));
  return max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
}

// The output of this warp's rows, times each row's f.
__device__ __forceinline__ void rescale(uint32_t col, float f) {
#pragma unroll 1
  for (int k = 0; k < 8; ++k) {
    uint32_t o[16];
    tmem_ld16(col + 16 * k, o);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j)
      o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
    tmem_st16(col + 16 * k, o);
  }
}

// ---------------------------------------------------------------------------
// The schedule
// ---------------------------------------------------------------------------
// An item is a block of up to kRows = 256 rows (token, head of the KV head)
// of one sequence and KV head; it spans the KV tiles up to its last row's
// position (one at least, so that rows that see nothing are written too).  It
// counts as kItemUnits units for its own (query, output: measured at some 6
// us against 2 us for a tile, whether half of its rows are used or all) and
// one for each tile.  The units of all items, in the order sequence, block,
// KV head, tile, are cut into equal shares, one per CTA; an item that is cut
// leaves partial results, which the merge kernel joins.  Every share has more
// than kItemUnits units, so that none in the middle of an item is without a
// tile.
// A cut costs two partial results (a full one: 133 KB written and read
// again).  So the end of a share within kSnap units of an item's end moves
// there.
constexpr int kRows = 256;
constexpr int kItemUnits = 3;
constexpr int kSnap = 2;

// Where a share's end at unit r of an item of `size` units falls.
__device__ __forceinline__ int snap(int r, int size) {
  if (min(r, size - r) > kSnap) return r;
  return r <= size - r ? 0 : size;
}

struct Seq {
  int q0, n, L;
};

__device__ __forceinline__ Seq seq_of(const ChunkParams& p, int b) {
  const int total = static_cast<int>(p.total_q);
  Seq s;
  s.q0 = min(max(__ldg(p.cu + b), 0), total);
  s.n = min(max(__ldg(p.cu + b + 1), s.q0), total) - s.q0;
  s.L = min(max(__ldg(p.lens + b), 0), p.len_cap);
  if (s.n <= p.skip) s.n = 0;
  return s;
}

// The blocks of a sequence, one after the other.  Block i ends with row
// min(256 (i + 1), n G) - 1, whose token sees L - n + row / G + 1 tokens:
// floor((row + G (L - n + 128)) / (128 G)) tiles.  From block to block the
// row grows by 256, and the quotient is carried along.  (Rows are below 2^29,
// contexts at most 2^26 tokens, groups at most 16: 32 bits.)
struct Blocks {
  int left;   // rows from this block on
  int step;   // 128 G
  int tiles;  // of the block, were it full
  int rest;   // of that division

  __device__ __forceinline__ void begin(const ChunkParams& p, const Seq& s,
                                        int i) {
    step = 128 * p.G;
    left = s.n * p.G - i * kRows;
    const int top = i * kRows + kRows - 1 + p.G * (s.L - s.n + 128);
    tiles = max(top, 0) / step;
    rest = top - tiles * step;
  }
  __device__ __forceinline__ void next() {
    left -= kRows;
    rest += kRows;
    while (rest >= step) {
      rest -= step;
      ++tiles;
    }
  }
  // Tiles of this block (a last block that is not full ends earlier).
  __device__ __forceinline__ int width() const {
    const int short_by = max(kRows - left, 0) - rest;
    return max(tiles - (short_by > 0) - (short_by > step), 1);
  }
  __device__ __forceinline__ int units() const {
    return kItemUnits + width();
  }
};

// Shares of U units: the first ones are one unit longer than the others.
__device__ __noinline__ int64_t share_begin(int64_t U, int cta, int* ctas) {
  const int64_t most = U / (kItemUnits + 2);
  const int n = static_cast<int>(
      min(static_cast<int64_t>(gridDim.x), max(most, int64_t{1})));
  *ctas = n;
  if (cta >= n) return U;
  const int64_t size = U / n;
  return size * cta + min(static_cast<int64_t>(cta), U - size * n);
}

// A position in a share: one segment, the tiles kv0 .. kv1 - 1 of one item.
struct Walk {
  int b, block, h;
  int rem, end;   // the segment's units, from the item's first one
  int64_t left;   // units of the share from here on
  Seq s;
  int W;          // tiles of the item
  int kv0, kv1;
  int two;        // it has two query tiles (more than 128 rows)
  int seg, tiles;  // segments and tiles of the share before this one
  int there;       // (in the ring) this segment exists

  __device__ __forceinline__ void enter(const ChunkParams& p) {
    Blocks k;
    k.begin(p, s, block);
    W = k.width();
    two = k.left > 128;
    end = static_cast<int>(min(static_cast<int64_t>(k.units()), rem + left));
    kv0 = max(rem - kItemUnits, 0);
    kv1 = max(end - kItemUnits, 0);
  }
  // To the next segment that has a tile (the first one: from a position with
  // rem set and kv0 == kv1); false: there is none.
  __device__ __forceinline__ bool next(const ChunkParams& p, bool first) {
    if (!first) {
      ++seg;
      tiles += kv1 - kv0;
    }
    do {
      if (!first) {
        left -= end - rem;
        rem = 0;
        if (left <= 0) return false;
        if (++h == p.Hkv) {
          h = 0;
          if (++block * kRows >= s.n * p.G) {
            block = 0;
            do {
              if (++b >= p.num_seqs) return false;
              s = seq_of(p, b);
            } while (s.n == 0);
          }
        }
      }
      first = false;
      enter(p);
    } while (kv0 >= kv1);
    return true;
  }
};

// The position of the product warp and of each filler is in shared memory,
// moved on by the warp's first lane, out of line: a copy of this code in
// each role would be larger than the loops it serves.  True for the whole
// warp if there is another segment.  (The softmax warps take theirs from the
// product warp, through a ring: a call would cost them registers.)
__device__ __noinline__ bool advance(const ChunkParams& p, Walk* walk) {
  bool more = false;
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    Walk w = *walk;
    more = w.next(p, false);
    *walk = w;
  }
  __syncwarp();
  return __shfl_sync(0xFFFFFFFFu, more, 0);
}

// What the merge kernel needs of an item that begins in a CTA's share and
// goes on in the next ones': partial results in this CTA's slot `slot` and
// in slot 0 of the `more` CTAs behind it.  And whether a wait of this CTA
// gave up: an item with a part of such a CTA is left out.
struct Cut {
  int32_t b, block, h, slot, more, gave_up, pad[2];
};
constexpr int kMaxCtas = 512;
constexpr int64_t kCutBytes = kMaxCtas * sizeof(Cut);
constexpr int64_t kSlotFloats = kRows * (kD + 2);  // output, reference, sum

__device__ __forceinline__ float* slot_of(const ChunkParams& p, int cta,
                                          int slot) {
  return reinterpret_cast<float*>(p.workspace + kCutBytes) +
         (2 * static_cast<int64_t>(cta) + slot) * kSlotFloats;
}

// A segment that begins an item and does not end it: which CTAs go on with
// it.
__device__ __noinline__ void note_cut(const ChunkParams& p, const Walk& w,
                                      int64_t U, int64_t share_end) {
  const int64_t begin = share_end - w.left - w.rem;
  const int size = kItemUnits + w.W;
  const int cta = blockIdx.x;
  int more = 0, ctas;
  int64_t end;
  do {
    ++more;
    end = share_begin(U, cta + more + 1, &ctas) - begin;
  } while (end < size && snap(static_cast<int>(end), size) < size);
  *(reinterpret_cast<Cut*>(p.workspace) + cta) = {
      w.b, w.block, w.h, w.seg > 0, more, 0, {0, 0}};
}

// ---------------------------------------------------------------------------
// Roles, barriers, shared memory
// ---------------------------------------------------------------------------
// Warps 0 .. 7: softmax, a warpgroup for each slot (query tile), one row per
// thread.  Warps 8 and 9 issue the products of slot 0 and 1: the tensor cores
// queue hardly more than one instruction, so what a warp spends between two
// batches of them (waits, commits) is hidden only by the other warp's.  Warps
// 10 .. 15 (fillers) dequantise.
// (16 warps of 128 registers fill the register file; a split of the registers
// by role, softmax 176 and the others 80, was 2 % slower, 420 us against 411
// at 2048 tokens over 8192, halves of the softmax not unrolled.)
constexpr int kSoftWarps = 8;
constexpr int kFillers = 6;
constexpr int kThreads = 32 * (kSoftWarps + 2 + kFillers);
constexpr int kStages = 2;
// Barriers that say that a tile's products are done, taken in turn by the
// tiles.  A filler has no quarter of K and V both in every tile and so does
// not look at every phase.  By a barrier for each stage it could take tile
// t - 4's product with V, still running for one slot while the other was
// ahead, for that of t - 2, and fill the tile under it.  With four barriers
// the one that it waits on last stood for tile t - 6, which was done before
// whatever the filler waited for at t - 2, where it had work.
constexpr int kEmpties = 4;
// Barriers that announce segments, taken in turn.  With one, slot 1's softmax
// warps could miss a phase: a product warp announces segment s + 2 once slot
// 0's query of s + 1 is there, while slot 1's warps may still be in the
// epilogue of s, and then wait for s + 1 by the parity that s + 2 has turned
// back (many short items, or a short one behind one of two query tiles: the
// waits gave up).  Segment s + 3 is announced only behind slot 1's warps'
// part in s + 1: two are enough.
constexpr int kAnnounced = 2;

enum Bar {
  kKFull = 0,                  // [stage] a tile of K is in shared memory
  kKEmpty = kKFull + kStages,  // [tile % kEmpties] its products are done
  kVFull = kKEmpty + kEmpties,
  kVEmpty = kVFull + kStages,
  kQFull = kVEmpty + kEmpties,  // [slot] the query rows are in shared memory
  kSFull = kQFull + 2,         // [slot] logits are in tensor memory
  kPFull = kSFull + 2,         // [slot][half] weights are in tensor memory
  kPDone = kPFull + 4,         // [slot] the first half is multiplied with V
  kODone = kPDone + 2,         // [slot] all of them are
  kTurn = kODone + 2,          // [slot] the tensor cores are this slot's
  kOFree = kTurn + 2,          // the segment's output has been read
  kSegment = kOFree + 1,       // [segment % kAnnounced] it is in the ring
  kLast = kSegment + kAnnounced,  // (a wait that gave up: products in flight)
  kBars = kLast + 1
};

constexpr int kQAt = 0;                       // 2 tiles
constexpr int kKAt = kQAt + 2 * kTile;        // kStages tiles
constexpr int kVAt = kKAt + kStages * kTile;  // kStages tiles
// The fillers' raw bytes: two slots each of 32 rows of 64 data bytes (by
// 16-byte piece, then lane) and 8 scale bytes.
constexpr int kRawSlot = 32 * 72;
constexpr int kRawBytes = 2 * kRawSlot;
constexpr int kRawAt = kVAt + kStages * kTile;
constexpr int kBarAt = kRawAt + kFillers * kRawBytes;
// Per tile and quarter: the tokens that are not left out ([8][4] words).  K
// of tile k waits for the logits of tile k - 2, whose product is issued after
// the weights of tile k - 4 at the latest: eight entries are enough.
constexpr int kValidAt = kBarAt + 8 * 32;
// Per segment, group and quarter: the first token whose V scale is NaN
// ([8][8][4] ints).  V of tile k waits for tile k - 2's product with V, and
// that one for the epilogues of all segments before its own: when segment s
// is filled, those up to s - 3 are over.
constexpr int kNanAt = kValidAt + 128;
// 16 ints: whether a wait gave up, the tensor memory's address, whether there
// is a segment; from kJoined on, one per softmax warp: the segments whose
// sums it has left for the other slot's warp.
constexpr int kMiscAt = kNanAt + 1024;
constexpr int kJoined = 4;
constexpr int kScanAt = kMiscAt + 64;    // 32 int64
constexpr int kUnitsAt = kScanAt + 256;  // 3 int64: all, share's end, begin
constexpr int kSumAt = kUnitsAt + 32;    // [slot][row] floats
constexpr int kRefAt = kSumAt + 1024;    // [slot][row] floats
// The segments for the softmax warps ([segment % 4]; when segment s begins,
// weights of segment s - 1 have been multiplied, so s - 3 is over), then the
// other warps' positions.
constexpr int kRingAt = kRefAt + 1024;
constexpr int kWalkAt = kRingAt + 4 * static_cast<int>(sizeof(Walk));
constexpr int kSmemBytes =
    kWalkAt + (kFillers + 2) * static_cast<int>(sizeof(Walk)) + 1024;
static_assert(kSmemBytes <= 227 * 1024 && kRawBytes % 16 == 0 &&
                  kBars <= 32 && kValidAt % 16 == 0 && kUnitsAt % 8 == 0 &&
                  sizeof(Walk) % 8 == 0,
              "");
// Tensor memory: logits (and, over them, weights) of the two slots, outputs
// of the two slots.
constexpr uint32_t kOCol = 256;

template <bool kF16>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ ChunkParams p) {
  extern __shared__ __align__(16) uint8_t raw_smem[];
  uint8_t* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* misc = reinterpret_cast<volatile int*>(smem + kMiscAt);
  volatile int* abort = misc;  // a wait gave up
  int* nan_at = reinterpret_cast<int*>(smem + kNanAt);
  volatile int64_t* units_kept =
      reinterpret_cast<volatile int64_t*>(smem + kUnitsAt);
  auto bar = [&](int i) { return base + kBarAt + 8 * i; };

  if (warp == 0) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
        ::"r"(base + kMiscAt + 4)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 32) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kKFull + s), 4);
      mbar_init(bar(kVFull + s), 4);
    }
    for (int t = 0; t < kEmpties; ++t) {
      mbar_init(bar(kKEmpty + t), 2);
      mbar_init(bar(kVEmpty + t), 2);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(bar(kQFull + m), 4);
      mbar_init(bar(kSFull + m), 1);
      mbar_init(bar(kPFull + 2 * m), 4);
      mbar_init(bar(kPFull + 2 * m + 1), 4);
      mbar_init(bar(kPDone + m), 1);
      mbar_init(bar(kTurn + m), 1);
      mbar_init(bar(kODone + m), 1);
    }
    mbar_init(bar(kOFree), kSoftWarps);
    for (int i = 0; i < kAnnounced; ++i) mbar_init(bar(kSegment + i), 2);
    mbar_init(bar(kLast), 2);
    misc[0] = 0;
    misc[2] = 0;
    for (int w = 0; w < kSoftWarps; ++w) misc[kJoined + w] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < 256) nan_at[tid] = INT32_MAX;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Cut* const own_cut = reinterpret_cast<Cut*>(p.workspace) + blockIdx.x;
  if (tid == 0)  // nothing to join, unless note_cut says so
    own_cut->more = own_cut->gave_up = 0;

  // --- this CTA's share -----------------------------------------------------
  // inclusive scan of the sequences' units, kThreads of them at a time; with
  // no more sequences than threads each is looked at once
  Walk* ring = reinterpret_cast<Walk*>(smem + kRingAt);
  {
    int64_t* scan = reinterpret_cast<int64_t*>(smem + kScanAt);
    const int rounds = (p.num_seqs + kThreads - 1) / kThreads;
    int64_t units = 0, incl = 0, U = 0, u0 = 0, u1 = 0;
    Seq s;
#pragma unroll 1
    for (int r = 0; r < (rounds > 1 ? 2 * rounds : 1); ++r) {
      if (r == rounds) U = 0;  // (second time over: the totals again)
      const int b = r % rounds * kThreads + tid;
      units = 0;
      if (b < p.num_seqs) {
        s = seq_of(p, b);
        if (s.n > 0) {
          Blocks k;
          k.begin(p, s, 0);
#pragma unroll 1
          for (; k.left > 0; k.next()) units += k.units();
        }
        units *= p.Hkv;
        if (r < rounds && blockIdx.x == 0) {
          const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1);
          if (c0 < 0 || c1 < c0 || c1 > p.total_q ||
              __ldg(p.lens + b) > p.len_cap)
            flag(p.dev_error, KVQ_DEVERR_SEQ);
        }
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
      incl = U + x;
#pragma unroll 1
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) incl += scan[w];
        U += scan[w];
      }
      if (r == rounds - 1) {  // the sum is known
        int ctas;
        u0 = share_begin(U, blockIdx.x, &ctas);
        u1 = share_begin(U, blockIdx.x + 1, &ctas);
        if (tid == 0) {
          units_kept[0] = U;
          units_kept[1] = units_kept[2] = U;  // (what no sequence holds)
        }
        __syncthreads();
      }
      // (r >= rounds - 1: u0 and u1 are known)
      if (r < rounds - 1 || (rounds > 1 && r < rounds) || units == 0)
        continue;
#pragma unroll 1
      for (int end = 0; end < 2; ++end) {
        const int64_t u = end ? u1 : u0;
        if (u < incl - units || u >= incl) continue;
        int64_t rem = u - (incl - units);
        Walk w = {};
        Blocks k;
        k.begin(p, s, 0);
#pragma unroll 1
        for (; rem >= static_cast<int64_t>(k.units()) * p.Hkv; k.next()) {
          rem -= static_cast<int64_t>(k.units()) * p.Hkv;
          ++w.block;
        }
        const int size = k.units();
        w.b = b;
        w.h = static_cast<int>(rem) / size;
        const int at = static_cast<int>(rem) - w.h * size;
        w.rem = snap(at, size);
        w.s = s;
        units_kept[2 - end] = u + w.rem - at;
        if (end == 0) ring[0] = w;
      }
    }
    __syncthreads();
    if (tid == 0 && units_kept[2] < units_kept[1]) {
      Walk w = ring[0];
      w.left = units_kept[1] - units_kept[2];
      w.there = w.next(p, true);
      ring[0] = w;
      misc[2] = w.there;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[1]);
  const bool any = misc[2] != 0;
  Walk* walk = reinterpret_cast<Walk*>(smem + kWalkAt) +
               (warp < kSoftWarps ? 0 : warp - kSoftWarps);
  if (any && warp >= kSoftWarps && lane == 0) *walk = ring[0];
  __syncwarp();

  if (warp < kSoftWarps) {
    // --- softmax ------------------------------------------------------------
    const int m = warp >> 2, row = tid & 127;
    const uint32_t lanes =
        tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = lanes + 128 * m, o_col = lanes + kOCol + 128 * m;
    const float c0 = p.scale * __ldg(p.k_scale);
    // (c0 == 0: a query of zeros, and any c > 0)
    const float c = c0 != 0.0f ? fabsf(c0) * kLog2e : 1.0f;
    uint32_t cnt0 = 0, cnt1 = 0;  // tiles of the slots so far
#pragma unroll 1
    for (uint32_t seg = 0; any;) {
      int kv0, kv1, pos, tiles, rows;
      {
        const Walk& w = ring[seg & 3];
        kv0 = w.kv0;
        kv1 = w.kv1;
        rows = min(kRows, w.s.n * p.G - w.block * kRows);
        // (tile kt of this segment is the CTA's (tiles + kt)-th)
        tiles = w.tiles - kv0;
        // two query tiles, or one whose KV tiles the slots share out
        const int at = (rows > 128 ? 128 * m : 0) + row;
        const int r = w.block * kRows + at;  // row of the sequence
        const int tok = r / p.G;
        // (a row that is none sees all, so that it does not slow the others)
        pos = at < rows ? w.s.L - w.s.n + tok : INT32_MAX;
        if (m == 0 || rows > 128) {
          // the query rows, rounded to fp16, their sign folded with the
          // scale's: two rows of the warp at a time, 16 bytes per lane (a
          // row per lane would touch 32 rows with every load)
          const int64_t from = at < rows ? (w.s.q0 + tok) * p.q_stride0 +
                                               (w.h * p.G + (r - tok * p.G)) *
                                                   kD
                                         : int64_t{-1};
          const uint32_t flip = c0 < 0.0f ? 0x80008000u : 0u;
          const int ch = lane & 15;
          uint4 v[16];
#pragma unroll
          for (int g = 0; g < 16; ++g) {
            const int64_t row_at =
                __shfl_sync(0xFFFFFFFFu, from, 2 * g + (lane >> 4));
            v[g] = make_uint4(0, 0, 0, 0);
            if (row_at >= 0 && c0 != 0.0f)
              v[g] = ldg128(p.q + row_at + 8 * ch);
          }
#pragma unroll
          for (int g = 0; g < 16; ++g) {
            uint32_t x[4] = {v[g].x, v[g].y, v[g].z, v[g].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[k] = (kF16 ? x[k] : bf16x2_to_f16x2(x[k])) ^ flip;
            const int to = (warp & 3) * 32 + 2 * g + (lane >> 4);
            sts128(base + kQAt + m * kTile + (ch >> 3) * kHalf + to * 128 +
                       (((ch & 7) ^ (to & 7)) << 4),
                   x);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kQFull + m));
        }
      }
      const bool two = rows > 128;
      float ref = -INFINITY, sum = 0.0f;
      uint32_t cnt = m == 0 ? cnt0 : cnt1;
      const int kt0 = two ? kv0 : kv0 + m, step = two ? 1 : 2;
#pragma unroll 1
      for (int kt = kt0; kt < kv1; kt += step, ++cnt) {
        if (!warp_wait(bar(kSFull + m), cnt & 1, abort)) goto done;
        fence_after();
        // Weights are exp2 of the scaled logits minus a reference: kBelow
        // less than the maximum of the first half of the first tile, so that
        // the weight there is 2^8.  They are rounded to fp16, which keeps 11
        // bits of those down to 2^-14, 2^-22 of that weight: behind one token
        // that takes nearly all of the weight (the first of a long context,
        // often) thousands of others may share the rest.  (With a weight of 1
        // there 30000 tokens with 0.1 to 1 % of the weight together came out
        // up to 22 % off.)
        // Later halves do without their maximum: as long as a row's weights
        // of half a tile sum up to less than kMost, fp16's largest number,
        // none is out of range; 64 of 2^8 are 2^14.  Where that fails the
        // half is done over, with its maximum for the new reference.  The
        // product of the first half with V begins while the second is made.
        // (Unrolled: 500 tokens over 131000 1.53 ms against 1.61.)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          bool look = kt == kt0 && half == 0;
          uint32_t s[64];
          float ts;
          for (;;) {
            tmem_ld32(s_col + 64 * half, s);
            tmem_ld32(s_col + 64 * half + 32, s + 32);
            const uint2 valid = *reinterpret_cast<const uint2*>(
                smem + kValidAt + ((tiles + kt) & 7) * 16 + 8 * half);
            // (the row sees columns 0 .. lim)
            const int lim = pos - kt * kKeys - 64 * half;
            tmem_wait_ld();
            if (!__all_sync(0xFFFFFFFFu,
                            lim >= 63 && (valid.x & valid.y) == ~0u)) {
              mask32(s, valid.x & first_bits(lim));
              mask32(s + 32, valid.y & first_bits(lim - 32));
            }
            if (look) {
              const float top = max64(s) * c - kBelow;
              const float f = top > ref ? ex2(ref - top) : 1.0f;
              ref = fmaxf(ref, top);
              sum *= f;
              if (kt > kt0 || half > 0) {
                // (every product of this slot so far)
                if (!warp_spin(bar((half ? kPDone : kODone) + m),
                               (half ? cnt : cnt - 1) & 1, abort))
                  goto done;
                fence_after();
                rescale(o_col, f);
              }
            }
            const float low = ref == -INFINITY ? 0.0f : ref;
            const uint64_t cc = pack2(c, c), ll = pack2(-low, -low);
            uint64_t add[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
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
            ts = e + o;
            // (a row that has seen nothing has no reference yet)
            const bool again = !(ts < kMost) || ref == -INFINITY;
            if (look || !__any_sync(0xFFFFFFFFu, again)) break;
            look = true;
          }
          tmem_st32(s_col + 32 * half, s);
          sum += ts;
          tmem_wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kPFull + 2 * m + half));
        }
      }
      // --- epilogue ---------------------------------------------------------
      const int n = kv1 - kv0;
      cnt0 += two ? n : (n + 1) >> 1;
      cnt1 += two ? n : n >> 1;
      float w0 = 1.0f, w1 = 0.0f;
      if (test_gives_up(warp, seg)) {
        *abort = 1;
        goto done;
      }
      if (two) {
        if (!warp_wait(bar(kODone + m), (cnt - 1) & 1, abort)) goto done;
      } else {
        // The slots' sums and references (a product of this segment with V
        // is done, so every warp has read those of the last segment).  Each
        // slot's warps wait for its own last product: of the other slot's
        // phases they have not looked at each, and could take an older one
        // for this.  Behind the joint barrier that one is over, and the wait
        // for it passes at once.
        const bool both = n > 1;
        const uint32_t last0 = cnt0 - 1, last1 = cnt1 - 1;
        float* x_sum = reinterpret_cast<float*>(smem + kSumAt) + row;
        float* x_ref = reinterpret_cast<float*>(smem + kRefAt) + row;
        const int own = m == 1 && both;
        if (!warp_wait(bar(kODone + own), (own ? last1 : last0) & 1, abort))
          goto done;
        x_sum[128 * m] = sum;
        x_ref[128 * m] = ref;
        // (a warp that has given up arrives at the end of the kernel, where
        // it does not count: without its sums this one has no rows either)
        if (lane == 0) misc[kJoined + warp] = static_cast<int>(seg) + 1;
        bar_sync(1 + (warp & 3), 64);
        if (uniform(misc[kJoined + (warp ^ 4)]) <= static_cast<int>(seg))
          goto gone;
        if (both && !warp_wait(bar(kODone + 1 - own),
                               (own ? last0 : last1) & 1, abort))
          goto done;
        const float r0 = x_ref[0], r1 = x_ref[128];
        ref = fmaxf(r0, r1);
        w0 = r0 == ref ? 1.0f : ex2(r0 - ref);
        w1 = r1 == ref ? 1.0f : ex2(r1 - ref);
        sum = x_sum[0] * w0 + x_sum[128] * w1;
      }
      fence_after();
      const Walk& w = ring[seg & 3];
      const int4* nan_row =
          reinterpret_cast<const int4*>(nan_at + (seg & 7) * 32);
      const int at = (two ? 128 * m : 0) + row;
      const bool whole = kv0 == 0 && kv1 == w.W;
      const float inv = sum > 0.0f ? __ldg(p.v_scale) / sum
                                   : (sum == 0.0f ? 0.0f : sum);
      float* slot = slot_of(p, blockIdx.x, seg > 0);
      const int r = w.block * kRows + at, tok = r / p.G;
      uint16_t* dst = p.out + (w.s.q0 + tok) * p.out_stride0 +
                      (w.h * p.G + (r - tok * p.G)) * kD;
      float* part = slot + at * kD;
      // whole 32-byte sectors (of half sectors the SM stores no more a cycle)
      const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0 &&
                        p.out_stride0 % 16 == 0;
      // columns: the row of the slot's own output, or half a row of the two
      // slots' joined ones
#pragma unroll 1
      for (int k = 0; k < (two ? 4 : 2); ++k) {
        const int col = two ? 32 * k : 64 * m + 32 * k;
        uint32_t o[32];
        __syncwarp();
        tmem_ld32(lanes + kOCol + (two ? 128 * m : 0) + col, o);
        if (!two && n > 1) {
          uint32_t o1[32];
          tmem_ld32(lanes + kOCol + 128 + col, o1);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j)
            o[j] = __float_as_uint(__uint_as_float(o[j]) * w0 +
                                   __uint_as_float(o1[j]) * w1);
        } else {
          tmem_wait_ld();
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int4 x = nan_row[col / 16 + g];
          if (min(min(x.x, x.y), min(x.z, x.w)) <= pos) {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[16 * g + j] = 0x7FFFFFFFu;
          }
        }
        if (at < rows && whole) {
          uint32_t x[16];
#pragma unroll
          for (int g = 0; g < 16; ++g) {
            const float a = __uint_as_float(o[2 * g]) * inv;
            const float b = __uint_as_float(o[2 * g + 1]) * inv;
            // (a row that sees nothing gets zeros whatever the scales are)
            x[g] = pos < 0 ? 0u
                           : kF16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
          }
          if (wide) {
            stg256(dst + col, x);
            stg256(dst + col + 16, x + 8);
          } else {
#pragma unroll
            for (int g = 0; g < 4; ++g)
              *reinterpret_cast<uint4*>(dst + col + 8 * g) = make_uint4(
                  x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]);
          }
        } else if (at < rows) {
#pragma unroll
          for (int g = 0; g < 4; ++g) stg256(part + col + 8 * g, o + 8 * g);
        }
      }
      if (!whole && at < rows && (two || m == 0)) {
        slot[kRows * kD + at] = ref;
        slot[kRows * (kD + 1) + at] = sum;
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kOFree));
      // (waited for here and not at the loop's head, where the registers fall
      // worse: 500 tokens over 131000 1536 us against 1570)
      ++seg;
      if (!warp_wait(bar(kSegment + seg % kAnnounced),
                     (seg - 1) / kAnnounced & 1, abort))
        goto done;
      if (!ring[seg & 3].there) break;
    }
  }
  if (warp >= kSoftWarps + 2) {
    // --- dequantise: a quarter (32 tokens) of a tile's K or V at a time ------
    // The quarters K 0..3, V 0..3 of the share's tiles, in order, are dealt
    // round-robin to the warps.  A warp has four in hand: the one that it
    // dequantises, whose raw bytes are in shared memory, two whose bytes are
    // on their way there (a slot each; every lane copies and reads its own
    // token's), and the one behind them, whose block id is on its way (`job`,
    // `kt` and `walk` are at that one).
    int job = warp - kSoftWarps - 2;  // 0..3: K quarters, 4..7: V quarters
    // (this segment: its sequence's length and table row, its head, its end)
    int kt = walk->kv0, kv1 = walk->kv1, len = walk->s.L, seg = 0;
    const int32_t* table = p.block_table + walk->b * p.bt_stride;
    int64_t data_h = walk->h * p.dhs;
    int64_t scale_h = p.scale_off + walk->h * p.shs;
    uint32_t cnt = 0;      // tile of the share
    bool more = any;       // there is a tile at kt
    bool first = true;     // it is the segment's first
    int32_t blk = -1;      // the block id of this thread's token
    int pos = 0, off = 0;  // the token, and its place in the page
    bool quad = false;     // its 4-token band is inside the context
    auto look_up = [&]() {
      pos = kt * kKeys + 32 * (job & 3) + lane;
      quad = more && (pos & ~3) < len;  // (a band is in one page)
      if (quad) {
        const int j = p.b_shift >= 0 ? pos >> p.b_shift : pos / p.B;
        off = pos - j * p.B;
        blk = __ldg(table + j);
      }
    };
    // The last job whose copies were issued, and the one before it.
    struct Job {
      bool some, first, in;
      int pos, job;
      uint32_t mask, cnt, seg;
    };
    Job next, after;
    const uint32_t raw = base + kRawAt + (warp - kSoftWarps - 2) * kRawBytes +
                         16 * lane;
    // copies of the job at (kt, job) into slot `slot`, and on to the next
    auto issue = [&](uint32_t slot) {
      Job n = {more, first, false, pos, job, 0, cnt,
               static_cast<uint32_t>(seg)};
      bool bad = false;
      const uint8_t *data = reinterpret_cast<const uint8_t*>(p.q),
                    *scales = data;
      if (quad) {
        bad = blk < 0 || blk >= p.num_blocks;
        const bool in = pos < len, v = job >= 4;
        if (!bad) {
          const uint8_t* page =
              (v ? p.side[1] : p.side[0]) + blk * p.page_stride;
          data = page + data_h + off * p.dts;
          // swizzled: row off % 4 of the band, other lanes' scales too
          scales = page + scale_h + off * p.sts;
          n.in = in;
        } else if (in && !v) {
          flag(p.dev_error, KVQ_DEVERR_BLOCK);
        }
      }
      n.mask = __ballot_sync(0xFFFFFFFFu, !bad);
      if (more) {
        // (a token that is not to be read: the query's first bytes, which
        // are scaled by 0)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           raw + slot * kRawSlot + 512 * i),
                       "l"(data + 16 * i)
                       : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(
                         raw + slot * kRawSlot + 2048 - 8 * lane),
                     "l"(scales)
                     : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (more) {
        job += kFillers;
        if (job >= 8) {
          job -= 8;
          ++cnt;
          first = false;
          if (++kt == kv1) {
            more = advance(p, walk);
            first = true;
            ++seg;
            kt = walk->kv0;
            kv1 = walk->kv1;
            len = walk->s.L;
            table = p.block_table + walk->b * p.bt_stride;
            data_h = walk->h * p.dhs;
            scale_h = p.scale_off + walk->h * p.shs;
          }
        }
        look_up();
      }
      return n;
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
    next = issue(0);
    after = issue(1);
    for (uint32_t slot = 0; next.some; slot ^= 1) {
      const int stage = next.cnt & 1;
      const bool is_v = next.job >= 4, in = next.in, first = next.first;
      const int quarter = next.job & 3, cur_pos = next.pos;
      const bool swz = is_v || p.swizzle_k;
      const uint32_t mask = next.mask, cur = next.cnt, cur_seg = next.seg;
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      // (of the tile before in this stage; a barrier as it was made counts as
      // one whose phase 1 is over: the first two tiles wait for nothing)
      const uint32_t old = cur - kStages;
      if (!warp_wait(bar((is_v ? kVEmpty : kKEmpty) + old % kEmpties),
                     old / kEmpties & 1, abort))
        goto done;
      const uint32_t from = raw + slot * kRawSlot;
      const uint2 sc = lds64(from + 2048 - 8 * lane);
      if (!is_v && lane == 0)
        reinterpret_cast<volatile uint32_t*>(
            smem + kValidAt)[(cur & 7) * 4 + quarter] = mask;
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
        lo = drop_nan(lo, nan_at + (cur_seg & 7) * 32 + quarter, cur_pos);
        hi = drop_nan(hi, nan_at + (cur_seg & 7) * 32 + 4 + quarter, cur_pos);
      }
      // (a row is 128-byte aligned: its swizzled chunks by XOR)
      const uint32_t dst =
          (base + (is_v ? kVAt : kKAt) + stage * kTile +
           (32 * quarter + lane) * 128) | ((lane & 7) << 4);
#pragma unroll
      for (int g = 0; g < 4; ++g) {  // groups 2g, 2g + 1
        const uint4 d = lds128(from + 512 * g);
        const uint32_t pair = swz ? prmt(lo, hi, g | ((g + 4) << 4))
                                  : (g < 2 ? lo : hi) >> (16 * (g & 1));
        const uint32_t sf = e4m3x2_to_f16x2(pair & 0xFFFFu);
        const uint32_t se = prmt(sf, sf, 0x1010u), so = prmt(sf, sf, 0x3232u);
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
          dequant_word(w[i], i < 2 ? se : so, o);
          const int ch = 4 * g + i;  // 16-byte chunk of the row
          sts128((dst ^ ((ch & 7) << 4)) + (ch >> 3) * kHalf, o);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar((is_v ? kVFull : kKFull) + stage));
      next = after;
      after = issue(slot);  // (this lane has read its bytes)
    }
  } else if (warp >= kSoftWarps && any) {
    // --- products of slot m: the warp waits, one lane issues -----------------
    // In order: logits of the slot's first tile, then its output with a tile
    // and its logits of the next one, so that the tensor cores work for this
    // slot while the other's weights come.  Both slots release a stage of K
    // or V; where they share one query tile, the slot that used it does so
    // twice.
    const int m = warp - kSoftWarps;
    uint32_t cnt = 0;                    // KV tiles before this segment
    uint32_t q1 = 0, p_cnt = 0;          // phases of query 1, of the weights
    uint32_t segs = 0, turns = 0;
    bool go = true;
    while (go) {
      const bool two = uniform(walk->two) != 0;
      const int n = uniform(walk->kv1 - walk->kv0);
      const int step = two ? 1 : 2, first = two ? 0 : m;
      const int q = two ? m : 0;
      // Both warps wait for slot 0's query, whether they use it or not: once
      // it is there, slot 0 is done with the last segment, and every tile of
      // it has come and gone.  Without that, a warp that had no tile in a
      // segment could run two phases ahead of a barrier, and take the phase
      // before the last for the one that it waits for.
      if (!warp_wait(bar(kQFull), segs & 1, abort)) goto done;
      if (q == 1 && !warp_wait(bar(kQFull + 1), q1 & 1, abort)) goto done;
      // product i - step with V, then the logits of tile i: everything is
      // waited for first, then the batch is issued in one go
#pragma unroll 1
      for (int i = first; i < n + step; i += step) {
        const bool pv = i >= first + step, qk = i < n;
        const uint32_t tv = cnt + i - step, tk = cnt + i;  // their tiles
        // (the weights after V: they come last, and every test on the way
        // from them to the products would add to the slot's round)
        const uint32_t a = desc_lo<16>(base + kQAt + q * kTile);
        const uint32_t k = desc_lo<16>(base + kKAt + (tk & 1) * kTile);
        const uint32_t v = desc_lo<kHalf>(base + kVAt + (tv & 1) * kTile);
        const uint32_t s_at = tmem + 128 * m, o_at = s_at + kOCol;
        if (pv) {
          if (!warp_wait(bar(kVFull + (tv & 1)), (tv >> 1) & 1, abort))
            goto done;
          // the output's columns are free once the last segment's are read
          // (after the weights: see the phases above)
          if (!warp_wait(bar(kPFull + 2 * m), p_cnt & 1, abort)) goto done;
          if (i == first + step && segs > 0 &&
              !warp_wait(bar(kOFree), (segs - 1) & 1, abort))
            goto done;
          fence_after();
          if (elect()) {
            mma_ts(o_at, s_at, v, kIdescBmn, i > first + step);
#pragma unroll
            for (int x = 1; x < 4; ++x)
              mma_ts(o_at, s_at + 8 * x, v + x * (2048 >> 4), kIdescBmn, 1);
            mma_commit(bar(kPDone + m));
          }
          __syncwarp();
        }
        if (qk && !warp_wait(bar(kKFull + (tk & 1)), (tk >> 1) & 1, abort))
          goto done;
        // Two query tiles take turns with the rest: batches that ran side by
        // side would end side by side, and leave the tensor cores idle while
        // both slots make their weights (1 % on long contexts).
        if (two && pv) {
          if (turns + m > 0 &&
              !warp_wait(bar(kTurn + m), (turns + m - 1) & 1, abort))
            goto done;
          ++turns;
        }
        if (pv && !warp_wait(bar(kPFull + 2 * m + 1), p_cnt++ & 1, abort))
          goto done;
        fence_after();
        if (elect()) {
          if (pv) {
#pragma unroll
            for (int x = 4; x < 8; ++x)
              mma_ts(o_at, s_at + 8 * x, v + x * (2048 >> 4), kIdescBmn, 1);
            mma_commit(bar(kODone + m));
            mma_commit(bar(kVEmpty + tv % kEmpties));
            if (!two) mma_commit(bar(kVEmpty + tv % kEmpties));
            if (two && !qk) mbar_arrive(bar(kTurn + 1 - m));
          }
          if (qk) {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const uint32_t at = ((x >> 2) * kHalf + (x & 3) * 32) >> 4;
              mma_ss(s_at, a + at, k + at, kIdesc, x > 0);
              // (what is left takes as long as the other warp to begin)
              if (x == 4 && two && pv) mbar_arrive(bar(kTurn + 1 - m));
            }
            mma_commit(bar(kSFull + m));
            mma_commit(bar(kKEmpty + tk % kEmpties));
            if (!two) mma_commit(bar(kKEmpty + tk % kEmpties));
          }
        }
        __syncwarp();
        if (i == first) {
          // while the first weights are made: the next segment (slot 0: for
          // the softmax warps too)
          if (m == 0 && lane == 0 && walk->kv0 == 0 && walk->kv1 < walk->W)
            note_cut(p, *walk, units_kept[0], units_kept[1]);
          go = advance(p, walk);
          if (lane == 0) {
            if (m == 0) {
              Walk* next = ring + ((segs + 1) & 3);
              *next = *walk;
              next->there = go;
            }
            // (from both warps: no query of the next segment is announced
            // before both have seen this one's)
            mbar_arrive(bar(kSegment + (segs + 1) % kAnnounced));
          }
          __syncwarp();
        }
      }
      if (two) ++q1;
      cnt += n;
      ++segs;
    }
  }
done:
  __syncwarp();
  if (*abort != 0) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    // whoever waits for this warp's sums goes on, finds that they are not
    // there and comes to no further barrier of this kind
    if (warp < kSoftWarps) bar_arrive(1 + (warp & 3), 64);
  }
gone:
  fence_before();
  __syncthreads();
  fence_after();
  if (*abort != 0) {  // (the same in every thread: all waits are over)
    // products in flight end by themselves; wait for them before the tensor
    // memory goes
    if (warp == kSoftWarps || warp == kSoftWarps + 1) {
      if (elect()) {
        mma_commit(bar(kLast));
        const uint64_t start = dev::global_ns();
        while (!mbar_try(bar(kLast), 0) &&
               dev::global_ns() - start < KVQ_WAIT_LIMIT_NS) {
        }
      }
      __syncwarp();
    }
    // the rows that this CTA has written are right, its parts may be missing
    if (tid == 0) {
      own_cut->gave_up = 1;
      flag(p.dev_error, KVQ_DEVERR_TIMEOUT);
    }
    fence_before();
    __syncthreads();
    fence_after();
  }
  if (warp == 0)
    asm volatile(
        "tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---------------------------------------------------------------------------
// The items that were cut: their parts joined
// ---------------------------------------------------------------------------
constexpr int kMergeRows = 32;  // rows of a CTA, four to a warp

template <bool kF16>
__global__ void __launch_bounds__(256)
    chunk_merge_kernel(const __grid_constant__ ChunkParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int cta = blockIdx.x;
  const Cut cut = *(reinterpret_cast<const Cut*>(p.workspace) + cta);
  if (cut.more == 0) return;
  int lost = 0;  // a part may be missing: the rows are left as they were
  for (int k = threadIdx.x; k <= cut.more; k += blockDim.x)
    lost |= (reinterpret_cast<const Cut*>(p.workspace) + cta + k)->gave_up;
  if (__syncthreads_or(lost)) return;
  const Seq s = seq_of(p, cut.b);
  const int row0 = cut.block * kRows;
  const int rows = min(kRows, s.n * p.G - row0);
  const int lane = threadIdx.x & 31;
  const float vs = __ldg(p.v_scale);
  const int blind = s.n - s.L;  // tokens that see nothing, whose rows are 0
  for (int i = 0; i < kMergeRows / 8; ++i) {
    const int row = blockIdx.y * kMergeRows + 8 * i + (threadIdx.x >> 5);
    if (row >= rows) return;
    float top = -INFINITY;
    for (int k = 0; k <= cut.more; ++k)
      top = fmaxf(top, slot_of(p, cta + k,
                               k == 0 ? cut.slot : 0)[kRows * kD + row]);
    float sum = 0.0f;
    float4 o = make_float4(0, 0, 0, 0);
    for (int k = 0; k <= cut.more; ++k) {
      const float* slot = slot_of(p, cta + k, k == 0 ? cut.slot : 0);
      const float ref = slot[kRows * kD + row];
      const float w = ref == top ? 1.0f : ex2(ref - top);
      sum += slot[kRows * (kD + 1) + row] * w;
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
    uint2 w = make_uint2(0, 0);
    if (tok < blind) {
      *reinterpret_cast<uint2*>(dst) = w;
      continue;
    }
    w.x = kF16 ? pack_f16x2(o.x * inv, o.y * inv)
               : pack_bf16x2(o.x * inv, o.y * inv);
    w.y = kF16 ? pack_f16x2(o.z * inv, o.w * inv)
               : pack_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(dst) = w;
  }
}

template <bool kF16>
cudaError_t launch(const ChunkParams& p, cudaStream_t stream) {
  const cudaError_t set = cudaFuncSetAttribute(
      chunk_kernel<kF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
      kSmemBytes);
  if (set != cudaSuccess) return set;
  const unsigned ctas = static_cast<unsigned>(sm_count());
  if (ctas > kMaxCtas) return cudaErrorInvalidConfiguration;
  const cudaError_t err = launch_kernel(chunk_kernel<kF16>, dim3(ctas),
                                        kThreads, kSmemBytes, stream, p.pdl,
                                        p);
  if (err != cudaSuccess) return err;
  return launch_kernel(chunk_merge_kernel<kF16>,
                       dim3(ctas, kRows / kMergeRows), 256, 0, stream, true,
                       p);
}

}  // namespace

int64_t chunk_workspace_bytes(int sms) {
  return kCutBytes + static_cast<int64_t>(sms) * 2 * kSlotFloats * 4;
}

// Short chunks go token by token through the decode kernel, which walks the
// context once for every token, but at three times the speed of a tile of
// 128 rows that is mostly padding, and with nothing to set up: 200 single
// tokens over 512 to 2560 tokens of context 73 us against 391 us by tiles,
// five tokens of 8 sequences 25 us against 34 us.  Up to four tokens always,
// up to eight where there are no more than one (sequence, KV head) per SM;
// single tokens beside longer chunks too.
static int short_chunk(const ChunkParams& p) {
  if (p.max_q_len <= 4) return p.max_q_len > 1 ? p.max_q_len : 1;
  const bool few = static_cast<int64_t>(p.num_seqs) * p.Hkv <= sm_count();
  return few && p.max_q_len <= 8 ? p.max_q_len : 1;
}

cudaError_t launch_chunk_attention(const ChunkParams& caller,
                                   cudaStream_t stream) {
  ChunkParams p = caller;
  p.skip = short_chunk(p);
  // the decode kernel's scratch: output, sum and maximum of each stretch
  constexpr int kPart = 512;
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.skip;
  const int64_t parts = (static_cast<int64_t>(p.len_cap) + kPart - 1) / kPart;
  const int64_t cells = rows * p.Hq * parts;
  if (rows * p.Hkv * (parts > 0 ? parts : 1) >= INT32_MAX ||
      (parts > 1 && cells * (kD + 2) * 4 > chunk_workspace_bytes(sm_count())))
    p.skip = 0;
  cudaError_t err = cudaSuccess;
  const bool tiles = p.skip == 0 || p.max_q_len > p.skip;
  if (tiles)
    err = p.f16 ? launch<true>(p, stream) : launch<false>(p, stream);
  if (err != cudaSuccess || p.skip == 0) return err;
  AttnParams a{};
  a.q = p.q;
  a.q_stride0 = p.q_stride0;
  a.side[0] = p.side[0];
  a.side[1] = p.side[1];
  a.page_stride = p.page_stride;
  a.num_blocks = p.num_blocks;
  a.scale_off = p.scale_off;
  a.dhs = p.dhs;
  a.dts = p.dts;
  a.shs = p.shs;
  a.sts = p.sts;
  a.block_table = p.block_table;
  a.bt_stride = p.bt_stride;
  a.lens = p.lens;
  a.k_scale = p.k_scale;
  a.v_scale = p.v_scale;
  a.scale = p.scale;
  a.tmp_out = reinterpret_cast<float*>(p.workspace);
  a.exp_sums = a.tmp_out + cells * kD;
  a.max_logits = a.exp_sums + cells;
  a.out = p.out;
  a.out_stride0 = p.out_stride0;
  a.dev_error = p.dev_error;
  a.num_seqs = static_cast<int32_t>(rows);
  a.Hq = p.Hq;
  a.Hkv = p.Hkv;
  a.G = p.G;
  a.B = p.B;
  a.b_shift = p.b_shift;
  a.part = kPart;
  a.max_parts = static_cast<int32_t>(parts > 0 ? parts : 1);
  a.len_cap = p.len_cap;
  a.swizzle_k = p.swizzle_k;
  a.f16 = p.f16;
  a.pdl = tiles || p.pdl;
  a.cu = p.cu;
  a.total_q = p.total_q;
  a.per_seq = p.skip;
  a.only_short = !tiles;
  return launch_paged_attention_mma(a, stream);
}

}  // namespace kvq
