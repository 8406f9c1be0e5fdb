// page_move.cu -- bytes of a paged cache from place to place, sm_103a:
// whole pages (kvq_copy_pages) and single NVFP4 tokens
// (kvq_move_tokens_nvfp4), in many caches (a model's layers) at once.
//
// Both read and write every byte once and compute nothing.  Measured: copies
// of 1.47 GB (read and written) 216 us, 6.8 TB/s, the HBM's rate; 2.2 us for
// a few pages, the launch's time.  Moves of 2.26 GB in an eviction round 433
// us with the state's two calls, 5.2 TB/s: bound by the memory's latency (a
// step's reads, barrier, writes), which more warps per SM cover best (see
// there), and by scales, whose 8 bytes per token and side are a quarter of
// the sector that they move (1.5 times the bytes written, by L2's counter).
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_internal.h"

namespace kvq {
namespace {

__device__ __forceinline__ void flag(int32_t* err, int32_t bits) {
  if (err != nullptr) atomicOr(err, bits);
}

struct alignas(32) Vec32 {
  uint64_t v[4];
};
__device__ __forceinline__ Vec32 load32(const uint8_t* p) {
  Vec32 r;
  asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];"
               : "=l"(r.v[0]), "=l"(r.v[1]), "=l"(r.v[2]), "=l"(r.v[3])
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ void store32(uint8_t* p, const Vec32& r) {
  asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p),
               "l"(r.v[0]), "l"(r.v[1]), "l"(r.v[2]), "l"(r.v[3])
               : "memory");
}
__device__ __forceinline__ uint4 load16(const uint8_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// ---------------------------------------------------------------------------
// whole pages: a warp copies kUnroll x 32 vectors of one (pair, cache)
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kUnroll = 4;

template <bool kVec32>
__global__ void __launch_bounds__(kCopyThreads)
    copy_pages_kernel(const __grid_constant__ CopyParams p) {
  pdl_prologue();
  constexpr int kBytes = kVec32 ? 32 : 16;
  const int lane = threadIdx.x & 31;
  const int64_t w =
      static_cast<int64_t>(blockIdx.x) * (kCopyThreads / 32) +
      (threadIdx.x >> 5);
  const int64_t unit = w / p.pieces;  // pair-major: a pair's caches together
  const int piece = static_cast<int>(w - unit * p.pieces);
  if (unit >= static_cast<int64_t>(p.num_pairs) * p.num_caches) return;
  const int pair = static_cast<int>(unit / p.num_caches);
  const int c = static_cast<int>(unit - static_cast<int64_t>(pair) *
                                            p.num_caches);
  const int32_t src = __ldg(p.src + pair), dst = __ldg(p.dst + pair);
  if (src < 0 || dst < 0 || src == dst) return;
  if (src >= p.num_blocks || dst >= p.num_blocks) {
    if (lane == 0) flag(p.err, KVQ_DEVERR_BLOCK);
    return;
  }
  const uint8_t* from = p.caches[c] + src * p.page_stride;
  uint8_t* to = p.caches[c] + dst * p.page_stride;
  const int64_t first =
      (static_cast<int64_t>(piece) * kUnroll * 32 + lane) * kBytes;
  if constexpr (kVec32) {
    Vec32 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = first + u * 32 * kBytes;
      if (at < p.page_bytes) v[u] = load32(from + at);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = first + u * 32 * kBytes;
      if (at < p.page_bytes) store32(to + at, v[u]);
    }
  } else {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = first + u * 32 * kBytes;
      if (at < p.page_bytes) v[u] = load16(from + at);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = first + u * 32 * kBytes;
      if (at < p.page_bytes) *reinterpret_cast<uint4*>(to + at) = v[u];
    }
  }
}

// ---------------------------------------------------------------------------
// single tokens: a CTA walks one list of one cache, for kHeads heads
// ---------------------------------------------------------------------------
// The tokens of a list may move within the same pages (a token's
// destination is then a place that an earlier token of the list left), so a
// list is walked in order: a step's tokens are all read before any of them
// is written.  A thread moves the 16-byte piece c of its token's rows (32
// elements) with its two group scales, K and V, of kHeads heads: what the
// slots cost (two divisions, the page's address) is spent once for 2 kHeads
// pieces.  A step has kTokens tokens per thread.  What bounds it is the wait
// for memory between a step's barriers (with four heads at three CTAs per SM
// the schedulers issued in 30 % of the cycles), so that warps matter most: a
// round of 2.26 GB by 4 heads at 3 CTAs per SM 511 us, at 4 457; by 2 heads
// at 5 433 (at 6, with spills, 445); by 1 head at 6 446.  Reading a step
// ahead takes more registers than it gives: 2 heads at 4 466, 4 heads 586.
// A V scale (and a swizzled K scale) of group j of a token at offset r of
// its 4-token band is byte 4j + r of the band's head tile, whose 4 rows are
// scale-row strides apart.
constexpr int kMoveThreads = 256;

template <int kHeads, int kTokens, int kCtas>
__global__ void __launch_bounds__(kMoveThreads, kCtas)
    move_tokens_kernel(const __grid_constant__ MoveParams p) {
  pdl_prologue();
  const int i = blockIdx.x;  // list
  const int h0 = blockIdx.y * kHeads;
  uint8_t* cache = p.caches[blockIdx.z];
  const int64_t begin = p.cu[i], end = p.cu[i + 1];
  if (begin < 0 || end < begin || end > p.total) {
    if (threadIdx.x == 0) flag(p.err, KVQ_DEVERR_SEQ);
    return;
  }
  const int vecs = p.D / 32;            // 16-byte pieces of a head row
  const int half = p.S / 4;             // scale groups in a swizzled row
  const int per = kMoveThreads / vecs;  // tokens of a round
  const int tok = threadIdx.x / vecs, c = threadIdx.x - tok * vecs;
  const bool works = tok < per;
  const int heads = min(kHeads, p.H - h0);

  // offsets in a page, from the head's first byte of the side: data, and
  // the scales of groups 2c and 2c + 1 (linear and swizzled)
  struct Place {
    int64_t data, linear, twisted0, twisted1;
  };
  auto place = [&](int64_t slot) {
    const int64_t blk = p.b_shift >= 0 ? slot >> p.b_shift : slot / p.B;
    const int off = static_cast<int>(slot - blk * p.B);
    const int64_t page = blk * p.page_stride;
    const int64_t tile = page + p.scale_off + h0 * p.shs;
    const int j = 2 * c;
    Place q;
    q.data = page + h0 * p.dhs + off * p.dts + 16 * c;
    q.linear = tile + off * p.sts + j;
    q.twisted0 = tile + ((off & ~3) + j / half) * p.sts + (j % half) * 4 +
                 (off & 3);
    q.twisted1 = tile + ((off & ~3) + (j + 1) / half) * p.sts +
                 ((j + 1) % half) * 4 + (off & 3);
    return q;
  };

  for (int64_t base = begin; base < end; base += kTokens * per) {
    uint4 kd[kTokens][kHeads], vd[kTokens][kHeads];
    uint16_t ks[kTokens][kHeads], vs[kTokens][kHeads];
    int64_t to[kTokens];
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
      const int64_t t = base + u * per + tok;
      to[u] = -1;
      if (!works || t >= end) continue;
      const int64_t src = p.src[t], dst = p.dst[t];
      if (src < 0 || dst < 0 || src == dst) continue;
      if (src >= p.num_slots || dst >= p.num_slots) {
        flag(p.err, KVQ_DEVERR_SLOT);
        continue;
      }
      to[u] = dst;
      const Place q = place(src);
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        if (h >= heads) break;
        const uint8_t* k = cache + h * p.dhs;
        const uint8_t* s = cache + h * p.shs;
        kd[u][h] = load16(k + q.data);
        vd[u][h] = load16(k + p.value_offset + q.data);
        ks[u][h] = p.swizzle_k
                       ? s[q.twisted0] | s[q.twisted1] << 8
                       : *reinterpret_cast<const uint16_t*>(s + q.linear);
        vs[u][h] = s[p.value_offset + q.twisted0] |
                   s[p.value_offset + q.twisted1] << 8;
      }
    }
    __syncthreads();  // all of the step is read
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
      if (to[u] < 0) continue;
      const Place q = place(to[u]);
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        if (h >= heads) break;
        uint8_t* k = cache + h * p.dhs;
        uint8_t* s = cache + h * p.shs;
        *reinterpret_cast<uint4*>(k + q.data) = kd[u][h];
        *reinterpret_cast<uint4*>(k + p.value_offset + q.data) = vd[u][h];
        if (p.swizzle_k) {
          s[q.twisted0] = ks[u][h] & 0xFF;
          s[q.twisted1] = ks[u][h] >> 8;
        } else {
          *reinterpret_cast<uint16_t*>(s + q.linear) = ks[u][h];
        }
        s[p.value_offset + q.twisted0] = vs[u][h] & 0xFF;
        s[p.value_offset + q.twisted1] = vs[u][h] >> 8;
      }
    }
  }
}

template <int kHeads, int kTokens, int kCtas>
cudaError_t launch_move(const MoveParams& p, cudaStream_t stream) {
  return launch_kernel(
      move_tokens_kernel<kHeads, kTokens, kCtas>,
      dim3(p.num_lists, (p.H + kHeads - 1) / kHeads, p.num_caches),
      kMoveThreads, 0, stream, p.pdl, p);
}

}  // namespace

cudaError_t launch_copy_pages(const CopyParams& p, bool vec32,
                              cudaStream_t stream) {
  const int64_t warps =
      static_cast<int64_t>(p.num_pairs) * p.num_caches * p.pieces;
  const int64_t ctas =
      (warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  return launch_kernel(vec32 ? copy_pages_kernel<true>
                             : copy_pages_kernel<false>,
                       dim3(static_cast<unsigned>(ctas)), kCopyThreads, 0,
                       stream, p.pdl, p);
}

int copy_piece_bytes(bool vec32) { return kUnroll * 32 * (vec32 ? 32 : 16); }

// One head to a CTA (four tokens deep, three CTAs per SM) while all of those
// run at once, else two heads (one token, five per SM).  Measured with 16
// lists of 8 heads, with the state's calls before: 384 CTAs of one head 93 us
// against 121 by two heads, 512 130 against 125, 2048 300 against 264.
cudaError_t launch_move_tokens(const MoveParams& p, cudaStream_t stream) {
  const int64_t ctas =
      static_cast<int64_t>(p.num_lists) * p.num_caches * p.H;
  return p.H == 1 || ctas <= 3 * sm_count()
             ? launch_move<1, 4, 3>(p, stream)
             : launch_move<2, 1, 5>(p, stream);
}

}  // namespace kvq
