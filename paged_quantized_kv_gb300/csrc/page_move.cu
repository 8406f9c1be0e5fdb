// page_move.cu -- bytes of a paged cache from place to place, sm_103a:
// whole pages (kvq_copy_pages) and single NVFP4 tokens
// (kvq_move_tokens_nvfp4), in many caches (a model's layers) at once.
//
// Both read and write every byte once and compute nothing: they are bound
// by HBM bandwidth, and for a few pages by the launch.
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
// single tokens: a CTA walks one list of one (cache, side, head)
// ---------------------------------------------------------------------------
// The tokens of a list may move within the same pages (a token's
// destination is then a place that an earlier token of the list left), so a
// list is walked in order: a step's tokens are all read before any of them
// is written.  A thread moves one 16-byte piece of a head row (32 elements)
// with its two group scales.  A V scale (and a swizzled K scale) of group j
// of a token at offset r of its 4-token band is byte 4j + r of the band's
// head tile, whose 4 rows are scale-row strides apart.
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

__global__ void __launch_bounds__(kMoveThreads)
    move_tokens_kernel(const __grid_constant__ MoveParams p) {
  pdl_prologue();
  const int i = blockIdx.x;             // list
  const int h = blockIdx.y >> 1, side = blockIdx.y & 1;
  uint8_t* cache = p.caches[blockIdx.z] + (side ? p.value_offset : 0);
  const int64_t begin = p.cu[i], end = p.cu[i + 1];
  if (begin < 0 || end < begin || end > p.total) {
    if (threadIdx.x == 0) flag(p.err, KVQ_DEVERR_SEQ);
    return;
  }
  const int vecs = p.D / 32;            // 16-byte pieces of a head row
  const bool swz = side == 1 || p.swizzle_k;
  const int half = p.S / 4;             // scale groups in a swizzled row
  const int per = kMoveThreads / vecs;  // tokens of a round
  const int tok = threadIdx.x / vecs, c = threadIdx.x - tok * vecs;
  const bool works = tok < per;

  auto data_at = [&](int64_t blk, int off) {
    return cache + blk * p.page_stride + h * p.dhs + off * p.dts + 16 * c;
  };
  auto scale_at = [&](int64_t blk, int off, int j) {
    const uint8_t* tile = cache + blk * p.page_stride + p.scale_off;
    const int row = swz ? (off & ~3) + j / half : off;
    const int col = swz ? (j % half) * 4 + (off & 3) : j;
    return const_cast<uint8_t*>(tile) + h * p.shs + row * p.sts + col;
  };

  for (int64_t base = begin; base < end; base += kMoveUnroll * per) {
    uint4 d[kMoveUnroll];
    uint8_t s0[kMoveUnroll], s1[kMoveUnroll];
    int64_t to_blk[kMoveUnroll];
    int to_off[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int64_t t = base + u * per + tok;
      to_blk[u] = -1;
      to_off[u] = 0;
      if (!works || t >= end) continue;
      const int64_t src = p.src[t], dst = p.dst[t];
      if (src < 0 || dst < 0 || src == dst) continue;
      if (src >= p.num_slots || dst >= p.num_slots) {
        flag(p.err, KVQ_DEVERR_SLOT);
        continue;
      }
      const int64_t blk = src / p.B;
      const int off = static_cast<int>(src - blk * p.B);
      d[u] = load16(data_at(blk, off));
      s0[u] = *scale_at(blk, off, 2 * c);
      s1[u] = *scale_at(blk, off, 2 * c + 1);
      to_blk[u] = dst / p.B;
      to_off[u] = static_cast<int>(dst - to_blk[u] * p.B);
    }
    __syncthreads();  // all of the step is read
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      if (to_blk[u] < 0) continue;
      *reinterpret_cast<uint4*>(data_at(to_blk[u], to_off[u])) = d[u];
      *scale_at(to_blk[u], to_off[u], 2 * c) = s0[u];
      *scale_at(to_blk[u], to_off[u], 2 * c + 1) = s1[u];
    }
  }
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

cudaError_t launch_move_tokens(const MoveParams& p, cudaStream_t stream) {
  return launch_kernel(move_tokens_kernel,
                       dim3(p.num_lists, 2 * p.H, p.num_caches),
                       kMoveThreads, 0, stream, p.pdl, p);
}

}  // namespace kvq
