// chunk_attention.cu -- attention of a chunk of new tokens over the NVFP4
// pages, sm_103a.
//
// A warp computes one output row (new token, query head): it walks the
// row's visible tokens once with a running maximum and sum.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kD = 128;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void flag(int32_t* err, int32_t bits) {
  if (err != nullptr) atomicOr(err, bits);
}

__device__ __forceinline__ float e4m3(uint8_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  float f;
  asm("{ .reg .f16 a, b;\n mov.b32 {a, b}, %1;\n cvt.f32.f16 %0, a; }"
      : "=f"(f) : "r"(h));
  return f;
}

__device__ __forceinline__ float e2m1(uint32_t q) {
  const uint32_t m = q & 7u;
  const float v = m < 2 ? 0.5f * m : (1.0f + 0.5f * (m & 1)) *
                                         static_cast<float>(1 << ((m >> 1) - 1));
  return (q & 8u) ? -v : v;
}

// The 4 elements 4 * lane .. + 3 of a head row.
__device__ __forceinline__ void load4(const ChunkParams& p, int side,
                                      int32_t blk, int off, int h, int lane,
                                      float (&x)[4]) {
  const uint8_t* page = p.side[side] + blk * p.page_stride;
  const uint16_t w = *reinterpret_cast<const uint16_t*>(
      page + h * p.dhs + off * p.dts + 2 * lane);
  const int j = lane >> 2;
  const bool swz = side == 1 || p.swizzle_k;
  const int row = swz ? (off & ~3) + j / 2 : off;
  const int col = swz ? (j % 2) * 4 + (off & 3) : j;
  const float sf =
      e4m3(page[p.scale_off + h * p.shs + row * p.sts + col]);
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = e2m1((w >> (4 * k)) & 15u) * sf;
}

__device__ __forceinline__ float half_bits(uint16_t v, bool f16) {
  float f;
  if (f16)
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(v));
  else
    f = __uint_as_float(static_cast<uint32_t>(v) << 16);
  return f;
}

__global__ void __launch_bounds__(256)
    chunk_kernel(const __grid_constant__ ChunkParams p) {
  pdl_prologue();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t r = w / p.Hq;
  const int hq = static_cast<int>(w - r * p.Hq);
  if (r >= p.total_q) return;
  // the sequence of the row
  int b = -1, q0 = 0, n = 0;
  for (int k = 0; k < p.num_seqs; ++k) {
    const int lo = max(p.cu[k], 0);
    const int hi = max(lo, static_cast<int>(min(
                               static_cast<int64_t>(p.cu[k + 1]), p.total_q)));
    if (lane == 0 && (lo != p.cu[k] || hi != p.cu[k + 1]))
      flag(p.dev_error, KVQ_DEVERR_SEQ);
    if (lo <= r && r < hi) {
      b = k;
      q0 = lo;
      n = hi - lo;
    }
  }
  if (b < 0) return;
  int L = p.lens[b];
  if (L > p.len_cap) {
    L = p.len_cap;
    if (lane == 0) flag(p.dev_error, KVQ_DEVERR_SEQ);
  }
  const int64_t last = static_cast<int64_t>(L) - n + (r - q0);
  float q[4];
  {
    const uint16_t* src = p.q + r * p.q_stride0 + hq * kD + 4 * lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = half_bits(src[k], p.f16);
  }
  const float c = p.scale * *p.k_scale * kLog2e;
  float m = -INFINITY, sum = 0.0f, o[4] = {0, 0, 0, 0};
  for (int64_t t = 0; t <= last; ++t) {
    const int32_t blk = p.block_table[b * p.bt_stride + t / p.B];
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0) flag(p.dev_error, KVQ_DEVERR_BLOCK);
      continue;
    }
    const int off = static_cast<int>(t % p.B), h = hq / p.G;
    float x[4];
    load4(p, 0, blk, off, h, lane, x);
    float s = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) s += q[k] * x[k];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    s *= c;
    const float mn = fmaxf(m, s);
    const float a = exp2f(m - mn), e = exp2f(s - mn);
    m = mn;
    sum = sum * a + e;
    load4(p, 1, blk, off, h, lane, x);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = o[k] * a + e * x[k];
  }
  const float f = sum > 0 ? *p.v_scale / sum : (sum == 0 ? 0.0f : sum);
  uint16_t* dst = p.out + r * p.out_stride0 + hq * kD + 4 * lane;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint16_t v;
    if (p.f16)
      asm("cvt.rn.f16.f32 %0, %1;" : "=h"(v) : "f"(o[k] * f));
    else
      asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(v) : "f"(o[k] * f));
    dst[k] = v;
  }
}

}  // namespace

int64_t chunk_workspace_bytes(int sms) {
  return static_cast<int64_t>(sms) * 2 * 256 * (kD + 4) * 4;
}

cudaError_t launch_chunk_attention(const ChunkParams& p,
                                   cudaStream_t stream) {
  const int64_t warps = p.total_q * p.Hq;
  return launch_kernel(chunk_kernel,
                       dim3(static_cast<unsigned>((warps + 7) / 8)), 256, 0,
                       stream, p.pdl, p);
}

}  // namespace kvq
