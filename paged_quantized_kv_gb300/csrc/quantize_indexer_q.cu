// quantize_indexer_q.cu -- the indexer's queries, bf16 / fp16 -> e4m3 with
// the scale of each head folded into its weight, sm_103a.
//
// For head h of row t: s = max |q| / 448, codes = e4m3(q / s), w = (weight *
// scale) * s, so that w * relu(codes . k) is weight * scale * relu(q . k) up
// to the rounding of the codes.  The rule of the codes is that of the
// indexer-K store.
//
// A lane takes 16 elements (32 bytes in, 16 out) of two heads, D / 16 lanes a
// head; the maximum goes over them by shuffles.  Bound by HBM: 2 D + 4 bytes
// read and D + 4 written per head.  6000 rows of 64 heads of 128 (150 MB): 27
// us, 5.6 TB/s, 84 % of the measured copy rate (an IEEE division for each
// element, and one head a thread: 37 us).
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_e4m3.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

using namespace e4m3;

constexpr int kThreads = 256;
constexpr int kUnroll = 2;

__device__ __forceinline__ void load16(const uint16_t* p, uint32_t (&w)[8],
                                       bool vec32) {
  if (vec32) {
    asm volatile(
        "ld.global.nc.L1::no_allocate.v8.u32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]),
          "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(p));
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

template <bool kF16, int L>
__global__ void __launch_bounds__(kThreads)
    quantize_q_kernel(const QuantizeQParams p) {
  pdl_prologue();
  constexpr int kHeads = kThreads / L;  // of a thread block at a time
  const int part = threadIdx.x % L, lane = threadIdx.x & 31;
  const int64_t first =
      static_cast<int64_t>(blockIdx.x) * (kUnroll * kHeads) + threadIdx.x / L;
  const int64_t n = p.total * p.heads;
  uint32_t raw[kUnroll][8];
  float weight[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = first + u * kHeads;  // row * heads + head
#pragma unroll
    for (int k = 0; k < 8; ++k) raw[u][k] = 0u;
    weight[u] = 0.0f;
    if (i >= n) continue;
    int64_t q = i * (16 * L), w = i;
    if (!p.dense) {
      const int64_t t = i / p.heads, h = i - t * p.heads;
      q = t * p.q_stride0 + h * (16 * L);
      w = t * p.w_stride0 + h;
    }
    load16(p.q + q + part * 16, raw[u], p.vec32);
    if (part == 0) weight[u] = __ldg(p.weights + w);
  }
  const uint32_t lanes = L == 32 ? ~0u : ((1u << L) - 1u) << (lane / L * L);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = first + u * kHeads;
    uint32_t m = raw[u][0] & 0x7FFF7FFFu;
#pragma unroll
    for (int k = 1; k < 8; ++k)
      m = half2_max<kF16>(m, raw[u][k] & 0x7FFF7FFFu);
    float lo, hi;
    widen2<kF16>(m, lo, hi);
    float amax = fmaxf(lo, hi);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, o));
    if (i >= n) continue;
    const float s = __fdiv_rn(amax, 448.0f);
    uint32_t c[4] = {0u, 0u, 0u, 0u};
    if (amax != 0.0f) codes16<kF16>(raw[u], s, c);
    *reinterpret_cast<uint4*>(p.q_fp8 + (i * L + part) * 16) =
        make_uint4(c[0], c[1], c[2], c[3]);
    if (part == 0)
      p.w_out[i] = __fmul_rn(__fmul_rn(weight[u], p.scale), s);
  }
}

template <bool kF16, int L>
cudaError_t launch(const QuantizeQParams& p, cudaStream_t stream) {
  constexpr int64_t kHeads = kUnroll * (kThreads / L);
  const int64_t ctas = (p.total * p.heads + kHeads - 1) / kHeads;
  return launch_kernel(quantize_q_kernel<kF16, L>,
                       dim3(static_cast<unsigned>(ctas)), kThreads, 0, stream,
                       p.pdl, p);
}

template <bool kF16>
cudaError_t launch_dim(const QuantizeQParams& p, cudaStream_t stream) {
  switch (p.D) {  // D / 16 lanes per head
    case 16: return launch<kF16, 1>(p, stream);
    case 32: return launch<kF16, 2>(p, stream);
    case 64: return launch<kF16, 4>(p, stream);
    case 128: return launch<kF16, 8>(p, stream);
    default: return launch<kF16, 16>(p, stream);  // 256
  }
}

}  // namespace

cudaError_t launch_quantize_q(const QuantizeQParams& p, cudaStream_t stream) {
  return p.f16 ? launch_dim<true>(p, stream) : launch_dim<false>(p, stream);
}

}  // namespace kvq
