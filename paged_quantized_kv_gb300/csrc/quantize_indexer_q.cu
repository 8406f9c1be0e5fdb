// quantize_indexer_q.cu -- the indexer's queries, bf16 / fp16 -> e4m3 with
// the scale of each head folded into its weight, sm_103a.
//
// For head h of row t: s = max |q| / 448, codes = e4m3(q / s), w = (weight *
// scale) * s, so that w * relu(codes . k) is weight * scale * relu(q . k) up
// to the rounding of the codes.  The rule of the codes is that of the
// indexer-K store.
//
// A lane takes 16 elements (32 bytes in, 16 out), D / 16 lanes a head; the
// maximum goes over them by shuffles.  Bound by HBM: 2 D + 4 bytes read and
// D + 4 written per head.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.h"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 256;

template <bool kF16>
__device__ __forceinline__ void widen2(uint32_t w, float& lo, float& hi) {
  if constexpr (kF16) {
    asm("{ .reg .f16 a, b;\n"
        "  mov.b32 {a, b}, %2;\n"
        "  cvt.f32.f16 %0, a;\n"
        "  cvt.f32.f16 %1, b; }"
        : "=f"(lo), "=f"(hi)
        : "r"(w));
  } else {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t pair;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(hi),
      "f"(lo));
  return pair;
}

template <bool kF16, int L>
__global__ void __launch_bounds__(kThreads)
    quantize_q_kernel(const QuantizeQParams p) {
  pdl_prologue();
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads +
                     threadIdx.x) / L;  // row * heads + head
  const int part = threadIdx.x % L;
  // (the lanes of a head leave together; shuffles name them only)
  if (i >= p.total * p.heads) return;
  const int64_t t = i / p.heads;
  const int h = static_cast<int>(i - t * p.heads);
  const uint4* src = reinterpret_cast<const uint4*>(
      p.q + t * p.q_stride0 + h * (16 * L) + part * 16);
  const uint4 a = __ldg(src), b = __ldg(src + 1);
  const float weight = part == 0 ? __ldg(p.weights + t * p.w_stride0 + h)
                                 : 0.0f;
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float x[16], amax = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    widen2<kF16>(w[k], x[2 * k], x[2 * k + 1]);
    amax = fmaxf(amax, fmaxf(fabsf(x[2 * k]), fabsf(x[2 * k + 1])));
  }
  const int lane = threadIdx.x & 31;
  const uint32_t lanes =
      L == 32 ? ~0u : ((1u << L) - 1u) << (lane / L * L);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1)
    amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, o));
  const float s = __fdiv_rn(amax, 448.0f);
  uint32_t c[4] = {0, 0, 0, 0};
  if (amax != 0.0f) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      c[k] = e4m3x2(__fdiv_rn(x[4 * k], s), __fdiv_rn(x[4 * k + 1], s)) |
             (e4m3x2(__fdiv_rn(x[4 * k + 2], s),
                     __fdiv_rn(x[4 * k + 3], s))
              << 16);
  }
  *reinterpret_cast<uint4*>(p.q_fp8 + (i * L + part) * 16) =
      make_uint4(c[0], c[1], c[2], c[3]);
  if (part == 0)
    p.w_out[i] = __fmul_rn(__fmul_rn(weight, p.scale), s);
}

template <bool kF16, int L>
cudaError_t launch(const QuantizeQParams& p, cudaStream_t stream) {
  const int64_t ctas = (p.total * p.heads * L + kThreads - 1) / kThreads;
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
