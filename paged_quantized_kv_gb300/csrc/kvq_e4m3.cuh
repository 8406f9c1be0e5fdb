// kvq_e4m3.cuh -- device helpers of the kernels that quantise rows to e4m3:
// 16 elements of a lane, their largest size, their codes at a scale.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kvq {
namespace e4m3 {

template <bool kF16>
__device__ __forceinline__ uint32_t half2_max(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (kF16)
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Packed pair -> two fp32 values (exact for both element types).
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

// Two fp32 -> e4m3 codes, rn, satfinite; `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t pair;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(hi),
      "f"(lo));
  return pair;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(lo)) |
         (static_cast<uint64_t>(__float_as_uint(hi)) << 32);
}

// Four elements (two packed pairs) -> their four e4m3 codes, element 0 in
// the low byte: q0 = k y, r = k + q0 (-scale), q1 = q0 + r y (P. Markstein's
// quotient correction, IBM J. Res. Dev. 34(1), 1990) as packed IEEE
// products and fused multiply-adds (two elements per f32x2 instruction),
// then cvt.rn.satfinite.e4m3x2.f32.  The codes are those of the IEEE quotients,
// which tests/quotient_exhaustive.c shows for every pair of inputs.  y2 = {y, y}, ns2 = {-scale, -scale}.
__device__ __forceinline__ uint32_t codes4(uint64_t x01, uint64_t x23,
                                           uint64_t y2, uint64_t ns2) {
  uint32_t out;
  asm("{ .reg .b64 p, q, r, t;\n"
      "  .reg .f32 p0, p1, q0, q1;\n"
      "  .reg .b16 c0, c1;\n"
      "  mul.rn.f32x2 p, %1, %3;\n"
      "  mul.rn.f32x2 q, %2, %3;\n"
      "  fma.rn.f32x2 r, p, %4, %1;\n"
      "  fma.rn.f32x2 t, q, %4, %2;\n"
      "  fma.rn.f32x2 p, r, %3, p;\n"
      "  fma.rn.f32x2 q, t, %3, q;\n"
      "  mov.b64 {p0, p1}, p;\n"
      "  mov.b64 {q0, q1}, q;\n"
      "  cvt.rn.satfinite.e4m3x2.f32 c0, p1, p0;\n"
      "  cvt.rn.satfinite.e4m3x2.f32 c1, q1, q0;\n"
      "  mov.b32 %0, {c0, c1}; }"
      : "=r"(out)
      : "l"(x01), "l"(x23), "l"(y2), "l"(ns2));
  return out;
}

// The sign bits of four packed 16-bit elements (two words, element 0 in the
// low half of wa) as the top bits of four bytes.
__device__ __forceinline__ uint32_t signs4(uint32_t wa, uint32_t wb) {
  return __byte_perm(wa, wb, 0x7531) & 0x80808080u;
}

// The rule written out for one lane's 16 elements: an IEEE division per
// element.  Out of line: it runs only for tokens whose scale is below
// 2^-90.
template <bool kF16>
__device__ __noinline__ uint4 codes16_exact(uint4 w0, uint4 w1,
                                            float scale) {
  const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float a, b, d, e;
    widen2<kF16>(w[2 * k], a, b);
    widen2<kF16>(w[2 * k + 1], d, e);
    c[k] = e4m3x2(__fdiv_rn(a, scale), __fdiv_rn(b, scale)) |
           (e4m3x2(__fdiv_rn(d, scale), __fdiv_rn(e, scale)) << 16);
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// The codes of a lane's 16 packed elements at `scale` = amax / 448 (0: codes
// of 0).
template <bool kF16>
__device__ __forceinline__ void codes16(const uint32_t (&raw)[8], float scale,
                                        uint32_t (&codes)[4]) {
  if (scale >= 0x1p-90f) {
    const float y = __frcp_rn(scale);
    const uint64_t y2 = pack2(y, y);
    const uint64_t ns2 = pack2(-scale, -scale);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a, b, d, e;
      widen2<kF16>(raw[2 * k], a, b);
      widen2<kF16>(raw[2 * k + 1], d, e);
      codes[k] = codes4(pack2(a, b), pack2(d, e), y2, ns2) |
                 signs4(raw[2 * k], raw[2 * k + 1]);
    }
  } else {
    const uint4 c =
        codes16_exact<kF16>(make_uint4(raw[0], raw[1], raw[2], raw[3]),
                            make_uint4(raw[4], raw[5], raw[6], raw[7]), scale);
    codes[0] = c.x;
    codes[1] = c.y;
    codes[2] = c.z;
    codes[3] = c.w;
  }
}

}  // namespace e4m3
}  // namespace kvq
