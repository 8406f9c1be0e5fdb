// paged_attention_mma.cu -- the decode attention's rows and the merge of long
// contexts; which kernel a launch's rows take.  (paged_attention_mma.cuh has
// the kernel; rows of chunks, and of trees and lists, are compiled in
// translation units of their own, side by side.)
#include "paged_attention_mma.cuh"

namespace kvq {
namespace {

// ---------------------------------------------------------------------------
// Merge of the partitions of contexts longer than one partition
// ---------------------------------------------------------------------------
// 16 rows (sequence, query head) per CTA of 256 threads, a half-warp per
// row and 8 head dims per lane, so that one wave of CTAs covers a whole
// decode batch.  The context length is read before the wait for the
// attention kernel, which writes none of it; every thread waits before it
// may leave.  Per dim, the sums run over the partitions in order.
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = kMergeThreads / 16;
// Rows of at most this many partitions issue all their loads at once.
constexpr int kMergeFew = 4;

// kLive: rows that a list on the device names (AttnParams::live), the grid's
// in turn.
template <bool kF16, int kOf, bool kLive>
__global__ void __launch_bounds__(kMergeThreads)
attention_merge_kernel(const AttnParams p) {
  const int sub = threadIdx.x & 15;  // dims 8 sub .. 8 sub + 7
  int64_t row =
      static_cast<int64_t>(blockIdx.x) * kMergeRows + (threadIdx.x >> 4);
  const int rows = kLive ? __ldg(p.live) : p.num_seqs;
  do {
    const bool live = row < static_cast<int64_t>(rows) * p.Hq;
    const int b = live ? static_cast<int>(row / p.Hq) : 0;
    const int h = live ? static_cast<int>(row - static_cast<int64_t>(b) * p.Hq)
                       : 0;
    const Row me = live ? row_of<kOf>(p, b) : Row{0, 0, 0, false, false, 0, 0u};
    pdl_prologue();
    const int L = me.live ? me.L : 0;
    const int nparts = (L + p.part - 1) / p.part;
    if (!live || (!kLive && nparts <= 1)) return;
    if (kLive && nparts <= 1) continue;
    const int64_t row0 = row * p.max_parts;
    float M = -INFINITY;
    float den = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto add = [&](float w, const float4& x, const float4& y) {
      den += w;
      acc[0] += w * x.x; acc[1] += w * x.y;
      acc[2] += w * x.z; acc[3] += w * x.w;
      acc[4] += w * y.x; acc[5] += w * y.y;
      acc[6] += w * y.z; acc[7] += w * y.w;
    };
    if (nparts <= kMergeFew) {
      // every load of the row in one round trip, then the same sums in order
      float ml[kMergeFew], es[kMergeFew];
      float4 xs[kMergeFew], ys[kMergeFew];
#pragma unroll
      for (int i = 0; i < kMergeFew; ++i) {
        if (i < nparts) {
          ml[i] = p.max_logits[row0 + i];
          es[i] = p.exp_sums[row0 + i];
          const float4* src = reinterpret_cast<const float4*>(
              p.tmp_out + (row0 + i) * kD + 8 * sub);
          xs[i] = src[0];
          ys[i] = src[1];
        }
      }
#pragma unroll
      for (int i = 0; i < kMergeFew; ++i)
        if (i < nparts) M = fmaxf(M, ml[i]);
#pragma unroll
      for (int i = 0; i < kMergeFew; ++i)
        if (i < nparts) add(es[i] * ex2(ml[i] - M), xs[i], ys[i]);
    } else {
#pragma unroll 4
      for (int i = 0; i < nparts; ++i) M = fmaxf(M, p.max_logits[row0 + i]);
#pragma unroll 2
      for (int i = 0; i < nparts; ++i) {
        const float4* src = reinterpret_cast<const float4*>(
            p.tmp_out + (row0 + i) * kD + 8 * sub);
        add(p.exp_sums[row0 + i] * ex2(p.max_logits[row0 + i] - M), src[0],
            src[1]);
      }
    }
    const bool some = has_weights<kOf != kDecodeRows>(den);
    const float f = some ? 1.0f / den : 0.f;
    const float vs = __ldg(p.v_scale);
    uint32_t packed[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float y0 = some ? acc[2 * k] * f * vs : 0.f;
      const float y1 = some ? acc[2 * k + 1] * f * vs : 0.f;
      packed[k] = static_cast<uint32_t>(float_to_out<kF16>(y0)) |
                  (static_cast<uint32_t>(float_to_out<kF16>(y1)) << 16);
    }
    *reinterpret_cast<uint4*>(p.out + me.q * p.out_stride0 + h * kD + 8 * sub) =
        make_uint4(packed[0], packed[1], packed[2], packed[3]);
  } while (kLive &&
           (row += static_cast<int64_t>(gridDim.x) * kMergeRows) > 0);
}

template <int kOf, bool kLive>
auto merge_of(bool f16) {
  return f16 ? attention_merge_kernel<true, kOf, kLive>
             : attention_merge_kernel<false, kOf, kLive>;
}

bool marked(const AttnParams& p) { return p.listed || p.mask != nullptr; }

}  // namespace

cudaError_t launch_attention_merge(const AttnParams& p, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.Hq;
  int64_t ctas = (rows + kMergeRows - 1) / kMergeRows;
  if (p.live != nullptr)
    ctas = std::min<int64_t>(ctas,
                             static_cast<int64_t>(kListedCtas) * sm_count());
  const dim3 grid(static_cast<unsigned>(ctas));
  auto kernel = merge_of<kDecodeRows, false>(p.f16);
  if (p.live != nullptr)
    kernel = merge_of<kMarkedRows, true>(p.f16);
  else if (marked(p))
    kernel = merge_of<kMarkedRows, false>(p.f16);
  else if (p.cu != nullptr)
    kernel = merge_of<kChunkRows, false>(p.f16);
  return launch_kernel(kernel, grid, kMergeThreads, 0, stream, true, p);
}

cudaError_t launch_paged_attention_mma(const AttnParams& p,
                                       cudaStream_t stream) {
  if (marked(p)) return launch_marked_rows(p, stream);
  if (p.cu != nullptr) return launch_chunk_rows(p, stream);
  return launch_rows<kDecodeRows>(p, stream);
}

}  // namespace kvq
