// attention_marked_rows.cu -- drafts of small trees and rows of block lists
// through the decode attention's kernel.
#include "paged_attention_mma.cuh"

namespace kvq {

cudaError_t launch_marked_rows(const AttnParams& p, cudaStream_t stream) {
  return launch_rows<kMarkedRows>(p, stream);
}

}  // namespace kvq
