// attention_chunk_rows.cu -- tokens of short chunks through the decode
// attention's kernel.
#include "paged_attention_mma.cuh"

namespace kvq {

cudaError_t launch_chunk_rows(const AttnParams& p, cudaStream_t stream) {
  return launch_rows<kChunkRows>(p, stream);
}

}  // namespace kvq
