// Attention over a paged cache, heads of 256 channels (see gdn_attn.cuh).

#include "gdn_attn.cuh"

namespace gdn {

cudaError_t launch_attn_256(const AttnArgs &P, bool bf16, cudaStream_t stream) {
  return attn::launch<256>(P, bf16, stream);
}

}  // namespace gdn
