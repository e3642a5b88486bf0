// Attention over a paged cache, heads of 128 channels (see gdn_attn.cuh).

#include "gdn_attn.cuh"

namespace gdn {

cudaError_t launch_attn_128(const AttnArgs &P, bool bf16, cudaStream_t stream) {
  return attn::launch<128>(P, bf16, stream);
}

// (the entry for every head size)
cudaError_t launch_attn(const AttnArgs &P, int hd, bool bf16, cudaStream_t stream) {
  return hd == 64    ? launch_attn_64(P, bf16, stream)
         : hd == 128 ? launch_attn_128(P, bf16, stream)
                     : launch_attn_256(P, bf16, stream);
}

size_t attn_workspace_bytes(int kind, int M, int group, int hd) {
  return attn::bytes(kind, M, group, hd);
}

}  // namespace gdn
