// Tensor-core attention of attn16.cuh in fp16.
#include "attn16.cuh"

namespace gqa {

cudaError_t launch_attn16_fp16(const Attn16Job& j, cudaStream_t stream) {
  return attn16::launch_type<__half>(j, stream);
}

}  // namespace gqa
