// Tensor-core attention of attn16.cuh in bf16, and how a shared prefix is split.
#include "attn16.cuh"

namespace gqa {

// As many splits as give every SM a block, of at least two key blocks each; twice that many
// partial results where the rows fill one tile only (a block's two halves then take every
// other key block each).
int shared_prefix_splits(int B, int H, int Hkv, int prefix_len) {
  const int TQ = attn16::kRows / (H / Hkv), tokens = 2 * TQ;
  const int units = Hkv * ((B + tokens - 1) / tokens);
  const int blocks = (prefix_len + attn16::kBK - 1) / attn16::kBK;
  int n = 152 / units;
  if (n > blocks / 2) n = blocks / 2;
  if (n < 1) n = 1;
  return B <= TQ ? 2 * n : n;
}

cudaError_t launch_attn16_bf16(const Attn16Job& j, cudaStream_t stream) {
  return attn16::launch_type<__nv_bfloat16>(j, stream);
}

}  // namespace gqa
