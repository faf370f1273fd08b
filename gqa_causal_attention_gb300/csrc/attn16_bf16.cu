// Tensor-core attention of attn16.cuh in bf16, and how a shared prefix is split.
#include "attn16.cuh"

namespace gqa {

// As many splits as give every SM a block, but no more than leave the longest its length. Rows that
// fill one tile only are split by twos within a block, unless every split is one key block.
PrefixPlan shared_prefix_plan(int B, int H, int Hkv, int prefix_len) {
  const int TQ = attn16::kRows / (H / Hkv), tokens = 2 * TQ;
  const int units = Hkv * ((B + tokens - 1) / tokens);
  const int blocks = (prefix_len + attn16::kBK - 1) / attn16::kBK;
  const int most = 152 / units < 1 ? 1 : 152 / units;
  const int per = (blocks + most - 1) / most;
  return {(blocks + per - 1) / per, B <= TQ && per > 1};
}

cudaError_t launch_attn16_bf16(const Attn16Job& j, cudaStream_t stream) {
  return attn16::launch_type<__nv_bfloat16>(j, stream);
}

}  // namespace gqa
