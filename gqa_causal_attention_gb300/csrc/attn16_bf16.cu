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

// No call of at most B rows and prefix_len positions has more partial rows. Splits x pairs of tiles
// are at most one block an SM, or there is one split; a block leaves 256 partial rows (two tiles of
// different rows, or the two halves of one tile's keys). And a row has at most a part for each
// key block and one more (an odd number of them split by twos), or two of each split.
size_t shared_prefix_rows(int B, int H, int Hkv, int prefix_len) {
  const int64_t tokens = 2 * (attn16::kRows / (H / Hkv)), rows = static_cast<int64_t>(B) * H;
  const int64_t units = Hkv * ((B + tokens - 1) / tokens);
  const int64_t blocks = (prefix_len + int64_t(attn16::kBK) - 1) / attn16::kBK;
  const int64_t splits = std::max(1, 152 / Hkv);
  return std::min(rows * std::min(blocks + 1, 2 * splits), 2 * attn16::kRows * std::max<int64_t>(units, 152));
}

cudaError_t launch_attn16_bf16(const Attn16Job& j, cudaStream_t stream) {
  return attn16::launch_type<__nv_bfloat16>(j, stream);
}

}  // namespace gqa
