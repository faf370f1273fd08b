// The 4-bit decode's split kernel for head dims above 128.
#include "decode_q4_kernel.cuh"

namespace gqa {

cudaError_t launch_decode_q4_wide(const DecodeQ4Job& j, const StepQ4Args& st, cudaStream_t stream) {
  switch (j.D / 32) {
    case 5: return launch_split<5>(j, st, stream);
    case 6: return launch_split<6>(j, st, stream);
    case 7: return launch_split<7>(j, st, stream);
    default: return launch_split<8>(j, st, stream);
  }
}

}  // namespace gqa
