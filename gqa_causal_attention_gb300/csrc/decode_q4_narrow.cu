// The 4-bit decode's split kernel for head dims up to 128.
#include "decode_q4_kernel.cuh"

namespace gqa {

cudaError_t launch_decode_q4_narrow(const DecodeQ4Job& j, const StepQ4Args& st, cudaStream_t stream) {
  switch (j.D / 32) {
    case 1: return launch_split<1>(j, st, stream);
    case 2: return launch_split<2>(j, st, stream);
    case 3: return launch_split<3>(j, st, stream);
    default: return launch_split<4>(j, st, stream);
  }
}

}  // namespace gqa
