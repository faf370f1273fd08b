// Device helpers shared by the kernels of this library.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gqa_attn.h"

namespace gqa {

__device__ __forceinline__ void report(int32_t* status, int32_t bits) {
  if (status) atomicOr(status, bits);
}

// True when the call's non-finite check found a bad input: every kernel of the
// call then returns at once (skip is the caller's status word, or nullptr when
// the check is off).
__device__ __forceinline__ bool gated_off(const int32_t* skip) {
  return skip && (*reinterpret_cast<const volatile int32_t*>(skip) & ATTN_DEV_NONFINITE);
}

// A kernel launched by launch_dependent may start while the one enqueued before it still
// runs, whatever that one is: it must call dependent_wait before its first access to global
// memory, which returns when everything before has ended and its writes are visible. What it
// reads may thus be written while it is already resident: no read-only loads (__ldg). With
// dependents_may_launch a kernel lets the next one be placed once all of its own blocks have
// got there. (Every kernel of the 4-bit cache waits this way: they are short, and between
// two of them the launch otherwise costs about 2 us.)
__device__ __forceinline__ void dependent_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependents_may_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem,
                             cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// c * tanh(s / c) written as c * (1 - 2 / (exp(2 s / c) + 1)), evaluated with
// the hardware base-2 exponential. Relative error of the tanh stays near
// fp32 rounding for every |s / c| (the cancellation near 0 costs a few bits
// of a value that is itself small); exp2 overflow to +inf gives exactly c.
__device__ __forceinline__ float softcap_apply(float s, float cap, float two_log2e_over_cap) {
  float e = exp2f(s * two_log2e_over_cap);
  return cap - 2.0f * cap / (e + 1.0f);
}

}  // namespace gqa
