// 16-bit tensors and the paged KV cache: what their kernels share.
//
// Rows of heads are token-major, x[token * token_stride + head * head_stride + d] (elements);
// the pools are [pages, Hkv, page, D] with a stride of their own between pages. Position p of
// row b lies in slot p % page of pool page block_table[b][p / page].
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace gqa {

constexpr float kLog2e16 = 1.4426950408889634f;

template <class T>
struct Rows {
  T* p;
  int64_t token, head;      // strides in elements
  __device__ __forceinline__ T* at(int64_t t, int h) const { return p + t * token + h * head; }
};
template <class T>
__host__ __device__ __forceinline__ Rows<T> rows_as(const RowsArg& r) {
  return {static_cast<T*>(r.p), r.token, r.head};
}

// The eight 16-bit values of a 16-byte granule as floats, and back (rounded to nearest even).
__device__ __forceinline__ float2 two(__nv_bfloat162 x) { return __bfloat1622float2(x); }
__device__ __forceinline__ float2 two(__half2 x) { return __half22float2(x); }
template <class T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct Pair<__half> {
  using type = __half2;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <class T>
__device__ __forceinline__ float2 unpack(uint32_t x) {
  return two(*reinterpret_cast<const typename Pair<T>::type*>(&x));
}
template <class T>
__device__ __forceinline__ void unpack8(const uint4& v, uint64_t (&x)[4]) {   // in pairs
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack<T>(w[i]);
    x[i] = tc::pack2(f.x, f.y);
  }
}
template <class T>
__device__ __forceinline__ uint32_t pack(uint64_t x) {
  float a, b;
  tc::unpack2(x, a, b);
  return Pair<T>::pack(a, b);
}
template <class T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(Pair<T>::pack(x[0], x[1]), Pair<T>::pack(x[2], x[3]),
                    Pair<T>::pack(x[4], x[5]), Pair<T>::pack(x[6], x[7]));
}
template <class T>
__device__ __forceinline__ uint4 pack8(const uint64_t (&x)[4]) {
  return make_uint4(pack<T>(x[0]), pack<T>(x[1]), pack<T>(x[2]), pack<T>(x[3]));
}

// The largest b in [0, n) with key(b) <= x for nondecreasing keys (-1: none), found by the whole
// warp, 32 keys at a time: two rounds of loads for up to 1024 keys.
template <class F>
__device__ __forceinline__ int warp_find_last(int n, int64_t x, F key) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool le = i < n && key(lo + i) <= x;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    if (c == 0) return -1;                   // only ever in the first round
    lo += (c - 1) * step;
    if (step == 1) return lo;
    n = min(step, n - (c - 1) * step);
  }
  return -1;
}

// cap tanh(scale x / cap) of a raw score x, in log2 units: where |scale x / cap| <= 0.4, tanh's series to
// the ninth power (the next term is 1e-6 of the value); past it, out (1 - 2 / (2^(in x) + 1)), which
// loses out's bits against a small x: a cap of 1e6 would leave a score of 1 off by 5%.
struct CapArgs {
  int on;
  float in, out;
  float series[5], limit;                      // limit: in a raw score; -1: no series
};
// A cap of 2^60 scales or more is none: it changes a score by fp32's rounding where that reaches 2^48,
// and by less below.
inline CapArgs cap_args(float softcap, float scale) {
  CapArgs a{};
  const double c = static_cast<double>(scale) / softcap;
  a.on = softcap > 0.f && c > 0x1p-60;
  if (!a.on) return a;
  a.in = static_cast<float>(std::fmin(2.0 * kLog2e16 * c, FLT_MAX));   // finite: 0 times it is 0
  a.out = kLog2e16 * softcap;
  a.limit = static_cast<float>(0.4 / c);
  // tanh u = u (1 - u^2/3 + 2 u^4/15 - 17 u^6/315 + 62 u^8/2835 - ...)
  const double series[5] = {1.0, -1.0 / 3, 2.0 / 15, -17.0 / 315, 62.0 / 2835};
  double power = static_cast<double>(scale) * 1.4426950408889634;
  for (int i = 0; i < 5; ++i, power *= c * c) {
    a.series[i] = static_cast<float>(series[i] * power);
    if (!std::isfinite(a.series[i])) a.limit = -1.f;   // a cap of next to nothing
  }
  return a;
}

// Sequence b's rows [first, first + n) of T packed rows; n < 0 where cu_seqlens breaks a rule.
struct SeqRows {
  int first, n;
};
__device__ __forceinline__ SeqRows seq_rows(const int32_t* cu, int b, int T) {
  const int a = cu[b], e = cu[b + 1];
  return {a, a < 0 || e < a || e > T ? -1 : e - a};
}

}  // namespace gqa
