// The 4-bit KV cache record, and what the kernels share to read and write it.
//
// One record holds one slot of one kv head: key and value of D = 32 M dims, in
// groups of 32 dims, each group M 4-bit codes c in [-7, 7] (stored as c + 8) with
// one bf16 scale s; the value is c * s, exact in fp32 (3 + 8 significant bits).
//   [0, 16 M)       key codes: 32-bit word w = a M + g holds dims 32 g + 8 a + i at bits 4 i
//   [16 M, 32 M)    value codes: 16-bit unit u = n M + g holds dims 32 g + 4 n + j at bits 4 j
//   [32 M, 34 M)    key scales, [34 M, 36 M) value scales (bf16), zero padding to 16 bytes
// The word order is the tensor-core fragment order of the decode: thread (n, a) of
// a warp (n = lane / 4, a = lane % 4) reads its M key words and its M value units
// of a record as one contiguous piece each. Records are multiples of 16 bytes, so
// any run of slots is one bulk copy; key and value share a record because a step
// always needs both, and because 18 M + 18 M bytes pad better than each alone
// (144 bytes, no padding, at D = 128; fp32 takes 1024).
#pragma once

#include <stdint.h>

namespace gqa {
namespace q4 {

__host__ __device__ constexpr int record_bytes(int M) { return (36 * M + 15) / 16 * 16; }

constexpr uint32_t kNanScale = 0x7fc0u;   // a group that held an inf or NaN: reads back as NaN

#ifdef __CUDACC__

__device__ __forceinline__ float bf16_to_float(uint32_t bits) { return __uint_as_float(bits << 16); }

__device__ __forceinline__ uint32_t group_max_u(uint32_t v) {      // over 8 aligned lanes
  v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
  v = max(v, __shfl_xor_sync(0xffffffffu, v, 2));
  return max(v, __shfl_xor_sync(0xffffffffu, v, 4));
}

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// x > 0 (finite) rounded once to bf16, ties to even; below 2^-126 to the subnormal grid.
__device__ __forceinline__ uint32_t bf16_bits_of(double x) {
  if (x < 0x1p-126) return static_cast<uint32_t>(__double2int_rn(x * 0x1p133));
  const unsigned long long b = __double_as_longlong(x);
  // 45 of the 52 stored bits go; the exponent is rebased from 1023 to 127
  const unsigned long long r = (b + ((1ull << 44) - 1) + ((b >> 45) & 1ull)) >> 45;
  return static_cast<uint32_t>(r - (896ull << 7));
}

// Four neighbouring dims of one row around RMSNorm and RoPE:
//   y[e] = a[e] * c[e] + b[e] * s[e],  a = own * inv * wo,  b = oth * inv * wt
// with own the dims' raw values, oth their rotary partners', inv the row's 1 / rms
// (1, and weights unused, without a norm). y is fp32, off by at most err.
struct Quad {
  float own[4], oth[4], c[4], s[4], wo[4], wt[4];
  float y[4], err[4];
};

// What four dims become: 16 bits of codes, and their group's scale (the same on the
// group's 8 lanes).
struct Coded {
  uint32_t codes, scale;
};

// Quantises the warp's row of D dims: lane l holds quads l + 32 k (k < NC) of its D / 4
// (zeros where there is none); a group is 8 aligned lanes. Codes and scales are those
// of the exact y (of own when PLAIN: no norm and no rotation): the scale is
// bf16(max|y| / 7), the code rint(y / scale), both rounded once, ties to even. fp32
// decides wherever it is further from a rounding border than its error; otherwise the
// warp works the row out again in fp64, whose rate is a thirtieth of fp32's here, so
// that all rows in fp64 would cost several times the memory traffic. At D = 128 that
// is under one row in a hundred with RoPE. Every lane of the warp must call it.
template <int NC, bool PLAIN>
__device__ __forceinline__ void quantise_row(const Quad (&q)[NC], bool norm, int D, float eps,
                                             Coded (&out)[NC]) {
  bool unsure = false;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const Quad& u = q[k];
    uint32_t top = 0, far = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      top = max(top, __float_as_uint(u.y[e]) & 0x7fffffffu);     // NaN above inf above the rest
      if (!PLAIN) far = max(far, __float_as_uint(u.err[e]));
    }
    top = group_max_u(top);
    if (!PLAIN) far = group_max_u(far);
    if (max(top, far) >= 0x7f800000u) {
      out[k].codes = 0x8888u;
      out[k].scale = kNanScale;
    } else if ((top | far) == 0) {
      out[k].codes = 0x8888u;
      out[k].scale = 0;
    } else {
      const float ferr = __uint_as_float(far);
      const float a7 = __uint_as_float(top) / 7.0f;
      const uint32_t bits = __float_as_uint(a7);
      const float mid = __uint_as_float((bits & 0xffff0000u) | 0x8000u);
      unsure |= a7 < 0x1p-120f || fabsf(a7 - mid) <= ferr * 0.15f + a7 * 0x1p-23f;
      const uint32_t sc = (bits + 0x7fffu + ((bits >> 16) & 1u)) >> 16;
      const float rs = 1.0f / bf16_to_float(sc);
      uint32_t codes = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // t is off by err / scale and by two roundings of 2^-24 of at most 7.04
        const float t = u.y[e] * rs, c = rintf(t);
        unsure |= 0.5f - fabsf(t - c) <= (PLAIN ? 0x1p-20f : fmaf(u.err[e], rs, 0x1p-20f));
        codes |= (static_cast<uint32_t>(static_cast<int>(c) + 8) & 15u) << (4 * e);
      }
      out[k].codes = codes;
      out[k].scale = sc;
    }
  }
  if (!__any_sync(0xffffffffu, unsure)) return;

  double inv = 1.0;
  if (!PLAIN && norm) {
    double ss = 0.0;
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) ss += static_cast<double>(q[k].own[e]) * q[k].own[e];
    inv = 1.0 / sqrt(warp_sum_d(ss) / D + static_cast<double>(eps));
  }
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const Quad& u = q[k];
    double y[4], amax = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (PLAIN) {
        y[e] = u.own[e];
      } else {
        double a = u.own[e], b = u.oth[e];
        if (norm) {
          a = a * inv * u.wo[e];
          b = b * inv * u.wt[e];
        }
        y[e] = a * u.c[e] + b * u.s[e];
      }
      amax = fmax(amax, fabs(y[e]));
    }
#pragma unroll
    for (int o = 1; o <= 4; o <<= 1) amax = fmax(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (out[k].scale != kNanScale) {
      const uint32_t sc = amax > 0.0 ? bf16_bits_of(amax / 7.0) : 0u;
      const double s = bf16_to_float(sc);
      uint32_t codes = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = sc ? max(-7, min(7, __double2int_rn(y[e] / s))) : 0;
        codes |= static_cast<uint32_t>(c + 8) << (4 * e);
      }
      out[k].codes = codes;
      out[k].scale = sc;
    }
  }
}

// Stores lane `lane`'s quads of a row into the record at rec: the key part (part = 0)
// or the value part (part = 1).
template <int M, int NC>
__device__ __forceinline__ void store_part(uint8_t* rec, int part, const Coded (&q)[NC], int lane) {
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int ch = lane + 32 * k;
    if (ch >= 8 * M) continue;
    const int g = ch >> 3, e = ch & 7;                  // group, quad within it
    const int at = part ? 16 * M + 2 * (e * M + g) : 4 * ((e >> 1) * M + g) + 2 * (e & 1);
    *reinterpret_cast<uint16_t*>(rec + at) = static_cast<uint16_t>(q[k].codes);
    if (e == 0)
      *reinterpret_cast<uint16_t*>(rec + (32 + 2 * part) * M + 2 * g) =
          static_cast<uint16_t>(q[k].scale);
  }
  if (part == 1) {                                      // zero padding
    constexpr int pad = (record_bytes(M) - 36 * M) / 2;
    if (pad > 0 && lane < pad) *reinterpret_cast<uint16_t*>(rec + 36 * M + 2 * lane) = 0;
  }
}

#endif  // __CUDACC__

}  // namespace q4
}  // namespace gqa
