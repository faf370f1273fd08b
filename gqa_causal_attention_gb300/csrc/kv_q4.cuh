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

// What four neighbouring dims become: 16 bits of codes, and their group's scale (the same
// on the group's 8 lanes).
struct Coded {
  uint32_t codes, scale;
};

// t in (-2^21, 2^21) to the nearest integer, ties to even, as the sum's low bits: the float
// 1.5 * 2^23 + 8 + t is rounded at its unit place. Its low four bits are then t's code + 8.
constexpr float kRound = 12582920.0f;

// Quantises a row held as quads y[k] (dims 4 (lane + 32 k) .. + 3; zeros where there are
// none), each off from the exact values by at most err[k]; a group is 8 aligned lanes. The
// scale is bf16(max|y| / 7), the code rint(y / scale), ties to even. Returns whether every
// rounding was further from its border than the error (warp-uniform): if not, the row has
// to be done again by quantise_exact. EXACT: y is the row itself, err is not read. Every
// lane of the warp must call it. About six instructions a value.
template <int NC, bool EXACT>
__device__ __forceinline__ bool quantise_fast(const float (&y)[NC][4], const float (&err)[NC],
                                              Coded (&out)[NC]) {
  bool unsure = false;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(y[k][e]) & 0x7fffffffu);
    top = group_max_u(top);                               // NaN above inf above the rest
    const uint32_t far = EXACT ? 0u : group_max_u(__float_as_uint(err[k]));
    const float amax = __uint_as_float(top), ferr = __uint_as_float(far);
    // amax / 7 to two roundings; far from a bf16 border that settles the scale
    const float a7 = amax * (1.0f / 7.0f);
    const uint32_t bits = __float_as_uint(a7);
    const float mid = __uint_as_float((bits & 0xffff0000u) | 0x8000u);
    const uint32_t sc = (bits + 0x7fffu + ((bits >> 16) & 1u)) >> 16;
    float rs;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(bf16_to_float(sc)));
    // t = y / scale is off by err / scale, by 2^-23 of at most 7.04 in rs and by its rounding
    const float near = 0.5f - (EXACT ? 0x1p-19f : fmaf(err[k], rs, 0x1p-19f));
    uint32_t b[4];
    float off = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float t = y[k][e] * rs, u = t + kRound;
      b[e] = __float_as_uint(u);
      off = fmaxf(off, fabsf(t - (u - kRound)));
    }
    // the four floats' high bits cancel below bit 16
    out[k].codes = b[0] + 16u * b[1] + 256u * b[2] + 4096u * b[3];
    out[k].scale = sc;
    bool doubt = a7 < 0x1p-120f || fabsf(a7 - mid) <= fmaf(ferr, 0.15f, a7 * 0x1p-22f) || off >= near;
    if (max(top, far) >= 0x7f800000u || (top | far) == 0) {   // inf or NaN; all zero
      out[k].codes = 0x8888u;
      out[k].scale = (top | far) == 0 ? 0u : kNanScale;
      doubt = false;
    }
    unsure |= doubt;
  }
  return !__any_sync(0xffffffffu, unsure);
}

// The same for the raw row x of D dims in fp64: y = RoPE(RMSNorm(x)) with the row's (cos,
// sin) table tab (NULL: no rotation) and norm weights nw (NULL: none). fp64 runs at a
// thirtieth of fp32's rate here, so all rows this way would cost several times the memory
// traffic; a few rows in a thousand come here.
template <int NC>
__device__ __noinline__ void quantise_exact(const float* x, const float2* tab, int R,
                                            const float* nw, float eps, int D, int lane,
                                            Coded (&out)[NC]) {
  double inv = 1.0;
  if (nw) {
    double ss = 0.0;
    for (int d = lane; d < D; d += 32) ss += static_cast<double>(x[d]) * x[d];
    inv = 1.0 / sqrt(warp_sum_d(ss) / D + static_cast<double>(eps));
  }
  auto at = [&](int d) {
    const double v = x[d];
    return nw ? v * inv * nw[d] : v;
  };
  const int half = R / 2;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    double y[4], amax = 0.0;
    bool bad = false;
    for (int e = 0; e < 4; ++e) {
      const int d = 4 * (lane + 32 * k) + e;
      y[e] = 0.0;
      if (d < D) {
        if (tab && d < R) {
          const int i = d < half ? d : d - half;
          const double a = at(i), b = at(i + half), c = tab[i].x, s = tab[i].y;
          y[e] = d < half ? a * c - b * s : b * c + a * s;
        } else {
          y[e] = at(d);
        }
      }
      bad |= !isfinite(y[e]);
      amax = fmax(amax, fabs(y[e]));
    }
    for (int o = 1; o <= 4; o <<= 1) amax = fmax(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    bad = group_max_u(bad ? 1u : 0u) != 0;
    const uint32_t sc = bad ? kNanScale : (amax > 0.0 ? bf16_bits_of(amax / 7.0) : 0u);
    const double s = bf16_to_float(sc);
    uint32_t codes = 0;
    for (int e = 0; e < 4; ++e) {
      const int c = sc == 0 || bad ? 0 : max(-7, min(7, __double2int_rn(y[e] / s)));
      codes |= static_cast<uint32_t>(c + 8) << (4 * e);
    }
    out[k].codes = codes;
    out[k].scale = sc;
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
