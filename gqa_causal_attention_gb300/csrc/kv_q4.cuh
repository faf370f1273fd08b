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

// Four neighbouring dims quantised: their codes in the low 16 bits, their group's scale (the
// same on the group's 8 lanes) in the high ones.

// t in (-2^21, 2^21) to the nearest integer, ties to even, as the sum's low bits: the float
// 1.5 * 2^23 + 8 + t is rounded at its unit place. Its low four bits are then t's code + 8.
constexpr float kRound = 12582920.0f;

// Quantises a row held as quads y[k] (dims 4 (lane + 32 k) .. + 3; zeros where there are
// none), each off from the exact values by at most err[k]; a group is 8 aligned lanes. The
// scale is bf16(max|y| / 7), the code rint(y / scale), ties to even. doubt[k] gets the lanes
// (warp-uniform) whose roundings were not further from their borders than the error: their
// groups have to be done again by quantise_exact. EXACT: y is the row itself, err is not
// read. Every lane of the warp must call it. About six instructions a value.
template <int NC, bool EXACT>
__device__ __forceinline__ void quantise_fast(const float (&y)[NC][4], const float (&err)[NC],
                                              uint32_t (&out)[NC], uint32_t (&doubt)[NC]) {
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
    out[k] = ((b[0] + 16u * b[1] + 256u * b[2] + 4096u * b[3]) & 0xffffu) | sc << 16;
    bool unsure = a7 < 0x1p-120f || fabsf(a7 - mid) <= fmaf(ferr, 0.15f, a7 * 0x1p-22f) || off >= near;
    if (max(top, far) >= 0x7f800000u || (top | far) == 0) {   // inf or NaN; all zero
      out[k] = 0x8888u | ((top | far) == 0 ? 0u : kNanScale << 16);
      unsure = false;
    }
    doubt[k] = __ballot_sync(0xffffffffu, unsure);
  }
}

// Quad e of group g into the key part (part = 0) or value part (1) of the record at rec.
template <int M>
__device__ __forceinline__ void store_quad(uint8_t* rec, int part, uint32_t q, int g, int e) {
  const int at = part ? 16 * M + 2 * (e * M + g) : 4 * ((e >> 1) * M + g) + 2 * (e & 1);
  *reinterpret_cast<uint16_t*>(rec + at) = static_cast<uint16_t>(q);
  if (e == 0)
    *reinterpret_cast<uint16_t*>(rec + (32 + 2 * part) * M + 2 * g) = static_cast<uint16_t>(q >> 16);
}

// A lane's quads of a row.
template <int M, int NC>
__device__ __forceinline__ void store_part(uint8_t* rec, int part, const uint32_t (&q)[NC], int lane) {
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int ch = lane + 32 * k;
    if (ch < 8 * M) store_quad<M>(rec, part, q[k], ch >> 3, ch & 7);
  }
  if (part == 1) {                                      // zero padding
    constexpr int pad = (record_bytes(M) - 36 * M) / 2;
    if (pad > 0 && lane < pad) *reinterpret_cast<uint16_t*>(rec + 36 * M + 2 * lane) = 0;
  }
}

// 1 / rms of a row in fp64.
template <int = 0>
__device__ __noinline__ double exact_inv_rms(const float* x, float eps, int D, int lane) {
  double ss = 0.0;
#pragma unroll 1
  for (int d = lane; d < D; d += 32) ss = fma(static_cast<double>(x[d]), static_cast<double>(x[d]), ss);
  return 1.0 / sqrt(warp_sum_d(ss) / D + static_cast<double>(eps));
}

// The doubtful groups (doubt: quantise_fast's lanes, of quads 0 .. 31 and 32 .. 63) of the raw
// row x again, in fp64, into part `part` of the record at rec: y = RoPE(RMSNorm(x)) with the
// row's (cos, sin) table tab (NULL: no rotation) and norm weights nw (NULL: none), a group at
// a time, one dim per lane. No quotient is formed: fp32 proposes the scale and the codes, and
// exact products with the borders next to them decide. A few rows in a thousand come here
// (with a norm about one in a hundred); kept short, since its instructions are not in the
// cache then (unrolled over a row, the first use on an SM took 3 us).
template <int M>
__device__ __noinline__ void quantise_exact(const float* x, const float2* tab, int R,
                                            const float* nw, float eps, int lane, uint2 doubt,
                                            uint8_t* rec, int part) {
  constexpr int D = 32 * M;
  const double inv = nw ? exact_inv_rms<>(x, eps, D, lane) : 1.0;
  const int half = R / 2;
#pragma unroll 1
  for (int g = 0; g < M; ++g) {
    if (!((g < 4 ? doubt.x : doubt.y) >> (8 * (g & 3)) & 0xffu)) continue;
    const int d = 32 * g + lane;
    double y = x[d];
    if (nw) y = y * inv * nw[d];
    if (tab && d < R) {
      const int i = d < half ? d : d - half, p = d < half ? d + half : i;
      const float2 t = tab[i];
      double b = x[p];
      if (nw) b = b * inv * nw[p];
      y = fma(y, static_cast<double>(t.x), b * (d < half ? -t.y : t.y));
    }
    double amax = fabs(y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmax(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // the scale's two borders, half a unit from the proposed one
    const uint32_t bits = __float_as_uint(static_cast<float>(amax) * (1.0f / 7.0f));
    uint32_t sc = (bits + 0x7fffu + ((bits >> 16) & 1u)) >> 16;
    const double above = 7.0 * __uint_as_float((sc << 16) | 0x8000u);
    const double below = sc ? 7.0 * __uint_as_float(((sc - 1u) << 16) | 0x8000u) : -1.0;
    if (amax > above || (amax == above && (sc & 1u)))
      ++sc;
    else if (amax < below || (amax == below && (sc & 1u)))
      --sc;
    // the code; tiny scales are lifted out of the subnormals for the proposal
    const double s = bf16_to_float(sc), lift = sc < 0x0800u ? 0x1p100 : 1.0;
    int c = sc ? __float2int_rn(static_cast<float>(y * lift) / static_cast<float>(s * lift)) : 0;
    const double rest = fma(static_cast<double>(-c), s, y), border = 0.5 * s;
    if (rest > border || (rest == border && (c & 1)))
      ++c;
    else if (rest < -border || (rest == -border && (c & 1)))
      --c;
    c = sc ? max(-7, min(7, c)) : 0;
    // back to quads: lane l of the group's eight takes dims 4 (l % 8) .. + 3
    uint32_t codes = static_cast<uint32_t>(c + 8) << (4 * (lane & 3));
    codes |= __shfl_xor_sync(0xffffffffu, codes, 1);
    codes |= __shfl_xor_sync(0xffffffffu, codes, 2);
    codes = __shfl_sync(0xffffffffu, codes, 4 * (lane & 7));
    if (lane >> 3 == (g & 3)) store_quad<M>(rec, part, codes | sc << 16, g, lane & 7);
  }
}

#endif  // __CUDACC__

}  // namespace q4
}  // namespace gqa
