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

// A warp's rows: four lanes a group, two quads of dims each, 4 M lanes a row, so one to eight
// rows side by side. Lane a of group g holds quads a and a + 4 of the group's eight, in odd
// groups the other way round: eight lanes' 16-byte accesses then meet all banks, and the
// lanes of a group always touch 64 bytes in a row.
template <int M>
struct Lanes {
  static constexpr int kRows = 32 / (4 * M);              // rows of a warp
  int row, l, g, q0;                                      // l: lane of the row
  bool in;                                                // whether the lane has a row
  __device__ __forceinline__ explicit Lanes(int lane) {
    row = lane / (4 * M);
    in = row < kRows;
    l = lane - row * 4 * M;
    g = l >> 2;
    q0 = (l & 3) + 4 * (g & 1);
  }
  __device__ __forceinline__ int quad(int i) const { return i ? q0 ^ 4 : q0; }
  __device__ __forceinline__ int dim(int i) const { return 32 * g + 4 * quad(i); }
};

__device__ __forceinline__ uint32_t group_max_u(uint32_t v) {      // over 4 aligned lanes
  v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return max(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// Sum over a row's 4 M lanes.
template <int M>
__device__ __forceinline__ float row_sum(float v, int lane) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  if constexpr ((M & (M - 1)) == 0) {
#pragma unroll
    for (int o = 4; o < 4 * M; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  } else {
    const int base = lane - lane % (4 * M);
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < M; ++g) t += __shfl_sync(0xffffffffu, v, min(base + 4 * g, 31));
    return t;
  }
}

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// t in (-2^21, 2^21) to the nearest integer, ties to even, as the sum's low bits: the float
// 1.5 * 2^23 + 8 + t is rounded at its unit place. Its low four bits are then t's code + 8.
constexpr float kRound = 12582920.0f;

// Quantises a lane's two quads y, four lanes a group, each value off from the
// exact one by at most err and rel times the group's largest: the scale is bf16(max|y| / 7),
// the code rint(y / scale), ties to even. Returns whether a rounding was not further from its
// border than the error: the group has to be done again by quantise_exact. Both distances
// from a border, max|y| - 7 (middle of two scales) and y - code * scale, are exact in fp32, so
// of exact values only ties and some borders' nearest neighbours are in doubt. EXACT: y is
// exact, err and rel are not read. Every lane of the warp must call it. About six
// instructions a value.
template <bool EXACT>
__device__ __forceinline__ bool quantise_fast(const float (&y)[8], float err, float rel,
                                              uint32_t& codes, uint32_t& scale) {
  float big = 0.f;                           // a NaN stays one, and its bits are above inf's
#pragma unroll
  for (int e = 0; e < 8; ++e) asm("max.NaN.f32 %0, %0, %1;" : "+f"(big) : "f"(fabsf(y[e])));
  const uint32_t top = group_max_u(__float_as_uint(big));
  const uint32_t far = EXACT ? 0u : group_max_u(__float_as_uint(err));
  const float amax = __uint_as_float(top);
  const float ferr = EXACT ? 0.f : fmaf(amax, rel, __uint_as_float(far));
  // amax / 7 to two roundings lies between two scales (or on one); their middle decides
  const float a7 = amax * (1.0f / 7.0f);
  const uint32_t bits = __float_as_uint(a7);
  const float past = fmaf(-7.f, __uint_as_float((bits & 0xffff0000u) | 0x8000u), amax);
  scale = (bits >> 16) + (past > 0.f);
  const float s = bf16_to_float(scale), near = fmaf(0.5f, s, -ferr);
  float rs;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(s));
  uint32_t b[8];
  float off = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float u = fmaf(y[e], rs, kRound);
    b[e] = __float_as_uint(u);
    off = fmaxf(off, fabsf(fmaf(kRound - u, s, y[e])));
  }
  // four codes a sum: the floats' high bits cancel below bit 16
  const uint32_t lo = b[0] + 16u * b[1] + 256u * b[2] + 4096u * b[3];
  const uint32_t hi = b[4] + 16u * b[5] + 256u * b[6] + 4096u * b[7];
  codes = __byte_perm(lo, hi, 0x5410);
  const bool special = max(top, far) >= 0x7f800000u || (top | far) == 0;   // inf, NaN; zeros
  if (special) {
    codes = 0x88888888u;
    scale = (top | far) == 0 ? 0u : kNanScale;
  }
  return !special && (a7 < 0x1p-120f || fabsf(past) <= ferr || off >= near);
}

// Quad q of group g at 16 bits of codes, in the key part (part = 0) or the value part (1) of
// a record.
template <int M>
__device__ __forceinline__ int quad_at(int part, int g, int q) {
  return part ? 16 * M + 2 * (q * M + g) : 4 * ((q >> 1) * M + g) + 2 * (q & 1);
}

// A lane's codes (its quads' in the low and high half) and its group's scale into a record.
template <int M>
__device__ __forceinline__ void store_codes(uint8_t* rec, int part, uint32_t codes, uint32_t scale,
                                            const Lanes<M>& at) {
  *reinterpret_cast<uint16_t*>(rec + quad_at<M>(part, at.g, at.quad(0))) = static_cast<uint16_t>(codes);
  *reinterpret_cast<uint16_t*>(rec + quad_at<M>(part, at.g, at.quad(1))) =
      static_cast<uint16_t>(codes >> 16);
  if ((at.l & 3) == 0)
    *reinterpret_cast<uint16_t*>(rec + (32 + 2 * part) * M + 2 * at.g) = static_cast<uint16_t>(scale);
}

// 1 / rms of a row in fp64.
template <int = 0>
__device__ __noinline__ double exact_inv_rms(const float* x, float eps, int D, int lane) {
  double ss = 0.0;
#pragma unroll 1
  for (int d = lane; d < D; d += 32) ss = fma(static_cast<double>(x[d]), static_cast<double>(x[d]), ss);
  return rsqrt(warp_sum_d(ss) / D + static_cast<double>(eps));
}

// The doubtful groups of the raw row x (doubt: four bits a group, any set) again, in fp64,
// into part `part` of the record at rec: y = RoPE(RMSNorm(x)) with the row's (cos, sin)
// table tab (NULL: no rotation) and norm weights nw (NULL: none), a group at a time, one dim
// per lane. No quotient is formed: fp32 proposes the scale and the codes, and exact products
// with the borders next to them decide. At D = 128 one row in 2500 comes here, with a norm one
// in 300 (with D = 256 twice as many); kept short, since its instructions are not in the cache
// then: about 3 us a use, which 64 rows of one token still see.
template <int M>
__device__ __noinline__ void quantise_exact(const float* x, const float2* tab, int R,
                                            const float* nw, float eps, int lane, uint32_t doubt,
                                            uint8_t* rec, int part) {
  constexpr int D = 32 * M;
  const double inv = nw ? exact_inv_rms<>(x, eps, D, lane) : 1.0;
  const int half = R / 2;
#pragma unroll 1
  for (int g = 0; g < M; ++g) {
    if (!(doubt >> (4 * g) & 15u)) continue;
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
    // the largest: of |y| as 64 bits, the upper half first
    const double ay = fabs(y);
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(__double2hiint(ay)));
    const uint32_t lo = __reduce_max_sync(
        0xffffffffu, __double2hiint(ay) == static_cast<int>(hi) ? static_cast<uint32_t>(__double2loint(ay)) : 0u);
    const double amax = __hiloint2double(static_cast<int>(hi), static_cast<int>(lo));
    // a seventh of it lies between two scales (or on one), whose middle decides
    const uint32_t bits = __float_as_uint(static_cast<float>(amax) * (1.0f / 7.0f));
    uint32_t sc = bits >> 16;
    const double past = fma(-7.0, static_cast<double>(__uint_as_float((bits & 0xffff0000u) | 0x8000u)), amax);
    if (past > 0.0 || (past == 0.0 && (sc & 1u))) ++sc;
    // the code; tiny scales are lifted out of the subnormals for the proposal
    const double s = bf16_to_float(sc);
    const float lift = sc < 0x0800u ? 0x1p100f : 1.0f;
    float rs;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(bf16_to_float(sc) * lift));
    int c = sc ? __float2int_rn(static_cast<float>(y * lift) * rs) : 0;
    const double rest = fma(static_cast<double>(-c), s, y), border = 0.5 * s;
    if (rest > border || (rest == border && (c & 1)))
      ++c;
    else if (rest < -border || (rest == -border && (c & 1)))
      --c;
    c = sc ? max(-7, min(7, c)) : 0;
    // four lanes' codes make a quad
    uint32_t codes = static_cast<uint32_t>(c + 8) << (4 * (lane & 3));
    codes |= __shfl_xor_sync(0xffffffffu, codes, 1);
    codes |= __shfl_xor_sync(0xffffffffu, codes, 2);
    if ((lane & 3) == 0)
      *reinterpret_cast<uint16_t*>(rec + quad_at<M>(part, g, lane >> 2)) = static_cast<uint16_t>(codes);
    if (lane == 0)
      *reinterpret_cast<uint16_t*>(rec + (32 + 2 * part) * M + 2 * g) = static_cast<uint16_t>(sc);
  }
}

#endif  // __CUDACC__

}  // namespace q4
}  // namespace gqa
