// Rows of keys and values on their way into 4-bit records: RMSNorm, RoPE and quantisation of
// a warp's rows, shared by the append and the decode step.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "kv_q4.cuh"

namespace gqa {

// How a row's rotation is read: not at all, in quads (half the rotary dims a multiple of
// four: a quad lies within one half, and so do its partners), in quads with every dim
// rotary, or dim by dim.
enum { kNoRope = 0, kRopeQuads = 1, kRopeDims = 2, kRopeAll = 3 };
inline int rope_kind(int R, int D) { return R % 8 ? kRopeDims : (R == D ? kRopeAll : kRopeQuads); }

__device__ __forceinline__ void load4(const float* p, float* r) {
  const float4 t = *reinterpret_cast<const float4*>(p);
  r[0] = t.x; r[1] = t.y; r[2] = t.z; r[3] = t.w;
}

// A lane's quads of a row. (Lanes without a row of their own have dims of a row too: they
// read along, and what they make of it is dropped.)
template <int M>
__device__ __forceinline__ void load_row(const float* x, const q4::Lanes<M>& at, float (&y)[8]) {
  load4(x + at.dim(0), y);
  load4(x + at.dim(1), y + 4);
}
template <int M>
__device__ __forceinline__ void store_row(float* x, const q4::Lanes<M>& at, const float (&y)[8]) {
  *reinterpret_cast<float4*>(x + at.dim(0)) = make_float4(y[0], y[1], y[2], y[3]);
  *reinterpret_cast<float4*>(x + at.dim(1)) = make_float4(y[4], y[5], y[6], y[7]);
}

// The part of rotate_row's error that goes with the values themselves: with a norm the
// common factor's 9 roundings (at most 12 in the sum of squares, one each in the quotient and
// the sum with eps, halved by the root; one each in the root and its reciprocal), without one
// what quantise_fast rounds in its own bounds.
__device__ __forceinline__ float row_error(const float* nw) { return nw ? 0x1.28p-21f : 0x1p-26f; }

// A lane's quads of the raw row x through RMSNorm (nw) and RoPE (tab: the row's angles;
// x and tab in any memory), in fp32, and a bound of their error (with row_error's). Every
// lane of the warp calls it.
template <int M, int ROPE>
__device__ __forceinline__ float rotate_row(const float* x, const float2* tab, int R,
                                            const float* nw, float eps, const q4::Lanes<M>& at,
                                            int lane, float (&y)[8]) {
  const int half = ROPE == kRopeAll ? 16 * M : R / 2;
  float c[8], s[8], b[8], w[8];
  if (ROPE != kRopeAll) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = w[e] = 1.f;
      s[e] = b[e] = 0.f;
    }
  }
  // y = a c + b s, b the rotary partner
#pragma unroll
  for (int q = 0; q < 8; q += 4) {
    const int d0 = at.dim(q / 4);
    if (ROPE != kRopeAll && d0 >= R) continue;
    if (ROPE != kRopeDims) {
      const bool low = d0 < half;
      const int i = low ? d0 : d0 - half, p = low ? d0 + half : i;
      const float sign = low ? -1.f : 1.f;
      const float4* ang = reinterpret_cast<const float4*>(tab + i);
      const float4 a0 = ang[0], a1 = ang[1];
      load4(x + p, b + q);
      c[q] = a0.x; c[q + 1] = a0.z; c[q + 2] = a1.x; c[q + 3] = a1.z;
      s[q] = a0.y * sign; s[q + 1] = a0.w * sign; s[q + 2] = a1.y * sign; s[q + 3] = a1.w * sign;
      if (nw) load4(nw + p, w + q);
    } else {
#pragma unroll
      for (int e = q; e < q + 4; ++e) {
        const int d = d0 + e - q;
        if (d >= R) continue;
        const bool low = d < half;
        const int i = low ? d : d - half, p = low ? d + half : i;
        const float2 a = tab[i];
        b[e] = x[p];
        c[e] = a.x;
        s[e] = low ? -a.y : a.y;
        if (nw) w[e] = nw[p];
      }
    }
  }
  load_row<M>(x, at, y);
  // Errors in roundings of 2^-24, |(a, b)| <= sqrt(2) of the larger: 1 of b s and 1 of y, 2.42 of
  // the larger. With a norm also two each in a and b, 5.25 in all, and the common factor's.
  float unit = 0x1.4p-23f;                   // 2.5
  if (nw) {
    float ss[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) ss[e] = fmaf(y[2 * e], y[2 * e], y[2 * e + 1] * y[2 * e + 1]);
    const float sum = q4::row_sum<M>((ss[0] + ss[1]) + (ss[2] + ss[3]), lane);
    const float inv = 1.0f / sqrtf(sum / static_cast<float>(32 * M) + eps);
    unit = 0x1.6p-22f;                       // 5.5
    float wo[8];
    load_row<M>(nw, at, wo);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = y[e] * inv * wo[e];
      b[e] = b[e] * inv * w[e];
    }
  }
  float mag = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    mag = fmaxf(mag, fmaxf(fabsf(y[e]), fabsf(b[e])));
    y[e] = fmaf(y[e], c[e], b[e] * s[e]);
  }
  return mag * unit;
}

// A warp's rows, side by side: each lane's own row x, v (raw) and angles tab in any memory;
// its record goes to rec (any memory) unless that is nullptr, the rotated key to k_out
// unless that is. Every lane of the warp calls it; those without a row pass on = false and
// any row's pointers. Groups whose rounding fp32 cannot settle come back as their lanes:
// (key, value).
template <int M, int ROPE>
__device__ __forceinline__ uint2 append_rows(const AppendQ4Job& j, const float* x, const float* v,
                                             const float2* tab, uint8_t* rec, float* k_out,
                                             const q4::Lanes<M>& at, int lane, bool on) {
  using namespace q4;
  float y[8];
  uint32_t codes, scale;
  bool doubt;
  uint2 r;
  load_row<M>(v, at, y);
  doubt = quantise_fast<true>(y, 0.f, 0.f, codes, scale);
  if (on && rec) {
    store_codes<M>(rec, 1, codes, scale, at);
    constexpr int pad = (record_bytes(M) - 36 * M) / 4;   // zero padding
    if (pad > 0 && at.l < pad) *reinterpret_cast<uint32_t*>(rec + 36 * M + 4 * at.l) = 0;
  }
  r.y = __ballot_sync(0xffffffffu, doubt && on && rec);
  if (ROPE != kNoRope) {
    const float err = rotate_row<M, ROPE>(x, tab, j.R, j.norm_w, j.norm_eps, at, lane, y);
    doubt = quantise_fast<false>(y, err, row_error(j.norm_w), codes, scale);
  } else {
    load_row<M>(x, at, y);
    doubt = quantise_fast<true>(y, 0.f, 0.f, codes, scale);
  }
  if (on && rec) store_codes<M>(rec, 0, codes, scale, at);
  r.x = __ballot_sync(0xffffffffu, doubt && on && rec);   // also: every lane has read its partners
  if (on && k_out) store_row<M>(k_out, at, y);
  return r;
}

}  // namespace gqa
