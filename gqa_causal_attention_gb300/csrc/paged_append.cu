// Append to a paged cache: RMSNorm and RoPE of packed queries and keys ("mojolearn.transformer",
// qk_norm before RoPE; "Core Layers -- Deep Reference", "RMSNorm", "RoPE"), keys and values to
// their pages.
//
//   y = x / sqrt(mean(x^2) + eps) * w            (with norm weights)
//   y[i], y[i + R/2] = y[i] c_i - y[i + R/2] s_i,  y[i + R/2] c_i + y[i] s_i   (i < R/2)
//
// in fp32 from the 16-bit values, rounded once to the call's type (half a step: what the
// type can hold). Every value is read and written once: memory bound for prompts, bound by
// its chain of loads (sequence -> start -> page -> store) for single tokens.
#include "paged.cuh"

namespace gqa {

namespace {

enum { kPlain = 0, kShuffle = 1, kAnyDims = 2 };   // how the rotary partner is reached
constexpr int kPasses = 4;

// A head row of D values is held by LPH lanes (a power of two >= D / 8), 16 bytes each, so a warp
// takes 32 / LPH heads in a pass and kPasses passes of one token: their loads are all on
// their way before the token's place in the cache is known. With half the rotary dims a
// multiple of 8 (kShuffle) the partner dims are another lane's whole granule.
template <class T, int LPH, int ROPE>
__global__ void __launch_bounds__(256) append_paged_kernel(const AppendPagedJob j, unsigned warps) {
  dependent_wait();
  dependents_may_launch();
  if (gated_off(j.skip)) return;
  const unsigned w = blockIdx.x * 8 + threadIdx.x / 32;
  if (w >= warps) return;
  constexpr int HPW = 32 / LPH;
  const int lane = threadIdx.x & 31;
  const int nq = j.q.p ? j.H : 0, heads = nq + 2 * j.Hkv;
  const int per_token = (heads + HPW * kPasses - 1) / (HPW * kPasses);
  const int t = w / per_token, h0 = (w % per_token) * HPW * kPasses + lane / LPH;
  const int d0 = 8 * (lane % LPH);
  const bool in_row = d0 < j.D;
  const Rows<T> q = rows_as<T>(j.q), k = rows_as<T>(j.k), v = rows_as<T>(j.v);

  uint4 raw[kPasses];
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int h = h0 + u * HPW;
    raw[u] = make_uint4(0, 0, 0, 0);
    if (!in_row || h >= heads) continue;
    const T* src = h < nq ? q.at(t, h) : (h < nq + j.Hkv ? k.at(t, h - nq) : v.at(t, h - nq - j.Hkv));
    raw[u] = *reinterpret_cast<const uint4*>(src + d0);
  }

  // The token's sequence, position and page.
  int b = t, i = 0, n = 1;
  if (j.cu) {
    b = warp_find_last(j.B, t, [&](int x) { return static_cast<int64_t>(j.cu[x]); });
    if (b < 0) return;                       // before the first sequence
    const SeqRows s = seq_rows(j.cu, b, j.T);
    if (s.n < 0) {
      if (lane == 0) report(j.status, ATTN_DEV_LENGTH);
      return;
    }
    i = t - s.first;
    n = s.n;
    if (i >= n) return;                      // behind the last sequence
  }
  const int64_t first = j.start[b];
  if (first < 0 || first + n - 1 > j.max_pos) {
    if (lane == 0) report(j.status, ATTN_DEV_POSITION);
    return;
  }
  const int pos = static_cast<int>(first) + i;
  const int page = j.block_table[static_cast<int64_t>(b) * j.width + (pos >> j.cache.page_shift)];
  if (page < 0 || page >= j.cache.pages) {
    if (lane == 0) report(j.status, ATTN_DEV_PAGE);
    return;
  }
  const int64_t slot = pos & ((1 << j.cache.page_shift) - 1);
  const int64_t head_stride = static_cast<int64_t>(j.D) << j.cache.page_shift;
  T* kc = static_cast<T*>(j.cache.k) + page * j.cache.page_stride + slot * j.D + d0;
  T* vc = static_cast<T*>(j.cache.v) + page * j.cache.page_stride + slot * j.D + d0;

  const int half = j.R / 2;
  float cs[8], sn[8];
  if (ROPE != kPlain) {
    const float2* row = j.table + static_cast<int64_t>(pos) * half;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cs[e] = 1.f;
      sn[e] = 0.f;
    }
    if (in_row && d0 < j.R) {
      if (ROPE == kShuffle) {
        const float4* r4 = reinterpret_cast<const float4*>(row + (d0 < half ? d0 : d0 - half));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 c = r4[e];
          cs[2 * e] = c.x; cs[2 * e + 1] = c.z;
          sn[2 * e] = c.y; sn[2 * e + 1] = c.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = d0 + e;
          if (d < j.R) {
            const float2 c = row[d < half ? d : d - half];
            cs[e] = c.x;
            sn[e] = c.y;
          }
        }
      }
      // y = x c + partner s: the first half's partner enters with a minus
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (d0 + e < half) sn[e] = -sn[e];
    }
  }

#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int h = h0 + u * HPW;
    const bool is_q = h < nq, is_v = h >= nq + j.Hkv, live = in_row && h < heads;
    uint4 y = raw[u];
    if (ROPE != kPlain) {
      float x[8], p[8];
      unpack8<T>(raw[u], x);
      const float* nw = is_v ? nullptr : (is_q ? j.q_norm_w : j.k_norm_w);
      float inv = 1.f;
      if (j.q_norm_w || j.k_norm_w) {        // sums over the row's lanes (all lanes take part)
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        inv = 1.0f / sqrtf(ss / static_cast<float>(j.D) + j.norm_eps);
      }
      if (ROPE == kAnyDims) {                // partner dims one by one from the raw row
        const T* src = is_q ? q.at(t, h) : k.at(t, min(h - nq, j.Hkv - 1));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = d0 + e;
          p[e] = 0.f;
          if (live && !is_v && d < j.R) {
            const int pd = d < half ? d + half : d - half;
            p[e] = static_cast<float>(src[pd]);
            if (nw) p[e] *= inv * nw[pd];
          }
        }
      }
      if (nw && live) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv * nw[d0 + e];
      }
      if (ROPE == kShuffle) {
        const int hl = half / 8;             // lanes of half the rotary dims
        const int from = (lane & ~(LPH - 1)) + ((lane % LPH) < hl ? (lane % LPH) + hl
                                                                  : (lane % LPH) - hl);
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = __shfl_sync(0xffffffffu, x[e], from & 31);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = d0 + e < j.R ? fmaf(x[e], cs[e], p[e] * sn[e]) : x[e];
      if (!is_v) y = pack8<T>(x);
      __syncwarp();                          // in place: every lane has read its partners
    }
    if (!live) continue;
    if (is_q) {
      *reinterpret_cast<uint4*>(rows_as<T>(j.q_out).at(t, h) + d0) = y;
    } else if (!is_v) {
      const int hk = h - nq;
      *reinterpret_cast<uint4*>(kc + hk * head_stride) = y;
      if (j.k_out.p) *reinterpret_cast<uint4*>(rows_as<T>(j.k_out).at(t, hk) + d0) = y;
    } else {
      *reinterpret_cast<uint4*>(vc + (h - nq - j.Hkv) * head_stride) = y;
    }
  }
}

template <class T, int LPH>
cudaError_t launch_lph(const AppendPagedJob& j, cudaStream_t stream) {
  const int heads = (j.q.p ? j.H : 0) + 2 * j.Hkv;
  const int per_warp = 32 / LPH * kPasses;
  const unsigned warps = static_cast<unsigned>(j.T) * ((heads + per_warp - 1) / per_warp);
  const unsigned grid = (warps + 7) / 8;
  const int rope = !j.table ? kPlain : (j.R % 16 == 0 ? kShuffle : kAnyDims);
  switch (rope) {
    case kPlain:
      return launch_dependent(append_paged_kernel<T, LPH, kPlain>, grid, 256, 0, stream, j, warps);
    case kShuffle:
      return launch_dependent(append_paged_kernel<T, LPH, kShuffle>, grid, 256, 0, stream, j, warps);
    default:
      return launch_dependent(append_paged_kernel<T, LPH, kAnyDims>, grid, 256, 0, stream, j, warps);
  }
}

template <class T>
cudaError_t launch_type(const AppendPagedJob& j, cudaStream_t stream) {
  if (j.D <= 32) return launch_lph<T, 4>(j, stream);
  if (j.D <= 64) return launch_lph<T, 8>(j, stream);
  return launch_lph<T, 16>(j, stream);
}

}  // namespace

cudaError_t launch_append_paged(const AppendPagedJob& j, cudaStream_t stream) {
  return j.bf16 ? launch_type<__nv_bfloat16>(j, stream) : launch_type<__half>(j, stream);
}

}  // namespace gqa
