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
// 9500 tokens of 32 + 2 x 8 heads of 128, norms: 2 passes a group and all of a token's 12 groups in
// one warp 65 us; 6 groups 71, 1 group 114; 4 passes (more registers, fewer warps) 74, 12 passes 118.
constexpr int kPasses = 2;
constexpr int kGroups = 12;
constexpr int64_t kManyWarps = 152 * 24;

// A head row of D values is held by LPH lanes (a power of two >= D / 8), 16 bytes each, so a warp
// takes 32 / LPH heads in a pass. It does `groups` groups of kPasses passes of one token; a
// group's loads are on their way before the group before it is worked on, the first before the
// token's place in the cache is known. The token's angles, times the norm's weights, stay in
// registers for all its queries, then all its keys. With half the rotary dims a multiple of 8 (kShuffle) the partner dims are another lane's whole granule.
template <class T, int LPH, int ROPE>
__global__ void __launch_bounds__(256, 3) append_paged_kernel(const AppendPagedJob j, unsigned warps,
                                                           int warps_per_token, int groups) {
  dependent_wait();
  dependents_may_launch();
  if (gated_off(j.skip)) return;
  const unsigned w = blockIdx.x * 8 + threadIdx.x / 32;
  if (w >= warps) return;
  constexpr int HPW = 32 / LPH;
  const int lane = threadIdx.x & 31;
  const int nq = j.q.p ? j.H : 0, heads = nq + 2 * j.Hkv;
  const int t = w / warps_per_token;
  int h0 = (w % warps_per_token) * groups * HPW * kPasses + lane / LPH;
  const int d0 = 8 * (lane % LPH);
  const bool in_row = d0 < j.D;
  const float inv_D = 1.0f / static_cast<float>(j.D);
  const Rows<T> q = rows_as<T>(j.q), k = rows_as<T>(j.k), v = rows_as<T>(j.v);
  auto row_of = [&](int h) -> const T* {
    return h < nq ? q.at(t, h) : (h < nq + j.Hkv ? k.at(t, h - nq) : v.at(t, h - nq - j.Hkv));
  };
  uint4 raw[kPasses], ahead[kPasses];
  auto load = [&](uint4 (&to)[kPasses], int h) {
#pragma unroll
    for (int u = 0; u < kPasses; ++u, h += HPW)
      to[u] = in_row && h < heads ? *reinterpret_cast<const uint4*>(row_of(h) + d0)
                                  : make_uint4(0, 0, 0, 0);
  };
  load(raw, h0);

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
  const int half = j.R / 2, hl = half / 8;   // hl: lanes of half the rotary dims
  const int from = (lane & ~(LPH - 1)) + ((lane % LPH) < hl ? lane % LPH + hl : lane % LPH - hl);
  // Factors of a rotated row's own and partner dims, with the norm's weights in them (the common
  // 1 / rms comes after): y = x own + x' other, of the kind (query or key) at hand.
  float own[8], other[8];
  int kind = -1;
  auto factors = [&](const float* nw) {
    const float2* row = j.table + static_cast<int64_t>(pos) * half;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      own[e] = 1.f;
      other[e] = 0.f;
    }
    if (!in_row) return;
    if (d0 < j.R) {
      if (ROPE == kShuffle) {
        const float4* r4 = reinterpret_cast<const float4*>(row + (d0 < half ? d0 : d0 - half));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 c = r4[e];
          own[2 * e] = c.x; own[2 * e + 1] = c.z;
          other[2 * e] = c.y; other[2 * e + 1] = c.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = d0 + e;
          if (d < j.R) {
            const float2 c = row[d < half ? d : d - half];
            own[e] = c.x;
            other[e] = c.y;
          }
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = d0 + e;
      if (d < half) other[e] = -other[e];    // the first half's partner enters with a minus
      if (nw) {
        own[e] *= nw[d];
        if (d < j.R) other[e] *= nw[d < half ? d + half : d - half];
      }
    }
  };
  if (page < 0 || page >= j.cache.pages) {
    if (lane == 0) report(j.status, ATTN_DEV_PAGE);
    return;
  }
  const int64_t slot = pos & ((1 << j.cache.page_shift) - 1);
  const int64_t head_stride = static_cast<int64_t>(j.D) << j.cache.page_shift;
  T* kc = static_cast<T*>(j.cache.k) + page * j.cache.page_stride + slot * j.D + d0;
  T* vc = static_cast<T*>(j.cache.v) + page * j.cache.page_stride + slot * j.D + d0;

#pragma unroll 1
  for (int g = 0; g < groups; ++g, h0 += HPW * kPasses) {
    if (g + 1 < groups) load(ahead, h0 + HPW * kPasses);
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      const int h = h0 + u * HPW;
      const bool is_q = h < nq, is_v = h >= nq + j.Hkv, live = in_row && h < heads;
      uint4 y = raw[u];
      if (ROPE != kPlain) {
        const float* nw = is_q ? j.q_norm_w : j.k_norm_w;
        if (!is_v && kind != is_q) {         // at most twice a warp and lane
          factors(nw);
          kind = is_q;
        }
        float x[8], p[8];
        unpack8<T>(raw[u], x);
        float inv = 1.f;
        if (j.q_norm_w || j.k_norm_w) {      // sums over the row's lanes (all lanes take part)
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (nw) inv = rsqrtf(fmaf(ss, inv_D, j.norm_eps));   // within 2 ulp of fp32
        }
        if (ROPE == kShuffle) {
          const uint4 o = make_uint4(__shfl_sync(0xffffffffu, raw[u].x, from & 31),
                                     __shfl_sync(0xffffffffu, raw[u].y, from & 31),
                                     __shfl_sync(0xffffffffu, raw[u].z, from & 31),
                                     __shfl_sync(0xffffffffu, raw[u].w, from & 31));
          unpack8<T>(o, p);
        } else {                             // partner dims one by one from the raw row
          const T* src = is_q ? q.at(t, h) : k.at(t, min(h - nq, j.Hkv - 1));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int d = d0 + e;
            p[e] = 0.f;
            if (live && !is_v && d < j.R) p[e] = static_cast<float>(src[d < half ? d + half : d - half]);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // past the rotary dims: no partner (its lane's value may be anything)
          const float r = fmaf(x[e], own[e], d0 + e < j.R ? p[e] * other[e] : 0.f);
          x[e] = r * inv;
        }
        if (!is_v) y = pack8<T>(x);
        __syncwarp();                        // in place: every lane has read its partners
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
#pragma unroll
    for (int u = 0; u < kPasses; ++u) raw[u] = ahead[u];
  }
}

template <class T, int LPH, int ROPE>
cudaError_t launch_rope(const AppendPagedJob& j, cudaStream_t stream) {
  const int heads = (j.q.p ? j.H : 0) + 2 * j.Hkv, per = 32 / LPH * kPasses;
  const int all = (heads + per - 1) / per;   // groups of a token
  // Few tokens: a warp for each group. Many: kGroups groups a warp, which share its search and angles.
  int groups = 1;
  if (static_cast<int64_t>(j.T) * all > kManyWarps) groups = all < kGroups ? all : kGroups;
  const int per_token = (all + groups - 1) / groups;
  const unsigned warps = static_cast<unsigned>(j.T) * per_token;
  return launch_dependent(append_paged_kernel<T, LPH, ROPE>, (warps + 7) / 8, 256, 0, stream, j,
                          warps, per_token, groups);
}

template <class T, int LPH>
cudaError_t launch_lph(const AppendPagedJob& j, cudaStream_t stream) {
  if (!j.table) return launch_rope<T, LPH, kPlain>(j, stream);
  return j.R % 16 == 0 ? launch_rope<T, LPH, kShuffle>(j, stream)
                       : launch_rope<T, LPH, kAnyDims>(j, stream);
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
