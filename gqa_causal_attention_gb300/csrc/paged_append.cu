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
// 9500 tokens of 32 + 2 x 8 heads of 128, norms, blocks of 8 warps: 2 passes a group and all of a
// token's 12 groups in one warp 51.3 us; 6 groups 54.0; 1 pass 57.5, 4 passes 54.1; four blocks an SM
// (64 registers) 55.1; two groups ahead 50.9. Blocks of 4 warps, which end less unevenly: 49.8.
constexpr int kPasses = 2;
constexpr int kGroups = 12;
constexpr int kWarps = 4, kBlocks = 6;       // a block's warps, blocks an SM
constexpr int64_t kManyWarps = 152 * kWarps * kBlocks;

// A head row of D values is held by LPH lanes (a power of two >= D / 8), 16 bytes each, so a warp
// takes 32 / LPH heads in a pass. It does `groups` groups of kPasses passes of one token, each of
// queries, keys or values alone, so that what differs between them is decided once a group (with
// heads of all kinds in one group, chosen lane by lane, and unpaired arithmetic 58.9 us: 213
// instructions for 8 values). A group's loads are on their way before the group before it is worked
// on, the first before the token's place in the cache is known. The token's angles, times the
// norm's weights, stay in registers for all its queries, then all its keys. With half the rotary
// dims a multiple of 8 (kShuffle) the partner dims are another lane's whole granule.
template <class T, int LPH, int ROPE>
__global__ void __launch_bounds__(32 * kWarps, kBlocks)
    append_paged_kernel(const AppendPagedJob j, unsigned warps, int warps_per_token, int groups) {
  dependent_wait();
  dependents_may_launch();
  if (gated_off(j.skip)) return;
  const unsigned w = blockIdx.x * kWarps + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (w >= warps) {
    // A warp of its own looks every sequence's bounds over: one may have no row to find it bad.
    if (w == warps && j.cu)
      for (int b = lane; b < j.B; b += 32)
        if (seq_rows(j.cu, b, j.T).n < 0) report(j.status, ATTN_DEV_LENGTH);
    return;
  }
  constexpr int HPW = 32 / LPH;
  constexpr int kPer = HPW * kPasses;        // heads of a group, all queries, keys or values
  const int nq = j.q.p ? j.H : 0;
  const int gq = (nq + kPer - 1) / kPer, gk = (j.Hkv + kPer - 1) / kPer;
  const int t = w / warps_per_token;
  int g = (w % warps_per_token) * groups;
  const int gend = min(g + groups, gq + 2 * gk);
  const int d0 = 8 * (lane % LPH);
  const bool in_row = d0 < j.D;
  const float inv_D = 1.0f / static_cast<float>(j.D);
  // Group g's first head on this lane, its kind's number of heads and its rows.
  auto group = [&](int g, int& h, int& n) -> Rows<T> {
    const int kind = g < gq ? 0 : (g < gq + gk ? 1 : 2);
    const RowsArg& r = kind == 0 ? j.q : (kind == 1 ? j.k : j.v);
    h = (kind == 0 ? g : (kind == 1 ? g - gq : g - gq - gk)) * kPer + lane / LPH;
    n = in_row ? (kind == 0 ? nq : j.Hkv) : 0;
    return rows_as<T>(r);
  };
  uint4 raw[kPasses], ahead[kPasses];
  auto load = [&](uint4 (&to)[kPasses], int g) {
    int h, n;
    const Rows<T> r = group(g, h, n);
    const T* p = r.at(t, h) + d0;
#pragma unroll
    for (int u = 0; u < kPasses; ++u, p += HPW * r.head)
      to[u] = h + u * HPW < n ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
  };
  load(raw, g);

  // The token's sequence, position and page.
  int b = t, i = 0, n = 1;
  if (j.cu) {
    b = warp_find_last(j.B, t, [&](int x) { return static_cast<int64_t>(j.cu[x]); });
    if (b < 0) return;                       // before the first sequence
    const SeqRows s = seq_rows(j.cu, b, j.T);
    // Bounds that decrease can name a sequence that begins behind the token.
    if (s.n < 0 || t < s.first) {
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
  const bool turned = d0 < j.R;              // past the rotary dims: no partner
  const int from = (lane & ~(LPH - 1)) +
                   (!turned ? lane % LPH : ((lane % LPH) < hl ? lane % LPH + hl : lane % LPH - hl));
  const uint32_t partner = turned ? 0xffffffffu : 0u;
  // Factors of a rotated row's own and partner dims, with the norm's weights in them (the common
  // 1 / rms comes after): y = x own + x' other, of the kind (query or key) at hand. In pairs.
  uint64_t own2[4], other2[4];
  int kind_at = -1;
  auto factors = [&](const float* nw) {
    float own[8], other[8];
    const float2* row = j.table + static_cast<int64_t>(pos) * half;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      own[e] = 1.f;
      other[e] = 0.f;
    }
    if (in_row && turned) {
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
      if (nw && in_row) {
        own[e] *= nw[d];
        if (d < j.R) other[e] *= nw[d < half ? d + half : d - half];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      own2[e] = tc::pack2(own[2 * e], own[2 * e + 1]);
      other2[e] = tc::pack2(other[2 * e], other[2 * e + 1]);
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
  for (; g < gend; ++g) {
    if (g + 1 < gend) load(ahead, g + 1);
    int h, n;
    const Rows<T> r = group(g, h, n);
    const bool is_q = g < gq, is_v = g >= gq + gk;
    if (ROPE != kPlain && !is_v) {
      const float* nw = is_q ? j.q_norm_w : j.k_norm_w;
      if (kind_at != is_q) {                 // at most twice a warp
        factors(nw);
        kind_at = is_q;
      }
#pragma unroll
      for (int u = 0; u < kPasses; ++u) {
        uint64_t x[4], p[4];
        unpack8<T>(raw[u], x);
        float inv = 1.f;
        if (nw) {                            // sums over the row's lanes (all lanes take part)
          uint64_t s2 = tc::mul2(x[0], x[0]);
#pragma unroll
          for (int e = 1; e < 4; ++e) s2 = tc::fma2(x[e], x[e], s2);
          float ss, hi;
          tc::unpack2(s2, ss, hi);
          ss += hi;
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          inv = rsqrtf(fmaf(ss, inv_D, j.norm_eps));           // within 2 ulp of fp32
        }
        if (ROPE == kShuffle) {              // (a lane without a partner takes zeros)
          const uint4 o = make_uint4(__shfl_sync(0xffffffffu, raw[u].x, from) & partner,
                                     __shfl_sync(0xffffffffu, raw[u].y, from) & partner,
                                     __shfl_sync(0xffffffffu, raw[u].z, from) & partner,
                                     __shfl_sync(0xffffffffu, raw[u].w, from) & partner);
          unpack8<T>(o, p);
        } else {                             // partner dims one by one from the raw row
          const T* src = r.at(t, h + u * HPW);
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int d = d0 + e;
            f[e] = h + u * HPW < n && d < j.R
                       ? static_cast<float>(src[d < half ? d + half : d - half])
                       : 0.f;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = tc::pack2(f[2 * e], f[2 * e + 1]);
        }
        const uint64_t inv2 = tc::pack2(inv, inv);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = tc::mul2(tc::fma2(x[e], own2[e], tc::mul2(p[e], other2[e])), inv2);
        raw[u] = pack8<T>(x);
      }
      if (ROPE == kAnyDims) __syncwarp();    // in place: every lane has read its partners
    }
    if (is_q) {
      const Rows<T> out = rows_as<T>(j.q_out);
      T* p = out.at(t, h) + d0;
#pragma unroll
      for (int u = 0; u < kPasses; ++u, p += HPW * out.head)
        if (h + u * HPW < n) *reinterpret_cast<uint4*>(p) = raw[u];
    } else {
      T* p = (is_v ? vc : kc) + h * head_stride;
#pragma unroll
      for (int u = 0; u < kPasses; ++u, p += HPW * head_stride)
        if (h + u * HPW < n) *reinterpret_cast<uint4*>(p) = raw[u];
      if (!is_v && j.k_out.p) {
        const Rows<T> out = rows_as<T>(j.k_out);
        T* o = out.at(t, h) + d0;
#pragma unroll
        for (int u = 0; u < kPasses; ++u, o += HPW * out.head)
          if (h + u * HPW < n) *reinterpret_cast<uint4*>(o) = raw[u];
      }
    }
#pragma unroll
    for (int u = 0; u < kPasses; ++u) raw[u] = ahead[u];
  }
}

template <class T, int LPH, int ROPE>
cudaError_t launch_rope(const AppendPagedJob& j, cudaStream_t stream) {
  const int per = 32 / LPH * kPasses;        // groups of a token, as the kernel counts them:
  const int all = ((j.q.p ? j.H : 0) + per - 1) / per + 2 * ((j.Hkv + per - 1) / per);
  // Few tokens: a warp for each group. Many: kGroups groups a warp, which share its search and angles.
  int groups = 1;
  if (static_cast<int64_t>(j.T) * all > kManyWarps) groups = all < kGroups ? all : kGroups;
  const int per_token = (all + groups - 1) / groups;
  const unsigned warps = static_cast<unsigned>(j.T) * per_token;
  const unsigned all_warps = warps + (j.cu ? 1 : 0);   // and the one for the bounds
  return launch_dependent(append_paged_kernel<T, LPH, ROPE>, (all_warps + kWarps - 1) / kWarps,
                          32 * kWarps, 0, stream, j, warps, per_token, groups);
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
