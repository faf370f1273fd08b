// Single-token attention over a cache held in 4 bits (record format: kv_q4.cuh),
// split over the key axis.
//
// Same operation as decode.cu ("mojolearn.transformer", TransformerBlock.step), with
//   key = ck * sk,  value = cv * sv     (codes c in [-7, 7], one scale per 32 dims)
//   s[h, n] = scale * sum_g sk[n, g] * (sum over the dims of group g of q * ck)
//   out[h, d] = sum_n (p[h, n] sv[n, g(d)]) cv[n, d] / sum_n p[h, n],  p = 2^(s log2(e) - ref)
//
// Why tensor cores: a record is 144 bytes at D = 128, an eighth of fp32's, but the
// products per key are as many. With 8 query heads that is 14 multiply-adds per byte
// read, twice what the CUDA cores could keep up with; unpacking comes on top. The
// codes are small integers, exact in fp16, so m16n8k16 products of fp16 pairs are
// exact, and q and p, split into a high and a low fp16 part (22 bits), keep fp32's
// accuracy. The 16 rows of the A operand are the 8 heads' high and low parts. (The
// operand is unpacked in registers and used once: staging it in shared memory for
// tcgen05 would cost more shared-memory traffic than the copy of the codes itself.)
//
// A pair of codes becomes a packed fp16 pair in two instructions: a nibble u = c + 8
// masked out of its 16-bit half and put under the exponent of 1024 is 1024 + u, or
// 1024 + 16 u for the odd nibbles, and a packed subtraction leaves c or 16 c; the 16
// goes into q (1 / 16) and into the output dims. (The masked nibble alone is the fp16
// subnormal u * 2^-24 and would do for a key without the subtraction, but the tensor
// core aligns its products by the operands' exponent fields: ten bits of the sum were
// lost, and outputs were off by 2.5e-6 instead of 3e-7.)
//
// Each warp owns whole 32-key tiles and a ring of bulk copies of its own; nothing in
// the loop waits for another warp. Products accumulate over one tile only (two
// m16n8k16 steps) and are then added to the fp32 sums with rounding to nearest: the
// tensor core truncates its sums, which over a long cache would drift.
//
// The reference of p is the running row maximum minus 14 plus the running exponent of
// the value scales, so that p * sv peaks near 2^14 whatever the values' magnitude and
// both fp16 parts keep their bits down to 2^-24.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "kv_q4.cuh"
#include "tc_ptx.cuh"

namespace gqa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 32;                    // keys per tile
constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kHeads = 8;                    // query heads per block

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D += A B, A 16 x 16 (row), B 16 x 8 (column), fp16 in, fp32 out.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// Two values to packed fp16 high parts and the fp16 of what is left of them.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = as_u32(h);
  lo = as_u32(__floats2half2_rn(x - f.x, y - f.y));
}

// The nibbles at bits 4 ODD of w's two halves as packed fp16 c (ODD = 0) or 16 c (1).
template <int ODD>
__device__ __forceinline__ uint32_t codes(uint32_t w) {
  const uint32_t u = (w & (ODD ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u;
  return as_u32(__hsub2(as_half2(u), as_half2(ODD ? 0x64806480u : 0x64086408u)));
}

// N 32-bit words from shared memory, aligned to their largest power-of-two divisor.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 t = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = t.x; w[4 * i + 1] = t.y; w[4 * i + 2] = t.z; w[4 * i + 3] = t.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint2 t = reinterpret_cast<const uint2*>(p)[i];
      w[2 * i] = t.x; w[2 * i + 1] = t.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}

// M 16-bit units at p into packed words.
template <int M>
__device__ __forceinline__ void load_units(const uint8_t* p, uint32_t (&w)[(M + 1) / 2]) {
  if constexpr (M % 2 == 0) {
    load_words<M / 2>(p, w);
  } else {
#pragma unroll
    for (int i = 0; i < (M + 1) / 2; ++i) {
      w[i] = reinterpret_cast<const uint16_t*>(p)[2 * i];
      if (2 * i + 1 < M)
        w[i] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[2 * i + 1]) << 16;
    }
  }
}

__device__ __forceinline__ float unit_scale(uint32_t w, int odd) {     // bf16 half of a word
  return __uint_as_float(odd ? w & 0xffff0000u : w << 16);
}

constexpr size_t split_smem(int M) {
  return static_cast<size_t>(kWarps) * kStages * kTile * q4::record_bytes(M) + 1024 * M;
}

// Live slots of row b (0: the row is invalid).
__device__ __forceinline__ int live_slots(const DecodeQ4Job& j, int b, bool lead) {
  const int n = j.cache_len[b];
  if (n < 1 || n > j.max_cache_len || (j.window == 0 && n > j.capacity)) {
    if (lead) report(j.status, ATTN_DEV_LENGTH);
    return 0;
  }
  return j.window > 0 ? min(n, j.window) : n;
}

// One block: up to 8 query heads of one kv head over the slots [split chunk, + chunk).
template <int M, bool WEIGHTS>
__global__ void __launch_bounds__(32 * kWarps, M <= 4 ? 3 : 2) decode_q4_kernel(DecodeQ4Job j) {
  constexpr int D = 32 * M, REC = q4::record_bytes(M), TILE_BYTES = kTile * REC, VW = (M + 1) / 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ float q_factor[kHeads];
  __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads];
  __shared__ int abort_flag;
  if (gated_off(j.skip)) return;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int G = j.H / j.Hkv, ngroups = (G + kHeads - 1) / kHeads;
  const int split = static_cast<int>(blockIdx.x % j.nsplit);
  const unsigned unit = blockIdx.x / j.nsplit;
  const int g0 = static_cast<int>(unit % ngroups) * kHeads;
  const long bh = unit / ngroups;
  const int b = static_cast<int>(bh / j.Hkv), hkv = static_cast<int>(bh - static_cast<long>(b) * j.Hkv);
  const int nlive = live_slots(j, b, threadIdx.x == 0 && split == 0 && g0 == 0 && hkv == 0);
  const int k0 = split * j.chunk;
  if (k0 >= nlive) return;
  const int k1 = min(k0 + j.chunk, nlive);
  const int tiles = (k1 - k0 + kTile - 1) / kTile;
  const int mine = tiles > warp ? (tiles - 1 - warp) / kWarps + 1 : 0;

  uint8_t* ring = smem + warp * kStages * TILE_BYTES;
  const uint8_t* records = j.cache + bh * j.capacity * REC;
  auto first_key = [&](int i) { return k0 + (i * kWarps + warp) * kTile; };
  auto issue = [&](int i) {                  // lane 0: tile i of this warp
    const int s = i % kStages, kb = first_key(i);
    const uint32_t bytes = static_cast<uint32_t>(min(kTile, k1 - kb)) * REC;
    tc::mbar_arrive_expect_tx(&full[warp][s], bytes);
    tc::bulk_load(ring + s * TILE_BYTES, records + static_cast<long>(kb) * REC, bytes,
                  &full[warp][s]);
  };
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) tc::mbar_init(&full[warp][s], 1);
    tc::fence_mbar_init();
    for (int i = 0; i < min(kStages, mine); ++i) issue(i);
  }
  if (threadIdx.x == 0) abort_flag = 0;

  // Queries as A fragments: a warp per head, lane g * 4 + a holds dims 32 g + 8 a .. + 7
  // (the dims of key word (a, g)). Scaled by a power of two so that the head's largest
  // element lies in [2^12, 2^13): both fp16 parts are then normal over 22 bits.
  uint32_t* frag = reinterpret_cast<uint32_t*>(smem + kWarps * kStages * TILE_BYTES);
  for (int h = warp; h < kHeads; h += kWarps) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    const bool there = lane < 4 * M;
    const int g = lane >> 2, a = lane & 3;
    if (there && g0 + h < G) {
      const float4* src = reinterpret_cast<const float4*>(
          j.q + (static_cast<long>(b) * j.H + hkv * G + g0 + h) * D + 8 * lane);
      const float4 t0 = __ldg(src), t1 = __ldg(src + 1);
      x[0] = t0.x; x[1] = t0.y; x[2] = t0.z; x[3] = t0.w;
      x[4] = t1.x; x[5] = t1.y; x[6] = t1.z; x[7] = t1.w;
    }
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    int ex = static_cast<int>(top >> 23) - 127 - 12;          // 2^12 <= |x| 2^-ex < 2^13
    ex = max(-120, ex);
    if (top >= 0x7f800000u) ex = 0;                           // inf or NaN: its head becomes NaN
    const float f = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
    uint32_t hi[4], lo[4];                   // pairs (2 st + odd): dims e and e + 4
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float w = e & 1 ? f * 0.0625f : f;
      split2(x[e] * w, x[e + 4] * w, hi[e], lo[e]);
    }
    if (there) {
#pragma unroll
      for (int st = 0; st < 2; ++st)         // thread (r = h, c = a) of step (g, st)
        *reinterpret_cast<uint4*>(frag + ((2 * g + st) * 32 + 4 * h + a) * 4) =
            make_uint4(hi[2 * st], lo[2 * st], hi[2 * st + 1], lo[2 * st + 1]);
    }
    // scores come out times 2^-ex; undo it, times the softmax scale, in log2 units
    if (lane == 0)
      q_factor[h] = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23) * j.scale *
                    (j.softcap > 0.f ? 1.f : kLog2e);
  }
  __syncthreads();

  const float qf = q_factor[r];
  const uint4* afrag = reinterpret_cast<const uint4*>(frag) + lane;
  float* score_row = nullptr;
  if (WEIGHTS && g0 + r < G)
    score_row = j.scores + (static_cast<long>(b) * j.H + hkv * G + g0 + r) * j.pitch;

  float m_run = -INFINITY, l_run = 0.f;
  int e_run = -60 - 14;                      // exponent of the reference beside the maximum
  float o[M][4][2];
#pragma unroll
  for (int g = 0; g < M; ++g)
#pragma unroll
    for (int q = 0; q < 4; ++q) o[g][q][0] = o[g][q][1] = 0.f;

  int i = 0;
  for (; i < mine; ++i) {
    const int st = i % kStages;
    const bool ok = tc::mbar_wait(&full[warp][st], (i / kStages) & 1, &abort_flag);
    if (__any_sync(0xffffffffu, !ok)) break;
    const uint8_t* tile = ring + st * TILE_BYTES;
    const int kb = first_key(i), valid = min(kTile, k1 - kb);

    // Scores. Thread (r, c) gets head r's of keys 8 t + 2 c and 8 t + 2 c + 1, t = 0 .. 3.
    // Their scales, M of the key and M of the value, come in one load where the registers
    // allow (M <= 4; odd M, whose halves share a word), else the value's later.
    constexpr bool kBoth = M <= 4 || M % 2 == 1;
    constexpr int SW = kBoth ? M : M / 2;
    float s[8];
    uint32_t sc[8][SW];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      s[x] = 0.f;
      load_words<SW>(tile + (8 * (x >> 1) + 2 * c + (x & 1)) * REC + 32 * M, sc[x]);
    }
    {
      uint32_t kw[4][M];
#pragma unroll
      for (int t = 0; t < 4; ++t) load_words<M>(tile + (8 * t + r) * REC + 4 * M * c, kw[t]);
#pragma unroll
      for (int g = 0; g < M; ++g) {
        const uint4 f0 = afrag[64 * g], f1 = afrag[64 * g + 32];
        const uint32_t a0[4] = {f0.x, f0.y, f0.z, f0.w}, a1[4] = {f1.x, f1.y, f1.z, f1.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          const uint32_t w = kw[t][g], w8 = w >> 8;
          mma(d, a0, codes<0>(w), codes<1>(w));
          mma(d, a1, codes<0>(w8), codes<1>(w8));
          s[2 * t] = fmaf(unit_scale(sc[2 * t][g / 2], g & 1), d[0] + d[2], s[2 * t]);
          s[2 * t + 1] = fmaf(unit_scale(sc[2 * t + 1][g / 2], g & 1), d[1] + d[3], s[2 * t + 1]);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) s[x] *= qf;
    if (j.softcap > 0.f) {
#pragma unroll
      for (int x = 0; x < 8; ++x) s[x] = tanhf(s[x] / j.softcap) * (j.softcap * kLog2e);
    }
    // The value scales, apart from the keys'.
    uint32_t vs[8][VW];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      if constexpr (!kBoth) {
        load_words<VW>(tile + (8 * (x >> 1) + 2 * c + (x & 1)) * REC + 34 * M, vs[x]);
      } else {
#pragma unroll
        for (int w = 0; w < VW; ++w)
          vs[x][w] = M % 2 == 0 ? sc[x][M / 2 + w]
                                : __funnelshift_r(sc[x][M / 2 + w],
                                                  M / 2 + w + 1 < M ? sc[x][M / 2 + w + 1] : 0u, 16);
      }
    }
    if (valid < kTile) {                     // slots past the live ones: whatever was there
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        if (8 * (x >> 1) + 2 * c + (x & 1) >= valid) {
          s[x] = -INFINITY;
#pragma unroll
          for (int w = 0; w < VW; ++w) vs[x][w] = 0;
        }
      }
    }
    if (WEIGHTS && score_row) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int k = 8 * t + 2 * c;
        if (k < valid) score_row[kb + k] = s[2 * t];
        if (k + 1 < valid) score_row[kb + k + 1] = s[2 * t + 1];
      }
    }
    // Reference: running maximum and running exponent of the value scales.
    float mx = s[0];
    uint32_t top = 0;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      mx = fmaxf(mx, s[x]);
#pragma unroll
      for (int w = 0; w < VW; ++w) top = __vmaxu2(top, vs[x][w]);
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    if (top >= 0x7f80u) {                    // a NaN group: the others keep their range
      top = 0;
#pragma unroll
      for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          const uint32_t lo = vs[x][w] & 0xffffu, hi = vs[x][w] >> 16;
          top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
      top = __reduce_max_sync(0xffffffffu, top);
    }
    const float m_new = fmaxf(m_run, mx);
    const int e_new = max(e_run, static_cast<int>(top >> 7) - 127 - 14);
    if (__any_sync(0xffffffffu, m_new > m_run) || e_new != e_run) {
      const float corr = m_new == -INFINITY
                             ? 1.f
                             : ex2((m_run - m_new) + static_cast<float>(e_run - e_new));
      l_run *= corr;
#pragma unroll
      for (int g = 0; g < M; ++g)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          o[g][q][0] *= corr;
          o[g][q][1] *= corr;
        }
      m_run = m_new;
      e_run = e_new;
    }
    const float ref = (m_run == -INFINITY ? 0.f : m_run) + static_cast<float>(e_run);
    float p[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      p[x] = ex2(s[x] - ref);
      l_run += p[x];
    }

    // P V. Keys of the two 16-key steps: 16 k + 2 c, + 1, + 8, + 9.
    uint32_t vw[8][VW];
#pragma unroll
    for (int x = 0; x < 8; ++x)
      load_units<M>(tile + (8 * (x >> 1) + 2 * c + (x & 1)) * REC + 16 * M + 2 * M * r, vw[x]);
#pragma unroll
    for (int g = 0; g < M; ++g) {
      uint32_t a[2][4], v[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int x = 4 * k + 2 * h;
          split2(p[x] * unit_scale(vs[x][g / 2], g & 1),
                 p[x + 1] * unit_scale(vs[x + 1][g / 2], g & 1), a[k][2 * h], a[k][2 * h + 1]);
          v[k][h] = __byte_perm(vw[x][g / 2], vw[x + 1][g / 2], g & 1 ? 0x7632 : 0x5410);
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t w0 = q & 2 ? v[k][0] >> 8 : v[k][0], w1 = q & 2 ? v[k][1] >> 8 : v[k][1];
          if (q & 1)
            mma(d, a[k], codes<1>(w0), codes<1>(w1));
          else
            mma(d, a[k], codes<0>(w0), codes<0>(w1));
        }
        o[g][q][0] += d[0] + d[2];
        o[g][q][1] += d[1] + d[3];
      }
    }
    __syncwarp();                            // every lane is done with the stage
    if (lane == 0 && i + kStages < mine) issue(i + kStages);
  }
  if (i < mine && lane == 0) {
    // A wait ran out: let the copies already issued land, then report.
    for (int u = i; u < min(mine, i + kStages); ++u) {
      const uint64_t t0 = tc::globaltimer();
      while (!tc::mbar_try_wait(&full[warp][u % kStages], (u / kStages) & 1))
        if (tc::globaltimer() - t0 > tc::kWaitLimitNs) break;
    }
    report(j.status, ATTN_DEV_TIMEOUT);
  }

  // The warps' sums, brought to one reference, meet in the (now idle) rings.
  l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
  l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
  const float m_ref = m_run + static_cast<float>(e_run);
  if (c == 0) {
    sm_m[warp][r] = m_ref;
    sm_l[warp][r] = l_run;
  }
  __syncthreads();
  float m_all = sm_m[0][r];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) m_all = fmaxf(m_all, sm_m[w][r]);
  const float mine_f = m_ref == -INFINITY ? 0.f : ex2(m_ref - m_all);
  float* ex = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int g = 0; g < M; ++g)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      *reinterpret_cast<float4*>(ex + r * D + 32 * g + 8 * c + 4 * u) =
          make_float4(o[g][0][u] * mine_f, o[g][1][u] * (mine_f * 0.0625f), o[g][2][u] * mine_f,
                      o[g][3][u] * (mine_f * 0.0625f));
  __syncthreads();
  if (abort_flag) return;
  const bool single = nlive <= j.chunk;
  const long hrow0 = static_cast<long>(b) * j.H + hkv * G + g0;
  const int heads = min(kHeads, G - g0);
  float* ml = j.partial + static_cast<long>(j.B) * j.H * j.nsplit * D;
  for (int t = threadIdx.x; t < heads * (D / 4); t += 32 * kWarps) {
    const int h = t / (D / 4), d = 4 * (t - h * (D / 4));
    float M_ = sm_m[0][h], L = 0.f;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M_ = fmaxf(M_, sm_m[w][h]);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (sm_m[w][h] != -INFINITY) L = fmaf(ex2(sm_m[w][h] - M_), sm_l[w][h], L);
      const float4 z = *reinterpret_cast<const float4*>(smem + w * kStages * TILE_BYTES +
                                                        (h * D + d) * 4);
      y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
    }
    if (single) {
      const float inv = 1.0f / L;
      *reinterpret_cast<float4*>(j.out + (hrow0 + h) * D + d) =
          make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
    } else {
      *reinterpret_cast<float4*>(j.partial + ((hrow0 + h) * j.nsplit + split) * D + d) = y;
    }
    if ((WEIGHTS || !single) && d == 0)
      *reinterpret_cast<float2*>(ml + 2 * ((hrow0 + h) * j.nsplit + split)) = make_float2(M_, L);
  }
}

// Maximum reference and sum of one query row over its ns splits, by one warp.
__device__ __forceinline__ float2 row_ml(const float* ml, int ns, int lane) {
  float m = -INFINITY;
  for (int s = lane; s < ns; s += 32) m = fmaxf(m, ml[2 * s]);
  m = warp_max(m);
  float l = 0.f;
  if (m != -INFINITY)
    for (int s = lane; s < ns; s += 32) l = fmaf(ex2(ml[2 * s] - m), ml[2 * s + 1], l);
  return make_float2(m, warp_sum(l));
}

// Blocks [0, rows): one query row's splits merged. Blocks after: with weights, 256
// slots of one kv head get the sum over its query heads of 2^(score - reference) / sum
// (one thread per slot, heads in order, so the result does not depend on timing).
__global__ void __launch_bounds__(256) decode_q4_finish_kernel(DecodeQ4Job j, unsigned rows,
                                                               unsigned slot_blocks) {
  __shared__ float2 sh[8];
  if (gated_off(j.skip)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float* ml = j.partial + static_cast<long>(j.B) * j.H * j.nsplit * j.D;
  if (blockIdx.x < rows) {
    const int b = static_cast<int>(blockIdx.x / j.H);
    const int nlive = live_slots(j, b, false);
    if (nlive <= j.chunk) return;            // finished by its one split, or invalid
    const int ns = (nlive + j.chunk - 1) / j.chunk;
    const long row = blockIdx.x;
    const float* rml = ml + 2 * row * j.nsplit;
    const float2 t = row_ml(rml, ns, lane);
    const float* part = j.partial + row * j.nsplit * j.D;
    const int d = threadIdx.x;
    if (d >= j.D) return;
    float y = 0.f;
    for (int s = 0; s < ns; ++s) {
      const float m = rml[2 * s];
      if (m != -INFINITY) y = fmaf(ex2(m - t.x), part[static_cast<long>(s) * j.D + d], y);
    }
    j.out[row * j.D + d] = y / t.y;
    return;
  }
  const unsigned blk = blockIdx.x - rows;
  const long bh = blk / slot_blocks;
  const int b = static_cast<int>(bh / j.Hkv), hkv = static_cast<int>(bh - static_cast<long>(b) * j.Hkv);
  const int nlive = live_slots(j, b, false);
  const int n = static_cast<int>(blk % slot_blocks) * 256 + threadIdx.x;
  if (static_cast<int>(blk % slot_blocks) * 256 >= nlive) return;
  const int ns = (nlive + j.chunk - 1) / j.chunk;
  const int G = j.H / j.Hkv;
  const long row0 = static_cast<long>(b) * j.H + hkv * G;
  float acc = 0.f;
  for (int g0 = 0; g0 < G; g0 += 8) {
    const int heads = min(8, G - g0);
    if (warp < heads) {
      const float2 t = row_ml(ml + 2 * (row0 + g0 + warp) * j.nsplit, ns, lane);
      if (lane == 0) sh[warp] = make_float2(t.x, 1.0f / t.y);
    }
    __syncthreads();
    if (n < nlive)
      for (int h = 0; h < heads; ++h)
        acc = fmaf(ex2(j.scores[(row0 + g0 + h) * j.pitch + n] - sh[h].x), sh[h].y, acc);
    __syncthreads();
  }
  if (n < nlive) j.weights[bh * j.capacity + n] += acc;
}

template <int M, bool W>
cudaError_t launch_split(const DecodeQ4Job& j, unsigned grid, cudaStream_t stream) {
  static PerContext<cudaError_t> allowed;    // the shared-memory size is per context
  const cudaError_t e = allowed.get(
      [] {
        return cudaFuncSetAttribute(decode_q4_kernel<M, W>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(split_smem(M)));
      },
      cudaErrorInvalidDevice, [](const cudaError_t& v) { return v == cudaSuccess; });
  if (e != cudaSuccess) return e;
  decode_q4_kernel<M, W><<<grid, 32 * kWarps, split_smem(M), stream>>>(j);
  return cudaGetLastError();
}

template <int M>
cudaError_t launch_split(const DecodeQ4Job& j, unsigned grid, cudaStream_t stream) {
  return j.weights ? launch_split<M, true>(j, grid, stream) : launch_split<M, false>(j, grid, stream);
}

int eff_len(int max_cache_len, int window) {
  return window > 0 && window < max_cache_len ? window : max_cache_len;
}

// The most splits of any length up to this one: it does not shrink as the length grows.
int split_bound(int B, int H, int Hkv, int max_cache_len, int window) {
  const int tiles = (eff_len(max_cache_len, window) - 1) / kTile + 1;
  const long units = static_cast<long>(B) * Hkv * ((H / Hkv + kHeads - 1) / kHeads);
  constexpr int resident = 152 * 3;          // blocks on the GPU at once
  const long want = units >= resident ? (4 * resident + units - 1) / units
                                      : (units < 1 ? 1 : resident / units);
  const long most = (tiles + kWarps - 1) / kWarps;            // a tile for every warp
  return static_cast<int>(want < most ? want : most);
}

}  // namespace

void decode_q4_plan(int B, int H, int Hkv, int max_cache_len, int window, int* nsplit,
                    int* chunk) {
  const int tiles = (eff_len(max_cache_len, window) - 1) / kTile + 1;
  const int n = split_bound(B, H, Hkv, max_cache_len, window);
  const int per = (tiles + n - 1) / n;
  *chunk = per * kTile;
  *nsplit = (tiles + per - 1) / per;
}

namespace {
struct Layout {
  size_t scores, total;
  int pitch;
};
Layout layout(int B, int H, int D, int nsplit, int eff, bool weights) {
  Layout y{};
  const size_t rows = static_cast<size_t>(B) * H;
  size_t p = nsplit > 1 || weights ? rows * nsplit * (D + 2) * sizeof(float) : 0;
  y.scores = p = (p + 255) / 256 * 256;
  y.pitch = (eff + 3) / 4 * 4;
  if (weights) p += rows * y.pitch * sizeof(float);
  y.total = p;
  return y;
}
}  // namespace

size_t decode_q4_bytes(int B, int H, int Hkv, int D, int max_cache_len, int window, bool weights,
                       bool bound) {
  int nsplit, chunk;
  decode_q4_plan(B, H, Hkv, max_cache_len, window, &nsplit, &chunk);
  if (bound) nsplit = split_bound(B, H, Hkv, max_cache_len, window);
  return layout(B, H, D, nsplit, eff_len(max_cache_len, window), weights).total;
}

void decode_q4_workspace(DecodeQ4Job* j, void* workspace) {
  decode_q4_plan(j->B, j->H, j->Hkv, j->max_cache_len, j->window, &j->nsplit, &j->chunk);
  const Layout y = layout(j->B, j->H, j->D, j->nsplit, eff_len(j->max_cache_len, j->window),
                          j->weights != nullptr);
  j->partial = static_cast<float*>(workspace);
  j->scores = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) + y.scores) : nullptr;
  j->pitch = y.pitch;
}

cudaError_t launch_decode_q4(const DecodeQ4Job& j, cudaStream_t stream) {
  const int G = j.H / j.Hkv;
  const unsigned units = static_cast<unsigned>(j.B) * j.Hkv * ((G + kHeads - 1) / kHeads);
  const unsigned grid = units * j.nsplit;
  cudaError_t e;
  switch (j.D / 32) {
    case 1: e = launch_split<1>(j, grid, stream); break;
    case 2: e = launch_split<2>(j, grid, stream); break;
    case 3: e = launch_split<3>(j, grid, stream); break;
    case 4: e = launch_split<4>(j, grid, stream); break;
    case 5: e = launch_split<5>(j, grid, stream); break;
    case 6: e = launch_split<6>(j, grid, stream); break;
    case 7: e = launch_split<7>(j, grid, stream); break;
    default: e = launch_split<8>(j, grid, stream); break;
  }
  if (e != cudaSuccess || (j.nsplit == 1 && !j.weights)) return e;
  const unsigned rows = j.nsplit > 1 ? static_cast<unsigned>(j.B) * j.H : 0;
  const unsigned per = j.weights ? (eff_len(j.max_cache_len, j.window) - 1) / 256 + 1 : 0;
  decode_q4_finish_kernel<<<rows + static_cast<unsigned>(j.B) * j.Hkv * per, 256, 0, stream>>>(
      j, rows, per ? per : 1);
  return cudaGetLastError();
}

}  // namespace gqa
