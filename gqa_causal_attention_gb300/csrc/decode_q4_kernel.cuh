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
// accuracy. (The codes are unpacked in registers and used once: staging them in shared
// memory for tcgen05 would cost more shared-memory traffic than the copy itself.)
//
// Keys (then value dims) are the 16 rows of the A operand. With up to 4 query heads (NT =
// 1) the 8 columns of B are their high and low parts, side by side in a thread, which sums
// them. With up to 8 (NT = 2) the columns are the heads, and a second product with the low
// parts adds to the first one's sums. Either way one 8 x 8 transpose (movmatrix) turns 8
// keys' packed weights into the next product's B operand.
//
// A pair of codes becomes a packed fp16 pair in two instructions: a nibble u = c + 8
// masked out of its 16-bit half and put under the exponent of 1024 is 1024 + u, or
// 1024 + 16 u for the odd nibbles, and a packed subtraction leaves c or 16 c; the 16
// goes into q (1 / 16) and into the output dims. (The masked nibble alone is the fp16
// subnormal u * 2^-24 and would do for a key without the subtraction, but the tensor
// core aligns its products by the operands' exponent fields: ten bits of the sum were
// lost, and outputs were off by 2.5e-6 instead of 1.1e-7.)
//
// Each warp owns whole 32-key tiles and a ring of bulk copies of its own; nothing in
// the loop waits for another warp. Products accumulate over one tile only (two
// m16n8k16 steps) and are then added to the fp32 sums: those round to nearest, the tensor
// core's do not, and over a long cache that would drift.
//
// What bounds it: no one unit. A 32-key tile at D = 128 takes 707 instructions of a warp, starts
// and ends among them (304 unpack); 32 rows of 8192 slots, 32 heads over 8 (302 MB, 4.7 TB/s):
// 2.8 of 4 instructions a cycle, ALU pipe at 58 %, memory at 59 %, tensor pipe at 25 %. The sixteen
// warps an SM that the registers leave wait for the ALU pipe and for their own results in turn, and
// 1280 blocks are two waves and a little. With 8 heads a kv head, twelve warps an SM, 881
// instructions a tile, 2.4 a cycle: one row of 131072 slots, 151 MB in 46 us, 3.3 TB/s. With few
// or ragged rows the blocks' uneven shares come on top: a row takes the same chunk whatever its
// length, so the last block of a short row has little, and some SMs hold two blocks, others one.
//
// p and its sum are relative to the running row maximum. For the products p is multiplied by
// 2^-e (exact), e the running exponent of the warp's value scales less 14, so that p * sv peaks
// near 2^14 and both fp16 parts keep their bits down to 2^-24: 22 bits of every weighted value
// within 2^16 of the largest scale the warp has met, fewer below. The output's sums stay in
// units of 2^e until they are normalised, so they neither overflow nor vanish: e reaches down to
// -127, where scales below 2^-126 (values below 1e-37) begin to lose bits.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "kv_q4_rows.cuh"
#include "tc_ptx.cuh"

namespace gqa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 32;                    // keys per tile
constexpr int kWarps = 4;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D += A B, A 16 x 16 (row), B 16 x 8 (column), fp16 in, fp32 out.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit elements (lane: row lane / 4, columns 2 (lane % 4), + 1) transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
  uint32_t u;                                // (w & mask) | 0x6400 in one instruction
  asm("lop3.b32 %0, %1, %2, %3, 0xea;"
      : "=r"(u)
      : "r"(w), "n"(ODD ? 0x00f000f0 : 0x000f000f), "r"(0x64006400u));
  return as_u32(__hsub2(as_half2(u), as_half2(ODD ? 0x64806480u : 0x64086408u)));
}

// 2^n, n <= 127: 0 below fp32's subnormals' first binary order.
__device__ __forceinline__ float pow2(int n) {
  return __uint_as_float(n >= -126 ? static_cast<uint32_t>(127 + n) << 23 : (n == -127 ? 0x400000u : 0u));
}

// The top eleven bits of x >= 0 below 2^16: exact in fp16, as is the rest in fp32. (Below
// 2^-14 fp16 keeps fewer bits: an error of 2^-25, of weights whose largest is near 2^14.)
__device__ __forceinline__ float high_part(float x) {
  return __uint_as_float(__float_as_uint(x) & 0xffffe000u);
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

constexpr int kStages = 2;

// Blocks an SM holds: what registers (124 a thread at D = 128 with NT = 1, 163 with 2) and,
// from D = 192, shared memory leave. Twenty warps an SM instead of sixteen were no faster at
// D = 128.
__host__ __device__ constexpr int resident_blocks(int M, int NT) {
  constexpr int blocks[2][8] = {{8, 6, 5, 4, 4, 3, 3, 2}, {5, 4, 3, 3, 3, 2, 2, 2}};
  return blocks[NT - 1][M - 1];
}

// Rings of all warps, then the queries' B fragments.
constexpr size_t split_smem(int M, int NT, int NW) {
  return static_cast<size_t>(NW) * kStages * kTile * q4::record_bytes(M) + 512 * M * NT;
}

// Live slots of row b, whose length is n (0: the row is invalid).
__device__ __forceinline__ int live_slots(const DecodeQ4Job& j, int n, bool lead) {
  if (n < 1 || n > j.max_cache_len || (j.window == 0 && n > j.capacity)) {
    if (lead) report(j.status, ATTN_DEV_LENGTH);
    return 0;
  }
  return j.window > 0 ? min(n, j.window) : n;
}

// A step's row b: its slot count with the new token (0: the row breaks a rule), slot and
// rotary position.
struct StepRow {
  int n, slot, pos;
};
__device__ __forceinline__ StepRow step_row(const StepQ4Args& st, int b, bool lead) {
  const AppendQ4Job& a = st.kv;
  const int s0 = a.start[b], p0 = a.pos ? a.pos[b] : s0;
  const bool placed = s0 >= 0 && p0 >= 0 && p0 < a.max_positions;
  const bool has_slot = a.window > 0 || s0 < a.capacity;
  if (lead) {
    if (!placed)
      report(a.status, ATTN_DEV_POSITION);
    else if (!has_slot)
      report(a.status, ATTN_DEV_CAPACITY);
    st.cache_len[b] = placed && has_slot ? s0 + 1 : 0;
  }
  return StepRow{placed && has_slot ? s0 + 1 : 0, a.window > 0 ? s0 % a.window : s0, p0};
}

// RMSNorm (nw) and RoPE at tab's angles of eight dims d0 .. + 7 of the raw row; the lanes of
// the warp hold the whole row (x; zeros past it).
__device__ __forceinline__ void rotate_query(const float* row, const float2* tab, int R,
                                             const float* nw, float eps, int D, int d0,
                                             float (&x)[8]) {
  float inv = 1.f;
  if (nw) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
    inv = 1.0f / sqrtf(warp_sum(ss) / static_cast<float>(D) + eps);
  }
  if (d0 >= D) return;
  const int half = R / 2;
  if (half % 8 == 0) {                       // the eight dims lie within one half
    float b[8], w[8], cs[16];
    const bool rotary = d0 < R, low = d0 < half;
    const int i = low ? d0 : d0 - half, p = low ? d0 + half : i;
    if (rotary) {
#pragma unroll
      for (int q = 0; q < 4; ++q) load4(reinterpret_cast<const float*>(tab + i) + 4 * q, cs + 4 * q);
      load4(row + p, b);
      load4(row + p + 4, b + 4);
    }
    if (nw) {
      load4(nw + d0, w);
      load4(nw + d0 + 4, w + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * w[e];
      if (rotary) {
        load4(nw + p, w);
        load4(nw + p + 4, w + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = b[e] * inv * w[e];
      }
    }
    if (rotary) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = fmaf(x[e], cs[2 * e], (low ? -b[e] : b[e]) * cs[2 * e + 1]);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int d = d0 + e;
    float a = nw ? x[e] * inv * nw[d] : x[e];
    if (d < R) {
      const int i = d < half ? d : d - half, p = d < half ? d + half : i;
      const float b = nw ? row[p] * inv * nw[p] : row[p];
      const float2 t = tab[i];
      a = d < half ? fmaf(a, t.x, -b * t.y) : fmaf(a, t.x, b * t.y);
    }
    x[e] = a;
  }
}

// One block: up to 4 NT query heads of one kv head over the slots [split chunk, + chunk).
// NW warps share its tiles.
template <int M, int NT, bool WEIGHTS, int NW>
__global__ void __launch_bounds__(32 * NW, NW > kWarps ? 1 : resident_blocks(M, NT))
decode_q4_kernel(DecodeQ4Job j, StepQ4Args st) {
  constexpr int D = 32 * M, REC = q4::record_bytes(M), TILE_BYTES = kTile * REC, VW = (M + 1) / 2;
  constexpr int kHeads = 4 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[NW][kStages];
  __shared__ float q_factor[kHeads];
  __shared__ float sm_m[NW][kHeads], sm_l[NW][kHeads];
  __shared__ int sm_e[NW];
  __shared__ int abort_flag;
  dependent_wait();
  if (gated_off(j.skip)) return;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int G = j.H / j.Hkv, ngroups = (G + kHeads - 1) / kHeads;
  const int split = static_cast<int>(blockIdx.x % j.nsplit);
  const unsigned unit = blockIdx.x / j.nsplit;
  const int g0 = static_cast<int>(unit % ngroups) * kHeads;
  const long bh = unit / ngroups;
  const int b = static_cast<int>(bh / j.Hkv), hkv = static_cast<int>(bh - static_cast<long>(b) * j.Hkv);
  const bool lead = threadIdx.x == 0 && split == 0 && g0 == 0 && hkv == 0;   // one a batch row
  // A warp's first query head is on its way while the row's length comes.
  const float* queries = j.q + (static_cast<long>(b) * j.H + hkv * G + g0) * D;
  float4 q0 = make_float4(0.f, 0.f, 0.f, 0.f), q1 = q0;
  auto load_query = [&](int h) {
    if (lane < 4 * M && h < min(kHeads, G - g0)) {
      const float4* src = reinterpret_cast<const float4*>(queries + h * D + 8 * lane);
      q0 = src[0];
      q1 = src[1];
    }
  };
  load_query(warp);
  const bool step = st.kv.k != nullptr;
  StepRow row{};
  if (step) row = step_row(st, b, lead);
  const int nlive = live_slots(j, step ? row.n : j.cache_len[b], lead);
  const int k0 = split * j.chunk;
  if (k0 >= nlive) return;
  const int k1 = k0 + min(j.chunk, nlive - k0);
  const int tiles = (k1 - k0 + kTile - 1) / kTile;
  const int mine = tiles > warp ? (tiles - 1 - warp) / NW + 1 : 0;

  uint8_t* ring = smem + warp * kStages * TILE_BYTES;
  const uint8_t* records = j.cache + bh * j.capacity * REC;
  auto first_key = [&](int i) { return k0 + (i * NW + warp) * kTile; };
  auto issue = [&](int i) {                  // lane 0: tile i of this warp
    const int s = i % kStages, kb = first_key(i);
    const uint32_t bytes = static_cast<uint32_t>(min(kTile, k1 - kb)) * REC;
    tc::mbar_arrive_expect_tx(&full[warp][s], bytes);
    tc::bulk_load(ring + s * TILE_BYTES, records + static_cast<long>(kb) * REC, bytes,
                  &full[warp][s]);
  };
  if (step && row.slot >= k0 && row.slot < k1 && (row.slot - k0) / kTile % NW == warp) {
    // This warp's tiles hold the new token's slot: it goes there first. With more than 8 heads
    // a kv head several blocks do this, so the record is finished in the (still idle) ring and
    // only its final bytes, the same in each, reach the cache. The fence orders the writes
    // there and the reads here before this warp's bulk copies.
    q4::Lanes<M> at(lane);
    at.in = at.in && at.row == 0;
    const float *x = st.kv.k + bh * D, *v = st.kv.v + bh * D;
    const float2* tab = st.kv.table + static_cast<long>(row.pos) * (st.kv.R / 2);
    const uint2 d = append_rows<M, kRopeDims>(st.kv, x, v, tab, ring, nullptr, at, lane, at.in);
    __syncwarp();
    if (d.x)
      q4::quantise_exact<M>(x, tab, st.kv.R, st.kv.norm_w, st.kv.norm_eps, lane, d.x, ring, 0);
    if (d.y) q4::quantise_exact<M>(v, nullptr, 0, nullptr, 0.f, lane, d.y, ring, 1);
    __syncwarp();
    if (lane < REC / 16)
      reinterpret_cast<uint4*>(st.kv.cache + (bh * j.capacity + row.slot) * REC)[lane] =
          reinterpret_cast<const uint4*>(ring)[lane];
    asm volatile("fence.proxy.async;" ::: "memory");
    __syncwarp();
  }
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) tc::mbar_init(&full[warp][s], 1);
    tc::fence_mbar_init();
    for (int i = 0; i < min(kStages, mine); ++i) issue(i);
  }
  if (threadIdx.x == 0) abort_flag = 0;

  // Queries as B fragments: a warp per head, lane g * 4 + a holds dims 32 g + 8 a .. + 7
  // (the dims of key word (a, g)). Scaled by a power of two so that the head's largest
  // element lies in [2^12, 2^13): both fp16 parts are then normal over 22 bits. Product
  // step (g, st) takes from thread (n, a) the pairs of dims 2 st, 2 st + 4 and 2 st + 1,
  // 2 st + 5 of the word. Column n = 2 h is head h's high part and 2 h + 1 its low part (NT
  // = 1), or n = h in two fragments, high and low.
  uint2* frag = reinterpret_cast<uint2*>(smem + NW * kStages * TILE_BYTES);
  for (int h = warp; h < kHeads; h += NW) {
    if (h > warp) {
      q0 = q1 = make_float4(0.f, 0.f, 0.f, 0.f);
      load_query(h);
    }
    float x[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
    const bool there = lane < 4 * M;
    const int g = lane >> 2, a = lane & 3;
    if (step)
      rotate_query(queries + h * D, st.kv.table + static_cast<long>(row.pos) * (st.kv.R / 2), st.kv.R,
                   st.q_norm_w, st.kv.norm_eps, D, g0 + h < G ? 8 * lane : D, x);
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    int ex = max(-120, static_cast<int>(top >> 23) - 127 - 12);   // 2^12 <= |x| 2^-ex < 2^13
    if (top >= 0x7f800000u) ex = 0;                           // inf or NaN: its head becomes NaN
    const float f = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float w = e & 1 ? f * 0.0625f : f;
      split2(x[e] * w, x[e + 4] * w, hi[e], lo[e]);
    }
    if (there) {
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        uint2* to = frag + (2 * g + st) * 32 + (NT == 1 ? 8 : 4) * h + a;
        to[0] = make_uint2(hi[2 * st], hi[2 * st + 1]);
        to[NT == 1 ? 4 : 64 * M] = make_uint2(lo[2 * st], lo[2 * st + 1]);
      }
    }
    // scores come out times 2^-ex; undo it, times the softmax scale, in log2 units
    if (lane == 0)
      q_factor[h] = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23) * j.scale *
                    (j.softcap > 0.f ? 1.f : kLog2e);
  }
  __syncthreads();

  const uint2* bfrag = frag + lane;
  float qf[NT];
  auto head = [&](int t) { return NT * c + t; };           // this thread's heads
  float* score_row[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int h = head(t);
    qf[t] = q_factor[h];
    score_row[t] = WEIGHTS && g0 + h < G
                       ? j.scores + (static_cast<long>(b) * j.H + hkv * G + g0 + h) * j.pitch
                       : nullptr;
  }

  float m_run[NT], l_run[NT];
  int e_run = -127;                          // o's unit is 2^e_run
  float o[NT][M][4];                         // head(t), dims 32 g + 4 r + (0 .. 3)
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m_run[t] = -INFINITY;
    l_run[t] = 0.f;
#pragma unroll
    for (int g = 0; g < M; ++g)
#pragma unroll
      for (int q = 0; q < 4; ++q) o[t][g][q] = 0.f;
  }

  int i = 0;
  for (; i < mine; ++i) {
    const int st = i % kStages;
    const bool ok = tc::mbar_wait(&full[warp][st], (i / kStages) & 1, &abort_flag);
    if (__any_sync(0xffffffffu, !ok)) break;
    const uint8_t* tile = ring + st * TILE_BYTES;
    const int kb = first_key(i), valid = min(kTile, k1 - kb);

    // Scores of keys r, r + 8, r + 16, r + 24 (x = 0 .. 3). Their scales, M of the key and
    // M of the value, come in one load where the registers allow (M <= 4; odd M, whose
    // halves share a word), else the value's later.
    constexpr bool kBoth = M <= 4 || M % 2 == 1;
    constexpr int SW = kBoth ? M : M / 2;
    float s[NT][4];
    uint32_t sc[4][SW];
    {
      uint32_t kw[4][M];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        load_words<M>(tile + (8 * x + r) * REC + 4 * M * c, kw[x]);
        load_words<SW>(tile + (8 * x + r) * REC + 32 * M, sc[x]);
#pragma unroll
        for (int t = 0; t < NT; ++t) s[t][x] = 0.f;
      }
#pragma unroll
      for (int g = 0; g < M; ++g) {
        uint2 f[NT][2];                      // NT = 2: high parts, low parts
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          f[t][0] = bfrag[((t * M + g) * 2) * 32];
          f[t][1] = bfrag[((t * M + g) * 2 + 1) * 32];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {        // keys 16 k .. 16 k + 15
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t w0 = q ? kw[2 * k][g] >> 8 : kw[2 * k][g];
            const uint32_t w1 = q ? kw[2 * k + 1][g] >> 8 : kw[2 * k + 1][g];
            const uint32_t a0 = codes<0>(w0), a1 = codes<0>(w1), a2 = codes<1>(w0), a3 = codes<1>(w1);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma(d, a0, a1, a2, a3, f[t][q].x, f[t][q].y);
          }
          const float s0 = unit_scale(sc[2 * k][g / 2], g & 1);
          const float s1 = unit_scale(sc[2 * k + 1][g / 2], g & 1);
          if (NT == 1) {
            s[0][2 * k] = fmaf(s0, d[0] + d[1], s[0][2 * k]);
            s[0][2 * k + 1] = fmaf(s1, d[2] + d[3], s[0][2 * k + 1]);
          } else {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              s[t][2 * k] = fmaf(s0, d[t], s[t][2 * k]);
              s[t][2 * k + 1] = fmaf(s1, d[2 + t], s[t][2 * k + 1]);
            }
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[t][x] *= qf[t];
    if (j.softcap > 0.f) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[t][x] = tanhf(s[t][x] / j.softcap) * (j.softcap * kLog2e);
    }
    // The value scales, apart from the keys'.
    uint32_t vs[4][VW];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if constexpr (!kBoth) {
        load_words<VW>(tile + (8 * x + r) * REC + 34 * M, vs[x]);
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
      for (int x = 0; x < 4; ++x) {
        if (8 * x + r >= valid) {
#pragma unroll
          for (int t = 0; t < NT; ++t) s[t][x] = -INFINITY;
#pragma unroll
          for (int w = 0; w < VW; ++w) vs[x][w] = 0;
        }
      }
    }
    if (WEIGHTS) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (score_row[t]) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (8 * x + r < valid) score_row[t][kb + 8 * x + r] = s[t][x];
        }
    }
    // Reference: each head's running maximum and the running exponent of the value scales.
    uint32_t top = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int w = 0; w < VW; ++w) top = __vmaxu2(top, vs[x][w]);
    top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    if (top >= 0x7f80u) {                    // a NaN group: the others keep their range
      top = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          const uint32_t lo = vs[x][w] & 0xffffu, hi = vs[x][w] >> 16;
          top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
      top = __reduce_max_sync(0xffffffffu, top);
    }
    const int e_new = max(e_run, static_cast<int>(top >> 7) - 127 - 14);
    float m_new[NT];
    bool moved = e_new != e_run;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float mx = fmaxf(fmaxf(s[t][0], s[t][1]), fmaxf(s[t][2], s[t][3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      m_new[t] = fmaxf(m_run[t], mx);
      moved |= m_new[t] > m_run[t];
    }
    if (__any_sync(0xffffffffu, moved)) {
      const float coarser = pow2(e_run - e_new);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float corr = m_new[t] == -INFINITY ? 1.f : ex2(m_run[t] - m_new[t]);
        l_run[t] *= corr;
        corr *= coarser;
#pragma unroll
        for (int g = 0; g < M; ++g)
#pragma unroll
          for (int q = 0; q < 4; ++q) o[t][g][q] *= corr;
        m_run[t] = m_new[t];
      }
      e_run = e_new;
    }
    float p[NT][4];
    const float lift = __uint_as_float(static_cast<uint32_t>(127 - e_run) << 23);   // 2^-e_run
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float ref = m_run[t] == -INFINITY ? 0.f : m_run[t];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        p[t][x] = ex2(s[t][x] - ref);
        l_run[t] += p[t][x];
        p[t][x] *= lift;
      }
    }

    // P V, 16 dims x 16 keys a product: thread (r, c) unpacks dims 32 g + 4 r + (0 .. 3) of
    // keys 16 k + 2 c, + 1, + 8, + 9.
    uint32_t vw[8][VW];
#pragma unroll
    for (int x = 0; x < 8; ++x)
      load_units<M>(tile + (8 * (x >> 1) + 2 * c + (x & 1)) * REC + 16 * M + 2 * M * r, vw[x]);
#pragma unroll
    for (int g = 0; g < M; ++g) {
      uint32_t w[4], pb[NT][4];              // per 8 keys: value codes of key pairs, weights
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        w[x] = __byte_perm(vw[2 * x][g / 2], vw[2 * x + 1][g / 2], g & 1 ? 0x7632 : 0x5410);
        const float sv = unit_scale(vs[x][g / 2], g & 1);
        if (NT == 1) {
          const float y = p[0][x] * sv, h = high_part(y);
          pb[0][x] = transpose8(as_u32(__floats2half2_rn(h, y - h)));
        } else {
          const float y0 = p[0][x] * sv, y1 = p[NT - 1][x] * sv, h0 = high_part(y0), h1 = high_part(y1);
          pb[0][x] = transpose8(as_u32(__floats2half2_rn(h0, h1)));
          pb[NT - 1][x] = transpose8(as_u32(__floats2half2_rn(y0 - h0, y1 - h1)));
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {          // dims 4 r + 2 q (rows 0 .. 7) and + 2 q + 1
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t w0 = q ? w[2 * k] >> 8 : w[2 * k], w1 = q ? w[2 * k + 1] >> 8 : w[2 * k + 1];
          const uint32_t a0 = codes<0>(w0), a1 = codes<1>(w0), a2 = codes<0>(w1), a3 = codes<1>(w1);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma(d, a0, a1, a2, a3, pb[t][2 * k], pb[t][2 * k + 1]);
        }
        if (NT == 1) {
          o[0][g][2 * q] += d[0] + d[1];
          o[0][g][2 * q + 1] += d[2] + d[3];
        } else {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            o[t][g][2 * q] += d[t];
            o[t][g][2 * q + 1] += d[2 + t];
          }
        }
      }
    }
    __syncwarp();                            // every lane is done with the stage
    if (lane == 0 && i + kStages < mine) issue(i + kStages);
  }
  if (i < mine && lane == 0) {
    // A wait ran out: let the copies already issued land, then report.
    for (int u = i; u < min(mine, i + kStages); ++u)
      tc::mbar_drain(&full[warp][u % kStages], (u / kStages) & 1);
    report(j.status, ATTN_DEV_TIMEOUT);
  }

  // Only now: blocks of the next kernel placed earlier would take the free places of the SMs
  // that got fewer of these, and spread unevenly themselves (one row of 131072 slots, 19
  // splits, repeated: 92 us instead of 60).
  dependents_may_launch();
  // The warps' sums, brought to one reference, meet in the (now idle) rings.
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l_run[t] += __shfl_xor_sync(0xffffffffu, l_run[t], off);
    // Scores that were all NaN have no maximum; any one keeps their sum in the merge.
    if (m_run[t] == -INFINITY && l_run[t] != l_run[t]) m_run[t] = 0.f;
    if (r == 0) {
      sm_m[warp][head(t)] = m_run[t];
      sm_l[warp][head(t)] = l_run[t];
    }
  }
  if (lane == 0) sm_e[warp] = e_run;
  __syncthreads();
  const int e_all = __reduce_max_sync(0xffffffffu, sm_e[lane % NW]);
  const float coarser = pow2(e_run - e_all);
  float* ex = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int h = head(t);
    float m_all = sm_m[0][h];
#pragma unroll
    for (int w = 1; w < NW; ++w) m_all = fmaxf(m_all, sm_m[w][h]);
    const float f = (m_run[t] == -INFINITY ? 0.f : ex2(m_run[t] - m_all)) * coarser, fo = f * 0.0625f;
#pragma unroll
    for (int g = 0; g < M; ++g)
      *reinterpret_cast<float4*>(ex + h * D + 32 * g + 4 * r) =
          make_float4(o[t][g][0] * f, o[t][g][1] * fo, o[t][g][2] * f, o[t][g][3] * fo);
  }
  __syncthreads();
  if (abort_flag) return;
  const bool single = nlive <= j.chunk;
  const long hrow0 = static_cast<long>(b) * j.H + hkv * G + g0;
  const int heads = min(kHeads, G - g0);
  float* ml = j.partial + static_cast<long>(j.B) * j.H * j.nsplit * D;
  for (int t = threadIdx.x; t < heads * (D / 4); t += 32 * NW) {
    const int h = t / (D / 4), d = 4 * (t - h * (D / 4));
    float M_ = sm_m[0][h], L = 0.f;
#pragma unroll
    for (int w = 1; w < NW; ++w) M_ = fmaxf(M_, sm_m[w][h]);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (sm_m[w][h] != -INFINITY) L = fmaf(ex2(sm_m[w][h] - M_), sm_l[w][h], L);
      const float4 z = *reinterpret_cast<const float4*>(smem + w * kStages * TILE_BYTES +
                                                        (h * D + d) * 4);
      y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
    }
    // Out of the unit only when normalised, a split's part by its own sum: a mean of values.
    // (A split without any weight counts for nothing; a row without any has no softmax.)
    const float inv = L == 0.f && !single ? 0.f : 1.0f / L, back = pow2(e_all);
    float* to = single ? j.out + (hrow0 + h) * D : j.partial + ((hrow0 + h) * j.nsplit + split) * D;
    *reinterpret_cast<float4*>(to + d) =
        make_float4(y.x * inv * back, y.y * inv * back, y.z * inv * back, y.w * inv * back);
    if ((WEIGHTS || !single) && d == 0)
      *reinterpret_cast<float2*>(ml + 2 * ((hrow0 + h) * j.nsplit + split)) = make_float2(M_, L);
  }
}

template <int M, int NT, bool W, int NW>
cudaError_t launch_split(const DecodeQ4Job& j, const StepQ4Args& st, unsigned grid, cudaStream_t stream) {
  static PerContext<cudaError_t> allowed;    // the shared-memory size is per context
  constexpr size_t smem = split_smem(M, NT, NW);
  auto kernel = decode_q4_kernel<M, NT, W, NW>;
  const cudaError_t e = allowed.get(
      [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(smem));
      },
      cudaErrorInvalidDevice, [](const cudaError_t& v) { return v == cudaSuccess; });
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, grid, 32 * NW, smem, stream, j, st);
}

// Query heads per block: 4 or 8.
inline int head_tiles(int H, int Hkv) { return H / Hkv <= 4 ? 1 : 2; }
inline long units_of(int B, int H, int Hkv) {
  const int per = 4 * head_tiles(H, Hkv);
  return static_cast<long>(B) * Hkv * ((H / Hkv + per - 1) / per);
}

// Short rows of few heads: one tile a warp, sixteen warps where the registers allow (the
// one block's rounds are the kernel's time: one row of 500 slots, 8 kv heads of 4 query
// heads, 6.1 us with 4 warps).
constexpr int kShortTiles = 16;

template <int M, int NT>
cudaError_t launch_split(const DecodeQ4Job& j, const StepQ4Args& st, cudaStream_t stream) {
  const long units = units_of(j.B, j.H, j.Hkv);
  const unsigned grid = static_cast<unsigned>(units) * j.nsplit;
  constexpr int kBig = M <= 4 && NT == 1 ? 16 : 8;
  const bool big = j.nsplit == 1 && j.chunk > kWarps * kTile && units <= 152;
  if (j.weights)
    return big ? launch_split<M, NT, true, kBig>(j, st, grid, stream)
               : launch_split<M, NT, true, kWarps>(j, st, grid, stream);
  return big ? launch_split<M, NT, false, kBig>(j, st, grid, stream)
             : launch_split<M, NT, false, kWarps>(j, st, grid, stream);
}

template <int M>
cudaError_t launch_split(const DecodeQ4Job& j, const StepQ4Args& st, cudaStream_t stream) {
  return head_tiles(j.H, j.Hkv) == 1 ? launch_split<M, 1>(j, st, stream)
                                     : launch_split<M, 2>(j, st, stream);
}

}  // namespace

}  // namespace gqa
