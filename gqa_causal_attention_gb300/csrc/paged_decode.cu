// Single-token attention over a paged 16-bit cache ("mojolearn.transformer", step; "Core Layers
// -- Deep Reference", "MHA and GQA"):
//
//   out[b,h] = sum_n w_n v_n / sum_n w_n,   w_n = 2^(c cap(q . k_n) - m),   n in [max(0, len - W), len)
//
// one pass over keys and values with a running reference m, sums in fp32.
//
// * Memory bound: every key and value is read once for the (up to 8) query heads of a unit, 4 D
//   bytes and 4 G D flops a position. Each warp has a ring of tiles (16 positions, their keys and
//   values) of its own in shared memory, filled by TMA two or three tiles ahead, so that 190 KB are on
//   their way to an SM at a time whatever its warps do (loads into registers, half as much:
//   64 rows of 512..8192 slots 197 us). In the 128-byte swizzle, with the tile's rows taken in an
//   order that keeps eight lanes on eight banks, a lane's 16 bytes are operands of m16n8k16
//   products as they lie: the products' inner and outer dims are taken in an order of their own,
//   and pairs of value rows made by one byte permutation a register.
//     scores S[key, head] = K Q^T      A = 16 keys, B = 8 heads of Q
//     O[dim, head] += V^T P^T          A = value pairs, B = P, its 8 x 8 blocks transposed by movmatrix
// * P is split in two 16-bit parts, so its rounding (2^-8 in bf16) does not add to the output's: a
//   weight is off by 2^-16 of itself, in fp16 by 2^-22 of itself and 2^-37 of the row's largest.
// * The tiles (16 positions) of all rows and heads, counted from the lengths on the device, are
//   dealt out to the blocks in shares of equal cost (tiles, and kStart for each row and head begun),
//   whatever the lengths; a block's share is one run of tiles, so at most its first and last unit
//   are shared with other blocks and joined by a second kernel, a warp per row and head. Where rows
//   are short, one block does each unit and nothing is left to join (see decode_paged_plan).
// * With a prefix that all rows share, either its partial results (from the tensor cores) are joined
//   here too, or, where it is read a few times only, its tiles come before the row's own.
#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "prefill_common.cuh"

namespace gqa {

namespace {

constexpr int kTile = 16;                     // positions per warp step (never across pages)
constexpr int kSms = 152;
// Warps of a block that takes a share, or one of many units, how many such blocks an SM holds, and
// those of a block alone on its SM; tiles on their way per warp: about 192 KB an SM. (8 rows of
// 32768 slots, 8 kv heads of 8 heads of 128: two blocks of 4 warps, three tiles 171.5 us, three and
// two 165. Heads of 64, where a tile is half as long: 15.7 and 18 for 23 rows of 1..5000.)
__host__ __device__ constexpr int warps_of(int D) { return D <= 64 ? 8 : 4; }
__host__ __device__ constexpr int wide_warps_of(int D) { return 2 * warps_of(D); }
__host__ __device__ constexpr int resident_of(int D) { return D <= 64 ? 2 : 3; }
__host__ __device__ constexpr int ring_of(int W, int D) {
  return W == warps_of(D) && D > 64 ? 2 : 3;
}
constexpr int kHeads = 8;                     // query heads of a unit
// What a block's start of a unit costs, in tiles: a chain of loads (length, page, tile) and the warps'
// merge. Shares are equal in tiles plus starts, or a block that meets many short rows ends last (64
// rows of 1..1000 slots, shared out: 0 48.5 us, 6 32.6, 16 31; of 1..2000 65.6, 53.9, 51.5).
constexpr unsigned kStart = 16;
// A row's reference lies kBias below the maximum that set it, in log2 units, and moves when exceeded by
// kGrow. fp16 has few small numbers: with a bias of 12 a weight of 2^-25 of that maximum is known to
// 2^-12 of itself (without one it came out as nothing, or twice its size), and what is lost of any is
// 2^-37 of the maximum. Weights are at most 2^15 then.
template <class T> constexpr float kBias = std::is_same<T, __half>::value ? 12.0f : 0.0f;
template <class T> constexpr float kGrow = std::is_same<T, __half>::value ? 15.0f : 8.0f;
constexpr int kMaxScanRows = 8192;            // rows whose tile counts a block keeps

struct DecodeArgs {
  const void* q;
  void* out;
  int64_t q_token, q_head, o_token, o_head;
  const void* k;
  const void* v;
  int64_t page_stride;
  int pages, page_shift;
  const int32_t* block_table;
  int64_t width;
  const int32_t* cache_len;
  int max_len, B, H, Hkv, D, G, HT;           // HT: units per kv head
  int window;
  float c_score;                              // log2 units
  CapArgs cap;
  const int32_t* prefix_table;                // prefix read here, before the row's own positions
  int prefix_len;
  PrefixParts prefix;                         // or its partial results
  float* part_o;                              // [blocks][2][8][D]
  float2* part_ml;                            // [blocks][2][8]
  int blocks;
  int32_t* status;
  const int32_t* skip;
};

// Row b's live positions [lo, n) of its own and its tiles: pt of the prefix, then its own from
// tile t0 on; n < 0 where the length breaks a rule.
struct Span {
  int lo, n, t0, pt, nt;
};
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b) {
  const int n = a.cache_len[b];
  if (n < 0 || n > a.max_len) return {0, -1, 0, 0, 0};
  const int lo = a.window > 0 ? max(0, n - a.window) : 0;
  const int pt = (a.prefix_len + kTile - 1) / kTile;
  return {lo, n, lo / kTile, pt, pt + (n > 0 ? (n - 1) / kTile + 1 - lo / kTile : 0)};
}

template <class T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1,
                                                        uint32_t a2, uint32_t a3, uint32_t b0,
                                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1,
                                                 uint32_t a2, uint32_t a3, uint32_t b0,
                                                 uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 block of 16-bit values, lane 4 g + t holding row g, columns 2 t and 2 t + 1: transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four raw scores capped: by the series, and where one of the warp's is past its limit, that one by
// 2^x and a reciprocal.
__device__ __forceinline__ void soft_cap(const CapArgs& c, float (&x)[4]) {
  float y[4];
  bool past = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float z = x[e] * x[e];
    float p = fmaf(c.series[4], z, c.series[3]);
    p = fmaf(p, z, c.series[2]);
    p = fmaf(p, z, c.series[1]);
    p = fmaf(p, z, c.series[0]);
    y[e] = p * x[e];
    past |= !(fabsf(x[e]) <= c.limit);
  }
  if (__any_sync(0xffffffffu, past)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float u = tc::ex2(x[e] * c.in);
      if (!(fabsf(x[e]) <= c.limit)) y[e] = fmaf(-2.0f * c.out, tc::rcp(u + 1.0f), c.out);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = y[e];
}

template <int W, int DP>
struct __align__(16) Merge {                  // one block's warps, then its result
  float o[W][kHeads][DP + 4];
  float m[W][kHeads], l[W][kHeads];
};

// A block's shared memory: rings, which the merge takes over once their tiles are done.
template <int W, int DP>
struct Smem {
  static constexpr int kRing = ring_of(W, DP);
  static constexpr int kBox = kTile * 128;    // 16 positions x 64 dims
  static constexpr int kStage = 2 * (DP / 64) * kBox;   // keys, then values
  union {
    uint8_t ring[W][kRing][kStage];
    Merge<W, DP> merge;
  };
  uint64_t full[W][kRing];
  int abort;
  static_assert(sizeof(Merge<W, DP>) <= W * kRing * kStage, "the merge fits in the rings");
};

// A warp's ring: tiles asked for and taken so far (stage: count % kRing, parity: of its turns).
struct Ring {
  uint32_t asked = 0, taken = 0;
};

// Output row of query head `head`, dims d .. d + 3.
template <class T>
__device__ __forceinline__ void store_out(const DecodeArgs& a, int b, int head, int d, float4 o) {
  T* p = static_cast<T*>(a.out) + b * a.o_token + head * a.o_head + d;
  *reinterpret_cast<uint2*>(p) =
      make_uint2(Pair<T>::pack(o.x, o.y), Pair<T>::pack(o.z, o.w));
}

// Adds `count` parts -- part(i, ml, o) says where the i-th's (reference, sum) and o / sum lie -- to a
// row's y = sum of weights x values, its reference `top` and sum. Whole warp, dims d .. d + 3 a lane.
// 32 parts at a time, a lane each; then their rows, eight loads on their way at once (one after
// the other 38 parts took 20 us).
template <class F>
__device__ __forceinline__ void add_parts(F part, unsigned count, int d, int D, float4& y, float& top,
                                          float& sum) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (unsigned s0 = 0; s0 < count; s0 += 32) {
    const unsigned n = min(32u, count - s0);
    const float2* ml;
    const float* o;
    part(s0 + min(static_cast<unsigned>(lane), n - 1), ml, o);
    const float2 mine = lane < n ? *ml : make_float2(-INFINITY, 0.f);
    const float before = top;
    top = fmaxf(top, warp_max(mine.x));
    const float f = mine.y == 0.f ? 0.f : tc::ex2(mine.x - top) * mine.y;
    if (before != top && before != -INFINITY) {
      const float r = tc::ex2(before - top);
      sum *= r;
      y.x *= r; y.y *= r; y.z *= r; y.w *= r;
    }
    sum += warp_sum(f);
#pragma unroll 1
    for (unsigned i = 0; i < n; i += 8) {
      float4 p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float* from = reinterpret_cast<const float*>(__shfl_sync(
            0xffffffffu, reinterpret_cast<unsigned long long>(o), min(i + e, n - 1)));
        p[e] = d < D ? *reinterpret_cast<const float4*>(from + d) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float fi = __shfl_sync(0xffffffffu, f, min(i + e, 31u));
        if (i + e < n) {
          y.x = fmaf(fi, p[e].x, y.x); y.y = fmaf(fi, p[e].y, y.y);
          y.z = fmaf(fi, p[e].z, y.z); y.w = fmaf(fi, p[e].w, y.w);
        }
      }
    }
  }
}

// The prefix's parts (PRE) of row b, query head `head`, and the row's output. (A kernel without
// them is one of its own: their code costs the others registers, 5% of the time.)
template <class T, bool PRE>
__device__ __forceinline__ void finish_row(const DecodeArgs& a, int b, int head, int d, float4 y,
                                           float top, float sum) {
  const int64_t row = static_cast<int64_t>(b) * a.H + head, rows = static_cast<int64_t>(a.B) * a.H;
  if (PRE) {
    dependent_wait();                         // for the prefix's kernel, if not yet
    add_parts(
        [&](unsigned i, const float2*& ml, const float*& o) {
          ml = a.prefix.ml + i * rows + row;
          o = a.prefix.o + (i * rows + row) * a.D;
        },
        a.prefix.nsplit, d, a.D, y, top, sum);
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;      // (a NaN stays one)
  if (d < a.D)
    store_out<T>(a, b, head, d, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
}

// Tiles [t0, t1) of row b's span for kv head hk, query heads [h0, h0 + nh): the block's result
// goes, with the prefix's parts, to the output when whole (slot < 0), else to partial slot `slot`
// of this block.
template <class T, int W, int DP, bool PRE>
__device__ void segment(const DecodeArgs& a, const CUtensorMap* tk, const CUtensorMap* tv,
                        Smem<W, DP>* sm, Ring& ring, int b, int hk, int h0, int nh, const Span& sp,
                        int t0, int t1, int slot) {
  constexpr int KC = DP / 32, VH = DP / 64, kBox = Smem<W, DP>::kBox, kRing = Smem<W, DP>::kRing;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int32_t* table = a.block_table + b * a.width;
  const int page_mask = (1 << a.page_shift) - 1;
  volatile int* abort = &sm->abort;

  int ids = -1, ids_at = -1;                  // page of the warp's tile ids_at + W * lane
  uint32_t bad = 0;                           // stages whose tile has no page
  // The first position of a tile in its table, the prefix's or the row's own.
  auto first_pos = [&](int tile) { return (tile < sp.pt ? tile : sp.t0 + tile - sp.pt) * kTile; };
  auto ask = [&](int tile) {
    if (ids_at < 0 || tile >= ids_at + 32 * W) {
      ids_at = tile;
      const int mine = tile + W * lane;
      ids = 0;
      if (mine < t1)
        ids = (mine < sp.pt ? a.prefix_table : table)[first_pos(mine) >> a.page_shift];
    }
    const int id = __shfl_sync(0xffffffffu, ids, (tile - ids_at) / W);
    const uint32_t st = ring.asked % kRing;
    const bool there = id >= 0 && id < a.pages;
    bad = there ? bad & ~(1u << st) : bad | 1u << st;
    if (lane == 0) {
      if (!there) report(a.status, ATTN_DEV_PAGE);   // page 0 is read and not used
      uint64_t* full = &sm->full[warp][st];
      uint8_t* dst = sm->ring[warp][st];
      const int at = first_pos(tile) & page_mask, page = there ? id : 0;
      tc::mbar_arrive_expect_tx(full, 2 * VH * kBox);
#pragma unroll
      for (int h = 0; h < VH; ++h) {
        tc::tma_load_4d(dst + h * kBox, tk, full, 64 * h, at, hk, page);
        tc::tma_load_4d(dst + (VH + h) * kBox, tv, full, 64 * h, at, hk, page);
      }
    }
    ++ring.asked;
  };
  int next = t0 + warp;                       // the next tile to ask for
  if (!__any_sync(0xffffffffu, *abort))
    for (int i = 0; i < kRing && next < t1; ++i, next += W) ask(next);

  uint4 qf[KC];
#pragma unroll
  for (int c = 0; c < KC; ++c) {
    const int d = 32 * c + 8 * t;
    qf[c] = g < nh && d < a.D
                ? *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + b * a.q_token +
                                                  (h0 + g) * a.q_head + d)
                : make_uint4(0, 0, 0, 0);
  }
  float o[VH][4][4];
#pragma unroll
  for (int h = 0; h < VH; ++h)
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[h][m][e] = 0.f;
  float m_ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // heads 2 t, 2 t + 1 (l: this lane's keys)

  // The products' key g is the tile's row g ^ 4 (g & 1) (and 8 more): rows of neighbouring g are then
  // four apart in the swizzle, and a quarter warp's reads of keys or values meet no bank twice.
  const int row_k = g ^ (g & 1) << 2;
  auto swizzled = [](int row, int c) { return row * 128 + ((c ^ (row & 7)) << 4); };
#pragma unroll 1
  for (int tile = t0 + warp; tile < t1; tile += W) {
    const uint32_t st = ring.taken % kRing;
    if (ring.taken == ring.asked) break;      // a wait ran out before
    const bool ok = tc::mbar_wait_short(&sm->full[warp][st], ring.taken / kRing & 1, abort);
    if (!__all_sync(0xffffffffu, ok)) break;
    ++ring.taken;
    const uint8_t* base = sm->ring[warp][st];
    const bool there = !(bad >> st & 1);
    float x[4] = {0.f, 0.f, 0.f, 0.f};        // keys of rows g, g, g + 8, g + 8, heads 2 t, 2 t + 1
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      const uint8_t* at = base + (c / 2) * kBox;
      const uint4 k0 = *reinterpret_cast<const uint4*>(at + swizzled(row_k, (c & 1) * 4 + t));
      const uint4 k1 = *reinterpret_cast<const uint4*>(at + swizzled(row_k + 8, (c & 1) * 4 + t));
      mma16816<T>(x, k0.x, k1.x, k0.y, k1.y, qf[c].x, qf[c].y);
      mma16816<T>(x, k0.z, k1.z, k0.w, k1.w, qf[c].z, qf[c].w);
    }
    uint4 vf[VH][4];
    const int row_v[4] = {2 * t, (2 * t + 1) ^ 4, 2 * t + 8, ((2 * t + 1) ^ 4) + 8};
#pragma unroll
    for (int h = 0; h < VH; ++h)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        vf[h][r] = *reinterpret_cast<const uint4*>(base + (VH + h) * kBox + swizzled(row_v[r], g));
    if (a.cap.on) {
      soft_cap(a.cap, x);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] *= a.c_score;
    }
    const int tile0 = first_pos(tile), lo = tile < sp.pt ? 0 : sp.lo;
    const int end = tile < sp.pt ? a.prefix_len : sp.n;
    if (tile0 < lo || tile0 > end - kTile || !there) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = tile0 + row_k + 8 * (e >> 1), mine = tile0 + row_v[e];
        if (key < lo || key >= end || !there) x[e] = -INFINITY;
        // an unused slot may hold anything, which a weight of 0 would still pass on
        if (mine < lo || mine >= end || !there) {
#pragma unroll
          for (int h = 0; h < VH; ++h) vf[h][e] = make_uint4(0, 0, 0, 0);
        }
      }
    }
    __syncwarp();                             // the stage has been read
    if (next < t1) {
      ask(next);
      next += W;
    }
    const float ref0 = m_ref[0] + kGrow<T>, ref1 = m_ref[1] + kGrow<T>;   // -inf stays -inf
    const float max0 = fmaxf(x[0], x[2]), max1 = fmaxf(x[1], x[3]);
    if (__any_sync(0xffffffffu, max0 > ref0 || max1 > ref1)) {
      const float ref[2] = {ref0, ref1};
      float top[2] = {max0, max1}, f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
        const float m_new = top[i] > ref[i] ? top[i] - kBias<T> : m_ref[i];
        f[i] = m_new == -INFINITY ? 1.0f : tc::ex2(m_ref[i] - m_new);
        m_ref[i] = m_new;
        l[i] *= f[i];
      }
#pragma unroll
      for (int h = 0; h < VH; ++h)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          o[h][m][0] *= f[0]; o[h][m][1] *= f[1];
          o[h][m][2] *= f[0]; o[h][m][3] *= f[1];
        }
    }
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[e] = tc::ex2(x[e] - (m_ref[e & 1] == -INFINITY ? 0.f : m_ref[e & 1]));
      l[e & 1] += p[e];
    }
    uint32_t hi[2], rest[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = Pair<T>::pack(p[2 * i], p[2 * i + 1]);
      const float2 r = unpack<T>(w);
      hi[i] = transpose8x8(w);
      rest[i] = transpose8x8(Pair<T>::pack(p[2 * i] - r.x, p[2 * i + 1] - r.y));
    }
#pragma unroll
    for (int h = 0; h < VH; ++h) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint32_t sel = m & 1 ? 0x7632u : 0x5410u;
        const int w = m / 2;
        auto word = [&](int r, int i) {
          const uint4& q4 = vf[h][r];
          return i == 0 ? q4.x : i == 1 ? q4.y : i == 2 ? q4.z : q4.w;
        };
        const uint32_t a0 = __byte_perm(word(0, w), word(1, w), sel);
        const uint32_t a1 = __byte_perm(word(0, 2 + w), word(1, 2 + w), sel);
        const uint32_t a2 = __byte_perm(word(2, w), word(3, w), sel);
        const uint32_t a3 = __byte_perm(word(2, 2 + w), word(3, 2 + w), sel);
        mma16816<T>(o[h][m], a0, a1, a2, a3, hi[0], hi[1]);
        mma16816<T>(o[h][m], a0, a1, a2, a3, rest[0], rest[1]);
      }
    }
  }
  // After a wait that ran out: copies still on their way land before the rings are used again.
  if (ring.taken != ring.asked) {
    for (; ring.taken != ring.asked; ++ring.taken)
      tc::mbar_drain(&sm->full[warp][ring.taken % kRing], ring.taken / kRing & 1);
    if (lane == 0) report(a.status, ATTN_DEV_TIMEOUT);
  }
  Merge<W, DP>* sh = &sm->merge;

  // The block's warps: weights, then dims.
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
  __syncthreads();                            // every warp is done with its ring
  if (g == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sh->m[warp][2 * t + i] = m_ref[i];
      sh->l[warp][2 * t + i] = l[i];
    }
  }
#pragma unroll
  for (int h = 0; h < VH; ++h)
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int d = 64 * h + 8 * g + m;
      sh->o[warp][2 * t][d] = o[h][m][0];
      sh->o[warp][2 * t + 1][d] = o[h][m][1];
      sh->o[warp][2 * t][d + 4] = o[h][m][2];
      sh->o[warp][2 * t + 1][d + 4] = o[h][m][3];
    }
  __syncthreads();
  const int d = 4 * lane;
#pragma unroll 1
  for (int h = warp; h < nh; h += W) {
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, sh->m[w][h]);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = sh->m[w][h] == -INFINITY ? 0.f : tc::ex2(sh->m[w][h] - top);
      const float4 p = d < DP ? *reinterpret_cast<const float4*>(&sh->o[w][h][d])
                              : make_float4(0.f, 0.f, 0.f, 0.f);
      sum = fmaf(f, sh->l[w][h], sum);
      y.x = fmaf(f, p.x, y.x); y.y = fmaf(f, p.y, y.y);
      y.z = fmaf(f, p.z, y.z); y.w = fmaf(f, p.w, y.w);
    }
    if (slot < 0) {
      finish_row<T, PRE>(a, b, h0 + h, d, y, top, sum);
      continue;
    }
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * kHeads + h;
    const float inv = top == -INFINITY ? 0.f : 1.0f / sum;
    if (d < a.D)
      *reinterpret_cast<float4*>(a.part_o + at * a.D + d) =
          make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
    if (lane == 0) a.part_ml[at] = make_float2(top, sum);
  }
}

// The rings' barriers; whole block.
template <int W, int DP>
__device__ __forceinline__ void init_rings(Smem<W, DP>* sm) {
  if (threadIdx.x < W * Smem<W, DP>::kRing) tc::mbar_init(&sm->full[0][0] + threadIdx.x, 1);
  if (threadIdx.x == 0) sm->abort = 0;
  tc::fence_mbar_init();
  __syncthreads();
}

// A row without any position of its own: zeros, or its prefix alone.
template <class T, bool PRE>
__device__ __noinline__ void empty_row(const DecodeArgs& a, int b) {
  for (int head = threadIdx.x / 32; head < a.H; head += blockDim.x / 32)
    finish_row<T, PRE>(a, b, head, 4 * (threadIdx.x & 31), make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f);
}

template <class S>
__device__ __forceinline__ S* aligned_smem(uint8_t* raw) {   // 1024 bytes: the swizzle's period
  return reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
}

// With the prefix's parts (PRE) the kernel before is the prefix's, which lets this one start only
// after its own wait, so all that came before it has ended. It writes nothing but those parts:
// rows of their own are read while it ends, and only what uses the parts waits for it (with the
// wait at the start, a prefix of 8192 and 64 rows of 1..500: 36.4 us for 34.1). Every block waits
// before it ends: who waits for this kernel has waited for the prefix's.

// One block per unit (row, kv head, group of up to 8 query heads).
template <class T, int W, int DP, bool PRE>
__global__ void __launch_bounds__(32 * W, W == warps_of(DP) ? resident_of(DP) : 1)
    decode_paged_units_kernel(const __grid_constant__ CUtensorMap tk,
                              const __grid_constant__ CUtensorMap tv, const DecodeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  auto* sm = aligned_smem<Smem<W, DP>>(smem_raw);
  if (threadIdx.x == 0) {
    tc::tma_prefetch(&tk);
    tc::tma_prefetch(&tv);
  }
  init_rings(sm);
  if (!PRE) dependent_wait();
  dependents_may_launch();
  if (gated_off(a.skip)) {
    if (PRE) dependent_wait();
    return;
  }
  const unsigned per_row = a.Hkv * a.HT;
  const int b = blockIdx.x / per_row, u = blockIdx.x % per_row;
  const Span sp = span_of(a, b);
  if (sp.n < 0) {
    if (threadIdx.x == 0) report(a.status, ATTN_DEV_LENGTH);
    if (PRE) dependent_wait();
    return;
  }
  if (sp.nt == 0) {
    if (u == 0) empty_row<T, PRE>(a, b);
    if (PRE) dependent_wait();
    return;
  }
  const int hk = u / a.HT, h0 = hk * a.G + (u % a.HT) * kHeads;
  Ring ring;
  segment<T, W, DP, PRE>(a, &tk, &tv, sm, ring, b, hk, h0, min(kHeads, (hk + 1) * a.G - h0), sp, 0,
                         sp.nt, -1);
  if (PRE) dependent_wait();
}

// prefix[b]: costs of a unit of each row before b; returns their total. Whole block of W warps.
template <int W>
__device__ unsigned scan_tiles(const DecodeArgs& a, unsigned* prefix, bool tell) {
  __shared__ unsigned warp_sum_of[W];
  __shared__ unsigned carry;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B; b0 += 32 * W) {
    const int b = b0 + threadIdx.x;
    unsigned n = 0;
    if (b < a.B) {
      const Span sp = span_of(a, b);
      if (sp.n < 0 && tell) report(a.status, ATTN_DEV_LENGTH);
      n = sp.nt > 0 ? kStart + sp.nt : 0;
    }
    unsigned s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    if (lane == 31) warp_sum_of[warp] = s;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += warp_sum_of[w];
    if (b < a.B) prefix[b] = before + s - n;
    if (threadIdx.x == 32 * W - 1) carry = before + s;
    __syncthreads();
    before = carry;
  }
  return before;
}

// Block i's share of a total cost begins at share_begin(i): the first total % blocks blocks have
// one more than the others.
__device__ __forceinline__ unsigned share_begin(unsigned total, unsigned blocks, unsigned i) {
  const unsigned q = total / blocks, r = total - q * blocks;
  return i * q + min(i, r);
}
__device__ __forceinline__ unsigned share_of(unsigned total, unsigned blocks, unsigned x) {
  const unsigned q = total / blocks, r = total - q * blocks, big = r * (q + 1);
  return x < big ? x / (q + 1) : r + (x - big) / q;   // q > 0 where x >= big
}

template <class T, int DP, bool PRE>
__global__ void __launch_bounds__(32 * warps_of(DP), resident_of(DP))
    decode_paged_share_kernel(const __grid_constant__ CUtensorMap tk,
                              const __grid_constant__ CUtensorMap tv, const DecodeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int W = warps_of(DP);
  auto* sm = aligned_smem<Smem<W, DP>>(smem_raw);
  unsigned* prefix = reinterpret_cast<unsigned*>(sm + 1);
  if (threadIdx.x == 0) {
    tc::tma_prefetch(&tk);
    tc::tma_prefetch(&tv);
  }
  init_rings(sm);
  if (!PRE) dependent_wait();
  dependents_may_launch();
  if (gated_off(a.skip)) {
    if (PRE) dependent_wait();
    return;
  }
  const unsigned per_row = a.Hkv * a.HT;
  const unsigned total = scan_tiles<W>(a, prefix, blockIdx.x == 0) * per_row;
  for (int b = blockIdx.x; b < a.B; b += a.blocks) {
    const Span sp = span_of(a, b);
    if (sp.n == 0 && sp.nt == 0) empty_row<T, PRE>(a, b);
  }
  Ring ring;
  unsigned x = share_begin(total, a.blocks, blockIdx.x);
  const unsigned end = share_begin(total, a.blocks, blockIdx.x + 1);
#pragma unroll 1
  while (x < end) {
    int b = 0, past = a.B;                    // the last row that begins at or before x
    while (past - b > 1) {
      const int mid = (b + past) / 2;
      if (prefix[mid] * per_row <= x) b = mid; else past = mid;
    }
    const Span sp = span_of(a, b);
    const unsigned cost = kStart + sp.nt, in_row = x - prefix[b] * per_row, u = in_row / cost;
    const unsigned c0 = in_row - u * cost, c1 = min(cost, c0 + (end - x));
    x += c1 - c0;
    if (c1 <= kStart) break;                  // the share ends before the unit's first tile
    const int t0 = c0 > kStart ? c0 - kStart : 0, t1 = c1 - kStart;
    const int hk = u / a.HT, h0 = hk * a.G + (u % a.HT) * kHeads;
    // Slot 0: a unit begun by an earlier block (the share's first); slot 1: one begun here and
    // continued by the next (its last).
    const int slot = t0 > 0 ? 0 : (t1 < sp.nt ? 1 : -1);
    segment<T, W, DP, PRE>(a, &tk, &tv, sm, ring, b, hk, h0, min(kHeads, (hk + 1) * a.G - h0), sp,
                           t0, t1, slot);
    tc::fence_proxy_async();                  // the merge's writes come before the next tiles
    __syncthreads();
  }
  if (PRE) dependent_wait();
}

// Joins the shares of a row and query head that several blocks had (nothing to do where one block
// finished it), and the prefix's parts. W warps each, taking every W-th share.
template <class T, int W, bool PRE>
__global__ void __launch_bounds__(256) decode_paged_join_kernel(const DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float4 rest_y[8][32];
  __shared__ float2 rest_ml[8];
  unsigned* prefix = reinterpret_cast<unsigned*>(smem);
  dependent_wait();
  dependents_may_launch();
  if (gated_off(a.skip)) return;
  const int lane = threadIdx.x & 31;
  const unsigned per_row = a.Hkv * a.HT;
  const unsigned total = scan_tiles<8>(a, prefix, false) * per_row;
  const int warp = threadIdx.x / 32, w = warp % W;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (8 / W) + warp / W;
  if (row >= static_cast<int64_t>(a.B) * a.H) return;   // with W = 8 all of a block or none
  const int b = row / a.H, head = row - static_cast<int64_t>(b) * a.H;
  const Span sp = span_of(a, b);
  if (sp.n < 0) return;
  const int hk = head / a.G, g = head - hk * a.G, h = g % kHeads;
  unsigned i0 = 0, own = 0;                   // first block, and how many had the unit
  if (sp.nt > 0) {
    const unsigned x0 = prefix[b] * per_row + (hk * a.HT + g / kHeads) * (kStart + sp.nt) + kStart;
    i0 = share_of(total, a.blocks, x0);
    own = share_of(total, a.blocks, x0 + sp.nt - 1) - i0 + 1;
  }
  if (own <= 1) return;                       // one block had it whole, or there is none
  const int d = 4 * lane;
  float top = -INFINITY, sum = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  add_parts(
      [&](unsigned i, const float2*& ml, const float*& o) {
        const unsigned p = w + W * i;
        const int64_t at = (static_cast<int64_t>(i0 + p) * 2 + (p == 0)) * kHeads + h;
        ml = a.part_ml + at;
        o = a.part_o + at * a.D;
      },
      w < own ? (own - w + W - 1) / W : 0, d, a.D, y, top, sum);
  if (W > 1) {
    rest_y[warp][lane] = y;
    if (lane == 0) rest_ml[warp] = make_float2(top, sum);
    __syncthreads();
    if (w > 0) return;
    const float2 ml = lane < W ? rest_ml[lane] : make_float2(-INFINITY, 0.f);
    top = warp_max(ml.x);
    const float f = ml.x == -INFINITY ? 0.f : tc::ex2(ml.x - top);
    sum = warp_sum(f * ml.y);
    y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
      const float4 p = rest_y[i][lane];
      y.x = fmaf(fi, p.x, y.x); y.y = fmaf(fi, p.y, y.y);
      y.z = fmaf(fi, p.z, y.z); y.w = fmaf(fi, p.w, y.w);
    }
  }
  finish_row<T, PRE>(a, b, head, d, y, top, sum);
}

// Shared memory past 48 KB is an attribute of the kernel in each device's context.
template <auto* Kernel>
cudaError_t allow_smem(size_t bytes) {
  static PerContext<cudaError_t> attr;
  return attr.get(
      [=] {
        return cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(bytes));
      },
      cudaErrorInvalidDevice, [](cudaError_t r) { return r == cudaSuccess; });
}

// A pool [pages, Hkv, page, D]: boxes of 64 dims x one tile.
bool map_tiles(CUtensorMap* m, const void* p, bool bf16, const DecodeArgs& a) {
  auto enc = prefill::encode_fn();
  if (!enc) return false;
  const cuuint64_t page = 1ull << a.page_shift;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.D), page, static_cast<cuuint64_t>(a.Hkv),
                              static_cast<cuuint64_t>(a.pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.D) * 2, page * a.D * 2,
                                 static_cast<cuuint64_t>(a.page_stride) * 2};
  const cuuint32_t box[4] = {64, kTile, 1, 1}, es[4] = {1, 1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int W, int DP, bool PRE>
cudaError_t launch_units(const DecodeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                         unsigned units, cudaStream_t stream) {
  constexpr size_t smem = sizeof(Smem<W, DP>) + 1024;
  const cudaError_t e = allow_smem<decode_paged_units_kernel<T, W, DP, PRE>>(smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(decode_paged_units_kernel<T, W, DP, PRE>, units, 32 * W, smem, stream, tk,
                          tv, a);
}

template <class T, int DP, bool PRE>
cudaError_t launch_dp(const DecodeArgs& a, int warps, cudaStream_t stream) {
  constexpr bool kBf16 = !std::is_same<T, __half>::value;
  CUtensorMap tk, tv;
  if (!map_tiles(&tk, a.k, kBf16, a) || !map_tiles(&tv, a.v, kBf16, a)) return cudaErrorInvalidValue;
  const unsigned units = static_cast<unsigned>(a.B) * a.Hkv * a.HT;
  cudaError_t e;
  size_t scan = 0;
  if (a.blocks == 0) {
    e = warps == wide_warps_of(DP)
            ? launch_units<T, wide_warps_of(DP), DP, PRE>(a, tk, tv, units, stream)
            : launch_units<T, warps_of(DP), DP, PRE>(a, tk, tv, units, stream);
  } else {
    constexpr int W = warps_of(DP);
    constexpr size_t smem = sizeof(Smem<W, DP>) + 1024;
    scan = static_cast<size_t>(a.B) * sizeof(unsigned);
    e = allow_smem<decode_paged_share_kernel<T, DP, PRE>>(smem + kMaxScanRows * sizeof(unsigned));
    if (e == cudaSuccess)
      e = launch_dependent(decode_paged_share_kernel<T, DP, PRE>, a.blocks, 32 * W, smem + scan,
                           stream, tk, tv, a);
  }
  if (e != cudaSuccess || a.blocks == 0) return e;
  // A unit's shares, about: past a dozen a row gets a block of its own.
  const int64_t rows = static_cast<int64_t>(a.B) * a.H;
  const bool wide = a.blocks / units > 12;
  return wide ? launch_dependent(decode_paged_join_kernel<T, 8, PRE>, static_cast<unsigned>(rows), 256,
                                 scan, stream, a)
              : launch_dependent(decode_paged_join_kernel<T, 1, PRE>,
                                 static_cast<unsigned>((rows + 7) / 8), 256, scan, stream, a);
}

}  // namespace

namespace {
template <class T>
cudaError_t launch_type(const DecodeArgs& a, int warps, cudaStream_t stream) {
  if (a.D <= 64)
    return a.prefix.nsplit ? launch_dp<T, 64, true>(a, warps, stream)
                           : launch_dp<T, 64, false>(a, warps, stream);
  return a.prefix.nsplit ? launch_dp<T, 128, true>(a, warps, stream)
                         : launch_dp<T, 128, false>(a, warps, stream);
}
}  // namespace

// One block per unit where no row can have more than 16 tiles a warp (8, in a block twice as wide,
// where that leaves each block an SM of its own), or 32 where there are units for every place; else
// blocks that share all tiles. Measured, 4 heads of 128 a kv head, 8 kv heads, us with a block a unit
// and shared out: one row of 500 slots 6.8, 9.7; of 1000 10.3, 11; of 2000 17, 11.1. 24 rows of 1000
// 18, 19.2; of 1..2000 26.9, 17.2. 64 rows of 1..1000 27.9, 30.8; of 1..2000 48.6, 51.5; 256 of those
// 148, 167. Heads of 64: 64 rows of 1..2000 29, 33; 23 rows of 1..5000 30, 21.
namespace {
struct PlanSizes {
  int64_t units, tiles, places, shares;       // (shares: blocks, where tiles are shared)
};
PlanSizes plan_sizes(int B, int H, int Hkv, int D, int max_len, int window, int prefix_len) {
  const int G = H / Hkv;
  const int64_t own = window > 0 && window < max_len ? window + kTile - 1 : max_len;
  PlanSizes s;
  s.units = static_cast<int64_t>(B) * Hkv * ((G + kHeads - 1) / kHeads);
  s.tiles = (own + kTile - 1) / kTile + (prefix_len + kTile - 1) / kTile;
  s.places = kSms * resident_of(D);
  s.shares = std::min((s.units * s.tiles + warps_of(D) - 1) / warps_of(D), s.places);
  return s;
}
}  // namespace

DecodePagedPlan decode_paged_plan(int B, int H, int Hkv, int D, int max_len, int window,
                                  int prefix_len) {
  const PlanSizes s = plan_sizes(B, H, Hkv, D, max_len, window, prefix_len);
  const int warps = warps_of(D), wide = wide_warps_of(D);
  if (s.tiles <= 8 * wide && s.units <= kSms) return {0, wide};
  if (s.tiles <= (s.units >= s.places ? 32 : 16) * warps || B > kMaxScanRows) return {0, warps};
  return {static_cast<int>(s.shares), warps};
}

// The partial results of the blocks' shares (part_ml follows part_o). Never shrinks as max_len or B
// grows, so it counts shares for batches that would do without too.
size_t decode_paged_bytes(int B, int H, int Hkv, int D, int max_len, int window, int prefix_len) {
  const PlanSizes s = plan_sizes(B, H, Hkv, D, max_len, window, prefix_len);
  if (s.tiles <= 16 * warps_of(D)) return 0;
  return static_cast<size_t>(s.shares) * 2 * kHeads * (D + 2) * sizeof(float);
}

cudaError_t launch_decode_paged(const DecodePagedJob& j, cudaStream_t stream) {
  DecodeArgs a{};
  a.q = j.q.p; a.q_token = j.q.token; a.q_head = j.q.head;
  a.out = j.out.p; a.o_token = j.out.token; a.o_head = j.out.head;
  a.k = j.cache.k; a.v = j.cache.v;
  a.page_stride = j.cache.page_stride;
  a.pages = j.cache.pages; a.page_shift = j.cache.page_shift;
  a.block_table = j.block_table; a.width = j.width;
  a.cache_len = j.cache_len; a.max_len = j.max_len;
  a.B = j.B; a.H = j.H; a.Hkv = j.Hkv; a.D = j.D;
  a.G = j.H / j.Hkv; a.HT = (a.G + kHeads - 1) / kHeads;
  a.window = j.window;
  a.c_score = j.scale * kLog2e16;
  a.cap = cap_args(j.softcap, j.scale);
  a.prefix_table = j.prefix_table;
  a.prefix_len = j.prefix_len;
  a.prefix = j.prefix;
  const DecodePagedPlan plan =
      decode_paged_plan(j.B, j.H, j.Hkv, j.D, j.max_len, j.window, j.prefix_len);
  // Shares are counted in 32 bits: rows that share pages could have more tiles than that.
  const int64_t most = (static_cast<int64_t>(j.max_len) + j.prefix_len) / kTile + 2 + kStart;
  a.blocks = static_cast<int64_t>(j.B) * j.Hkv * a.HT * most < (int64_t(1) << 32) ? plan.blocks : 0;
  a.part_o = j.partial;
  a.part_ml = reinterpret_cast<float2*>(j.partial + static_cast<size_t>(a.blocks) * 2 * kHeads * j.D);
  a.status = j.status; a.skip = j.skip;
  return j.bf16 ? launch_type<__nv_bfloat16>(a, plan.warps, stream)
                : launch_type<__half>(a, plan.warps, stream);
}

}  // namespace gqa
