// Attention on the tensor cores in 16 bits ("Core Layers -- Deep Reference", "Flash Attention",
// "MHA and GQA"): the whole prompts of a packed batch, causal or windowed; and the part of a
// batch's single-token attention that falls on a prefix all rows share.
//
//   S = Q K^T,  P = 2^(c cap(S) - m),  O = sum P V,  l = sum P,  out = O / l
//
// over blocks of 128 keys with a running reference m per query row; products of 16-bit operands
// with fp32 accumulation, softmax and sums in fp32, P rounded once to 16 bits for the second
// product (half a step of the type, the size of the output's own rounding).
//
// How, on GB300:
//  * A tile is 128 rows: TQ = 128 / G tokens x the G query heads of one kv head, which share
//    every key, value and almost all of the mask. A block works on two tiles at once (tokens
//    t0 .. t0 + TQ - 1 and the TQ after): while one tile's softmax runs, the tensor core does
//    the other's products, and both read each K and V block once.
//  * TMA brings Q tiles (boxes of 64 dims x G heads x TQ tokens), K and V blocks (128 keys; from
//    pages, box by page) through one ring of stages in the 128-byte swizzle. V is the
//    MN-major operand of the second product as it lies: no transposition.
//  * Tensor memory: S0 | S1 (128 fp32 columns each), O0 | O1. P overwrites S's first half in
//    16 bits and is the A operand of O += P V.
//  * One warp issues all products, in the order P V (tile 0), next S (tile 0), P V (tile 1),
//    next S (tile 1): the tensor pipe runs them in that order, so S may be written over the
//    P before it without a wait.
//  * Softmax: a thread per row, 4 warps per tile. The reference is the row's first maximum and stands until a half's sum shows that some weight exceeded
//    2^8 (then the half is redone against a new maximum and O rescaled): no maximum is
//    taken in the common case.
//  * Values behind the last key (another sequence's, an unused slot's) are zeroed in shared memory:
//    whatever lies there, NaNs included, has no part in the result.
//  * Every wait is bounded; one that runs out raises ATTN_DEV_TIMEOUT and the block winds down.
#pragma once

#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "prefill_common.cuh"

namespace gqa {
namespace attn16 {

using prefill::drain_wait;
using prefill::kRescaleLog2;
using prefill::kSmemLimit;
using prefill::kTmemCols;

constexpr int kBK = 128;                       // keys per block
constexpr int kRows = 128;                     // query rows per tile

struct Args {
  int T, B, max_len;                           // packed prompts
  const int32_t* cu;
  const int32_t* prefix_table;                 // shared prefix
  int prefix_len, pages, page_shift;
  int H, Hkv, D, G, TQ;
  int units, splits, split_keys;               // shared: pairs of tiles, splits of the key blocks
  int window, softcap_on;
  float c_score, c_cap_in, c_cap_out;          // log2 units
  void* out;
  int64_t o_token, o_head;
  float* part_o;
  float2* part_ml;
  int32_t* status;
  const int32_t* skip;
};

template <class T_, int DP_, bool SHARED_>
struct Cfg {
  using T = T_;
  static constexpr int DP = DP_;               // head dim padded to whole 64-dim chunks
  static constexpr bool SHARED = SHARED_;
  static constexpr bool BF16 = sizeof(T) == 2 && !std::is_same<T, __half>::value;
  static constexpr int kChunks = DP / 64;
  static constexpr int kChunk = 128 * 128;     // 128 rows x 64 dims (128 bytes)
  static constexpr int kTileBytes = kChunks * kChunk;   // a Q tile, a K block or a V block
  static constexpr int kNSraw = (kSmemLimit - 2048 - 2 * kTileBytes) / kTileBytes;
  static constexpr int NS = kNSraw > 8 ? 8 : kNSraw;
  static constexpr int kSmem = (NS + 2) * kTileBytes + 2048;
  static constexpr int kSCol = 0, kOCol = 256;
  // fp16 has few small numbers and P's range is [0, 2^(8 + kBias)]: shifted up, weights down
  // to 2^-21 of the largest keep all their bits.
  static constexpr float kBias = BF16 ? 0.f : 7.f;
};
// 2 x 4 softmax warps; producer, products and two idle warps. The block starts with 168
// registers a thread; a row's 128 scores take more, so the last four warps hand theirs on.
constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "the block's registers");

struct Bars {
  uint64_t unit_full[2], unit_empty[2];
  uint64_t q_full, q_empty;
  uint64_t kv_full[8], kv_empty[8];
  uint64_t s_full[2];
  uint64_t p_ready[2][2];                      // [tile][half]
  uint64_t o_half[2], o_done[2], o_free[2];
  uint64_t v_fixed;                            // the last block's V is zeroed behind the last key
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  struct {
    int hk, row0, q0, ntok, kbase, nk, jlo, jhi, nt, la, part;   // nt 0: no more units
  } unit[2];
};
using Unit = std::remove_extent<decltype(Bars::unit)>::type;

// The block's r-th unit, read by a consumer (count of unit_empty: the products' thread and
// one lane of each softmax warp).
__device__ __forceinline__ bool next_unit(Bars* bars, uint32_t r, Unit& u) {
  if (!tc::mbar_wait(&bars->unit_full[r & 1], (r >> 1) & 1, &bars->abort)) return false;
  u = bars->unit[r & 1];
  return u.nt > 0;
}

// Tile t's key blocks [lo, hi] of the unit's (la 2: every other one of them, from jlo + t).
template <class C>
__device__ __forceinline__ void tile_blocks(const Args& a, const Unit& u, int t, int& lo, int& hi) {
  lo = u.jlo;
  hi = u.jhi;
  if (u.la == 1 && t >= u.nt) {
    hi = lo - 1;
  } else if (!C::SHARED) {
    const int first = u.q0 + t * a.TQ, last = min(first + a.TQ, u.q0 + u.ntok) - 1;
    lo = a.window > 0 ? max(0, first - a.window + 1) / kBK : 0;
    hi = last / kBK;
  }
}

// ---------------------------------------------------------------- producer (one warp)
// The blocks walk one list of units, heaviest first, in snake order: unit x of round r for block c.
__device__ __forceinline__ unsigned unit_at(unsigned c, unsigned r, unsigned blocks) {
  return r * blocks + ((r & 1) ? blocks - 1 - c : c);
}

// Tiles (of 2 TQ tokens) of sequence b; 0 where its bounds break a rule.
__device__ __forceinline__ int seq_tiles(const Args& a, int b, bool tell) {
  const SeqRows s = seq_rows(a.cu, b, a.T);
  if (s.n < 0 || s.n > a.max_len) {
    if (tell) report(a.status, ATTN_DEV_LENGTH);
    return 0;
  }
  return (s.n + 2 * a.TQ - 1) / (2 * a.TQ);
}

// Tiles of all sequences with index >= i (whole warp; cu_seqlens stays in L1).
__device__ __forceinline__ int tiles_from(const Args& a, int i, bool tell) {
  int n = 0;
  for (int b = threadIdx.x & 31; b < a.B; b += 32) n += max(0, seq_tiles(a, b, tell) - i);
  return __reduce_add_sync(0xffffffffu, n);
}

// Unit x of the list; false past its end. Whole warp. Packed prompts: tiles by their index within
// their sequence, last first (a tile's keys grow with it), the kv heads of a tile side by
// side. `top`: no tile of index top or above is left (kept from unit to unit).
template <class C>
__device__ bool find_unit(const Args& a, unsigned x, int& top, Unit& u) {
  u.hk = x % a.Hkv;
  const int y = x / a.Hkv, tokens = 2 * a.TQ;
  if (C::SHARED) {
    const int pair = y / a.splits, blocks = (a.prefix_len + kBK - 1) / kBK;
    if (pair >= a.units) return false;
    u.part = y % a.splits;
    u.row0 = pair * tokens;
    u.q0 = 0;
    u.ntok = min(tokens, a.B - u.row0);
    u.kbase = 0;
    u.nk = a.prefix_len;
    u.jlo = static_cast<int>(static_cast<int64_t>(u.part) * blocks / a.splits);
    u.jhi = static_cast<int>(static_cast<int64_t>(u.part + 1) * blocks / a.splits) - 1;
    u.nt = u.ntok > a.TQ ? 2 : 1;
    u.la = a.split_keys ? 2 : 1;
    return true;
  }
  // The largest index i < top with more than y tiles of index >= i.
  if (tiles_from(a, 0, false) <= y) return false;
  int lo = 0, hi = top;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (tiles_from(a, mid, false) > y) lo = mid; else hi = mid;
  }
  top = lo + 1;
  int k = y - tiles_from(a, lo + 1, false);    // among the sequences that have a tile lo
  int b = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int mine = b0 + (threadIdx.x & 31);
    const bool has = mine < a.B && seq_tiles(a, mine, false) > lo;
    const uint32_t all = __ballot_sync(0xffffffffu, has);
    if (k < __popc(all)) {                     // the lane with k others before it
      const int before = __popc(all & ((1u << (threadIdx.x & 31)) - 1));
      b = b0 + __ffs(__ballot_sync(0xffffffffu, has && before == k)) - 1;
      break;
    }
    k -= __popc(all);
  }
  const SeqRows s = seq_rows(a.cu, b, a.T);
  u.q0 = lo * tokens;
  u.ntok = min(tokens, s.n - u.q0);
  u.row0 = s.first + u.q0;
  u.kbase = s.first;
  u.nk = s.n;
  u.nt = u.ntok > a.TQ ? 2 : 1;
  u.la = 1;
  u.part = 0;
  u.jlo = a.window > 0 ? max(0, u.q0 - a.window + 1) / kBK : 0;
  u.jhi = (u.q0 + u.ntok - 1) / kBK;
  return true;
}

// Finds the block's units, publishes each and loads it. The next one's search and loads run while
// the products are still at this one's.
template <class C>
__device__ void producer(const Args& a, const CUtensorMap* tq, const CUtensorMap* tk,
                         const CUtensorMap* tv, uint8_t* sq, uint8_t* skv, Bars* bars, int lane) {
  volatile int* abort = &bars->abort;
  int stage = 0;
  uint32_t phase = 0, loaded = 0;              // loads so far
  uint32_t units = 0;
  Unit u{};
  // The last block of a sequence may hold fewer than 128 keys: its V is zeroed behind them.
  auto load = [&](bool is_v, int j) -> bool {
    bool ok = true;
    uint64_t* full = &bars->kv_full[stage];
    uint8_t* dst = skv + stage * C::kTileBytes;
    int rows = kBK, id = 0;
    const int page = 1 << a.page_shift, box = min(page, kBK);
    if (C::SHARED) {
      // one lane per page of the block
      const int n = min(kBK, u.nk - j * kBK), boxes = (n + box - 1) / box;
      if (lane < boxes) {
        id = a.prefix_table[(static_cast<int64_t>(j) * kBK + lane * box) >> a.page_shift];
        if (id < 0 || id >= a.pages) {
          report(a.status, ATTN_DEV_PAGE);
          id = -1;
        }
      }
      rows = boxes * box;
    }
    if (lane == 0) ok = tc::mbar_wait(&bars->kv_empty[stage], phase ^ 1u, abort);
    if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
    const CUtensorMap* map = is_v ? tv : tk;
    if (C::SHARED) {
      // A page that does not exist is read as page 0 (the result is without meaning).
      if (lane == 0) tc::mbar_arrive_expect_tx(full, C::kChunks * 128 * rows);
      __syncwarp();
      if (lane < rows / box) {
        const int at = (j * kBK + lane * box) & (page - 1);
        for (int c = 0; c < C::kChunks; ++c)
          tc::tma_load_4d(dst + c * C::kChunk + lane * box * 128, map, full, 64 * c, at, u.hk,
                          max(id, 0));
      }
    } else if (lane == 0) {
      tc::mbar_arrive_expect_tx(full, C::kTileBytes);
      for (int c = 0; c < C::kChunks; ++c)
        tc::tma_load_3d(dst + c * C::kChunk, map, full, 64 * c, u.hk, u.kbase + j * kBK);
    }
    ++loaded;
    const int last_keys = u.nk - j * kBK;
    if (is_v && last_keys < kBK) {
      ok = tc::mbar_wait(full, phase, abort);
      if (!__all_sync(0xffffffffu, ok)) return false;
      for (int e = lane; e < (kBK - last_keys) * 8 * C::kChunks; e += 32) {
        const int c = e / ((kBK - last_keys) * 8), r = e % ((kBK - last_keys) * 8);
        *reinterpret_cast<uint4*>(dst + c * C::kChunk + last_keys * 128 + r * 16) =
            make_uint4(0, 0, 0, 0);
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->v_fixed);
    }
    if (++stage == C::NS) {
      stage = 0;
      phase ^= 1u;
    }
    return true;
  };
  auto publish = [&]() -> bool {               // u, as the units-th
    bool ok = true;
    if (lane == 0) {
      ok = tc::mbar_wait(&bars->unit_empty[units & 1], ((units >> 1) & 1) ^ 1u, abort);
      if (ok) {
        bars->unit[units & 1] = u;
        tc::mbar_arrive(&bars->unit_full[units & 1]);
      }
    }
    return __shfl_sync(0xffffffffu, ok, 0);
  };
  bool ok = true;
  int top = 0x7fffffff;
  if (!C::SHARED) {
    int most = 0;
    for (int b = lane; b < a.B; b += 32) most = max(most, seq_tiles(a, b, blockIdx.x == 0));
    top = __reduce_max_sync(0xffffffffu, most);
  }
  while (ok) {
    if (!find_unit<C>(a, unit_at(blockIdx.x, units, gridDim.x), top, u)) {
      u.nt = 0;
      publish();
      break;
    }
    if (!(ok = publish())) break;
    if (lane == 0) {
      const int tiles = u.la == 2 ? 1 : u.nt;
      ok = tc::mbar_wait(&bars->q_empty, (units & 1) ^ 1u, abort);
      if (ok) {
        tc::mbar_arrive_expect_tx(&bars->q_full, tiles * C::kChunks * 128 * a.G * a.TQ);
        for (int t = 0; t < tiles; ++t)
          for (int c = 0; c < C::kChunks; ++c)
            tc::tma_load_3d(sq + t * C::kTileBytes + c * C::kChunk, tq, &bars->q_full, 64 * c,
                            u.hk * a.G, u.row0 + t * a.TQ);
      }
    }
    if (!(ok = __shfl_sync(0xffffffffu, ok, 0))) break;
    ++units;
    for (int e = 0; ok && e < u.la && u.jlo + e <= u.jhi; ++e) ok = load(false, u.jlo + e);
    for (int j = u.jlo; ok && j <= u.jhi; ++j) {
      ok = load(true, j);
      if (ok && j + u.la <= u.jhi) ok = load(false, j + u.la);
    }
  }
  // Every copy this block started lands before the block may exit.
  if (lane == 0) {
    if (units > 0) drain_wait(&bars->q_full, (units - 1) & 1);
    for (uint32_t s = 0; s < C::NS && s < loaded; ++s) {
      const uint32_t fill = (loaded - 1 - s) / C::NS;   // the last load into stage s
      drain_wait(&bars->kv_full[s], fill & 1);
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------- products (one warp, one lane issues)
// The tensor pipe takes a product every 64 cycles, so the warp that issues them has to be lean: it
// stays converged with every operand the same in all lanes (uniform registers), its loops over
// a block's products are unrolled, and where a wait runs out it goes on (on data that is then
// without meaning, all of it this block's) to the block's end, where the warp leaves together.
template <class C>
__device__ void products(const Args& a, uint32_t tmem, uint8_t* sq, uint8_t* skv, Bars* bars) {
  volatile int* abort = &bars->abort;
  constexpr uint32_t id_s = tc::idesc_f16(kRows, kBK, C::BF16, false);
  constexpr uint32_t id_o = tc::idesc_f16(kRows, C::DP, C::BF16, true);
  const uint64_t qd = tc::sdesc_sw128(tc::smem_u32(sq), 16, 1024);
  const uint64_t kd = tc::sdesc_sw128(tc::smem_u32(skv), 16, 1024);
  // V [keys][dims], dims contiguous: the next 64 dims are a chunk away, the next 8 keys 1024 bytes
  const uint64_t vd = tc::sdesc_sw128(tc::smem_u32(skv), C::kChunk, 1024);
  uint32_t stage = 0, phase = 0, fixed = 0;
  uint32_t done[2] = {0, 0}, outputs[2] = {0, 0};   // blocks, and units, of each tile so far
  bool bad = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) { bad |= !tc::mbar_wait(bar, parity, abort); };
  auto take = [&]() -> uint32_t {
    wait(&bars->kv_full[stage], phase);
    const uint32_t st = stage;
    if (++stage == C::NS) {
      stage = 0;
      phase ^= 1u;
    }
    return st;
  };
  for (uint32_t r = 0;; ++r) {
    Unit u;
    if (!__all_sync(0xffffffffu, next_unit(bars, r, u))) break;
    if (threadIdx.x % 32 == 0) tc::mbar_arrive(&bars->unit_empty[r & 1]);
    const int la = __shfl_sync(0xffffffffu, u.la, 0), nk = __shfl_sync(0xffffffffu, u.nk, 0);
    const int jlo = __shfl_sync(0xffffffffu, u.jlo, 0), jhi = __shfl_sync(0xffffffffu, u.jhi, 0);
    int lo[2], hi[2];                          // each tile's blocks
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      int l = 0, h = 0;
      tile_blocks<C>(a, u, t, l, h);
      lo[t] = __shfl_sync(0xffffffffu, l, 0);
      hi[t] = __shfl_sync(0xffffffffu, h, 0);
    }
    auto active = [&](int t, int j) { return j >= lo[t] && j <= hi[t] && (la == 1 || ((j - jlo) & 1) == t); };
    auto scores = [&](int t, uint32_t st) {
      const uint64_t q = qd + ((la == 2 ? 0 : t) * C::kTileBytes >> 4);
      const uint64_t k = kd + (st * C::kTileBytes >> 4);
#pragma unroll
      for (int s = 0; s < C::DP / 16; ++s) {
        const uint32_t off = ((s >> 2) * C::kChunk + (s & 3) * 32) >> 4;
        tc::mma_f16_ss(tmem + C::kSCol + t * kBK, q + off, k + off, id_s, s > 0);
      }
      tc::mma_commit_warp(&bars->s_full[t]);
    };
    wait(&bars->q_full, r & 1);
    for (int e = 0; e < la && jlo + e <= jhi; ++e) {
      const uint32_t st = take();
      tc::fence_after_sync();
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (active(t, jlo + e)) scores(t, st);
      tc::mma_commit_warp(&bars->kv_empty[st]);
    }
    if (jlo + la > jhi) tc::mma_commit_warp(&bars->q_empty);
    for (int j = jlo; j <= jhi; ++j) {
      const uint32_t vs = take();
      const bool next = j + la <= jhi;
      uint32_t ks = 0;
      if (next) ks = take();
      if (nk - j * kBK < kBK) wait(&bars->v_fixed, fixed++ & 1);
      const uint64_t v = vd + (vs * C::kTileBytes >> 4);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (active(t, j)) {
          const bool first = la == 2 ? j - jlo == t : j == lo[t];
          if (first) {
            if (outputs[t] > 0) wait(&bars->o_free[t], (outputs[t] - 1) & 1);
            ++outputs[t];
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            wait(&bars->p_ready[t][h], done[t] & 1);
            tc::fence_after_sync();
#pragma unroll
            for (int s = 4 * h; s < 4 * h + 4; ++s)
              tc::mma_f16_ts(tmem + C::kOCol + t * C::DP, tmem + C::kSCol + t * kBK + 8 * s,
                             v + (s * 2048 >> 4), id_o, (!first || s > 0) ? 1u : 0u);
            if (h == 0) tc::mma_commit_warp(&bars->o_half[t]);
          }
          tc::mma_commit_warp(&bars->o_done[t]);
          ++done[t];
        }
        if (next && active(t, j + la)) scores(t, ks);
      }
      tc::mma_commit_warp(&bars->kv_empty[vs]);
      if (next) tc::mma_commit_warp(&bars->kv_empty[ks]);
      if (j + la == jhi) tc::mma_commit_warp(&bars->q_empty);   // the unit's last S
      if (__any_sync(0xffffffffu, bad)) break;
    }
    if (__any_sync(0xffffffffu, bad)) break;
  }
  tc::mma_commit_warp(&bars->drain);           // nothing may still run when the block frees its TMEM
  drain_wait(&bars->drain, 0);
}

// ---------------------------------------------------------------- softmax (4 warps a tile)
template <class C>
__device__ bool softmax(const Args& a, const Unit& u, uint32_t tmem, Bars* bars, int t, int quarter,
                        int lane, uint32_t& n) {
  using T = typename C::T;
  volatile int* abort = &bars->abort;
  const uint32_t n0 = n;                       // this tile's blocks before this unit
  const int row = quarter * 32 + lane, tok = row / a.G, head = u.hk * a.G + row % a.G;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const int tile = C::SHARED && u.la == 2 ? 0 : t;
  const int local = tile * a.TQ + tok;         // token of the unit
  const bool live = tok < a.TQ && local < u.ntok;
  const int qpos = u.q0 + local;
  const float cs = a.softcap_on ? 1.0f : a.c_score;
  constexpr float kLimit = C::BF16 ? 256.0f : 32768.0f;   // 2^(8 + kBias)
  float m_ref = -INFINITY, l = 0.f;            // P = 2^(score - m_ref) with the bias inside m_ref
  // The warp's rows' first and last visible keys are ordered as their tokens are.
  const int tok0 = 32 * quarter / a.G, tok1 = min((32 * quarter + 31) / a.G, a.TQ - 1);
  const int q_lo = u.q0 + tile * a.TQ + tok0, q_hi = u.q0 + tile * a.TQ + tok1;
  int j_lo, j_hi;
  tile_blocks<C>(a, u, t, j_lo, j_hi);
  bool ok = true, started = false;             // started: every live row has a reference
  for (int j = u.la == 2 ? j_lo + t : j_lo; j <= j_hi; j += u.la) {
    ok = tc::mbar_wait(&bars->s_full[t], n & 1, abort);
    if (__any_sync(0xffffffffu, !ok)) {        // leave together: tcgen05.ld is warp-wide
      ok = false;
      break;
    }
    tc::fence_after_sync();
    const uint32_t scol = lane_base + C::kSCol + t * kBK;
    float s[128];
    tc::tmem_ld128(scol, s);
    const int k0 = j * kBK;
    if (a.softcap_on) {
#pragma unroll
      for (int c = 0; c < 128; ++c) {
        const float e = tc::ex2(s[c] * a.c_cap_in);
        s[c] = fmaf(-2.0f * a.c_cap_out, tc::rcp(e + 1.0f), a.c_cap_out);
      }
    }
    // Blocks that the mask crosses: keys c <= hi and c >= lo are visible.
    if (k0 + kBK > u.nk || (!C::SHARED && (k0 + kBK - 1 > q_lo ||
                                           (a.window > 0 && k0 < q_hi - a.window + 1)))) {
      const int hi = (C::SHARED ? u.nk - 1 : min(qpos, u.nk - 1)) - k0;
      const int lo = !C::SHARED && a.window > 0 ? qpos - a.window + 1 - k0 : 0;
#pragma unroll
      for (int c = 0; c < 128; ++c) s[c] = c > hi || c < lo ? -INFINITY : s[c];
    }
    // P in two halves of 64 columns, each released to the products as soon as it is written.
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      uint32_t p[32];
      float lsum;
      bool slow = !started;
#pragma unroll 1
      while (true) {
        if (slow) {                            // a new reference from this half's maximum
          const float m_new = fmaxf(m_ref, fmaf(prefill::tq_max<64>(s + 64 * hh), cs, -C::kBias));
          const bool grow = m_ref != -INFINITY && m_new - m_ref > kRescaleLog2;
          if (__any_sync(0xffffffffu, grow)) {
            if (n > n0 || hh > 0) {            // once every product that wrote O is done
              ok = hh == 0 ? tc::mbar_wait(&bars->o_done[t], (n - 1) & 1, abort)
                           : tc::mbar_wait(&bars->o_half[t], n & 1, abort);
              if (__any_sync(0xffffffffu, !ok)) {
                ok = false;
                break;
              }
              tc::fence_after_sync();
              const float f = grow ? tc::ex2(m_ref - m_new) : 1.0f;
#pragma unroll 1
              for (int c = 0; c < C::DP; c += 16) {
                float o[16];
                tc::tmem_ld16(lane_base + C::kOCol + t * C::DP + c, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= f;
                tc::tmem_st16(lane_base + C::kOCol + t * C::DP + c, o);
              }
              l *= f;
            }
            if (grow) m_ref = m_new;
          }
          if (m_ref == -INFINITY) m_ref = m_new;
        }
        // -inf only while every key so far was masked; then every score is -inf
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        const uint64_t c2 = tc::pack2(cs, cs), m2 = tc::pack2(-m_use, -m_use);
        uint64_t acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = tc::pack2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          float x0, x1;
          tc::unpack2(tc::fma2(tc::pack2(s[64 * hh + c], s[64 * hh + c + 1]), c2, m2), x0, x1);
          x0 = tc::ex2(x0);
          x1 = tc::ex2(x1);
          p[c / 2] = Pair<T>::pack(x0, x1);
          acc[(c / 2) % 4] = tc::add2(acc[(c / 2) % 4], tc::pack2(x0, x1));
        }
        float a0, a1;
        tc::unpack2(tc::add2(tc::add2(acc[0], acc[1]), tc::add2(acc[2], acc[3])), a0, a1);
        lsum = a0 + a1;
        if (slow || !__any_sync(0xffffffffu, live && !(lsum <= kLimit))) break;
        slow = true;
      }
      if (!ok) break;
      l += lsum;
      tc::tmem_st32(scol + 32 * hh, reinterpret_cast<const float*>(p));
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->p_ready[t][hh]);
      if (!started && hh == 1) started = !__any_sync(0xffffffffu, live && m_ref == -INFINITY);
    }
    if (!ok) break;
    ++n;
  }
  if (!ok) return false;

  const bool has = n > n0;                     // the tile had blocks: its O waits to be read
  if (has) {
    ok = tc::mbar_wait(&bars->o_done[t], (n - 1) & 1, abort);
    if (__any_sync(0xffffffffu, !ok || *abort)) return false;
    tc::fence_after_sync();
  }
  const bool any = has && m_ref != -INFINITY;
  const float inv = any ? 1.0f / l : 0.f;
  if constexpr (C::SHARED) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.H;
    const int part = u.la == 2 ? 2 * u.part + t : u.part;
    if (u.la == 1 && t >= u.nt) return true;
    const int64_t at = part * rows + static_cast<int64_t>(u.row0 + local) * a.H + head;
    if (live) a.part_ml[at] = make_float2(any ? m_ref : -INFINITY, any ? l : 0.f);
#pragma unroll 1
    for (int c = 0; c < C::DP; c += 32) {
      float o[32];
      if (has) tc::tmem_ld32(lane_base + C::kOCol + t * C::DP + c, o);
      float* dst = a.part_o + at * a.D + c;
#pragma unroll
      for (int e = 0; e < 32; e += 4)
        if (live && c + e < a.D)
          *reinterpret_cast<float4*>(dst + e) =
              any ? make_float4(o[e] * inv, o[e + 1] * inv, o[e + 2] * inv, o[e + 3] * inv)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  } else {
    if (t >= u.nt) return true;
    T* dst = static_cast<T*>(a.out) + (u.row0 + local) * a.o_token + head * a.o_head;
#pragma unroll 1
    for (int c = 0; c < C::DP; c += 32) {
      float o[32];
      tc::tmem_ld32(lane_base + C::kOCol + t * C::DP + c, o);
#pragma unroll
      for (int e = 0; e < 32; e += 8)
        if (live && c + e < a.D) {
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = o[e + i] * inv;
          *reinterpret_cast<uint4*>(dst + c + e) = pack8<T>(x);
        }
    }
  }
  if (has) {
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&bars->o_free[t]);
  }
  return true;
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
    attn16_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const Args a) {
  dependent_wait();
  if (gated_off(a.skip)) return;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sq = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint8_t* skv = sq + 2 * C::kTileBytes;
  Bars* bars = reinterpret_cast<Bars*>(skv + C::NS * C::kTileBytes);
  static_assert(sizeof(Bars) <= 1024, "barriers fit behind the ring");
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  if (warp == 9) {
    tc::tmem_alloc(&bars->tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->q_full, 1);
    tc::mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < C::NS; ++s) {
      tc::mbar_init(&bars->kv_full[s], 1);
      tc::mbar_init(&bars->kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(&bars->s_full[t], 1);
      tc::mbar_init(&bars->p_ready[t][0], 4);
      tc::mbar_init(&bars->p_ready[t][1], 4);
      tc::mbar_init(&bars->o_half[t], 1);
      tc::mbar_init(&bars->o_done[t], 1);
      tc::mbar_init(&bars->o_free[t], 4);
      tc::mbar_init(&bars->unit_full[t], 1);
      tc::mbar_init(&bars->unit_empty[t], 9);
    }
    tc::mbar_init(&bars->v_fixed, 1);
    tc::mbar_init(&bars->drain, 1);
    bars->abort = 0;
    tc::fence_mbar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8) {
      producer<C>(a, &tm_q, &tm_k, &tm_v, sq, skv, bars, lane);
    } else if (warp == 9) {
      products<C>(a, tmem, sq, skv, bars);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    uint32_t n = 0;
    for (uint32_t r = 0;; ++r) {
      Unit u;
      const bool any = next_unit(bars, r, u);
      if (!__all_sync(0xffffffffu, any)) break;    // every lane has read it
      if (lane == 0) tc::mbar_arrive(&bars->unit_empty[r & 1]);
      if (!softmax<C>(a, u, tmem, bars, warp / 4, warp % 4, lane, n)) break;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && bars->abort) report(a.status, ATTN_DEV_TIMEOUT);
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- launch
// [tokens, heads, D] rows: boxes of 64 dims x box_heads x box_tokens.
inline bool map_rows(CUtensorMap* m, const RowsArg& r, bool bf16, int D, int heads, int T,
                     int box_heads, int box_tokens) {
  auto enc = prefill::encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(r.head) * 2,
                                 static_cast<cuuint64_t>(r.token) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads),
                             static_cast<cuuint32_t>(box_tokens)};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, r.p,
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A pool [pages, Hkv, page, D]: boxes of 64 dims x min(page, 128) slots.
inline bool map_pool(CUtensorMap* m, void* p, bool bf16, int D, int Hkv, const PagedKv& c) {
  auto enc = prefill::encode_fn();
  if (!enc) return false;
  const cuuint64_t page = 1ull << c.page_shift;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), page, static_cast<cuuint64_t>(Hkv),
                              static_cast<cuuint64_t>(c.pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, page * D * 2,
                                 static_cast<cuuint64_t>(c.page_stride) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(page < kBK ? page : kBK), 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, p,
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C>
cudaError_t launch(const Attn16Job& j, cudaStream_t stream) {
  static PerContext<cudaError_t> attr;
  const cudaError_t e = attr.get(
      [] {
        return cudaFuncSetAttribute(attn16_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    C::kSmem);
      },
      cudaErrorInvalidDevice, [](cudaError_t r) { return r == cudaSuccess; });
  if (e != cudaSuccess) return e;
  Args a{};
  a.T = j.T; a.B = j.B; a.max_len = j.max_len; a.cu = j.cu;
  a.prefix_table = j.prefix_table; a.prefix_len = j.prefix_len;
  a.pages = j.cache.pages; a.page_shift = j.cache.page_shift;
  a.H = j.H; a.Hkv = j.Hkv; a.D = j.D; a.G = j.H / j.Hkv; a.TQ = kRows / a.G;
  a.window = j.window;
  a.softcap_on = j.softcap > 0.f;
  a.c_score = j.scale * kLog2e16;
  a.c_cap_in = j.softcap > 0.f ? 2.0f * kLog2e16 * j.scale / j.softcap : 0.f;
  a.c_cap_out = kLog2e16 * j.softcap;
  a.out = j.out.p; a.o_token = j.out.token; a.o_head = j.out.head;
  a.part_o = j.part_o; a.part_ml = j.part_ml;
  a.status = j.status; a.skip = j.skip;
  const int tokens = 2 * a.TQ;
  int64_t grid;                                // units at most: no more blocks than SMs
  CUtensorMap tq, tk, tv;
  if (C::SHARED) {
    a.split_keys = a.B <= a.TQ;
    a.splits = shared_prefix_splits(a.B, a.H, a.Hkv, a.prefix_len) / (a.split_keys ? 2 : 1);
    a.units = (a.B + tokens - 1) / tokens;
    grid = static_cast<int64_t>(a.Hkv) * a.units * a.splits;
    if (!map_rows(&tq, j.q, j.bf16, a.D, a.H, a.B, a.G, a.TQ) ||
        !map_pool(&tk, j.cache.k, j.bf16, a.D, a.Hkv, j.cache) ||
        !map_pool(&tv, j.cache.v, j.bf16, a.D, a.Hkv, j.cache))
      return cudaErrorInvalidValue;
  } else {
    const int64_t tiles = (static_cast<int64_t>(a.max_len) + tokens - 1) / tokens;
    grid = static_cast<int64_t>(a.Hkv) * std::min<int64_t>(a.T / tokens + a.B, tiles * a.B);
    if (!map_rows(&tq, j.q, j.bf16, a.D, a.H, a.T, a.G, a.TQ) ||
        !map_rows(&tk, j.k, j.bf16, a.D, a.Hkv, a.T, 1, kBK) ||
        !map_rows(&tv, j.v, j.bf16, a.D, a.Hkv, a.T, 1, kBK))
      return cudaErrorInvalidValue;
  }
  grid = std::max<int64_t>(1, std::min<int64_t>(grid, prefill::sm_count()));
  return launch_dependent(attn16_kernel<C>, static_cast<unsigned>(grid), kThreads, C::kSmem, stream, tq, tk, tv, a);
}

template <class T>
cudaError_t launch_type(const Attn16Job& j, cudaStream_t stream) {
  if (j.cu)
    return j.D <= 64 ? launch<Cfg<T, 64, false>>(j, stream) : launch<Cfg<T, 128, false>>(j, stream);
  return j.D <= 64 ? launch<Cfg<T, 64, true>>(j, stream) : launch<Cfg<T, 128, true>>(j, stream);
}

}  // namespace attn16
}  // namespace gqa
