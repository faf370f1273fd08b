// Attention on the tensor cores in 16 bits ("Core Layers -- Deep Reference", "Flash Attention",
// "MHA and GQA"): the whole prompts of a packed batch, causal or windowed; and the part of a
// batch's single-token attention that falls on a prefix all rows share.
//
//   S = Q K^T,  P = 2^(c cap(S) - m),  O = sum P V,  l = sum P,  out = O / l
//
// over blocks of 128 keys with a running reference m per query row; products of 16-bit operands
// with fp32 accumulation, softmax and sums in fp32, P rounded once to 16 bits for the second
// product: half a step of the type, the size of the output's own rounding (one prompt of 77 tokens in
// fp16, against 64 bits: 2.2e-4 in norm, 2.0e-4 with fp32 weights). In two 16-bit parts it would cost
// half as many products again.
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
//  * Each tile's products are issued by a warp of its own, P V before the next S: the tensor
//    pipe runs a warp's products in order, so S may be written over the P before it without a
//    wait. (One warp for both spent a third of its time on barriers that were long complete,
//    about 150 cycles each, with the pipe running dry: 8192 tokens 394 us.)
//  * Softmax: a thread per row, 4 warps per tile. The reference is the row's first maximum and
//    stands until a block's weights sum to more than 2^15 (then the block is redone against a
//    new maximum and O rescaled): no maximum is taken in the common case.
//  * Values behind the last key (another sequence's, an unused slot's) are zeroed in shared memory:
//    whatever lies there, NaNs included, has no part in the result.
//  * Sixteen warps: softmax (2 x 4), loads, products (2), the list of units with the zeroing of V
//    behind the last key, and four that bring finished rows out of tensor memory, so that the
//    next unit's products and softmax run meanwhile. The blocks walk one list of units (a
//    pair of tiles each).
//  * Every wait is bounded; one that runs out raises ATTN_DEV_TIMEOUT and the block winds down.
//
// Measured (32 heads of 128 over 8): one prompt of 8192 tokens 353 us at 2070 MHz, 1560 TFLOP/s of
// products that are needed, 0.82 of the library product's rate measured on such a GPU; call after
// call for seconds, where the power limit takes the clock to 1927 MHz, 379 us. Tensor pipe at 68 % of
// its cycles, the rest lost where a tile's softmax and its products wait for one another. 8 prompts of
// 134..2013 tokens and 8 empty sequences 117..120 us (tensor pipe 53 %): the start and the end of each
// unit.
#pragma once

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "paged.cuh"
#include "prefill_common.cuh"

namespace gqa {
namespace attn16 {

using prefill::drain_wait;
using prefill::kSmemLimit;
using prefill::kTmemCols;

constexpr int kBK = 128;                       // keys per block
constexpr int kSums = 2 * 128 * 8;             // (sum, reference) of each row, behind the barriers
constexpr int kRows = 128;                     // query rows per tile

struct Args {
  int T, B, max_len;                           // packed prompts
  const int32_t* cu;
  const int32_t* prefix_table;                 // shared prefix
  int prefix_len, pages, page_shift;
  int H, Hkv, D, G, TQ;
  uint64_t inv_tokens;                         // floor(2^64 / (2 TQ)) + 1: n / (2 TQ) by the product's high half
  uint32_t inv_G;                              // floor(2^16 / G) + 1: row / G, row < 128
  int units, splits, split_keys;               // shared: pairs of tiles, splits of the key blocks
  int window;
  float c_score;                               // log2 units
  CapArgs cap;
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
  static constexpr int kOut = 16384;           // output rows on their way out (a share per warp)
  static constexpr int kNSraw = (kSmemLimit - 2048 - kSums - kOut - 2 * kTileBytes) / kTileBytes;
  static constexpr int NS = kNSraw > 8 ? 8 : kNSraw;
  static constexpr int kSmem = (NS + 2) * kTileBytes + kOut + kSums + 2048;
  static constexpr int kSCol = 0, kOCol = 256;
  // fp16 has few small numbers: with the first maximum's weight at 2^7, weights down to 2^-21 of
  // it keep all their bits, and there is room for weights 2^8 times as large.
  static constexpr float kBias = BF16 ? 0.f : 7.f;
};
// Warps 0-7 softmax, 8 loads, 9 and 10 products, 11 units and V's tails, 12-15 output rows. The block starts
// with 128 registers a thread; a row's 128 scores take more, so the last eight warps hand theirs on.
constexpr int kThreads = 512;
constexpr int kRegsSoftmax = 184, kRegsOther = 72;
static_assert(256 * kRegsSoftmax + 256 * kRegsOther <= kThreads * 128, "the block's registers");
constexpr int kUnits = 4;                      // units ahead

struct Bars {
  uint64_t unit_full[kUnits], unit_empty[kUnits];
  uint64_t q_full, q_empty;
  uint64_t kv_full[8], kv_empty[8];
  uint64_t landed[8];                          // V that is zeroed behind the last key before it is full
  uint64_t s_full[2];
  uint64_t p_ready[2], o_done[2];
  uint64_t turn[2];                            // the tiles' products of a block are issued in turn
  uint64_t l_ready[2], o_final[2], o_free[2];  // once a unit
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort;
  struct {
    int hk, row0, q0, ntok, kbase, nk, jlo, jhi, nt, la, part;   // nt 0: no more units
  } unit[kUnits];
};
using Unit = std::remove_extent<decltype(Bars::unit)>::type;

// The block's r-th unit, read by a whole warp; false: there is none (or a wait ran out).
__device__ __forceinline__ bool next_unit(Bars* bars, uint32_t r, int lane, Unit& u) {
  const bool ok = tc::mbar_wait_short(&bars->unit_full[r % kUnits], (r / kUnits) & 1, &bars->abort);
  if (ok) u = bars->unit[r % kUnits];
  if (!__all_sync(0xffffffffu, ok)) return false;              // every lane has read it
  if (lane == 0) tc::mbar_arrive(&bars->unit_empty[r % kUnits]);
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
// The blocks walk one list of units in snake order: unit x of round r for block c.
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
  return static_cast<int>(__umul64hi(s.n + 2 * a.TQ - 1, a.inv_tokens));
}

// Tiles of all sequences with index >= i (whole warp; cu_seqlens stays in L1).
__device__ __forceinline__ int tiles_from(const Args& a, int i) {
  int n = 0;
#pragma unroll 1
  for (int b = threadIdx.x & 31; b < a.B; b += 32) n += max(0, seq_tiles(a, b, false) - i);
  return __reduce_add_sync(0xffffffffu, n);
}

// Where the search for a block's next unit stands (they come in order).
struct Search {
  int top = 0, past = 0;                       // sorted: `past` tiles have an index of top or above
  int b0 = 0;                                  // else: `past` tiles are of sequences before b0
};

// Unit x of the list; false past its end. Whole warp. Packed prompts: the kv heads of a tile side by
// side. Up to kSorted sequences, tiles by their index within their sequence, last first (a tile's keys
// grow with it), so that the blocks end together; each unit's search then reads every sequence's
// bounds a few times. Past that many the sequences come in their own order, each one's last tile
// first, and a block reads their bounds once in all. 32 heads of 128 over 8, us sorted and in order:
// 16 of 1..2048 tokens 150, 163; 64 of 1..200 47, 43; 63 of 100 and one of 8192 385, 448; 96 such 403,
// 400; 256 of 1..200 187, 136; 4096 22900, 1980; 16384 of 4 tokens, 8 heads of 64: 124000, 2840.
constexpr int kSorted = 64;
template <class C>
__device__ bool find_unit(const Args& a, unsigned x, Search& at, Unit& u) {
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
  int lo = -1, b = 0;                          // the unit is tile lo of sequence b
  const int lane = threadIdx.x & 31;
  if (a.B <= kSorted) {
    // The largest index lo < top with more than y tiles of index >= lo; then top = lo + 1.
#pragma unroll 1
    while (at.top - lo > 1) {
      const int mid = (lo + at.top) / 2, n = tiles_from(a, mid);
      if (n > y) {
        lo = mid;
      } else {
        at.top = mid;
        at.past = n;
      }
    }
    if (lo < 0) return false;
    int k = y - at.past;                       // among the sequences that have a tile lo
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int mine = b0 + lane;
      const bool has = mine < a.B && seq_tiles(a, mine, false) > lo;
      const uint32_t all = __ballot_sync(0xffffffffu, has);
      if (k < __popc(all)) {                   // the lane with k others before it
        const int before = __popc(all & ((1u << lane) - 1));
        b = b0 + __ffs(__ballot_sync(0xffffffffu, has && before == k)) - 1;
        break;
      }
      k -= __popc(all);
    }
  } else {
#pragma unroll 1
    for (;; at.b0 += 32) {
      if (at.b0 >= a.B) return false;
      const int mine = at.b0 + lane, n = mine < a.B ? seq_tiles(a, mine, blockIdx.x == 0) : 0;
      int to = n;                              // tiles of the lanes up to this one
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int before = __shfl_up_sync(0xffffffffu, to, o);
        if (lane >= o) to += before;
      }
      const int k = y - at.past, all = __shfl_sync(0xffffffffu, to, 31);
      if (k < all) {                           // the first lane whose tiles pass k
        const int src = __ffs(__ballot_sync(0xffffffffu, to > k)) - 1;
        b = at.b0 + src;
        lo = __shfl_sync(0xffffffffu, to, src) - 1 - k;
        break;
      }
      at.past += all;
    }
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

// ---------------------------------------------------------------- units, and V behind the last key (one warp)
// The last block of a sequence may hold fewer than 128 keys: once its V has landed, the rows
// behind them are zeroed, and only then is the stage full.
template <class C>
__device__ __forceinline__ bool zero_tail(const Unit& u, uint8_t* skv, Bars* bars, int lane,
                                          uint32_t& loaded, uint32_t& fills) {
  loaded += 2 * (u.jhi - u.jlo + 1);           // as the loads count them: the unit's last is its last V
  const int keys = u.nk - u.jhi * kBK, stage = (loaded - 1) % C::NS;
  if (keys >= kBK) return true;
  const bool ok = tc::mbar_wait_short(&bars->landed[stage], fills >> stage & 1, &bars->abort);
  if (!__all_sync(0xffffffffu, ok)) return false;
  fills ^= 1u << stage;
  uint8_t* v = skv + stage * C::kTileBytes;
#pragma unroll 1
  for (int c = 0; c < C::kChunks; ++c)
#pragma unroll 2
    for (int e = 8 * keys + lane; e < 8 * kBK; e += 32)
      *reinterpret_cast<uint4*>(v + c * C::kChunk + e * 16) = make_uint4(0, 0, 0, 0);
  tc::fence_proxy_async();
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(&bars->kv_full[stage]);
  return true;
}

// Publishes the block's units; a unit's tail is done once the next one is published.
template <class C>
__device__ void scheduler(const Args& a, uint8_t* skv, Bars* bars, int lane) {
  volatile int* abort = &bars->abort;
  Search at;
  uint32_t loaded = 0, fills = 0;
  if (!C::SHARED && a.B <= kSorted) {
#pragma unroll 1
    for (int b = lane; b < a.B; b += 32) at.top = max(at.top, seq_tiles(a, b, blockIdx.x == 0));
    at.top = __reduce_max_sync(0xffffffffu, at.top);
  }
  Unit before{};
  for (uint32_t r = 0;; ++r) {
    Unit u{};
    const bool any = find_unit<C>(a, unit_at(blockIdx.x, r, gridDim.x), at, u);
    if (!any) u.nt = 0;
    bool ok = true;
    if (lane == 0) {
      ok = tc::mbar_wait_short(&bars->unit_empty[r % kUnits], ((r / kUnits) & 1) ^ 1u, abort);
      if (ok) {
        bars->unit[r % kUnits] = u;
        tc::mbar_arrive(&bars->unit_full[r % kUnits]);
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok && r > 0) ok = zero_tail<C>(before, skv, bars, lane, loaded, fills);
    if (!any || !ok) return;
    before = u;
  }
}

// ---------------------------------------------------------------- loads (one warp)
// A unit's ring order: K of its first block (first la blocks), then V and the K that is la ahead.
template <class C>
__device__ void loads(const Args& a, const CUtensorMap* tq, const CUtensorMap* tk,
                      const CUtensorMap* tv, uint8_t* sq, uint8_t* skv, Bars* bars, int lane) {
  volatile int* abort = &bars->abort;
  int stage = 0;
  uint32_t phase = 0, loaded = 0, units = 0;
  uint32_t to_land = 0, fills = 0;             // stages whose last load lands apart; landings' parities
  Unit u{};
  auto load = [&](bool is_v, int j) -> bool {
    bool ok = true;
    const bool apart = is_v && u.nk - j * kBK < kBK;   // zeroed behind the last key, then full
    uint64_t* full = apart ? &bars->landed[stage] : &bars->kv_full[stage];
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
    if (lane == 0) ok = tc::mbar_wait_short(&bars->kv_empty[stage], phase ^ 1u, abort);
    if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
    const CUtensorMap* map = is_v ? tv : tk;
    if (C::SHARED) {
      // A page that does not exist is read as page 0 (the result is without meaning).
      if (lane == 0) tc::mbar_arrive_expect_tx(full, C::kChunks * 128 * rows);
      __syncwarp();
      if (lane < rows / box) {
        const int at = (j * kBK + lane * box) & (page - 1);
#pragma unroll 1
        for (int c = 0; c < C::kChunks; ++c)
          tc::tma_load_4d(dst + c * C::kChunk + lane * box * 128, map, full, 64 * c, at, u.hk,
                          max(id, 0));
      }
    } else if (lane == 0) {
      tc::mbar_arrive_expect_tx(full, C::kTileBytes);
#pragma unroll 1
      for (int c = 0; c < C::kChunks; ++c)
        tc::tma_load_3d(dst + c * C::kChunk, map, full, 64 * c, u.hk, u.kbase + j * kBK);
    }
    ++loaded;
    if (apart) {
      fills ^= 1u << stage;
      to_land |= 1u << stage;
    } else {
      to_land &= ~(1u << stage);
    }
    if (++stage == C::NS) {
      stage = 0;
      phase ^= 1u;
    }
    return true;
  };
  bool ok = true;
  while (ok && next_unit(bars, units, lane, u)) {
    if (lane == 0) {
      const int tiles = u.la == 2 ? 1 : u.nt;
      ok = tc::mbar_wait_short(&bars->q_empty, (units & 1) ^ 1u, abort);
      if (ok) {
        tc::mbar_arrive_expect_tx(&bars->q_full, tiles * C::kChunks * 128 * a.G * a.TQ);
#pragma unroll 1
        for (int t = 0; t < tiles; ++t)
#pragma unroll 1
          for (int c = 0; c < C::kChunks; ++c)
            tc::tma_load_3d(sq + t * C::kTileBytes + c * C::kChunk, tq, &bars->q_full, 64 * c,
                            u.hk * a.G, u.row0 + t * a.TQ);
      }
    }
    if (!(ok = __shfl_sync(0xffffffffu, ok, 0))) break;
    ++units;
    // K, V by turns: item i is K of block jlo + i for the first la, then V and K alternate
    const int blocks = u.jhi - u.jlo + 1;
#pragma unroll 1
    for (int i = 0, nk = 0, nv = 0; ok && i < 2 * blocks; ++i) {
      const bool is_k = nk < blocks && nk < nv + u.la;
      ok = load(!is_k, u.jlo + (is_k ? nk++ : nv++));
    }
  }
  // Every copy this block started lands before the block may exit.
  if (lane == 0) {
    if (units > 0) drain_wait(&bars->q_full, (units - 1) & 1);
#pragma unroll 1
    for (uint32_t s = 0; s < C::NS && s < loaded; ++s) {
      const uint32_t fill = (loaded - 1 - s) / C::NS;   // the last load into stage s
      if (to_land >> s & 1)
        drain_wait(&bars->landed[s], (fills >> s & 1) ^ 1u);
      else
        drain_wait(&bars->kv_full[s], fill & 1);
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------- products (a warp per tile, one lane issues)
// The tensor pipe takes a product every 64 cycles, so the warps that issue them have to be lean:
// they stay converged with every operand the same in all lanes (uniform registers), the loops
// over a block's products are unrolled, and where a wait runs out a warp goes on (on data that
// is then without meaning, all of it this block's) to the block's end, where it leaves together.
// Both warps walk the whole ring, whether a block is their tile's or not, and take turns: one
// tile's softmax then runs while the other's products do (left to themselves the tiles fell
// into step, 3500 cycles a block instead of 2800).
template <class C>
__device__ void products(const Args& a, uint32_t tmem, uint8_t* sq, uint8_t* skv, Bars* bars,
                         const int t) {
  volatile int* abort = &bars->abort;
  constexpr uint32_t id_s = tc::idesc_f16(kRows, kBK, C::BF16, false);
  constexpr uint32_t id_o = tc::idesc_f16(kRows, C::DP, C::BF16, true);
  const uint64_t qd = tc::sdesc_sw128(tc::smem_u32(sq), 16, 1024);
  const uint64_t kd = tc::sdesc_sw128(tc::smem_u32(skv), 16, 1024);
  // V [keys][dims], dims contiguous: the next 64 dims are a chunk away, the next 8 keys 1024 bytes
  const uint64_t vd = tc::sdesc_sw128(tc::smem_u32(skv), C::kChunk, 1024);
  const uint32_t s_col = tmem + C::kSCol + t * kBK, o_col = tmem + C::kOCol + t * C::DP;
  uint32_t stage = 0, phase = 0;
  uint32_t done = 0, outputs = 0, turns = 0;   // the tile's blocks, units and turns so far
  bool bad = false;
  // Most of these are complete by now: asked first without leave to sleep (8192 tokens 369 -> 351 us).
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!tc::mbar_try_wait(bar, parity)) bad |= !tc::mbar_wait_short(bar, parity, abort);
  };
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
    if (!next_unit(bars, r, threadIdx.x % 32, u)) break;
    const int la = __shfl_sync(0xffffffffu, u.la, 0);
    const int jlo = __shfl_sync(0xffffffffu, u.jlo, 0), jhi = __shfl_sync(0xffffffffu, u.jhi, 0);
    int lo = 0, hi = 0;                        // the tile's blocks
    tile_blocks<C>(a, u, t, lo, hi);
    lo = __shfl_sync(0xffffffffu, lo, 0);
    hi = __shfl_sync(0xffffffffu, hi, 0);
    auto active = [&](int j) { return j >= lo && j <= hi && (la == 1 || ((j - jlo) & 1) == t); };
    const uint64_t q = qd + ((la == 2 ? 0 : t) * C::kTileBytes >> 4);
    auto scores = [&](uint32_t st) {
      const uint64_t k = kd + (st * C::kTileBytes >> 4);
#pragma unroll
      for (int s = 0; s < C::DP / 16; ++s) {
        const uint32_t off = ((s >> 2) * C::kChunk + (s & 3) * 32) >> 4;
        tc::mma_f16_ss(s_col, q + off, k + off, id_s, s > 0);
      }
      tc::mma_commit_warp(&bars->s_full[t]);
    };
    wait(&bars->q_full, r & 1);
    for (int e = 0; e < la && jlo + e <= jhi; ++e) {
      const uint32_t st = take();
      tc::fence_after_sync();
      if (active(jlo + e)) scores(st);
      tc::mma_commit_warp(&bars->kv_empty[st]);
    }
    if (jlo + la > jhi) tc::mma_commit_warp(&bars->q_empty);
    for (int j = jlo; j <= jhi; ++j, ++turns) {
      const uint32_t vs = take();
      const bool next = j + la <= jhi, mine = active(j), first = la == 2 ? j - jlo == t : j == lo;
      uint32_t ks = 0;
      if (next) ks = take();
      if (mine) {
        if (first) {
          if (outputs > 0) wait(&bars->o_free[t], (outputs - 1) & 1);
          ++outputs;
        }
        wait(&bars->p_ready[t], done & 1);
        ++done;
      }
      // In turn: tile 0's products of this block, then tile 1's, then tile 0's of the next.
      if (t == 1 || turns > 0) wait(&bars->turn[t], (turns - 1 + t) & 1);
      tc::fence_after_sync();
      if (mine) {
        const uint64_t v = vd + (vs * C::kTileBytes >> 4);
        // (Leaving out the steps of 16 keys that no row of the tile sees, at a tile's last
        // block, made these branches of and the whole kernel 9% slower.)
#pragma unroll
        for (int s = 0; s < 8; ++s)
          tc::mma_f16_ts(o_col, s_col + 8 * s, v + (s * 2048 >> 4), id_o,
                         (!first || s > 0) ? 1u : 0u);
        tc::mma_commit_warp(&bars->o_done[t]);
        if (j + la > hi) tc::mma_commit_warp(&bars->o_final[t]);
      }
      tc::mma_commit_warp(&bars->kv_empty[vs]);
      if (next) {
        if (active(j + la)) scores(ks);
        tc::mma_commit_warp(&bars->kv_empty[ks]);
      }
      if (threadIdx.x % 32 == 0) tc::mbar_arrive(&bars->turn[1 - t]);
      __syncwarp();
      if (j + la == jhi) tc::mma_commit_warp(&bars->q_empty);   // the unit's last S
      if (__any_sync(0xffffffffu, bad)) break;
    }
    if (__any_sync(0xffffffffu, bad)) break;
  }
  tc::mma_commit_warp(&bars->drain[t]);        // nothing may still run when the block frees its TMEM
  drain_wait(&bars->drain[t], 0);
}

// ---------------------------------------------------------------- softmax (4 warps a tile)
// 2^(s cs - m) of N scores, packed to 16 bits; returns their sum.
template <class T, int N>
__device__ __forceinline__ float exp_pack(const float* s, float cs, float m, uint32_t* p) {
  const uint64_t c2 = tc::pack2(cs, cs), m2 = tc::pack2(-m, -m);
  uint64_t acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = tc::pack2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    float x0, x1;
    tc::unpack2(tc::fma2(tc::pack2(s[c], s[c + 1]), c2, m2), x0, x1);
    x0 = tc::ex2(x0);
    x1 = tc::ex2(x1);
    p[c / 2] = Pair<T>::pack(x0, x1);
    acc[(c / 2) % 4] = tc::add2(acc[(c / 2) % 4], tc::pack2(x0, x1));
  }
  float a0, a1;
  tc::unpack2(tc::add2(tc::add2(acc[0], acc[1]), tc::add2(acc[2], acc[3])), a0, a1);
  return a0 + a1;
}

// A shared prefix: the softmax warps bring their rows out themselves (a block has one unit, as a rule,
// and eight warps are faster than four): O / l in fp32, 64 bytes of a row at a time through
// shared memory, with the row's reference and sum.
template <class C>
__device__ bool partial_rows(const Args& a, const Unit& u, uint32_t tmem, uint8_t* stage, Bars* bars,
                             int t, int quarter, int lane, bool has, uint32_t n, float l, float m_ref) {
  if (u.la == 1 && t >= u.nt) return true;
  if (has) {
    const bool ok = tc::mbar_wait_short(&bars->o_done[t], (n - 1) & 1, &bars->abort);
    if (!__all_sync(0xffffffffu, ok)) return false;
    tc::fence_after_sync();
  }
  const int row = quarter * 32 + lane, tok = row * a.inv_G >> 16;
  const int local = (u.la == 2 ? 0 : t * a.TQ) + tok, head = u.hk * a.G + row - tok * a.G;
  const int part = u.la == 2 ? 2 * u.part + t : u.part;
  const int64_t at = (static_cast<int64_t>(part) * a.B + u.row0 + local) * a.H + head;
  float* dst = nullptr;
  if (tok < a.TQ && local < u.ntok) {
    a.part_ml[at] = make_float2(m_ref, l);     // (-inf, 0) for a split without blocks
    dst = a.part_o + at * a.D;
  }
  float* rows[4];                              // where the lane's 16 bytes of 4 rows go
#pragma unroll
  for (int i = 0; i < 4; ++i)
    rows[i] = reinterpret_cast<float*>(__shfl_sync(
        0xffffffffu, reinterpret_cast<unsigned long long>(dst), 8 * i + lane / 4));
  const float inv = has && m_ref != -INFINITY ? 1.0f / l : 0.f;
  const uint32_t col = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + C::kOCol + t * C::DP;
  float4* s = reinterpret_cast<float4*>(stage);
#pragma unroll 1
  for (int c = 0; c < C::DP; c += 16) {
    float o[16];
    if (has) {
      tc::tmem_ld16(col + c, o);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s[lane * 4 + (e ^ (lane >> 1 & 3))] = make_float4(o[4 * e] * inv, o[4 * e + 1] * inv,
                                                        o[4 * e + 2] * inv, o[4 * e + 3] * inv);
    __syncwarp();
    const int e = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int from = 8 * i + lane / 4;
      const float4 x = s[from * 4 + (e ^ (from >> 1 & 3))];
      if (rows[i] && c + 4 * e < a.D) *reinterpret_cast<float4*>(rows[i] + c + 4 * e) = x;
    }
    __syncwarp();
  }
  if (has) {
    tc::fence_before_sync();
    if (lane == 0) tc::mbar_arrive(&bars->o_free[t]);
  }
  return true;
}

// The cap of 32 raw scores of a row. They are mostly well below it: while none is past the series'
// limit, the series on the paired multiply-add, 3 instructions a score, in place of two on the
// exponential's pipe, four cycles each (9 prompts of 100..1800, window 512, 16 heads of 64: 68 us
// with those alone, 63 with the series). Row by row: the other form is off by 2^-22 of the cap,
// which only a row that holds such a large score can do without.
__device__ __forceinline__ void soft_cap(const Args& a, float (&x)[32], bool live) {
  float most = 0.f;
#pragma unroll
  for (int c = 0; c < 32; c += 2) most = tc::max3(most, fabsf(x[c]), fabsf(x[c + 1]));
  if (!live || most <= a.cap.limit) {
    uint64_t k[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) k[i] = tc::pack2(a.cap.series[i], a.cap.series[i]);
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      const uint64_t v = tc::pack2(x[c], x[c + 1]), z = tc::mul2(v, v);
      uint64_t p = tc::fma2(k[4], z, k[3]);
      p = tc::fma2(p, z, k[2]);
      p = tc::fma2(p, z, k[1]);
      p = tc::fma2(p, z, k[0]);
      tc::unpack2(tc::mul2(p, v), x[c], x[c + 1]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const float e = tc::ex2(x[c] * a.cap.in);
      x[c] = fmaf(-2.0f * a.cap.out, tc::rcp(e + 1.0f), a.cap.out);
    }
  }
  __syncwarp();                                // what follows is for the whole warp
}

// The n lowest bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u);
}

// Only a block's common path and its mask are unrolled; what is rarer (softcap, a block done again)
// works on 32 columns at a time in rolled loops, on S in tensor memory: the roles' loops together
// have to stay in the instruction caches (with all paths unrolled the kernel took 1.2 times as long).
template <class C>
__device__ bool softmax(const Args& a, const Unit& u, uint32_t tmem, float2* sums, uint8_t* stage,
                        Bars* bars, int t, int quarter, int lane, uint32_t& n, uint32_t& outputs) {
  using T = typename C::T;
  volatile int* abort = &bars->abort;
  const uint32_t n0 = n;                       // this tile's blocks before this unit
  const int row = quarter * 32 + lane, tok = row * a.inv_G >> 16;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const int tile = C::SHARED && u.la == 2 ? 0 : t;
  const int local = tile * a.TQ + tok;         // token of the unit
  const bool live = tok < a.TQ && local < u.ntok;
  const int qpos = u.q0 + local;
  const float cs = a.cap.on ? 1.0f : a.c_score;
  constexpr float kLimit = 32768.0f;           // no weight can then be past fp16's range
  float m_ref = -INFINITY, l = 0.f;            // P = 2^(score - m_ref) with the bias inside m_ref
  // The warp's rows' first and last visible keys are ordered as their tokens are.
  const int tok0 = 32 * quarter * a.inv_G >> 16;
  const int tok1 = min(static_cast<int>((32 * quarter + 31) * a.inv_G >> 16), a.TQ - 1);
  const int q_lo = u.q0 + tile * a.TQ + tok0, q_hi = u.q0 + tile * a.TQ + tok1;
  const int tile_keys = C::SHARED ? u.nk : u.q0 + min((t + 1) * a.TQ, u.ntok);
  int j_lo, j_hi;
  tile_blocks<C>(a, u, t, j_lo, j_hi);
  bool ok = true, started = false;             // started: every live row has a reference
  const uint32_t scol = lane_base + C::kSCol + t * kBK;
  for (int j = u.la == 2 ? j_lo + t : j_lo; j <= j_hi; j += u.la) {
    ok = tc::mbar_try_wait(&bars->s_full[t], n & 1) ||
         tc::mbar_wait_short(&bars->s_full[t], n & 1, abort);
    if (!__all_sync(0xffffffffu, ok)) return false;   // together: tcgen05.ld is warp-wide
    tc::fence_after_sync();
    const int k0 = j * kBK;
    // Blocks that the mask crosses: keys c <= hi and c >= lo are visible.
    const bool edge = k0 + kBK > u.nk ||
                      (!C::SHARED && (k0 + kBK - 1 > q_lo ||
                                      (a.window > 0 && k0 < q_hi - a.window + 1)));
    const int hi = !edge ? kBK : (C::SHARED ? u.nk - 1 : min(qpos, u.nk - 1)) - k0;
    const int lo = edge && !C::SHARED && a.window > 0 ? qpos - a.window + 1 - k0 : 0;
    auto seen = [&](int c0) { return bits_below(hi + 1 - c0) & ~bits_below(lo - c0); };   // of 32 columns
    if (a.cap.on) {                        // in place, in tensor memory, where the tile has keys
      const int chunks = min(4, (tile_keys - k0 + 31) / 32);
#pragma unroll 1
      for (int i = 0; i < chunks; ++i) {
        float x[32];
        tc::tmem_ld32(scol + 32 * i, x);
        soft_cap(a, x, live);
        tc::tmem_st32(scol + 32 * i, x);
      }
    }
    float x[128];
    uint32_t p[64];
    tc::tmem_ld128(scol, x);
    if (edge) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t m = seen(32 * w);
#pragma unroll
        for (int c = 0; c < 32; ++c) x[32 * w + c] = m >> c & 1 ? x[32 * w + c] : -INFINITY;
      }
    }
    if (!started) {                            // rows without a reference take the block's maximum
      const float top = prefill::tq_max<128>(x);
      if (m_ref == -INFINITY) m_ref = fmaf(top, cs, -C::kBias);
      started = !__any_sync(0xffffffffu, live && m_ref == -INFINITY);
    }
    // -inf only while every key so far was masked; then every score is -inf
    float m_use = m_ref == -INFINITY ? 0.f : m_ref;
    float lsum = exp_pack<T, 64>(x, cs, m_use, p);
    lsum += exp_pack<T, 64>(x + 64, cs, m_use, p + 32);
    if (!__any_sync(0xffffffffu, live && !(lsum <= kLimit))) {
      l += lsum;
      tc::tmem_st64(scol, reinterpret_cast<const float*>(p));
    } else {                                   // a new reference, and all of it again
      float y[32], top = -INFINITY;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        tc::tmem_ld32(scol + 32 * i, y);
        const uint32_t m = seen(32 * i);
#pragma unroll
        for (int c = 0; c < 32; ++c) top = m >> c & 1 ? fmaxf(top, y[c]) : top;
      }
      const float m_new = fmaxf(m_ref, fmaf(top, cs, -C::kBias));
      const bool grow = m_ref != -INFINITY && m_new > m_ref;
      if (n > n0 && __any_sync(0xffffffffu, grow)) {   // O once every product that wrote it is done
        ok = tc::mbar_wait_short(&bars->o_done[t], (n - 1) & 1, abort);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tc::fence_after_sync();
        const float f = grow ? tc::ex2(m_ref - m_new) : 1.0f;
#pragma unroll 1
        for (int c = 0; c < C::DP; c += 32) {
          tc::tmem_ld32(lane_base + C::kOCol + t * C::DP + c, y);
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] *= f;
          tc::tmem_st32(lane_base + C::kOCol + t * C::DP + c, y);
        }
        l *= f;
      }
      if (grow) m_ref = m_new;
      m_use = m_ref == -INFINITY ? 0.f : m_ref;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {            // P's columns lie below those still to be read
        uint32_t q[16];
        tc::tmem_ld32(scol + 32 * i, y);
        const uint32_t m = seen(32 * i);
#pragma unroll
        for (int c = 0; c < 32; ++c) y[c] = m >> c & 1 ? y[c] : -INFINITY;
        l += exp_pack<T, 32>(y, cs, m_use, q);
        tc::tmem_st16(scol + 16 * i, reinterpret_cast<const float*>(q));
      }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&bars->p_ready[t]);
    ++n;
  }
  if constexpr (C::SHARED)
    return partial_rows<C>(a, u, tmem, stage, bars, t, quarter, lane, n > n0, n, l, m_ref);
  if (n == n0) return true;                    // the tile had no blocks
  // The row's sum and reference for those who bring it out, once they have read the last.
  if (outputs > 0) {
    ok = tc::mbar_wait_short(&bars->o_free[t], (outputs - 1) & 1, abort);
    if (!__all_sync(0xffffffffu, ok)) return false;
  }
  ++outputs;
  sums[t * 128 + row] = make_float2(l, m_ref);
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(&bars->l_ready[t]);
  return true;
}

// ---------------------------------------------------------------- output rows (4 warps)
// O / l of a finished tile: 128 bytes of a row at a time through shared memory, so that 8 lanes
// write them at once (a lane writing its own row touched 32 lines an instruction).
template <class C>
__device__ void outputs(const Args& a, uint32_t tmem, uint8_t* stage, const float2* sums, Bars* bars,
                        int quarter, int lane) {
  using T = typename C::T;
  volatile int* abort = &bars->abort;
  const int row = quarter * 32 + lane, tok = row * a.inv_G >> 16;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  uint4* s = reinterpret_cast<uint4*>(stage);
  uint32_t done = 0;                           // bit t: parity of the tile's outputs
  for (uint32_t r = 0;; ++r) {
    Unit u;
    if (!next_unit(bars, r, lane, u)) return;
#pragma unroll 1
    for (int t = 0; t < u.nt; ++t) {
      bool ok = tc::mbar_wait_short(&bars->l_ready[t], done >> t & 1, abort);
      ok = ok && tc::mbar_wait_short(&bars->o_final[t], done >> t & 1, abort);
      if (!__all_sync(0xffffffffu, ok)) return;
      done ^= 1u << t;
      tc::fence_after_sync();
      const float inv = 1.0f / sums[t * 128 + row].x;   // every live row sees itself
      const int local = t * a.TQ + tok, head = u.hk * a.G + row - tok * a.G;
      char* dst = nullptr;                     // the lane's row, where it is one
      if (tok < a.TQ && local < u.ntok)
        dst = reinterpret_cast<char*>(static_cast<T*>(a.out) + (u.row0 + local) * a.o_token +
                                      head * a.o_head);
      char* rows[8];                           // where the lane's 16 bytes of 8 rows go
#pragma unroll
      for (int i = 0; i < 8; ++i)
        rows[i] = reinterpret_cast<char*>(__shfl_sync(
            0xffffffffu, reinterpret_cast<unsigned long long>(dst), 4 * i + lane / 8));
#pragma unroll 1
      for (int c = 0; c < C::DP; c += 64) {
#pragma unroll 1
        for (int h = 0; h < 64; h += 16) {
          float o[16];
          tc::tmem_ld16(lane_base + C::kOCol + t * C::DP + c + h, o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= inv;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            s[lane * 8 + ((h / 8 + e) ^ (lane & 7))] =
                pack8<T>(*reinterpret_cast<float(*)[8]>(o + 8 * e));
        }
        __syncwarp();
        if (c + 64 >= C::DP) {                 // O may be written again
          tc::fence_before_sync();
          if (lane == 0) tc::mbar_arrive(&bars->o_free[t]);
        }
        const int e = lane & 7;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int from = 4 * i + lane / 8;
          const uint4 x = s[from * 8 + (e ^ (from & 7))];
          if (rows[i] && c + 8 * e < a.D) *reinterpret_cast<uint4*>(rows[i] + 2 * c + 16 * e) = x;
        }
        __syncwarp();
      }
    }
  }
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
    attn16_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sq = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint8_t* skv = sq + 2 * C::kTileBytes;
  uint8_t* sout = skv + C::NS * C::kTileBytes;
  Bars* bars = reinterpret_cast<Bars*>(sout + C::kOut);
  float2* sums = reinterpret_cast<float2*>(sout + C::kOut + 1024);
  static_assert(sizeof(Bars) <= 1024, "barriers fit behind the ring");
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  if (threadIdx.x == 32) {                     // ahead of the first loads, which would wait for them
    tc::tma_prefetch(&tm_q);
    tc::tma_prefetch(&tm_k);
    tc::tma_prefetch(&tm_v);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kUnits; ++i) {
      tc::mbar_init(&bars->unit_full[i], 1);
      tc::mbar_init(&bars->unit_empty[i], C::SHARED ? 11 : 15);   // warps that read it
    }
    tc::mbar_init(&bars->q_full, 1);
    tc::mbar_init(&bars->q_empty, 2);
    for (int s = 0; s < C::NS; ++s) {
      tc::mbar_init(&bars->kv_full[s], 1);
      tc::mbar_init(&bars->kv_empty[s], 2);
      tc::mbar_init(&bars->landed[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(&bars->s_full[t], 1);
      tc::mbar_init(&bars->p_ready[t], 4);
      tc::mbar_init(&bars->turn[t], 1);
      tc::mbar_init(&bars->o_done[t], 1);
      tc::mbar_init(&bars->l_ready[t], 4);
      tc::mbar_init(&bars->o_final[t], 1);
      tc::mbar_init(&bars->o_free[t], 4);
      tc::mbar_init(&bars->drain[t], 1);
    }
    bars->abort = 0;
    tc::fence_mbar_init();
  }
  dependent_wait();
  if (gated_off(a.skip)) return;
  // The rows' own kernel finds room as these blocks end (after the wait: see paged_decode.cu). Another
  // prefill that waits in these blocks' places gains nothing: 8 prompts of 134..2013, repeated, 118 -> 126 us.
  if (C::SHARED) dependents_may_launch();
  if (warp == 9) {
    tc::tmem_alloc(&bars->tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8) {
      loads<C>(a, &tm_q, &tm_k, &tm_v, sq, skv, bars, lane);
    } else if (warp <= 10) {
      products<C>(a, tmem, sq, skv, bars, warp - 9);
    } else if (warp == 11) {
      scheduler<C>(a, skv, bars, lane);
    } else {
      if (!C::SHARED) outputs<C>(a, tmem, sout + (warp - 12) * 4096, sums, bars, warp - 12, lane);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    uint32_t n = 0, outs = 0;
    Unit u;
    for (uint32_t r = 0; next_unit(bars, r, lane, u); ++r)
      if (!softmax<C>(a, u, tmem, sums, sout + warp * 2048, bars, warp / 4, warp % 4, lane, n, outs))
        break;
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
  a.inv_tokens = ~0ull / (2 * a.TQ) + 1;
  a.inv_G = 65536 / a.G + 1;
  a.window = j.window;
  a.c_score = j.scale * kLog2e16;
  a.cap = cap_args(j.softcap, j.scale);
  a.out = j.out.p; a.o_token = j.out.token; a.o_head = j.out.head;
  a.part_o = j.part_o; a.part_ml = j.part_ml;
  a.status = j.status; a.skip = j.skip;
  const int tokens = 2 * a.TQ;
  int64_t grid;                                // units at most: no more blocks than SMs
  CUtensorMap tq, tk, tv;
  if (C::SHARED) {
    const PrefixPlan plan = shared_prefix_plan(a.B, a.H, a.Hkv, a.prefix_len);
    a.split_keys = plan.split_keys;
    a.splits = plan.splits;
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
