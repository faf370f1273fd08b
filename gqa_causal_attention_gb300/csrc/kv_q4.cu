// Writing, reading back and trimming the 4-bit KV cache (record format: kv_q4.cuh).
//
// The cache is the caller-owned TransformerState of "mojolearn.transformer" with
// quantised storage ("dew.nn.backbones.causal_transformer": caches dense or paged,
// full or quantized); slots follow the same rules as kv_cache_append's.
//
// All of it is memory-bound: a warp per row with 16-byte reads of fp32 rows, and the
// records moved in 16-byte pieces.
#include "common.cuh"
#include "kernels.h"
#include "kv_q4_rows.cuh"
#include "tc_ptx.cuh"

namespace gqa {

namespace {

// Calls f(std::integral_constant-like tag) for the runtime group count m = D / 32.
template <int M>
struct Groups {
  static constexpr int value = M;
};
template <class F>
cudaError_t with_groups(int m, F f) {
  switch (m) {
    case 1: return f(Groups<1>{});
    case 2: return f(Groups<2>{});
    case 3: return f(Groups<3>{});
    case 4: return f(Groups<4>{});
    case 5: return f(Groups<5>{});
    case 6: return f(Groups<6>{});
    case 7: return f(Groups<7>{});
    case 8: return f(Groups<8>{});
    default: return cudaErrorInvalidValue;
  }
}

// Blocks of the row passes: four warps and up to sixteen rows, so that several are in
// flight on an SM in different stages.
constexpr int kRowThreads = 128, kMaxRows = 16;

struct RowAt {
  long bh;      // b * Hkv + hkv
  int b, l;
};
__device__ __forceinline__ RowAt row_at(long row, long rows, int Hkv, int L) {
  RowAt r;
  if (rows < (1L << 31)) {
    const uint32_t h = static_cast<uint32_t>(row) / static_cast<uint32_t>(L);
    r.l = static_cast<int>(static_cast<uint32_t>(row) - h * static_cast<uint32_t>(L));
    r.bh = h;
    r.b = static_cast<int>(h / static_cast<uint32_t>(Hkv));
  } else {
    r.bh = row / L;
    r.l = static_cast<int>(row - r.bh * L);
    r.b = static_cast<int>(r.bh / Hkv);
  }
  return r;
}

// Where row (bh, l) of an append goes: its record, or nullptr where it is not stored; ok:
// whether the row's positions are valid (one thread reports a batch row that is not).
struct Target {
  bool ok;
  uint8_t* rec;
  long angle;               // row of the angle table
};
template <int M, bool ROT>
__device__ __forceinline__ Target append_target(const AppendQ4Job& j, const RowAt& at, bool one) {
  const int s0 = j.start[at.b], p0 = j.pos ? j.pos[at.b] : s0;
  const bool first = one && at.l == j.l0 && at.bh % j.Hkv == 0;
  Target t{false, nullptr, static_cast<long>(p0) + at.l};
  if (s0 < 0 || p0 < 0 || (ROT && static_cast<long>(p0) + j.L > j.max_positions)) {
    if (first) report(j.status, ATTN_DEV_POSITION);
    return t;
  }
  if (j.window == 0 && static_cast<long>(s0) + j.L > j.capacity) {
    if (first) report(j.status, ATTN_DEV_CAPACITY);
    return t;
  }
  t.ok = true;
  if (j.window == 0 || at.l >= j.L - j.window) {
    const long p = static_cast<long>(s0) + at.l;
    t.rec = j.cache + (at.bh * j.capacity + (j.window > 0 ? p % j.window : p)) *
                          q4::record_bytes(M);
  }
  return t;
}

// Rows of k and v through shared memory: a block bulk-copies `tr` consecutive rows of each
// (rows are contiguous whatever L is), its warps quantise them into records in shared memory,
// and the records leave in 16-byte pieces. The bytes in flight are then bounded by shared
// memory, not by registers. Rows come in segments of seg_rows (the whole tensor, or, of a
// chunk longer than its ring, the last rows of each head), seg_tiles blocks each.
// 4 x 2048 tokens, 8 heads, D = 128, RoPE, rotated keys kept (111 MB): 25 us, 4.4 TB/s; bound
// by issue (225 instructions for a row's 256 values, 2.4 of 4 a cycle). Sixteen rows and seven
// blocks an SM: with 32 rows in 256 threads 8 % slower, eight rows 6 %; six blocks 2 % slower,
// eight the same.
template <int M, int ROPE>
__global__ void __launch_bounds__(kRowThreads, 7) append_q4_kernel(AppendQ4Job j, int tr,
                                                                   long seg_rows, int seg_tiles) {
  constexpr int D = 32 * M, REC = q4::record_bytes(M), P = REC / 16;
  constexpr int RW = q4::Lanes<M>::kRows, kWarps = kRowThreads / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full;
  __shared__ int abort_flag;
  __shared__ Target to[kMaxRows];
  __shared__ uint2 later[kMaxRows];
  dependents_may_launch();
  dependent_wait();
  if (gated_off(j.skip)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long seg = blockIdx.x / seg_tiles;
  const long in_seg = static_cast<long>(blockIdx.x % seg_tiles) * tr;
  const int n = static_cast<int>(min(static_cast<long>(tr), seg_rows - in_seg));
  // a segment's first row: heads are j.L rows apart, of which the last seg_rows count
  const long row0 = seg * j.L + j.l0 + in_seg;
  float* xk = reinterpret_cast<float*>(smem);
  float* xv = xk + tr * D;
  uint8_t* recs = smem + 2 * tr * D * 4;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    tc::mbar_init(&full, 1);
    tc::fence_mbar_init();
    const uint32_t bytes = static_cast<uint32_t>(n) * D * 4;
    tc::mbar_arrive_expect_tx(&full, 2 * bytes);
    tc::bulk_load(xk, j.k + row0 * D, bytes, &full);
    tc::bulk_load(xv, j.v + row0 * D, bytes, &full);
  }
  if (warp == 1 && lane < n)                 // meanwhile: where the rows go
    to[lane] = append_target<M, ROPE != kNoRope>(
        j, row_at(row0 + lane, static_cast<long>(j.B) * j.Hkv * j.L, j.Hkv, j.L), true);
  __syncthreads();
  if (!tc::mbar_wait(&full, 0, &abort_flag)) abort_flag = 1;
  __syncthreads();
  if (abort_flag) {                          // the copies are late
    if (threadIdx.x == 0) {
      tc::mbar_drain(&full, 0);
      report(j.status, ATTN_DEV_TIMEOUT);
    }
    return;
  }
  const q4::Lanes<M> at(lane);
  uint32_t doubts = 0;
  for (int i0 = warp * RW; i0 < n; i0 += kWarps * RW) {
    const int i = min(i0 + at.row, n - 1);   // lanes past the last row follow it
    const Target t = to[i];
    const bool on = at.in && i0 + at.row < n && t.ok;
    const uint2 d = append_rows<M, ROPE>(
        j, xk + i * D, xv + i * D, ROPE != kNoRope && t.ok ? j.table + t.angle * (j.R / 2) : j.table,
        t.rec ? recs + i * REC : nullptr, j.k_out ? j.k_out + (row0 + i) * D : nullptr, at, lane, on);
    doubts |= d.x | d.y;
    if (at.in && at.l == 0 && i0 + at.row < n) {
      const int sh = at.row * 4 * M;
      const uint32_t mask = M == 8 ? 0xffffffffu : (1u << (4 * M & 31)) - 1u;
      later[i] = make_uint2(d.x >> sh & mask, d.y >> sh & mask);
    }
  }
  // Second pass, rarely anything: kept out of the loop above, whose registers a call there
  // would have cost. A row's second pass is its own warp's.
  __syncwarp();
#pragma unroll 1
  for (int i0 = doubts ? warp * RW : n; i0 < n; i0 += kWarps * RW) {
#pragma unroll 1
    for (int i = i0; i < min(i0 + RW, n); ++i) {
      const uint2 d = later[i];
      const bool rot = ROPE != kNoRope;
      if (d.x)
        q4::quantise_exact<M>(xk + i * D, rot ? j.table + to[i].angle * (j.R / 2) : nullptr, j.R,
                              rot ? j.norm_w : nullptr, j.norm_eps, lane, d.x, recs + i * REC, 0);
      if (d.y)
        q4::quantise_exact<M>(xv + i * D, nullptr, 0, nullptr, 0.f, lane, d.y, recs + i * REC, 1);
    }
  }
  __syncthreads();
  for (int p = threadIdx.x; p < n * P; p += kRowThreads) {
    const int i = p / P;
    if (to[i].rec)
      reinterpret_cast<uint4*>(to[i].rec)[p - i * P] = reinterpret_cast<const uint4*>(recs)[p];
  }
}

// Records back to fp32: a block brings `tr` rows' records to shared memory in 16-byte
// pieces, then its warps write eight dims of key and value per lane. Bound by its stores: 4 x
// 2048 tokens, 8 heads, D = 128 (76 MB) 11.5 us, 6.6 TB/s.
template <int M>
__global__ void __launch_bounds__(kRowThreads) read_q4_kernel(ReadQ4Job j, int tr) {
  constexpr int D = 32 * M, REC = q4::record_bytes(M), P = REC / 16, RW = q4::Lanes<M>::kRows;
  __shared__ __align__(16) uint8_t recs[kMaxRows * REC];
  __shared__ const uint8_t* from[kMaxRows];
  dependents_may_launch();
  dependent_wait();
  if (gated_off(j.skip)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long rows = static_cast<long>(j.B) * j.Hkv * j.L;
  const long row0 = static_cast<long>(blockIdx.x) * tr;
  const int n = static_cast<int>(min(static_cast<long>(tr), rows - row0));
  if (threadIdx.x < n) {
    const RowAt at = row_at(row0 + threadIdx.x, rows, j.Hkv, j.L);
    const int s0 = j.start[at.b];
    const bool first = at.l == 0 && at.bh % j.Hkv == 0;
    const uint8_t* src = nullptr;
    if (s0 < 0) {
      if (first) report(j.status, ATTN_DEV_POSITION);
    } else if (j.window == 0 && static_cast<long>(s0) + j.L > j.capacity) {
      if (first) report(j.status, ATTN_DEV_CAPACITY);
    } else {
      const long p = static_cast<long>(s0) + at.l;
      src = j.cache + (at.bh * j.capacity + (j.window > 0 ? p % j.window : p)) * REC;
    }
    from[threadIdx.x] = src;
  }
  __syncthreads();
  for (int p = threadIdx.x; p < n * P; p += kRowThreads) {
    const int i = p / P;
    if (from[i])
      reinterpret_cast<uint4*>(recs)[p] = reinterpret_cast<const uint4*>(from[i])[p - i * P];
  }
  __syncthreads();
  const q4::Lanes<M> at(lane);
  for (int i0 = warp * RW; i0 < n; i0 += kRowThreads / 32 * RW) {
    const int i = i0 + at.row;
    if (!at.in || i >= n || !from[i]) continue;
    const uint8_t* rec = recs + i * REC;
    const uint16_t* sc = reinterpret_cast<const uint16_t*>(rec + 32 * M);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const float s = q4::bf16_to_float(sc[part * M + at.g]);
      float y[8];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t u =
            *reinterpret_cast<const uint16_t*>(rec + q4::quad_at<M>(part, at.g, at.quad(q)));
#pragma unroll
        for (int e = 0; e < 4; ++e)          // 2^23 + code + 8, less 2^23 + 8
          y[4 * q + e] = (__uint_as_float(0x4b000000u | (u >> (4 * e) & 15u)) - 8388616.0f) * s;
      }
      store_row<M>((part ? j.v : j.k) + (row0 + i) * D, at, y);
    }
  }
}

// ---------------------------------------------------------------- eviction

// Order of weights as unsigned keys, never 0: larger weight, larger key; -0 and +0 alike; NaN
// above everything (a slot whose weight is unknown is kept). The sum makes +0 of -0 and
// 0x7fffffff of every NaN.
__device__ __forceinline__ uint32_t weight_key(float w) {
  float c;
  asm("add.f32 %0, %1, 0f00000000;" : "=f"(c) : "f"(w));
  const uint32_t b = __float_as_uint(c);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_weight(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

constexpr int kFew = 256;                    // keys sharing the threshold's top bits, at most
constexpr int kSelItems = 8;                 // slots per thread and compaction tile
constexpr int kSelKeys = 40960;              // keys held in shared memory at most (160 KB)

// What the warps before this one counted (own: one value a warp), and all. wsum [32].
template <int kSelThreads>
__device__ __forceinline__ uint32_t warps_before(uint32_t own, uint32_t* wsum, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) wsum[warp] = own;
  __syncthreads();
  const uint32_t w = lane < kSelThreads / 32 ? wsum[lane] : 0u;
  total = __reduce_add_sync(0xffffffffu, w);
  return __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u);
}

// `parts` blocks per (row, head), each for a share of the kept slots: the need-th largest of
// the old slots' keys, then one ordered pass that writes the kept slots' numbers and weights.
// The largest by its top 11 or 13 bits (sign, exponent and two or four bits more: a histogram
// of them, summed from the top); then among the few keys that share those, gathered, by
// counting for each how many are larger; where they are not few, by histograms of the next
// bits first. The weights are read once where their keys fit in shared memory, the first of
// them before the length is known, else again from L2 in each pass. Bound by one block's issue
// and its chain of barriers: every instruction counts 16 or 32 times a pass (128 heads of up
// to 8192 slots: 8 us).
// With several parts, where the heads alone would leave SMs idle, every block finds the whole
// threshold for itself, writes its share and moves its records too: no second launch.
template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictQ4Job j, int held, int parts) {
  constexpr int kTopBits = kSelThreads == 1024 ? 13 : 11, kBins = 1 << kTopBits;
  constexpr int kPer = kBins / kSelThreads, kTileSlots = kSelThreads * kSelItems;
  constexpr int kShare = kSelThreads / kFew;     // threads that count for one of the few keys
  extern __shared__ __align__(16) uint32_t keys[];         // of the old slots, if they fit
  __shared__ __align__(16) uint32_t hist[kBins];
  __shared__ __align__(16) uint32_t few[kFew];
  __shared__ uint32_t wsum[32];
  __shared__ uint32_t found_bin, found_left, found_count, gathered;
  dependents_may_launch();
  dependent_wait();
  if (gated_off(j.skip)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = blockIdx.x / parts, part = blockIdx.x - head * parts;
  const long bh = head;
  const int b = head / j.Hkv;
  const bool lead = tid == 0 && part == 0 && head % j.Hkv == 0;            // one a batch row
  const float* w = j.weights + bh * j.capacity;
  float ahead[kSelItems];
#pragma unroll
  for (int e = 0; e < kSelItems; ++e) {
    const int i = tid + e * kSelThreads;
    ahead[e] = i < j.max_cache_len ? w[i] : 0.f;           // <= capacity
  }
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i)
      reinterpret_cast<uint4*>(hist)[tid + i * kSelThreads] = make_uint4(0, 0, 0, 0);
    if (tid == 0) gathered = 0;
    __syncthreads();
  };
  clear();
  const int n = j.cache_len[b];
  if (n < 0 || n > j.max_cache_len || n > j.capacity) {
    if (lead) report(j.status, ATTN_DEV_LENGTH);
    return;
  }
  float* wo = j.weights_out + bh * j.capacity_out;
  int32_t* index = j.index + bh * j.budget;
  const int kept = min(n, j.budget);
  if (lead) j.len_out[b] = kept;
  if (part == parts - 1) {
    for (long i = kept + tid; i < j.capacity_out; i += kSelThreads) wo[i] = 0.f;
    for (int i = kept + tid; i < j.budget; i += kSelThreads) index[i] = -1;
  }
  // Kept whatever its weight: all, or the recent slots, behind the others (`need` old ones).
  const int old = n <= j.budget ? 0 : n - j.recent, need = n <= j.budget ? 0 : j.budget - j.recent;

  // Keys of whole tiles, 0 behind the last; their histogram.
  const bool in_smem = old <= held;
  for (int i0 = 0; need > 0 && i0 < old; i0 += kTileSlots) {
#pragma unroll
    for (int e = 0; e < kSelItems; ++e) {
      const int i = i0 + tid + e * kSelThreads;
      if (i0 > 0) ahead[e] = i < old ? w[i] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < kSelItems; ++e) {
      const int i = i0 + tid + e * kSelThreads;
      const uint32_t k = i < old ? weight_key(ahead[e]) : 0u;
      if (in_smem) keys[i] = k;
      if (i < old) atomicAdd(&hist[k >> (32 - kTopBits)], 1u);
    }
  }
  __syncthreads();
  auto key_of = [&](int i) { return in_smem ? keys[i] : (i < old ? weight_key(w[i]) : 0u); };

  // Threshold: keys above T are kept, and the first `left` of those equal to it.
  uint32_t T = 0, left = static_cast<uint32_t>(need);
#pragma unroll 1
  for (int shift = 32 - kTopBits; need > 0;) {
    // bins from the top: thread t holds kPer of them, from kBins - 1 - kPer t down
    uint32_t h[kPer], mine = 0, total;
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
      const uint4 q = reinterpret_cast<const uint4*>(hist)[(kBins - kPer * tid - i) / 4 - 1];
      h[i] = q.w; h[i + 1] = q.z; h[i + 2] = q.y; h[i + 3] = q.x;
      mine += q.x + q.y + q.z + q.w;
    }
    // only the warp that holds the bin scans its own
    const uint32_t own = __reduce_add_sync(0xffffffffu, mine);
    uint32_t at = warps_before<kSelThreads>(own, wsum, total);
    if (at < left && at + own >= left) {
      uint32_t upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      at += upto - mine;
      if (at < left && at + mine >= left) {   // one thread
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (at < left && at + h[i] >= left) {
            found_bin = kBins - 1 - kPer * tid - i;
            found_left = left - at;
            found_count = h[i];
          }
          at += h[i];
        }
      }
    }
    __syncthreads();
    T |= found_bin << shift;
    left = found_left;
    const int count = static_cast<int>(found_count);
    if (shift == 0) break;
    if (count > kFew) {                      // the next ten bits (at most) of those
      const int next = shift > 10 ? shift - 10 : 0;
      clear();
      for (int i = tid; i < old; i += kSelThreads) {
        const uint32_t k = key_of(i);
        if (k >> shift == T >> shift)
          atomicAdd(&hist[(k >> next) & ((1u << (shift - next)) - 1)], 1u);
      }
      __syncthreads();
      shift = next;
      continue;
    }
    for (int i = tid; i < old; i += kSelThreads) {
      const uint32_t k = key_of(i);
      if (k >> shift == T >> shift) {        // (in bounds even if a weight has changed since)
        const uint32_t at = atomicAdd(&gathered, 1u);
        if (at < kFew) few[at] = k;
      }
    }
    if (tid >= count && tid < (count + 3) / 4 * 4) few[tid] = 0;           // below every key
    __syncthreads();
    if (warp * (32 / kShare) < count) {
      const int mine_at = tid / kShare;
      const uint32_t k = mine_at < count ? few[mine_at] : 0u;
      uint32_t more = 0, same = 0;
      for (int i = 4 * (tid % kShare); i < count; i += 4 * kShare) {
        const uint4 f = *reinterpret_cast<const uint4*>(few + i);
        more += (f.x > k) + (f.y > k) + (f.z > k) + (f.w > k);
        same += (f.x == k) + (f.y == k) + (f.z == k) + (f.w == k);
      }
#pragma unroll
      for (int o = 1; o < kShare; o <<= 1) {
        more += __shfl_xor_sync(0xffffffffu, more, o);
        same += __shfl_xor_sync(0xffffffffu, same, o);
      }
      if (mine_at < count && more < left && more + same >= left) {
        found_bin = k;                       // threads that agree on the key
        found_left = left - more;
      }
    }
    __syncthreads();
    T = found_bin;
    left = found_left;
    break;
  }

  // This block's share of the kept slots; their numbers take the histogram's place.
  const int share = (j.budget + parts - 1) / parts, lo = part * share, hi = min(lo + share, kept);
  auto keep = [&](int at, int slot, float weight) {
    if (at < lo || at >= hi) return;
    index[at] = slot;
    wo[at] = weight;
    if (parts > 1) hist[at - lo] = static_cast<uint32_t>(slot);
  };
  for (int i = old + tid; i < n; i += kSelThreads) keep(need + i - old, i, w[i]);

  // Ordered pass. Kept before a slot: those above T, and at most `left` equal to it. A warp's
  // slots are consecutive, 32 at a time, so its writes are too.
  uint32_t base_up = 0, base_eq = 0;
  const uint32_t below = (1u << lane) - 1u;
  for (int t0 = 0; need > 0 && t0 < old; t0 += kTileSlots) {
    const int i0 = t0 + warp * 32 * kSelItems + lane;
    uint32_t k[kSelItems], up[kSelItems], eq[kSelItems], own = 0, total;   // own: eq in the upper half
#pragma unroll
    for (int e = 0; e < kSelItems; ++e) {
      k[e] = key_of(i0 + 32 * e);
      up[e] = __ballot_sync(0xffffffffu, k[e] > T);
      eq[e] = __ballot_sync(0xffffffffu, k[e] == T);
      own += __popc(up[e]) + (__popc(eq[e]) << 16);        // at most 8192 of each a block
    }
    const uint32_t before = warps_before<kSelThreads>(own, wsum, total);
    uint32_t nup = base_up + (before & 0xffffu), neq = base_eq + (before >> 16);
#pragma unroll
    for (int e = 0; e < kSelItems; ++e) {
      const uint32_t u = nup + __popc(up[e] & below), q = neq + __popc(eq[e] & below);
      if (k[e] > T || (k[e] == T && q < left))
        keep(static_cast<int>(u + min(q, left)), i0 + 32 * e, key_weight(k[e]));
      nup += __popc(up[e]);
      neq += __popc(eq[e]);
    }
    base_up += total & 0xffffu;
    base_eq += total >> 16;
    __syncthreads();
  }
  if (parts == 1) return;                    // the records are moved by the next kernel
  __syncthreads();
  const int P = q4::record_bytes(j.D / 32) / 16, pieces = max(hi - lo, 0) * P;
  const uint4* src = reinterpret_cast<const uint4*>(j.cache) + bh * j.capacity * P;
  uint4* dst = reinterpret_cast<uint4*>(j.cache_out) + (bh * j.capacity_out + lo) * P;
  constexpr int U = 4;
  for (int i0 = tid; i0 < pieces; i0 += kSelThreads * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + kSelThreads * u;
      if (i < pieces) {
        const int r = i / P;                 // (and here)
        const uint32_t slot = min(hist[r], static_cast<uint32_t>(j.capacity - 1));
        v[u] = src[static_cast<long>(slot) * P + (i - r * P)];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + kSelThreads * u < pieces) dst[i0 + kSelThreads * u] = v[u];
  }
}

// The kept records, 16 bytes a thread, four in flight: 128 heads' 4096 of 8192 records of 144
// bytes (151 MB) in 27 us, 5.6 TB/s (two in flight 2.3 us more, eight 3.2; streaming loads and
// stores the same).
template <int M>
__global__ void __launch_bounds__(256) evict_move_kernel(EvictQ4Job j, unsigned per_head) {
  dependents_may_launch();
  dependent_wait();
  if (gated_off(j.skip)) return;
  constexpr int P = q4::record_bytes(M) / 16, U = 4;
  const long bh = blockIdx.x / per_head;
  const int b = static_cast<int>(bh / j.Hkv);
  const int n = j.cache_len[b];
  if (n < 0 || n > j.max_cache_len || n > j.capacity) return;
  const long pieces = static_cast<long>(min(n, j.budget)) * P;
  const uint4* src = reinterpret_cast<const uint4*>(j.cache) + bh * j.capacity * P;
  uint4* dst = reinterpret_cast<uint4*>(j.cache_out) + bh * j.capacity_out * P;
  const int32_t* index = j.index + bh * j.budget;
  for (long i0 = static_cast<long>(blockIdx.x % per_head) * 256 * U + threadIdx.x; i0 < pieces;
       i0 += static_cast<long>(per_head) * 256 * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long i = i0 + 256 * u;
      if (i < pieces) {
        const uint32_t r = static_cast<uint32_t>(i / P);
        // (in bounds even if the length has changed since the selection)
        const uint32_t slot = min(static_cast<uint32_t>(index[r]), static_cast<uint32_t>(j.capacity - 1));
        v[u] = src[static_cast<long>(slot) * P + (i - static_cast<long>(r) * P)];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long i = i0 + 256 * u;
      if (i < pieces) dst[i] = v[u];
    }
  }
}

}  // namespace

namespace {
template <int M, int ROPE>
cudaError_t launch_append(const AppendQ4Job& j, int tr, long seg_rows, int seg_tiles, unsigned grid,
                          cudaStream_t stream) {
  static PerContext<cudaError_t> allowed;    // the shared-memory size is per context
  const cudaError_t e = allowed.get(
      [] {
        return cudaFuncSetAttribute(append_q4_kernel<M, ROPE>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kMaxRows * (256 * M + q4::record_bytes(M)));
      },
      cudaErrorInvalidDevice, [](const cudaError_t& v) { return v == cudaSuccess; });
  if (e != cudaSuccess) return e;
  return launch_dependent(append_q4_kernel<M, ROPE>, grid, kRowThreads,
                          tr * (256 * M + q4::record_bytes(M)), stream, j, tr, seg_rows, seg_tiles);
}
}  // namespace

cudaError_t launch_append_q4(const AppendQ4Job& job, cudaStream_t stream) {
  AppendQ4Job j = job;
  const long heads = static_cast<long>(j.B) * j.Hkv;
  // The rows that leave anything: all, or of a chunk longer than its ring the last ones.
  const bool cut = !j.k_out && j.window > 0 && j.L > j.window;
  const int used = cut ? j.window : j.L;
  j.l0 = j.L - used;
  const long segs = cut ? heads : 1, seg_rows = cut ? used : heads * j.L;
  // Rows per block: 16 (8 wide ones: 18 KB), fewer while that leaves SMs without a block.
  int tr = j.D <= 128 ? 16 : 8;
  while (tr > 4 && (segs * seg_rows + tr - 1) / tr < 2 * 152) tr /= 2;
  const long tiles = (seg_rows + tr - 1) / tr;
  if (tiles * segs > 0x7fffffffL) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(tiles * segs);
  return with_groups(j.D / 32, [&](auto g) {
    constexpr int M = decltype(g)::value;
    const int t = static_cast<int>(tiles);
    if (!j.table) return launch_append<M, kNoRope>(j, tr, seg_rows, t, grid, stream);
    switch (rope_kind(j.R, j.D)) {
      case kRopeAll: return launch_append<M, kRopeAll>(j, tr, seg_rows, t, grid, stream);
      case kRopeQuads: return launch_append<M, kRopeQuads>(j, tr, seg_rows, t, grid, stream);
      default: return launch_append<M, kRopeDims>(j, tr, seg_rows, t, grid, stream);
    }
  });
}

cudaError_t launch_read_q4(const ReadQ4Job& j, cudaStream_t stream) {
  const long rows = static_cast<long>(j.B) * j.Hkv * j.L;
  int tr = kMaxRows;
  while (tr > 4 && (rows + tr - 1) / tr < 4 * 152) tr /= 2;
  const long blocks = (rows + tr - 1) / tr;
  if (blocks > 0x7fffffffL) return cudaErrorInvalidValue;
  return with_groups(j.D / 32, [&](auto g) {
    return launch_dependent(read_q4_kernel<decltype(g)::value>, static_cast<unsigned>(blocks),
                            kRowThreads, 0, stream, j, tr);
  });
}

namespace {
template <int T>
cudaError_t launch_select(const EvictQ4Job& j, unsigned heads, int parts, cudaStream_t stream) {
  static PerContext<cudaError_t> allowed;    // the shared-memory size is per context
  const cudaError_t e = allowed.get(
      [] {
        return cudaFuncSetAttribute(evict_select_kernel<T>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
      },
      cudaErrorInvalidDevice, [](const cudaError_t& v) { return v == cudaSuccess; });
  if (e != cudaSuccess) return e;
  constexpr int tile = T * kSelItems;        // whole tiles are held
  static_assert(kSelKeys % tile == 0, "");
  const int held = j.max_cache_len < kSelKeys ? (j.max_cache_len + tile - 1) / tile * tile : kSelKeys;
  return launch_dependent(evict_select_kernel<T>, heads * parts, T, held * 4, stream, j, held, parts);
}
}  // namespace

cudaError_t launch_evict_q4(const EvictQ4Job& j, cudaStream_t stream) {
  const unsigned heads = static_cast<unsigned>(j.B) * j.Hkv;
  // Short heads are chains of barriers, cheaper among 16 warps than among 32 (8 heads of 1100
  // slots: 7.3 us with the move as a second kernel, 8.8 with 32 warps); long ones are work on
  // the keys (128 heads of up to 8192: 38.5 and 35.2).
  const bool short_heads = j.max_cache_len <= 4096;
  // Heads that leave most SMs idle get several blocks, which move the records too (8 heads of
  // 1100 slots 6.7 us instead of 7.3, 16 of 8192 9.3 instead of 12.1, 32 of 4000 10.4 instead
  // of 11.3; with two blocks a head it was 64 of 4000 16.3 instead of 15.5).
  int parts = heads > 38 ? 1 : static_cast<int>(152 / heads);
  if (parts > 16) parts = 16;
  if ((j.budget + parts - 1) / parts > (short_heads ? 2048 : 8192)) parts = 1;
  const cudaError_t e = short_heads ? launch_select<512>(j, heads, parts, stream)
                                    : launch_select<1024>(j, heads, parts, stream);
  if (e != cudaSuccess || parts > 1) return e;
  return with_groups(j.D / 32, [&](auto g) {
    constexpr int M = decltype(g)::value;
    const long pieces = static_cast<long>(j.max_cache_len < j.budget ? j.max_cache_len : j.budget) *
                        (q4::record_bytes(M) / 16);
    if (pieces == 0) return cudaSuccess;
    // heads <= 65535 (host check)
    const long per = (pieces + 1023) / 1024, most = 0x7fffffffL / heads;
    const unsigned per_head = static_cast<unsigned>(per < most ? per : most);
    return launch_dependent(evict_move_kernel<M>, heads * per_head, 256, 0, stream, j, per_head);
  });
}

}  // namespace gqa
