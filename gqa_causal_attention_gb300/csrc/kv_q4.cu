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
#include "kv_q4.cuh"
#include "tc_ptx.cuh"

namespace gqa {

namespace {

__host__ __device__ constexpr int quads_per_lane(int M) { return (8 * M + 31) / 32; }

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

// A lane's angles of a row: (cos, +-sin) of its quads' dims, the sign that of the partner's
// term; (1, 0) past the rotary dims.
template <int M, int NC>
__device__ __forceinline__ void load_angles(const float2* tab, int R, int lane,
                                            float (&c)[NC][4], float (&s)[NC][4]) {
  const int half = R / 2;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int d0 = 4 * (lane + 32 * k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[k][e] = 1.f;
      s[k][e] = 0.f;
    }
    if (d0 >= R) continue;
    if (half % 4 == 0) {                     // the quad lies within one half
      const bool low = d0 < half;
      const float4* ang = reinterpret_cast<const float4*>(tab + (low ? d0 : d0 - half));
      const float4 a0 = __ldg(ang), a1 = __ldg(ang + 1);
      const float sign = low ? -1.f : 1.f;
      c[k][0] = a0.x; c[k][1] = a0.z; c[k][2] = a1.x; c[k][3] = a1.z;
      s[k][0] = a0.y * sign; s[k][1] = a0.w * sign; s[k][2] = a1.y * sign; s[k][3] = a1.w * sign;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = d0 + e;
        if (d < R) {
          const float2 a = __ldg(tab + (d < half ? d : d - half));
          c[k][e] = a.x;
          s[k][e] = d < half ? -a.y : a.y;
        }
      }
    }
  }
}

// A lane's quads of the raw row x through RMSNorm (nw) and RoPE (angles c, s), in fp32, and
// a bound of their error. Every lane of the warp calls it.
template <int M, int NC>
__device__ __forceinline__ void rotate_quads(const float* x, const float (&c)[NC][4],
                                             const float (&s)[NC][4], int R, const float* nw,
                                             float eps, int lane, float (&y)[NC][4],
                                             float (&err)[NC]) {
  constexpr int D = 32 * M;
  const int half = R / 2;
  float a[NC][4];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int d0 = 4 * (lane + 32 * k);
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (d0 < D) t = *reinterpret_cast<const float4*>(x + d0);
    a[k][0] = t.x; a[k][1] = t.y; a[k][2] = t.z; a[k][3] = t.w;
    ss = fmaf(t.x, t.x, fmaf(t.y, t.y, fmaf(t.z, t.z, fmaf(t.w, t.w, ss))));
  }
  // y = a c + b s, b the rotary partner. Without a norm its error is below four roundings of
  // 2^-24 of the larger of a and b (the products' and the sum's); with one, below sixteen of
  // either: at most nine in the sum of squares, halved by the root, and one each in the
  // quotient, the root, its reciprocal and two products come on top.
  float inv = 1.f, unit = 0x1p-22f;
  if (nw) {
    inv = 1.0f / sqrtf(warp_sum(ss) / static_cast<float>(D) + eps);
    unit = 0x1p-19f;
  }
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int d0 = 4 * (lane + 32 * k);
    float b[4] = {0.f, 0.f, 0.f, 0.f};
    if (nw && d0 < D) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(nw + d0));
      a[k][0] = a[k][0] * inv * w.x; a[k][1] = a[k][1] * inv * w.y;
      a[k][2] = a[k][2] * inv * w.z; a[k][3] = a[k][3] * inv * w.w;
    }
    if (d0 < R) {
      if (half % 4 == 0) {
        const int p = d0 < half ? d0 + half : d0 - half;
        const float4 o = *reinterpret_cast<const float4*>(x + p);
        b[0] = o.x; b[1] = o.y; b[2] = o.z; b[3] = o.w;
        if (nw) {
          const float4 w = __ldg(reinterpret_cast<const float4*>(nw + p));
          b[0] = b[0] * inv * w.x; b[1] = b[1] * inv * w.y;
          b[2] = b[2] * inv * w.z; b[3] = b[3] * inv * w.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = d0 + e, p = d < half ? d + half : d - half;
          if (d < R) b[e] = nw ? x[p] * inv * __ldg(nw + p) : x[p];
        }
      }
    }
    float mag = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[k][e] = fmaf(a[k][e], c[k][e], b[e] * s[k][e]);
      mag = fmaxf(mag, fmaxf(fabsf(a[k][e]), fabsf(b[e])));
    }
    err[k] = mag * unit;
  }
}

// A lane's quads of a row as they are.
template <int M, int NC>
__device__ __forceinline__ void plain_quads(const float* x, int lane, float (&y)[NC][4]) {
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int d0 = 4 * (lane + 32 * k);
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (d0 < 32 * M) t = *reinterpret_cast<const float4*>(x + d0);
    y[k][0] = t.x; y[k][1] = t.y; y[k][2] = t.z; y[k][3] = t.w;
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

// One row by one warp: x, v the raw rows (any memory); the record goes to rec (any memory)
// unless it is nullptr, the rotated key to k_out unless that is. Groups whose rounding fp32
// cannot settle are noted in later[0 .. 3] (their lanes, key then value) for a second pass,
// or with later == nullptr done at once.
template <int M, bool ROT>
__device__ __forceinline__ void append_row(const AppendQ4Job& j, const float* x, const float* v,
                                           long angle, uint8_t* rec, float* k_out, int lane,
                                           uint32_t* later) {
  using namespace q4;
  constexpr int D = 32 * M, NC = quads_per_lane(M);
  const float2* tab = ROT ? j.table + angle * (j.R / 2) : nullptr;
  const float* nw = ROT ? j.norm_w : nullptr;
  float y[NC][4], err[NC], c[NC][4], s[NC][4];
  uint32_t q[NC], doubt[NC];
  auto settle = [&](int part) {
    const uint2 d = make_uint2(doubt[0], NC > 1 ? doubt[NC - 1] : 0u);
    store_part<M>(rec, part, q, lane);
    if (later) {
      if (lane == 0) *reinterpret_cast<uint2*>(later + 2 * part) = d;
    } else if (d.x | d.y) {
      quantise_exact<M>(part ? v : x, part ? nullptr : tab, j.R, part ? nullptr : nw, j.norm_eps,
                        lane, d, rec, part);
    }
  };
  if (ROT) load_angles<M>(tab, j.R, lane, c, s);           // on their way while v is done
  if (rec) {
    plain_quads<M>(v, lane, y);
    quantise_fast<NC, true>(y, err, q, doubt);
    settle(1);
  }
  if (ROT)
    rotate_quads<M>(x, c, s, j.R, nw, j.norm_eps, lane, y, err);
  else
    plain_quads<M>(x, lane, y);
  if (rec) {
    quantise_fast<NC, !ROT>(y, err, q, doubt);
    settle(0);
  }
  if (k_out) {
    __syncwarp();                            // in place: every lane has read its partners
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int d0 = 4 * (lane + 32 * k);
      if (d0 < D)
        *reinterpret_cast<float4*>(k_out + d0) = make_float4(y[k][0], y[k][1], y[k][2], y[k][3]);
    }
  }
}

// Rows of k and v through shared memory: a block bulk-copies `tr` consecutive rows of each
// (rows are contiguous whatever L is), its warps quantise them row by row into records in
// shared memory, and the records leave in 16-byte pieces. The bytes in flight are then
// bounded by shared memory, not by registers. Rows come in segments of seg_rows (the whole
// tensor, or, of a chunk longer than its ring, the last rows of each head), seg_tiles blocks
// each.
template <int M, bool ROT>
__global__ void __launch_bounds__(kRowThreads, M <= 4 ? 6 : 4) append_q4_kernel(AppendQ4Job j, int tr, long seg_rows,
                                                        int seg_tiles) {
  constexpr int D = 32 * M, REC = q4::record_bytes(M), P = REC / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full;
  __shared__ int abort_flag;
  __shared__ Target to[kMaxRows];
  __shared__ __align__(8) uint32_t later[kMaxRows][4];
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
    to[lane] = append_target<M, ROT>(
        j, row_at(row0 + lane, static_cast<long>(j.B) * j.Hkv * j.L, j.Hkv, j.L), true);
  __syncthreads();
  if (!tc::mbar_wait(&full, 0, &abort_flag)) abort_flag = 1;
  __syncthreads();
  if (abort_flag) {                          // the copies never came
    if (threadIdx.x == 0) report(j.status, ATTN_DEV_TIMEOUT);
    return;
  }
  for (int i = warp; i < n; i += kRowThreads / 32) {
    const Target t = to[i];
    if (t.ok && (t.rec || j.k_out))
      append_row<M, ROT>(j, xk + i * D, xv + i * D, t.angle, t.rec ? recs + i * REC : nullptr,
                         j.k_out ? j.k_out + (row0 + i) * D : nullptr, lane, later[i]);
  }
  // Second pass, rarely anything: kept out of the loop above, whose registers a call there
  // would have cost (and 6 us at 4 x 2048 tokens). A row's second
  // pass is its own warp's.
  __syncwarp();
  for (int i = warp; i < n; i += kRowThreads / 32) {
    if (!to[i].rec) continue;
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
      const uint2 d = *reinterpret_cast<const uint2*>(&later[i][2 * part]);
      if (!(d.x | d.y)) continue;
      const bool rot = ROT && part == 0;
      q4::quantise_exact<M>((part ? xv : xk) + i * D,
                            rot ? j.table + to[i].angle * (j.R / 2) : nullptr, j.R,
                            rot ? j.norm_w : nullptr, j.norm_eps, lane, d, recs + i * REC, part);
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
// pieces, then a warp per row writes four dims of key and value per lane.
template <int M>
__global__ void __launch_bounds__(kRowThreads) read_q4_kernel(ReadQ4Job j, int tr) {
  constexpr int D = 32 * M, NC = quads_per_lane(M), REC = q4::record_bytes(M), P = REC / 16;
  __shared__ __align__(16) uint8_t recs[kMaxRows * REC];
  __shared__ const uint8_t* from[kMaxRows];
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
  for (int i = warp; i < n; i += kRowThreads / 32) {
    if (!from[i]) continue;
    const uint8_t* rec = recs + i * REC;
    const long row = row0 + i;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int ch = lane + 32 * k;
      if (ch >= 8 * M) continue;
      const int g = ch >> 3, e = ch & 7;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const int off = part ? 16 * M + 2 * (e * M + g) : 4 * ((e >> 1) * M + g) + 2 * (e & 1);
        const uint32_t c = *reinterpret_cast<const uint16_t*>(rec + off);
        const float s = q4::bf16_to_float(
            *reinterpret_cast<const uint16_t*>(rec + (32 + 2 * part) * M + 2 * g));
        // 2^23 + u, less 2^23 + 8
        auto value = [&](uint32_t u) {
          return (__uint_as_float(0x4b000000u | (u & 15u)) - 8388616.0f) * s;
        };
        const float4 y = make_float4(value(c), value(c >> 4), value(c >> 8), value(c >> 12));
        *reinterpret_cast<float4*>((part ? j.v : j.k) + row * D + 4 * ch) = y;
      }
    }
  }
}

// A step's first pass: a warp per row, the q rows (normed, rotated, fp32) first, then
// the k and v rows.
template <int M>
__global__ void __launch_bounds__(256) prep_q4_kernel(PrepQ4Job j) {
  if (gated_off(j.kv.skip)) return;
  constexpr int D = 32 * M, NC = quads_per_lane(M);
  const AppendQ4Job& a = j.kv;
  const int lane = threadIdx.x & 31;
  const long qrows = static_cast<long>(a.B) * j.H, kvrows = static_cast<long>(a.B) * a.Hkv;
  const long step = static_cast<long>(gridDim.x) * 8;
  for (long row = static_cast<long>(blockIdx.x) * 8 + threadIdx.x / 32; row < qrows + kvrows;
       row += step) {
    if (row >= qrows) {
      const RowAt at = row_at(row - qrows, kvrows, a.Hkv, 1);
      const Target t = append_target<M, true>(a, at, lane == 0);
      if (t.ok)
        append_row<M, true>(a, a.k + at.bh * D, a.v + at.bh * D, t.angle, t.rec, nullptr, lane,
                            nullptr);
      continue;
    }
    const int b = static_cast<int>(row / j.H);
    const int s0 = a.start[b], p0 = a.pos ? a.pos[b] : s0;
    const bool ok = s0 >= 0 && p0 >= 0 && p0 < a.max_positions &&
                    (a.window > 0 || s0 < a.capacity);
    if (row % j.H == 0 && lane == 0) j.cache_len[b] = ok ? s0 + 1 : 0;
    if (!ok) continue;                       // the row's key rows report it
    float y[NC][4], err[NC], c[NC][4], s[NC][4];
    load_angles<M>(a.table + static_cast<long>(p0) * (a.R / 2), a.R, lane, c, s);
    rotate_quads<M>(j.q + row * D, c, s, a.R, j.q_norm_w, a.norm_eps, lane, y, err);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int d0 = 4 * (lane + 32 * k);
      if (d0 < D)
        *reinterpret_cast<float4*>(j.qrot + row * D + d0) =
            make_float4(y[k][0], y[k][1], y[k][2], y[k][3]);
    }
  }
}

// ---------------------------------------------------------------- eviction

// Order of weights as unsigned keys: larger weight, larger key; -0 and +0 alike; NaN
// above everything (a slot whose weight is unknown is kept).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr int kSelThreads = 1024;
constexpr int kSelItems = 4;                 // slots per thread and compaction tile
constexpr int kSelKeys = 40960;              // keys held in shared memory at most (160 KB)

// One block per (row, head): the need-th largest of the old slots' keys by three radix
// passes (11, 11, 10 bits from the top), then one ordered pass that writes the kept
// slots' numbers and weights. The keys are read once from memory where they fit in
// shared memory, else again from L2 in each pass.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictQ4Job j, int held) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t wsum[32];
  __shared__ uint32_t found_bin, found_left;
  if (gated_off(j.skip)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long bh = blockIdx.x;
  const int b = static_cast<int>(bh / j.Hkv);
  const int n = j.cache_len[b];
  if (n < 0 || n > j.max_cache_len || n > j.capacity) {
    if (tid == 0 && bh % j.Hkv == 0) report(j.status, ATTN_DEV_LENGTH);
    return;
  }
  const float* w = j.weights + bh * j.capacity;
  float* wo = j.weights_out + bh * j.capacity_out;
  int32_t* index = j.index + bh * j.budget;
  const int kept = min(n, j.budget);
  if (tid == 0 && bh % j.Hkv == 0) j.len_out[b] = kept;
  for (long i = kept + tid; i < j.capacity_out; i += kSelThreads) wo[i] = 0.f;
  for (int i = kept + tid; i < j.budget; i += kSelThreads) index[i] = -1;
  if (n <= j.budget) {
    for (int i = tid; i < n; i += kSelThreads) {
      index[i] = i;
      wo[i] = w[i];
    }
    return;
  }
  const int old = n - j.recent;              // recent <= budget < n
  const bool in_smem = old <= held;
  if (in_smem) {
    for (int i = tid; i < old; i += kSelThreads) keys[i] = weight_key(w[i]);
    __syncthreads();
  }
  auto key_of = [&](int i) { return in_smem ? keys[i] : weight_key(w[i]); };

  // Threshold: keys above T are kept, and the first `left` of those equal to it.
  uint32_t T = 0, left = static_cast<uint32_t>(j.budget - j.recent);
  const bool any_old = left > 0;
  if (any_old) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const int bits = pass == 2 ? 10 : 11;
      const uint32_t above = pass == 0 ? 0u : 0xffffffffu << (shift + bits);
      for (int i = tid; i < 2048; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < old; i += kSelThreads) {
        const uint32_t k = key_of(i);
        if ((k & above) == (T & above)) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
      }
      __syncthreads();
      // bins from the top: thread t holds bins 2047 - 2 t and 2046 - 2 t
      const uint32_t h0 = hist[2047 - 2 * tid], h1 = hist[2046 - 2 * tid];
      uint32_t incl = h0 + h1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) wsum[warp] = incl;
      __syncthreads();
      uint32_t base = 0;
      for (int i = 0; i < warp; ++i) base += wsum[i];
      const uint32_t end = base + incl, begin = end - h0 - h1;
      if (begin < left && end >= left) {      // exactly one thread
        const bool second = begin + h0 < left;
        found_bin = second ? 2046 - 2 * tid : 2047 - 2 * tid;
        found_left = left - begin - (second ? h0 : 0);
      }
      __syncthreads();
      T |= found_bin << shift;
      left = found_left;
    }
  }
  // Ordered pass. Kept before a slot: those above T, and at most `left` equal to it.
  uint32_t base_up = 0, base_eq = 0;
  for (int t0 = 0; t0 < n; t0 += kSelThreads * kSelItems) {
    const int i0 = t0 + tid * kSelItems;
    uint32_t up = 0, eq = 0;                  // bit e: slot i0 + e
#pragma unroll
    for (int e = 0; e < kSelItems; ++e) {
      const int i = i0 + e;
      if (i >= old) {
        if (i < n) up |= 1u << e;
      } else if (any_old) {
        const uint32_t k = key_of(i);
        if (k > T) up |= 1u << e;
        if (k == T) eq |= 1u << e;
      }
    }
    // counts of both in one word: at most 4096 each
    const uint32_t own = __popc(up) | static_cast<uint32_t>(__popc(eq)) << 16;
    uint32_t incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();                          // wsum of the tile before is read
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    uint32_t before = incl - own, total = 0;
    for (int i = 0; i < 32; ++i) {
      if (i < warp) before += wsum[i];
      total += wsum[i];
    }
    uint32_t nup = base_up + (before & 0xffffu), neq = base_eq + (before >> 16);
#pragma unroll
    for (int e = 0; e < kSelItems; ++e) {
      const bool is_up = up >> e & 1u, is_eq = eq >> e & 1u;
      if (is_up || (is_eq && neq < left)) {
        const uint32_t at = nup + min(neq, left);
        index[at] = i0 + e;
        wo[at] = w[i0 + e];
      }
      nup += is_up;
      neq += is_eq;
    }
    base_up += total & 0xffffu;
    base_eq += total >> 16;
  }
}

// The kept records, 16 bytes a thread.
template <int M>
__global__ void __launch_bounds__(256) evict_move_kernel(EvictQ4Job j) {
  if (gated_off(j.skip)) return;
  constexpr int P = q4::record_bytes(M) / 16, U = 4;
  const long bh = blockIdx.y;
  const int b = static_cast<int>(bh / j.Hkv);
  const int n = j.cache_len[b];
  if (n < 0 || n > j.max_cache_len || n > j.capacity) return;
  const long pieces = static_cast<long>(min(n, j.budget)) * P;
  const uint4* src = reinterpret_cast<const uint4*>(j.cache) + bh * j.capacity * P;
  uint4* dst = reinterpret_cast<uint4*>(j.cache_out) + bh * j.capacity_out * P;
  const int32_t* index = j.index + bh * j.budget;
  for (long i0 = static_cast<long>(blockIdx.x) * 256 * U + threadIdx.x; i0 < pieces;
       i0 += static_cast<long>(gridDim.x) * 256 * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long i = i0 + 256 * u;
      if (i < pieces) {
        const uint32_t r = static_cast<uint32_t>(i / P);
        v[u] = src[static_cast<long>(index[r]) * P + (i - static_cast<long>(r) * P)];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long i = i0 + 256 * u;
      if (i < pieces) dst[i] = v[u];
    }
  }
}

unsigned row_blocks(long rows) {
  const long blocks = (rows + 7) / 8;
  return static_cast<unsigned>(blocks < 152L * 64 ? blocks : 152L * 64);
}

}  // namespace

namespace {
template <int M, bool ROT>
cudaError_t launch_append(const AppendQ4Job& j, int tr, long seg_rows, int seg_tiles, unsigned grid,
                          cudaStream_t stream) {
  static PerContext<cudaError_t> allowed;    // the shared-memory size is per context
  const cudaError_t e = allowed.get(
      [] {
        return cudaFuncSetAttribute(append_q4_kernel<M, ROT>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kMaxRows * (256 * M + q4::record_bytes(M)));
      },
      cudaErrorInvalidDevice, [](const cudaError_t& v) { return v == cudaSuccess; });
  if (e != cudaSuccess) return e;
  append_q4_kernel<M, ROT><<<grid, kRowThreads, tr * (256 * M + q4::record_bytes(M)), stream>>>(
      j, tr, seg_rows, seg_tiles);
  return cudaGetLastError();
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
    return j.table ? launch_append<M, true>(j, tr, seg_rows, static_cast<int>(tiles), grid, stream)
                   : launch_append<M, false>(j, tr, seg_rows, static_cast<int>(tiles), grid, stream);
  });
}

cudaError_t launch_read_q4(const ReadQ4Job& j, cudaStream_t stream) {
  const long rows = static_cast<long>(j.B) * j.Hkv * j.L;
  int tr = kMaxRows;
  while (tr > 4 && (rows + tr - 1) / tr < 4 * 152) tr /= 2;
  const long blocks = (rows + tr - 1) / tr;
  if (blocks > 0x7fffffffL) return cudaErrorInvalidValue;
  return with_groups(j.D / 32, [&](auto g) {
    read_q4_kernel<decltype(g)::value><<<static_cast<unsigned>(blocks), kRowThreads, 0, stream>>>(j, tr);
    return cudaGetLastError();
  });
}

cudaError_t launch_prep_q4(const PrepQ4Job& j, cudaStream_t stream) {
  const unsigned grid = row_blocks(static_cast<long>(j.kv.B) * (j.H + j.kv.Hkv));
  return with_groups(j.kv.D / 32, [&](auto g) {
    prep_q4_kernel<decltype(g)::value><<<grid, 256, 0, stream>>>(j);
    return cudaGetLastError();
  });
}

cudaError_t launch_evict_q4(const EvictQ4Job& j, cudaStream_t stream) {
  static PerContext<cudaError_t> allowed;    // the shared-memory size is per context
  const cudaError_t e = allowed.get(
      [] {
        return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSelKeys * 4);
      },
      cudaErrorInvalidDevice, [](const cudaError_t& v) { return v == cudaSuccess; });
  if (e != cudaSuccess) return e;
  const int held = j.max_cache_len < kSelKeys ? j.max_cache_len : kSelKeys;
  const unsigned heads = static_cast<unsigned>(j.B) * j.Hkv;
  evict_select_kernel<<<heads, kSelThreads, held * 4, stream>>>(j, held);
  if (const cudaError_t l = cudaGetLastError(); l != cudaSuccess) return l;
  return with_groups(j.D / 32, [&](auto g) {
    constexpr int M = decltype(g)::value;
    const long pieces = static_cast<long>(j.max_cache_len < j.budget ? j.max_cache_len : j.budget) *
                        (q4::record_bytes(M) / 16);
    if (pieces == 0) return cudaSuccess;
    long blocks = (pieces + 1023) / 1024;
    if (blocks > 65536) blocks = 65536;
    // heads on the y axis: the host check keeps B * Hkv <= 65535
    evict_move_kernel<M><<<dim3(static_cast<unsigned>(blocks), heads), 256, 0, stream>>>(j);
    return cudaGetLastError();
  });
}

}  // namespace gqa
