// Planning and finishing of single-token attention over a 4-bit cache: how many splits a
// row gets, the merge of its splits and the per-slot attention weights. The split kernel is
// in decode_q4_kernel.cuh.
#include "decode_q4_kernel.cuh"

namespace gqa {

namespace {

constexpr int kSms = 152;
constexpr int kMaxSplits = 8 * kSms;           // of one row: no more than blocks on the GPU at once

constexpr int kFewSplits = 8;
// Slots whose weights one block adds up: the rows' sums, which every block needs, then weigh
// little (8 rows of up to 4000 slots, 64 heads over 8, with weights: 256 24.6 us, 512 22.7,
// 1024 21.1, 2048 21.7).
constexpr int kSlots = 1024;

// One query row's few splits by one warp: every load is on its way before the first factor is
// known, and no barrier is met.
__device__ __forceinline__ void merge_few(const DecodeQ4Job& j, const float2* ml, long row, int lane) {
  const int nlive = live_slots(j, j.cache_len[row / j.H], false);
  if (nlive <= j.chunk) return;              // finished by its one split, or invalid
  const int ns = (nlive - 1) / j.chunk + 1;
  const float* part = j.partial + row * j.nsplit * j.D;
  const float2 t = lane < ns ? ml[row * j.nsplit + lane] : make_float2(-INFINITY, 0.f);
  for (int d0 = 0; d0 < j.D; d0 += 128) {
    const int d = d0 + 4 * lane;
    float4 p[kFewSplits];
#pragma unroll
    for (int s = 0; s < kFewSplits; ++s)
      if (s < ns && d < j.D)
        p[s] = *reinterpret_cast<const float4*>(part + static_cast<long>(s) * j.D + d);
    const float m = warp_max(t.x);
    float f = t.x == -INFINITY ? 0.f : ex2(t.x - m) * t.y;
    f *= 1.0f / warp_sum(f);                 // a split's share of the row
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < kFewSplits; ++s) {
      const float fs = __shfl_sync(0xffffffffu, f, s);
      if (s < ns) {                          // a factor of 0 still passes on a NaN
        y.x = fmaf(fs, p[s].x, y.x); y.y = fmaf(fs, p[s].y, y.y);
        y.z = fmaf(fs, p[s].z, y.z); y.w = fmaf(fs, p[s].w, y.w);
      }
    }
    if (d < j.D)
      *reinterpret_cast<float4*>(j.out + row * j.D + d) = y;
  }
}

// Blocks [0, rows): one query row's splits merged, a split per warp at a time; with few
// splits eight rows, one a warp. Blocks after: with weights, kSlots slots of one kv head get
// the sum over its query heads of 2^(score - reference) / sum (one thread for each, heads in
// order, so the result does not depend on timing). A few us, bound by its chain of loads:
// merging 64 splits one after the other in a thread took 19 us, a warp per split 5.
__global__ void __launch_bounds__(256) decode_q4_finish_kernel(DecodeQ4Job j, unsigned rows,
                                                               unsigned slot_blocks) {
  __shared__ float factor[kMaxSplits];
  __shared__ float red[8], sums[8];
  __shared__ __align__(16) float acc[8][kMaxHeadDim];
  __shared__ float2 sh[8];
  dependent_wait();
  if (gated_off(j.skip)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float2* ml = reinterpret_cast<const float2*>(j.partial + static_cast<long>(j.B) * j.H * j.nsplit * j.D);
  if (blockIdx.x < rows) {
    if (j.nsplit <= kFewSplits) {
      const long r = static_cast<long>(blockIdx.x) * 8 + warp;
      if (r < static_cast<long>(j.B) * j.H) merge_few(j, ml, r, lane);
      return;
    }
    const long row = blockIdx.x;
    const int nlive = live_slots(j, j.cache_len[row / j.H], false);
    if (nlive <= j.chunk) return;            // finished by its one split, or invalid
    const int ns = (nlive - 1) / j.chunk + 1;
    ml += row * j.nsplit;
    float m = -INFINITY;
    for (int s = threadIdx.x; s < ns; s += 256) m = fmaxf(m, ml[s].x);
    m = warp_max(m);
    if (lane == 0) red[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
    float l = 0.f;
    for (int s = threadIdx.x; s < ns; s += 256) {
      const float2 t = ml[s];
      const float f = t.x == -INFINITY ? 0.f : ex2(t.x - m) * t.y;
      factor[s] = f;
      l += f;
    }
    l = warp_sum(l);
    if (lane == 0) sums[warp] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) l += sums[w];
    const float inv = 1.0f / l;
    const float* part = j.partial + row * j.nsplit * j.D;
    for (int d = 4 * lane; d < j.D; d += 128) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int s = warp; s < ns; s += 8) {
        const float f = factor[s] * inv;     // a split's share of the row
        const float4 t = *reinterpret_cast<const float4*>(part + static_cast<long>(s) * j.D + d);
        y.x = fmaf(f, t.x, y.x); y.y = fmaf(f, t.y, y.y);
        y.z = fmaf(f, t.z, y.z); y.w = fmaf(f, t.w, y.w);
      }
      *reinterpret_cast<float4*>(&acc[warp][d]) = y;
    }
    __syncthreads();
    if (threadIdx.x >= j.D) return;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) y += acc[w][threadIdx.x];
    j.out[row * j.D + threadIdx.x] = y;
    return;
  }
  const unsigned blk = blockIdx.x - rows;
  const long bh = blk / slot_blocks;
  const int b = static_cast<int>(bh / j.Hkv), hkv = static_cast<int>(bh - static_cast<long>(b) * j.Hkv);
  const int nlive = live_slots(j, j.cache_len[b], false);
  const int n0 = static_cast<int>(blk % slot_blocks) * kSlots + threadIdx.x;
  if (n0 - static_cast<int>(threadIdx.x) >= nlive) return;
  const int ns = (nlive - 1) / j.chunk + 1;
  const int G = j.H / j.Hkv;
  const long row0 = static_cast<long>(b) * j.H + hkv * G;
  float* w = j.weights + bh * j.capacity + n0;
  float before[kSlots / 256], sum[kSlots / 256];
#pragma unroll
  for (int u = 0; u < kSlots / 256; ++u) {
    before[u] = n0 + 256 * u < nlive ? w[256 * u] : 0.f;
    sum[u] = 0.f;
  }
  for (int g0 = 0; g0 < G; g0 += 8) {
    const int heads = min(8, G - g0);
    float s[kSlots / 256][8];
#pragma unroll
    for (int u = 0; u < kSlots / 256; ++u)
#pragma unroll
      for (int h = 0; h < 8; ++h)
        s[u][h] = h < heads && n0 + 256 * u < nlive
                      ? j.scores[(row0 + g0 + h) * j.pitch + n0 + 256 * u] : 0.f;
    if (warp < heads) {
      const float2* r = ml + (row0 + g0 + warp) * j.nsplit;
      float m = -INFINITY, l = 0.f;
      for (int i = lane; i < ns; i += 32) {
        const float2 t = r[i];
        const float top = fmaxf(m, t.x);
        if (top != -INFINITY) l = l * ex2(m - top) + ex2(t.x - top) * t.y;
        m = top;
      }
      const float top = warp_max(m);
      l = warp_sum(m == -INFINITY ? 0.f : l * ex2(m - top));
      if (lane == 0) sh[warp] = make_float2(top, 1.0f / l);
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h < heads) {
#pragma unroll
        for (int u = 0; u < kSlots / 256; ++u) sum[u] = fmaf(ex2(s[u][h] - sh[h].x), sh[h].y, sum[u]);
      }
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < kSlots / 256; ++u)
    if (n0 + 256 * u < nlive) w[256 * u] = before[u] + sum[u];
}

int eff_len(int max_cache_len, int window) {
  return window > 0 && window < max_cache_len ? window : max_cache_len;
}

// The most splits a plan takes: one wave of blocks, or up to twenty blocks an SM in at most
// twenty splits.
int most_splits(int B, int H, int Hkv, int D) {
  const long units = units_of(B, H, Hkv);
  if (units < 1) return 1;
  const long resident = kSms * resident_blocks(D / 32, head_tiles(H, Hkv));
  long n = resident / units, many = 20 * kSms / units;
  if (many > 20) many = 20;
  if (n < many) n = many;
  return static_cast<int>(n < 1 ? 1 : n);
}

// Two splits where one would hold more slots than an int counts in whole tiles.
int least_splits(int tiles) { return tiles > (1 << 30) / kTile ? 2 : 1; }

// The most splits of any length up to this one: it does not shrink as the length grows.
// Up to 16 tiles stay in one block: the second launch costs what the split saves. With
// weights it comes anyway (one row of 500 slots: 8.3 us in one block, 6.2 in four splits).
int split_bound(int B, int H, int Hkv, int D, int max_cache_len, int window, bool weights) {
  const int tiles = (eff_len(max_cache_len, window) - 1) / kTile + 1;
  if (tiles <= kShortTiles && !weights) return 1;
  const int most = (tiles + kWarps - 1) / kWarps;             // a tile for every warp
  const int want = most_splits(B, H, Hkv, D);
  return want < least_splits(tiles) ? least_splits(tiles) : (want < most ? want : most);
}

}  // namespace

// The split count whose time, in tiles of one SM at full load, comes out least:
//   k (per + 6) / r   k blocks on the busiest SM, each of `per` tiles (whole rounds of its
//                     warps) and a start and an end worth 6; r: what one block alone (0.65)
//                     or two (0.93) reach of an SM's rate
//   x 1.25            for a last wave that is not full: its blocks go to whichever SMs end first
//   + 6 or 12         the second launch, with few splits or many.
// Measured (us): one row of 131072 slots, 8 kv heads of 8: 38 splits 48.1, 57 46.8, 76 60.7;
// 8 rows of up to 4000: 2 21.8, 4 18.8, 7 17.6, 14 25.3; 64 rows of 512..8192, 8 kv heads of
// 4: 1 89.3, 2 82.5, 4 72.8, 8 73.8, 16 90.9; 8 rows of 4096, D = 256, 8 kv heads of 2: 2 27.3,
// 4 23.8, 6 31.8, 8 27.1.
void decode_q4_plan(int B, int H, int Hkv, int D, int max_cache_len, int window, bool weights,
                    int* nsplit, int* chunk) {
  const int tiles = (eff_len(max_cache_len, window) - 1) / kTile + 1;
  const int bound = split_bound(B, H, Hkv, D, max_cache_len, window, weights);
  const long units = units_of(B, H, Hkv);
  const int resident = resident_blocks(D / 32, head_tiles(H, Hkv));
  double least = 1e30;
  int best = tiles;
  for (int n = least_splits(tiles), per = tiles; n <= bound;
       n = per > 1 ? (tiles + per - 2) / (per - 1) : bound + 1) {
    per = (tiles + n - 1) / n;               // the next n is the first with fewer tiles a block
    const long k = (units * n + kSms - 1) / kSms;
    const double rate = k == 1 ? 0.65 : (k == 2 ? 0.93 : 1.0);
    const double wave = k > resident && k < 2 * resident ? 1.25 : 1.0;
    const double time = k * ((per + kWarps - 1) / kWarps * kWarps + 6) / rate * wave +
                        (n == 1 && !weights ? 0 : (n <= kFewSplits ? 6 : 12));
    if (time < least) {
      least = time;
      best = per;
    }
  }
  *chunk = best * kTile;
  *nsplit = (tiles + best - 1) / best;
}

namespace {
struct Layout {
  size_t scores, total;
  long pitch;
};
Layout layout(int B, int H, int D, int nsplit, int eff, bool weights) {
  Layout y{};
  const size_t rows = static_cast<size_t>(B) * H;
  size_t p = nsplit > 1 || weights ? rows * nsplit * (D + 2) * sizeof(float) : 0;
  y.scores = p = (p + 255) / 256 * 256;
  y.pitch = (eff + 3L) / 4 * 4;
  if (weights) p += rows * y.pitch * sizeof(float);
  y.total = p;
  return y;
}
}  // namespace

size_t decode_q4_bytes(int B, int H, int Hkv, int D, int max_cache_len, int window, bool weights) {
  return layout(B, H, D, split_bound(B, H, Hkv, D, max_cache_len, window, weights),
                eff_len(max_cache_len, window), weights).total;
}

size_t decode_q4_prepare(DecodeQ4Job* j) {
  decode_q4_plan(j->B, j->H, j->Hkv, j->D, j->max_cache_len, j->window, j->weights != nullptr,
                 &j->nsplit, &j->chunk);
  const Layout y = layout(j->B, j->H, j->D, j->nsplit, eff_len(j->max_cache_len, j->window),
                          j->weights != nullptr);
  j->pitch = y.pitch;
  j->scores_at = y.scores;
  return y.total;
}

void decode_q4_workspace(DecodeQ4Job* j, void* workspace) {
  j->partial = static_cast<float*>(workspace);
  j->scores = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) + j->scores_at)
                        : nullptr;
}

cudaError_t launch_decode_q4(const DecodeQ4Job& j, const StepQ4Args& st, cudaStream_t stream) {
  const cudaError_t e = j.D <= 128 ? launch_decode_q4_narrow(j, st, stream)
                                   : launch_decode_q4_wide(j, st, stream);
  if (e != cudaSuccess || (j.nsplit == 1 && !j.weights)) return e;
  const unsigned heads = static_cast<unsigned>(j.B) * j.H;
  const unsigned rows = j.nsplit == 1 ? 0 : (j.nsplit <= kFewSplits ? (heads + 7) / 8 : heads);
  const unsigned per = j.weights ? (eff_len(j.max_cache_len, j.window) - 1) / kSlots + 1 : 0;
  return launch_dependent(decode_q4_finish_kernel, rows + static_cast<unsigned>(j.B) * j.Hkv * per,
                          256, 0, stream, j, rows, per ? per : 1u);
}

}  // namespace gqa
