// Embedding: rows of a vocabulary matrix, scaled, and the matrix's gradient by sorted tokens.
//
//   y_i = s W[id_i]                        (a row of zeros where id_i is outside [0, V))
//   dW_v = s sum_{i : id_i = v} dy_i       (v other than the padding id), or added to dW
//
// Both are bound by memory: the forward pass reads the distinct rows and writes N H elements, the
// gradient reads N H elements and writes V H (or reads and writes the distinct rows).
//
// The gradient's sums have one order, whatever the schedule: the tokens are sorted by (key,
// position), the key a permutation of the id, and cut into tiles; a row of dW is the sum over its
// tokens in that order in fp32, one part for each tile that it has tokens in, the parts added in
// order, and rounded once.
//   bucket  every block sorts its stretch of positions by range of the vocabulary (every 512th id)
//   sort    every block gathers one range's tokens, which the stretches hold in order, and sorts
//           them by key.  No block waits for another, no atomics in global memory.
//           Few tokens are sorted in one launch, whose blocks each read all ids and keep their
//           range's: 8 us for 5003 and 9 for 8192, where the two launches take 12 and 13; 48 for
//           131072, where they take 24.
//   tiles   every tile's tokens, 256 columns a warp: rows that lie within the tile are finished,
//           the others leave a part; beside them, zeros for the rows without a token
//   join    the rows with several parts
#include <type_traits>

#include "flce_device.cuh"
#include "flce_internal.h"
#include "flce_launch.cuh"

namespace flce {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ----------------------------------------------------------------------------- 8 elements of a row

// A warp holds 256 columns of a row, a lane 8 of them.  Where 16-byte accesses divide the rows
// (ALIGNED) they are 8 consecutive ones; else every 32nd, by accesses of one element each that
// are consecutive across the lanes: a warp's access then takes 2 or 4 sectors whatever the row's
// alignment, a fifth of what shifting the words of unaligned 16-byte chunks into place takes.
constexpr int kCols = 256;

//   LANES: of a row's group of columns, 32 but where the forward pass has several rows in a warp.
template <bool ALIGNED, int LANES = 32>
struct Place {
  int c;  // the lane's first column
  __device__ __forceinline__ Place(int group, int lane) : c(group * (8 * LANES) + (ALIGNED ? lane * 8 : lane)) {}
  __device__ __forceinline__ bool in(int e, int h) const { return ALIGNED ? c < h : c + LANES * e < h; }
  __device__ __forceinline__ int col(int e) const { return c + (ALIGNED ? e : LANES * e); }
};

// As they lie in memory: loads are issued together and their words taken apart after the last.
template <typename T, bool ALIGNED>
struct Words {
  static constexpr bool kPacked = ALIGNED && sizeof(T) == 2;
  uint32_t u[kPacked ? 4 : 8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < (kPacked ? 4 : 8); ++e) u[e] = 0;
  }
  // Lanes past the row's end load its last elements, which nobody uses: without a branch among them
  // the loads of several rows are under way together (the gradient of 131072 x 1001 bf16 in 128 us
  // for 273, of 131072 x 4096 in 259 for 343).
  template <int LANES>
  __device__ __forceinline__ void load(const T* row, const Place<ALIGNED, LANES>& at, int h) {
    if (ALIGNED) {
      const uint4* p = reinterpret_cast<const uint4*>(row + min(at.c, h - 8));
      const uint4 a = *p;
      u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w;
      if (!kPacked) {
        const uint4 b = p[1];
        u[kPacked ? 0 : 4] = b.x, u[kPacked ? 0 : 5] = b.y, u[kPacked ? 0 : 6] = b.z, u[kPacked ? 0 : 7] = b.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const T* p = row + min(at.col(e), h - 1);
        if (sizeof(T) == 2) u[kPacked ? 0 : e] = static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << 16;
        else u[kPacked ? 0 : e] = *reinterpret_cast<const uint32_t*>(p);
      }
    }
  }
  __device__ __forceinline__ float value(int e) const {
    if (kPacked) return __uint_as_float((e & 1) ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
    return __uint_as_float(u[kPacked ? 0 : e]);
  }
};

template <bool ALIGNED, int LANES>
__device__ __forceinline__ void store8(__nv_bfloat16* row, const Place<ALIGNED, LANES>& at, int h, const float (&x)[8]) {
  if (ALIGNED) {
    if (at.c < h)
      __stcs(reinterpret_cast<uint4*>(row + at.c), make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at.in(e, h)) row[at.col(e)] = __float2bfloat16_rn(x[e]);
  }
}
template <bool ALIGNED, int LANES>
__device__ __forceinline__ void store8(float* row, const Place<ALIGNED, LANES>& at, int h, const float (&x)[8]) {
  if (ALIGNED) {
    if (at.c < h) {
      __stcs(reinterpret_cast<float4*>(row + at.c), make_float4(x[0], x[1], x[2], x[3]));
      __stcs(reinterpret_cast<float4*>(row + at.c) + 1, make_float4(x[4], x[5], x[6], x[7]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at.in(e, h)) row[at.col(e)] = x[e];
  }
}

// ----------------------------------------------------------------------------- forward

constexpr int kFwdThreads = 256;
constexpr int kFwdUnits = 4;  // of a warp, as many rows' columns in flight
constexpr int64_t kScanIds = 16384;  // of a block

// Blocks below `scans` look the ids over, ahead of the rows so that none of it is left at the end:
// one writes the status word, several (for many ids) record errors in a word that was cleared.  In
// the others LANES threads take kFwdUnits consecutive (row, 8 LANES columns).
//   Bound by memory: 131072 x 4096 bf16, a vocabulary's frequencies, 216 us (1.36 GB through DRAM).
//   Several rows in a warp where they are short: 131072 x 64 in 13 us for 18, 2^20 x 64 in 30 for 89.
//   Times with one scanning block behind the rows, one ahead of them, and with these: 131072 x 512
// in 55, 39, 38 us, 131072 x 64 in 31, 33, 18, 131072 x 4096 in 338, 317, 318; 20000 x 512 in 14, 12, 13.
template <typename T, bool ALIGNED, int LANES>
__global__ void __launch_bounds__(kFwdThreads) embed_forward_kernel(int64_t n, int h, int64_t v, float scale,
                                                                    const int32_t* __restrict__ ids,
                                                                    const T* __restrict__ w, T* __restrict__ y,
                                                                    int groups, int scans, int* status) {
  griddep_begin();
  if (blockIdx.x < scans) {
    const int64_t to = min((static_cast<int64_t>(blockIdx.x) + 1) * kScanIds, n);
    int bad = 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kScanIds + threadIdx.x; i < to; i += 8 * kFwdThreads) {
      uint32_t id[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) id[k] = i + k * kFwdThreads < to ? static_cast<uint32_t>(ids[i + k * kFwdThreads]) : 0u;
#pragma unroll
      for (int k = 0; k < 8; ++k) bad |= id[k] >= static_cast<uint64_t>(v);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0 && (bad || scans == 1)) *status = bad ? kErrLabel : kOk;
    return;
  }
  const int lane = threadIdx.x % LANES;
  const int64_t first = (static_cast<int64_t>(blockIdx.x - scans) * (kFwdThreads / LANES) + threadIdx.x / LANES) * kFwdUnits;
  int64_t row = first / groups;
  int group = static_cast<int>(first - row * groups);
  int64_t rows[kFwdUnits], id[kFwdUnits];
  int cols[kFwdUnits];
#pragma unroll
  for (int k = 0; k < kFwdUnits; ++k) {
    rows[k] = row;
    cols[k] = group;
    id[k] = row < n ? ids[row] : -1;
    if (++group == groups) group = 0, ++row;
  }
  Words<T, ALIGNED> x[kFwdUnits];
#pragma unroll
  for (int k = 0; k < kFwdUnits; ++k) {
    x[k].zero();
    if (id[k] >= 0 && id[k] < v) x[k].load(w + id[k] * h, Place<ALIGNED, LANES>(cols[k], lane), h);
  }
#pragma unroll
  for (int k = 0; k < kFwdUnits; ++k) {
    if (rows[k] >= n) return;
    float z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = x[k].value(e) * scale;
    store8<ALIGNED, LANES>(y + rows[k] * h, Place<ALIGNED, LANES>(cols[k], lane), h, z);
  }
}

// ----------------------------------------------------------------------------- sort

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRound = 4096;  // tokens of a block's shared memory; a range with more takes several rounds
constexpr int kSearchStep = 256;  // the first of a search among the stretches
static_assert(2 * kSearchStep > kEmbedStretches, "steps of 256, 128, ... reach each");
constexpr int kPerMost = kEmbedIdsMost / kEmbedRanges;  // ids of a range

// Inclusive sum over the block's threads; *all gets the total.  `part` holds a word for each warp.
__device__ __forceinline__ int block_scan(int x, int* part, int* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(kFull, x, d);
    if (lane >= d) x += up;
  }
  __syncthreads();
  if (lane == 31) part[warp] = x;
  __syncthreads();
  const int w = lane < kSortWarps ? part[lane] : 0;
  const int before = __reduce_add_sync(kFull, lane < warp ? w : 0);
  *all = __reduce_add_sync(kFull, w);
  return x + before;
}

// The lane's place among the warp's lanes with its key, behind row[key] earlier ones; row[key]
// moves on.  Lanes of `some` alone call it.
__device__ __forceinline__ int take_rank(uint32_t some, int key, int32_t* row, int lane) {
  const uint32_t same = __match_any_sync(some, key);
  const int rank = row[key] + __popc(same & ((1u << lane) - 1));
  __syncwarp(some);
  if ((same >> lane) == 1u) row[key] = rank + 1;  // the highest of them
  __syncwarp(some);
  return rank;
}

// Block s: positions [s len, (s + 1) len), sorted by range (stable) into tokens[s len ..] as (id,
// position); off[r stretches + s] is where range r starts in it, the last entry how many tokens
// it holds.  Padding and ids outside the vocabulary are left out.
__global__ void __launch_bounds__(kSortThreads) embed_bucket_kernel(int n, int v, int len, int pad,
                                                                    const int32_t* __restrict__ ids,
                                                                    int2* __restrict__ tokens,
                                                                    int32_t* __restrict__ off, int32_t* __restrict__ bad) {
  __shared__ int32_t count[kSortWarps][kEmbedRanges];
  __shared__ int part[kSortWarps];
  griddep_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int stretches = static_cast<int>(gridDim.x);
  for (int i = tid; i < kSortWarps * kEmbedRanges; i += kSortThreads) (&count[0][0])[i] = 0;
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * len;
  const int mine = static_cast<int>(min(static_cast<int64_t>(len), n - first));
  const int each = (mine + kSortThreads - 1) / kSortThreads * 32;  // of a warp
  const int w0 = warp * each, w1 = min(w0 + each, mine);
  int32_t* row = count[warp];
  int outside = 0;
  for (int i0 = w0; i0 < w1; i0 += 32) {  // count
    const int id = i0 + lane < w1 ? ids[first + i0 + lane] : -1;
    const bool in = static_cast<uint32_t>(id) < static_cast<uint32_t>(v);
    outside |= i0 + lane < w1 && !in;
    if (in && id != pad) atomicAdd(row + (id & (kEmbedRanges - 1)), 1);
  }
  outside = __syncthreads_or(outside);
  if (tid == 0) bad[blockIdx.x] = outside;
  // exclusive sums over (range, warp)
  int base = 0;
  for (int r0 = 0; r0 < kEmbedRanges; r0 += kSortThreads) {
    const int r = r0 + tid;
    int total = 0, all;
    if (r < kEmbedRanges)
      for (int k = 0; k < kSortWarps; ++k) total += count[k][r];
    int at = base + block_scan(total, part, &all) - total;
    base += all;
    if (r < kEmbedRanges) off[static_cast<int64_t>(r) * stretches + blockIdx.x] = at;
    if (r < kEmbedRanges)
      for (int k = 0; k < kSortWarps; ++k) {
        const int c = count[k][r];
        count[k][r] = at;
        at += c;
      }
  }
  if (tid == 0) off[static_cast<int64_t>(kEmbedRanges) * stretches + blockIdx.x] = base;
  __syncthreads();
  for (int i0 = w0; i0 < w1; i0 += 32) {  // place
    const int id = i0 + lane < w1 ? ids[first + i0 + lane] : -1;
    const bool in = static_cast<uint32_t>(id) < static_cast<uint32_t>(v) && id != pad;
    const uint32_t some = __ballot_sync(kFull, in);
    if (in) {
      const int at = take_rank(some, id & (kEmbedRanges - 1), row, lane);
      tokens[first + at] = make_int2(id, static_cast<int>(first) + i0 + lane);
    }
    __syncwarp();
  }
}

// Block r: range r's ids, r and every kEmbedRanges-th after it.
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(int n, int per, int stretches, int len,
                                                                  const int2* __restrict__ tokens,
                                                                  const int32_t* __restrict__ off,
                                                                  const int32_t* __restrict__ bad,
                                                                  int32_t* __restrict__ start,
                                                                  int32_t* __restrict__ order,
                                                                  int32_t* __restrict__ sorted_id, int* status) {
  extern __shared__ __align__(16) int32_t sort_smem[];
  __shared__ int part[kSortWarps];
  __shared__ int32_t seg_first[2 * kSearchStep], seg_off[kEmbedStretches];  // of the range's tokens, of the stretch's
  int2* list = reinterpret_cast<int2*>(sort_smem);
  int32_t* running = sort_smem + 2 * kSortRound;  // [per]: where an id's next token goes
  int32_t* count = running + per;                 // [kSortWarps][per]
  griddep_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = blockIdx.x, lo = r * per;
  int all, wrong = 0;
  // the range's tokens of each stretch, and all tokens of the ranges before
  static_assert(kEmbedStretches <= kSortThreads, "a thread for each stretch");
  const int at = tid < stretches ? off[static_cast<int64_t>(r) * stretches + tid] : 0;
  const int to = tid < stretches ? off[static_cast<int64_t>(r + 1) * stretches + tid] : 0;
  if (r == 0 && tid < stretches) wrong = bad[tid];
  const int incl = block_scan(to - at, part, &all);
  const int m = all;
  static_assert(2 * kSearchStep <= kSortThreads, "a thread for each entry");
  if (tid < 2 * kSearchStep) seg_first[tid] = tid < stretches ? incl - (to - at) : INT32_MAX;
  if (tid < stretches) seg_off[tid] = at;
  block_scan(at, part, &all);
  int begin = all;
  wrong = __syncthreads_or(wrong);
  if (r == 0 && tid == 0) *status = wrong ? kErrLabel : kOk;
  constexpr int kEach = kSortRound / kSortThreads;
  // the range's tokens from i0 on, in the order of positions: the thread's are tid, tid + kSortThreads, ...
  auto fetch = [&](int i0, int2 (&t)[kEach]) {
    auto some = [&](auto count) {  // of the thread's
      constexpr int number = decltype(count)::value;
      int a[number];
#pragma unroll
      for (int k = 0; k < number; ++k) a[k] = 0;
#pragma unroll
      for (int step = kSearchStep; step; step >>= 1) {  // the last stretch that starts at or before it
#pragma unroll
        for (int k = 0; k < number; ++k) a[k] += seg_first[a[k] + step] <= i0 + k * kSortThreads + tid ? step : 0;
      }
#pragma unroll
      for (int k = 0; k < number; ++k) {
        const int i = i0 + k * kSortThreads + tid;
        t[k] = i < m ? tokens[static_cast<int64_t>(a[k]) * len + seg_off[a[k]] + (i - seg_first[a[k]])] : make_int2(-1, 0);
      }
    };
#pragma unroll
    for (int k = 1; k < kEach; ++k) t[k] = make_int2(-1, 0);
    if (m - i0 > kSortThreads) some(std::integral_constant<int, kEach>());
    else some(std::integral_constant<int, 1>());
  };
  // ids' totals, and where each one's tokens start
  for (int j = tid; j < per; j += kSortThreads) running[j] = 0;
  __syncthreads();
  for (int i0 = 0; i0 < m; i0 += kSortRound) {
    int2 t[kEach];
    fetch(i0, t);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      if (i0 + k * kSortThreads >= m) break;
      if (i0 == 0) list[k * kSortThreads + tid] = t[k];
      const uint32_t same = __match_any_sync(kFull, t[k].x);
      if (t[k].x >= 0 && (same >> lane) == 1u) atomicAdd(running + (t[k].x >> kEmbedRangeBits), __popc(same));
    }
  }
  __syncthreads();
  for (int j0 = 0; j0 < per; j0 += kSortThreads) {
    const int j = j0 + tid, c = j < per ? running[j] : 0;
    const int first = begin + block_scan(c, part, &all) - c;
    begin += all;
    if (j < per) start[lo + j] = running[j] = first;
  }
  if (r == kEmbedRanges - 1 && tid == 0) start[lo + per] = begin;
  __syncthreads();
  for (int i0 = 0; i0 < m; i0 += kSortRound) {
    const int here = min(kSortRound, m - i0);
    for (int j = tid; j < kSortWarps * per; j += kSortThreads) count[j] = 0;
    if (i0 > 0) {
      int2 t[kEach];
      fetch(i0, t);
#pragma unroll
      for (int k = 0; k < kEach; ++k) list[k * kSortThreads + tid] = t[k];
    }
    __syncthreads();
    // each token's rank among its warp's with its id
    const int each = (here + kSortThreads - 1) / kSortThreads * 32;
    const int w0 = warp * each, w1 = min(w0 + each, here);
    int32_t* row = count + warp * per;
    int rank[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = w0 + 32 * k + lane;
      const uint32_t some = __ballot_sync(kFull, i < w1);
      rank[k] = i < w1 ? take_rank(some, list[i].x >> kEmbedRangeBits, row, lane) : 0;
      __syncwarp();
    }
    __syncthreads();
    for (int j = tid; j < per; j += kSortThreads) {  // (warp, id) counts to places
      int next = running[j];
      for (int k = 0; k < kSortWarps; ++k) {
        const int c = count[k * per + j];
        count[k * per + j] = next;
        next += c;
      }
      running[j] = next;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = w0 + 32 * k + lane;
      if (i >= w1) continue;
      const int2 t = list[i];
      const int where = row[t.x >> kEmbedRangeBits] + rank[k];
      if (in_bounds(where, n, status)) {
        order[where] = t.y;
        sorted_id[where] = t.x;
      }
    }
    __syncthreads();
  }
}

constexpr int kFewThreads = 1024;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewBatch = 16;  // loads of ids in flight
constexpr int kFewMostPer = 1536;  // ids of a block: their counts fit its shared memory
constexpr int32_t kNoToken = INT32_MIN;  // behind a stretch's end: outside every range

// Block b owns ids [b per, (b + 1) per).  Warp w counts and places the positions of its stretch
// [w seg, (w + 1) seg), so that (id, warp, position) is the sorted order.
__global__ void __launch_bounds__(kFewThreads) embed_sort_few_kernel(int n, int v, int per, int seg, int pad,
                                                                  const int32_t* __restrict__ ids,
                                                                  int32_t* __restrict__ start,
                                                                  int32_t* __restrict__ order,
                                                                  int32_t* __restrict__ sorted_id, int* status) {
  extern __shared__ int32_t count[];  // [kFewWarps][per]
  __shared__ int32_t warp_sum[kFewWarps];
  __shared__ int32_t below_sum[kFewWarps];
  griddep_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lo = blockIdx.x * per;
  const int mine = min(per, v - lo);
  for (int i = tid; i < kFewWarps * per; i += kFewThreads) count[i] = 0;
  __syncthreads();
  int32_t* row = count + warp * per;
  const int64_t p0 = static_cast<int64_t>(warp) * seg;
  const int64_t p1 = min(p0 + seg, static_cast<int64_t>(n));
  const uint32_t ulo = static_cast<uint32_t>(lo), umine = static_cast<uint32_t>(mine);
  int below = 0, bad = 0;
  for (int64_t p = p0; p < p1; p += 32 * kFewBatch) {
    int32_t id[kFewBatch];
#pragma unroll
    for (int k = 0; k < kFewBatch; ++k) {
      const int64_t i = p + 32 * k + lane;
      id[k] = i < p1 ? __ldg(ids + i) : kNoToken;
    }
    uint32_t hits = 0;  // few: the block owns a small part of the vocabulary
#pragma unroll
    for (int k = 0; k < kFewBatch; ++k) {
      const uint32_t u = static_cast<uint32_t>(id[k]);  // (an id below 0 is above every range)
      below += u < ulo && id[k] != pad;
      hits |= (u - ulo < umine ? 1u : 0u) << k;
      if (blockIdx.x == 0) bad |= u >= static_cast<uint32_t>(v) && p + 32 * k + lane < p1;
    }
    if (hits) {
#pragma unroll
      for (int k = 0; k < kFewBatch; ++k)
        if ((hits >> k & 1) && id[k] != pad) atomicAdd(row + (id[k] - lo), 1);
    }
  }
  below = __reduce_add_sync(kFull, below);
  if (lane == 0) below_sum[warp] = below;
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && tid == 0) *status = bad ? kErrLabel : kOk;
  below = __reduce_add_sync(kFull, below_sum[lane]);
  // exclusive sums: of an id's counts over the warps, then of the ids (in turns of a block's threads)
  for (int j0 = 0; j0 < mine; j0 += kFewThreads) {
    const int j = j0 + tid;
    int total = 0;
    if (j < mine) {
      for (int k = 0; k < kFewWarps; ++k) {
        const int c = count[k * per + j];
        count[k * per + j] = total;
        total += c;
      }
    }
    int incl = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(kFull, incl, d);
      if (lane >= d) incl += up;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    const int ws = warp_sum[lane];
    int before = __reduce_add_sync(kFull, lane < warp ? ws : 0);
    const int all = __reduce_add_sync(kFull, ws);
    const int first = below + before + incl - total;
    if (j < mine) {
      start[lo + j] = first;
      for (int k = 0; k < kFewWarps; ++k) count[k * per + j] += first;
    }
    below += all;
    __syncthreads();
  }
  if (lo + mine == v && tid == 0) start[v] = below;
  __syncthreads();
  for (int64_t p = p0; p < p1; p += 32 * kFewBatch) {
    int32_t id[kFewBatch];
#pragma unroll
    for (int k = 0; k < kFewBatch; ++k) {
      const int64_t i = p + 32 * k + lane;
      id[k] = i < p1 ? __ldg(ids + i) : kNoToken;
    }
#pragma unroll
    for (int k = 0; k < kFewBatch; ++k) {
      const bool in = static_cast<uint32_t>(id[k]) - ulo < umine && id[k] != pad;
      const uint32_t some = __ballot_sync(kFull, in);
      if (!some) continue;
      if (in) {
        const int j = id[k] - lo;
        const uint32_t same = __match_any_sync(some, j);
        const int at = row[j] + __popc(same & ((1u << lane) - 1));
        __syncwarp(some);
        if ((same >> lane) == 1u) row[j] = at + 1;  // the highest of them
        if (in_bounds(at, n, status)) {
          order[at] = static_cast<int32_t>(p + 32 * k + lane);
          sorted_id[at] = id[k];
        }
      }
      __syncwarp();
    }
  }
}

// ----------------------------------------------------------------------------- sums

// dW's row: x scale, added to what it held where ADD.
template <typename TW, bool ALIGNED, bool ADD>
__device__ __forceinline__ void finish(TW* row, const Place<ALIGNED>& at, int h, float scale,
                                       const Words<TW, ALIGNED>& old, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = ADD ? fmaf(x[e], scale, old.value(e)) : x[e] * scale;
  store8<ALIGNED>(row, at, h, x);
}

// A part is a row of `groups` times 256 fp32, in the order of the lanes' elements.
template <bool ALIGNED>
__device__ __forceinline__ void part_store(float* p, int lane, const float (&x)[8]) {
  if (ALIGNED) {
    reinterpret_cast<float4*>(p)[2 * lane] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[2 * lane + 1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[32 * e + lane] = x[e];
  }
}
template <bool ALIGNED>
__device__ __forceinline__ void part_load(const float* p, int lane, float (&x)[8]) {
  if (ALIGNED) {
    const float4 a = reinterpret_cast<const float4*>(p)[2 * lane], b = reinterpret_cast<const float4*>(p)[2 * lane + 1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = p[32 * e + lane];
  }
}

constexpr int kZeroRows = 8;  // of a warp of the zeros' blocks

// Tile t has two parts: 2 t of a row that starts before it, 2 t + 1 of one that starts in it and
// goes on.
//   Blocks below `tile_blocks` take tiles, the others the rows without a token.  A batch of
// tokens' rows is in flight at once, with the rows of dW that they complete.
//   Bound by memory where there is enough of it: 131072 x 4096 added to dW in 241 us (1.53 GB, 80% of
// DRAM's nominal rate), 8192 x 2048 for 32000 rows in 28 (102 MB of them reach DRAM), 5003 x 1031 fp32
// for 40009 rows in 31.
template <typename T, typename TW, bool ALIGNED, bool ADD, int kTile>
__global__ void __launch_bounds__(256) embed_tiles_kernel(int n, int h, int v, EmbedKeys keys, float scale, int64_t tile_blocks,
                                                          const int32_t* __restrict__ start,
                                                          const int32_t* __restrict__ order,
                                                          const int32_t* __restrict__ sorted_id,
                                                          const T* __restrict__ dy, float* __restrict__ part,
                                                          TW* __restrict__ dw, int groups, int* status) {
  constexpr int kBatch = Words<T, ALIGNED>::kPacked ? 8 : 4;
  griddep_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x >= tile_blocks) {
    const int64_t first = ((static_cast<int64_t>(blockIdx.x) - tile_blocks) * 8 + warp) * kZeroRows;
    const int key = static_cast<int>(first) + lane, id = keys.id(min(key, keys.count() - 1));
    const int at = key <= keys.count() ? start[key] : 0;  // (lane 8: where the last one ends)
    const int to = __shfl_down_sync(kFull, at, 1);
    const uint32_t none = __ballot_sync(kFull, lane < kZeroRows && key < keys.count() && id < v && at == to);
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (uint32_t left = none; left; left &= left - 1) {
      TW* row = dw + static_cast<int64_t>(__shfl_sync(kFull, id, __ffs(left) - 1)) * h;
      for (int g = 0; g < groups; ++g) store8<ALIGNED>(row, Place<ALIGNED>(g, lane), h, zero);
    }
    return;
  }
  const int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  const int64_t t = u / groups;
  const int group = static_cast<int>(u % groups);
  const Place<ALIGNED> place(group, lane);
  const int total = start[keys.count()];
  if (t * kTile >= total) return;
  const int s0 = static_cast<int>(t) * kTile, tokens = min(kTile, total - s0);
  int my_id[kTile / 32], my_at[kTile / 32];
#pragma unroll
  for (int k = 0; k < kTile / 32; ++k) {
    const int i = 32 * k + lane;
    my_id[k] = i < tokens ? sorted_id[s0 + i] : -1;
    my_at[k] = i < tokens ? order[s0 + i] : 0;
  }
  const int before = s0 > 0 ? sorted_id[s0 - 1] : -1, after = s0 + tokens < total ? sorted_id[s0 + tokens] : -1;
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll 1
  for (int b = 0; b < tokens; b += kBatch) {
    Words<T, ALIGNED> y[kBatch];
    Words<TW, ALIGNED> old[ADD ? kBatch : 1];
    int id[kBatch + 1];
#pragma unroll
    for (int k = 0; k <= kBatch; ++k) {  // ids of the batch and of the token behind it
      int held = my_id[0];
#pragma unroll
      for (int j = 1; j < kTile / 32; ++j)
        if ((b + k) / 32 == j) held = my_id[j];
      id[k] = __shfl_sync(kFull, held, (b + k) & 31);
      if (b + k >= tokens) id[k] = after;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      int held = my_at[0];
#pragma unroll
      for (int j = 1; j < kTile / 32; ++j)
        if ((b + k) / 32 == j) held = my_at[j];
      const int64_t at = static_cast<int64_t>(__shfl_sync(kFull, held, (b + k) & 31)) * h;
      y[k].zero();
      if (ADD) old[ADD ? k : 0].zero();
      if (!in_bounds(at, static_cast<int64_t>(n) * h, status)) continue;
      y[k].load(dy + at, place, h);  // (behind the tile's last token: row 0, not added)
    }
    if (ADD) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (b + k < tokens && id[k + 1] != id[k] && id[k] != before) old[ADD ? k : 0].load(dw + static_cast<int64_t>(id[k]) * h, place, h);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (b + k >= tokens) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += y[k].value(e);
      const bool ends = id[k + 1] != id[k];
      if (!ends && b + k + 1 < tokens) continue;
      // the row's last token in this tile; it began here unless the token before the tile is its own
      const bool began = before != id[k];
      if (began && ends) {
        finish<TW, ALIGNED, ADD>(dw + static_cast<int64_t>(id[k]) * h, place, h, scale, old[ADD ? k : 0], x);
      } else {
        const int64_t to = ((2 * t + (began ? 1 : 0)) * groups + group) * kCols;
        if (in_bounds(to + kCols - 1, embed_part_floats(n, h), status))
          part_store<ALIGNED>(part + to, lane, x);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
  }
}

constexpr int kJoinGroups = 4;  // of 256 columns, a block's: one after the other where a row has many parts
constexpr int kJoinAlone = 16;  // parts that a warp adds up by itself; more are cut into a run for each warp

// Block (t, g): kJoinGroups times 256 columns of the row that starts in tile t and goes on, if there
// is one.  The row with the most parts is the end of it: 131072 x 4096 in tiles of 64, a vocabulary's
// frequencies, 30 us, with 8 groups a block 42 (and eight parts in flight in place of four 51); 8192 x 2048 8.
template <typename TW, bool ALIGNED, bool ADD, int kTile>
__global__ void __launch_bounds__(256) embed_join_kernel(int h, EmbedKeys keys, float scale, const int32_t* __restrict__ start,
                                                         const int32_t* __restrict__ sorted_id,
                                                         const float* __restrict__ part, TW* __restrict__ dw, int groups) {
  __shared__ float run[8][32][9];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wide = (groups + kJoinGroups - 1) / kJoinGroups;
  const int64_t t = blockIdx.x / wide;
  const int g0 = static_cast<int>(blockIdx.x % wide) * kJoinGroups;
  // The sorted order is older than the launch before, which waited for it: it is read ahead of the
  // wait, from L2.  Every block waits before it leaves, so that whatever follows this launch follows
  // that one.
  const int total = __ldcg(start + keys.count());
  const int64_t s0 = t * kTile, s1 = s0 + kTile;
  int id = 0, a = 0, b = 0;
  if (s1 < total) {
    id = __ldcg(sorted_id + s1 - 1);
    a = __ldcg(start + keys.of(id));
    b = __ldcg(start + keys.of(id) + 1);
  }
  griddep_begin();
  if (a < s0 || b <= s1) return;
  const int parts = static_cast<int>((b - 1) / kTile - t) + 1;  // part 0 is 2 t + 1, part i is 2 (t + i)
  TW* row = dw + static_cast<int64_t>(id) * h;
  auto sum = [&](int g, int from, int to, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll 4
    for (int i = from; i < to; ++i) {
      float q[8];
      part_load<ALIGNED>(part + ((2 * (t + i) + (i == 0)) * groups + g) * kCols, lane, q);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += q[e];
    }
  };
  Words<TW, ALIGNED> old;
  if (parts <= kJoinAlone) {
    const int g = g0 + warp;
    if (warp >= kJoinGroups || g >= groups) return;
    const Place<ALIGNED> place(g, lane);
    float x[8];
    old.zero();
    if (ADD) old.load(row, place, h);
    sum(g, 0, parts, x);
    finish<TW, ALIGNED, ADD>(row, place, h, scale, old, x);
    return;
  }
  const int each = (parts + 7) / 8;
  for (int g = g0; g < min(g0 + kJoinGroups, groups); ++g) {
    float x[8];
    sum(g, warp * each, min(parts, (warp + 1) * each), x);
    __syncthreads();  // (the runs of the group before have been read)
#pragma unroll
    for (int e = 0; e < 8; ++e) run[warp][lane][e] = x[e];
    __syncthreads();
    if (warp == 0) {
      const Place<ALIGNED> place(g, lane);
      old.zero();
      if (ADD) old.load(row, place, h);
      for (int k = 1; k < 8; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += run[k][lane][e];
      finish<TW, ALIGNED, ADD>(row, place, h, scale, old, x);
    }
  }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int groups_of(int h) { return (h + kCols - 1) / kCols; }

template <typename T, int LANES>
cudaError_t forward_by(const EmbedParams& q, const int32_t* ids, const void* w, void* y, int* status, cudaStream_t s) {
  const bool al = q.h % 8 == 0 && aligned16(w) && aligned16(y);
  const int groups = (q.h + 8 * LANES - 1) / (8 * LANES);
  constexpr int kPerBlock = kFwdThreads / LANES * kFwdUnits;
  const int64_t scans = (q.n + kScanIds - 1) / kScanIds;
  const int64_t blocks = (q.n * groups + kPerBlock - 1) / kPerBlock + scans;
  if (blocks > INT_MAX) return cudaErrorInvalidValue;
  if (scans > 1) {
    const cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int), s);
    if (e != cudaSuccess) return e;
  }
  auto* k = al ? embed_forward_kernel<T, true, LANES> : embed_forward_kernel<T, false, LANES>;
  return launch_k(k, dim3(static_cast<unsigned>(blocks)), dim3(kFwdThreads), 0, s, q.n, q.h, q.v, q.scale, ids,
                  static_cast<const T*>(w), static_cast<T*>(y), groups, static_cast<int>(scans), status);
}

template <typename T>
cudaError_t forward_of(const EmbedParams& q, const int32_t* ids, const void* w, void* y, int* status, cudaStream_t s) {
  return q.h <= 64    ? forward_by<T, 8>(q, ids, w, y, status, s)
         : q.h <= 128 ? forward_by<T, 16>(q, ids, w, y, status, s)
                      : forward_by<T, 32>(q, ids, w, y, status, s);
}

template <typename T, typename TW, bool ALIGNED, bool ADD, int TILE>
cudaError_t backward_by(const EmbedParams& q, const void* dy, const EmbedSorted& o, void* dw, cudaStream_t s) {
  const int groups = groups_of(q.h);
  const int n = static_cast<int>(q.n), v = static_cast<int>(q.v);
  const EmbedKeys keys = embed_keys(q.n, q.v);
  const int64_t tiles = (q.n + TILE - 1) / TILE, tile_blocks = (tiles * groups + 7) / 8;
  const int64_t zero_blocks = ADD ? 0 : (keys.count() + 8 * kZeroRows - 1) / (8 * kZeroRows);
  const int64_t join_blocks = (tiles - 1) * ((groups + kJoinGroups - 1) / kJoinGroups);
  if (tile_blocks + zero_blocks > INT_MAX || join_blocks > INT_MAX) return cudaErrorInvalidValue;
  TW* out = static_cast<TW*>(dw);
  cudaError_t e = launch_k(embed_tiles_kernel<T, TW, ALIGNED, ADD, TILE>,
                           dim3(static_cast<unsigned>(tile_blocks + zero_blocks)), dim3(256), 0, s, n, q.h, v, keys, q.scale,
                           tile_blocks, o.start, o.order, o.sorted_id, static_cast<const T*>(dy), o.part, out, groups,
                           o.status);
  if (e != cudaSuccess || join_blocks == 0) return e;
  return launch_k(embed_join_kernel<TW, ALIGNED, ADD, TILE>, dim3(static_cast<unsigned>(join_blocks)), dim3(256), 0, s,
                  q.h, keys, q.scale, o.start, o.sorted_id, o.part, out, groups);
}

template <typename T, typename TW, bool ALIGNED, bool ADD>
cudaError_t backward_as(const EmbedParams& q, const void* dy, const EmbedSorted& o, void* dw, cudaStream_t s) {
  return embed_tile(q.n, q.h) == kEmbedTile ? backward_by<T, TW, ALIGNED, ADD, kEmbedTile>(q, dy, o, dw, s)
                                            : backward_by<T, TW, ALIGNED, ADD, kEmbedTileMany>(q, dy, o, dw, s);
}

template <typename T, typename TW>
cudaError_t backward_of(const EmbedParams& q, const void* dy, const EmbedSorted& o, void* dw, bool add,
                        cudaStream_t s) {
  if (q.h % 8 == 0 && aligned16(dy) && aligned16(dw))
    return add ? backward_as<T, TW, true, true>(q, dy, o, dw, s) : backward_as<T, TW, true, false>(q, dy, o, dw, s);
  return add ? backward_as<T, TW, false, true>(q, dy, o, dw, s) : backward_as<T, TW, false, false>(q, dy, o, dw, s);
}

}  // namespace

cudaError_t launch_embed_forward(const EmbedParams& q, const int32_t* ids, const void* w, void* y, int* status,
                                 cudaStream_t s) {
  return q.w_f32 ? forward_of<float>(q, ids, w, y, status, s)
                 : forward_of<__nv_bfloat16>(q, ids, w, y, status, s);
}

static cudaError_t sort_few(const EmbedParams& q, int pad, const int32_t* ids, const EmbedSorted& o, int sms,
                            cudaStream_t s) {
  // a range for each SM, or as many as keep a block's counts within its shared memory
  const int64_t ranges = std::max<int64_t>(std::min<int64_t>(sms, q.v), (q.v + kFewMostPer - 1) / kFewMostPer);
  const int per = static_cast<int>((q.v + ranges - 1) / ranges);
  const int64_t blocks = (q.v + per - 1) / per;
  const int seg = static_cast<int>((q.n + kFewThreads - 1) / kFewThreads) * 32;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(embed_sort_few_kernel, sizeof(int32_t) * kFewWarps * kFewMostPer, done);
  if (e != cudaSuccess) return e;
  return launch_k(embed_sort_few_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kFewThreads),
                  sizeof(int32_t) * kFewWarps * static_cast<size_t>(per), s, static_cast<int>(q.n), static_cast<int>(q.v),
                  per, seg, pad, ids, o.start, o.order, o.sorted_id, o.status);
}

cudaError_t launch_embed_sort(const EmbedParams& q, int pad, const int32_t* ids, const EmbedSorted& o, int sms,
                              cudaStream_t s) {
  if (q.n <= kEmbedFew) return sort_few(q, pad, ids, o, sms, s);
  const int per = embed_keys(q.n, q.v).per;
  const int len = static_cast<int>((q.n + kEmbedStretches - 1) / kEmbedStretches);
  const int stretches = static_cast<int>((q.n + len - 1) / len);
  const int n = static_cast<int>(q.n), v = static_cast<int>(q.v);
  cudaError_t e = launch_k(embed_bucket_kernel, dim3(stretches), dim3(kSortThreads), 0, s, n, v, len, pad,
                           ids, static_cast<int2*>(o.tokens), o.off, o.bad);
  if (e != cudaSuccess) return e;
  auto smem = [](int ids_of_range) {
    return sizeof(int32_t) * (2 * kSortRound + static_cast<size_t>(kSortWarps + 1) * static_cast<size_t>(ids_of_range));
  };
  static std::atomic<uint64_t> done{0};
  e = allow_smem(embed_sort_kernel, smem(kPerMost), done);
  if (e != cudaSuccess) return e;
  return launch_k(embed_sort_kernel, dim3(kEmbedRanges), dim3(kSortThreads), smem(per), s, n, per, stretches, len,
                  static_cast<const int2*>(o.tokens), o.off, o.bad, o.start, o.order, o.sorted_id, o.status);
}

cudaError_t launch_embed_backward(const EmbedParams& q, const void* dy, const EmbedSorted& o, void* dw, bool add,
                                  cudaStream_t s) {
  if (q.y_f32)
    return q.w_f32 ? backward_of<float, float>(q, dy, o, dw, add, s)
                   : backward_of<float, __nv_bfloat16>(q, dy, o, dw, add, s);
  return q.w_f32 ? backward_of<__nv_bfloat16, float>(q, dy, o, dw, add, s)
                 : backward_of<__nv_bfloat16, __nv_bfloat16>(q, dy, o, dw, add, s);
}

}  // namespace flce
