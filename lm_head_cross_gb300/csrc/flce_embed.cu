// Embedding: rows of a vocabulary matrix, scaled, and the matrix's gradient by sorted tokens.
//
//   y_i = s W[id_i]                        (a row of zeros where id_i is outside [0, V))
//   dW_v = s sum_{i : id_i = v} dy_i       (v other than the padding id), or added to dW
//
// Both are bound by memory: the forward pass reads the distinct rows and writes N H elements, the
// gradient reads N H elements and writes V H (or reads and writes the distinct rows).
//
// The gradient's sums have one order, whatever the schedule: the tokens are sorted by (id,
// position) and cut into tiles of kTile; a row of dW is the sum over its tokens in that order in
// fp32, one part for each tile that it has tokens in, the parts added in order, and rounded once.
//   sort   every block owns a range of the vocabulary and reads all ids twice (they stay in L2):
//          once to count, a count for each (warp's stretch of positions, id), and once to place
//          its tokens.  No block waits for another, no atomics in global memory, one launch.
//   tiles  every tile's tokens, 32 chunks of columns a warp: rows that lie within the tile are
//          finished, the others leave a part; beside them, zeros for the rows without a token
//   join   the rows with several parts
#include "flce_device.cuh"
#include "flce_internal.h"
#include "flce_launch.cuh"

namespace flce {

namespace {

constexpr int kTile = kEmbedTile;
constexpr uint32_t kFull = 0xffffffffu;

// ----------------------------------------------------------------------------- 8 elements of a row

// 8 consecutive elements at any element alignment: two-byte elements that start at an odd one are
// taken from aligned words and shifted.
template <bool ALIGNED>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  uint32_t w[4];
  if (ALIGNED) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint32_t* q = reinterpret_cast<const uint32_t*>(a & ~uintptr_t{3});
    if (a & 2) {
      uint32_t u[5];
#pragma unroll
      for (int e = 0; e < 5; ++e) u[e] = __ldg(q + e);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __funnelshift_r(u[e], u[e + 1], 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __ldg(q + e);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

template <bool ALIGNED>
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  if (ALIGNED) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __ldg(p + e);
  }
}

// 8 elements whose first is at a multiple of 8 elements (from a 16-byte boundary on).
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                 pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// A row that is written is cut at the 8-element boundaries of its memory, so that only its first
// and last chunk can be short: `lead` elements of the first chunk belong to the row before.
template <typename T, bool ALIGNED>
__device__ __forceinline__ int lead_of(const T* row) {
  return ALIGNED ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 7);
}

}  // namespace

// Chunks that cover any row of h elements.
static int chunks_of(int h, bool aligned) { return aligned ? h / 8 : (h + 7 + 7) / 8; }

namespace {

// ----------------------------------------------------------------------------- forward

constexpr int kFwdThreads = 256;
constexpr int kFwdChunks = 4;  // of a thread: as many loads in flight

// Blocks 0 .. gridDim - 2 take kFwdThreads * kFwdChunks consecutive chunks of y; the last one
// looks all ids over and writes the status word, so that nothing has to clear it first.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kFwdThreads) embed_forward_kernel(int64_t n, int h, int64_t v, float scale,
                                                                    const int32_t* __restrict__ ids,
                                                                    const T* __restrict__ w, T* __restrict__ y,
                                                                    int cpr, int* status) {
  griddep_begin();
  const int tid = threadIdx.x;
  if (blockIdx.x == gridDim.x - 1) {
    int bad = 0;
    for (int64_t i = tid; i < n; i += kFwdThreads) bad |= static_cast<uint32_t>(ids[i]) >= static_cast<uint64_t>(v);
    bad = __syncthreads_or(bad);
    if (tid == 0) *status = bad ? kErrLabel : kOk;
    return;
  }
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kFwdThreads * kFwdChunks);
  const int64_t row0 = first / cpr;
  const uint32_t off0 = static_cast<uint32_t>(first - row0 * cpr);
  float x[kFwdChunks][8];
  int64_t row[kFwdChunks];
  int col[kFwdChunks];
  int64_t id[kFwdChunks];
#pragma unroll
  for (int k = 0; k < kFwdChunks; ++k) {
    const uint32_t at = off0 + static_cast<uint32_t>(tid + k * kFwdThreads);
    row[k] = row0 + at / static_cast<uint32_t>(cpr);
    col[k] = static_cast<int>(at % static_cast<uint32_t>(cpr)) * 8;
    if (row[k] >= n) {
      col[k] = INT_MAX;
      continue;
    }
    id[k] = ids[row[k]];
    col[k] -= lead_of<T, ALIGNED>(y + row[k] * h);
  }
#pragma unroll
  for (int k = 0; k < kFwdChunks; ++k) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[k][e] = 0.f;
    if (col[k] >= h || id[k] < 0 || id[k] >= v) continue;
    const T* src = w + id[k] * h;
    if (ALIGNED || (col[k] >= 0 && col[k] + 8 <= h)) {
      load8<ALIGNED>(src + col[k], x[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col[k] + e >= 0 && col[k] + e < h) x[k][e] = to_f32(src[col[k] + e]);
    }
  }
#pragma unroll
  for (int k = 0; k < kFwdChunks; ++k) {
    if (col[k] >= h) continue;
    T* dst = y + row[k] * h;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[k][e] *= scale;
    if (ALIGNED || (col[k] >= 0 && col[k] + 8 <= h)) {
      store8(dst + col[k], x[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col[k] + e >= 0 && col[k] + e < h) put(dst + col[k] + e, x[k][e]);
    }
  }
}

// ----------------------------------------------------------------------------- sort

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBatch = 16;  // loads of ids in flight
constexpr int32_t kNoToken = INT32_MIN;  // behind a stretch's end: outside every range

// Block b owns ids [b per, (b + 1) per).  Warp w counts and places the positions of its stretch
// [w seg, (w + 1) seg), so that (id, warp, position) is the sorted order.
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(int n, int v, int per, int seg, int pad,
                                                                  const int32_t* __restrict__ ids,
                                                                  int32_t* __restrict__ start,
                                                                  int32_t* __restrict__ order,
                                                                  int32_t* __restrict__ sorted_id, int* status) {
  extern __shared__ int32_t count[];  // [kSortWarps][per]
  __shared__ int32_t warp_sum[kSortWarps];
  __shared__ int32_t below_sum[kSortWarps];
  griddep_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lo = blockIdx.x * per;
  const int mine = min(per, v - lo);
  for (int i = tid; i < kSortWarps * per; i += kSortThreads) count[i] = 0;
  __syncthreads();
  int32_t* row = count + warp * per;
  const int64_t p0 = static_cast<int64_t>(warp) * seg;
  const int64_t p1 = min(p0 + seg, static_cast<int64_t>(n));
  const uint32_t ulo = static_cast<uint32_t>(lo), umine = static_cast<uint32_t>(mine);
  int below = 0, bad = 0;
  for (int64_t p = p0; p < p1; p += 32 * kSortBatch) {
    int32_t id[kSortBatch];
#pragma unroll
    for (int k = 0; k < kSortBatch; ++k) {
      const int64_t i = p + 32 * k + lane;
      id[k] = i < p1 ? __ldg(ids + i) : kNoToken;
    }
    uint32_t hits = 0;  // few: the block owns a small part of the vocabulary
#pragma unroll
    for (int k = 0; k < kSortBatch; ++k) {
      const uint32_t u = static_cast<uint32_t>(id[k]);  // (an id below 0 is above every range)
      below += u < ulo && id[k] != pad;
      hits |= (u - ulo < umine ? 1u : 0u) << k;
      if (blockIdx.x == 0) bad |= u >= static_cast<uint32_t>(v) && p + 32 * k + lane < p1;
    }
    if (hits) {
#pragma unroll
      for (int k = 0; k < kSortBatch; ++k)
        if ((hits >> k & 1) && id[k] != pad) atomicAdd(row + (id[k] - lo), 1);
    }
  }
  below = __reduce_add_sync(kFull, below);
  if (lane == 0) below_sum[warp] = below;
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && tid == 0) *status = bad ? kErrLabel : kOk;
  below = __reduce_add_sync(kFull, below_sum[lane]);
  // exclusive sums: of an id's counts over the warps, then of the ids (in turns of a block's threads)
  for (int j0 = 0; j0 < mine; j0 += kSortThreads) {
    const int j = j0 + tid;
    int total = 0;
    if (j < mine) {
      for (int k = 0; k < kSortWarps; ++k) {
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
      for (int k = 0; k < kSortWarps; ++k) count[k * per + j] += first;
    }
    below += all;
    __syncthreads();
  }
  if (lo + mine == v && tid == 0) start[v] = below;
  __syncthreads();
  for (int64_t p = p0; p < p1; p += 32 * kSortBatch) {
    int32_t id[kSortBatch];
#pragma unroll
    for (int k = 0; k < kSortBatch; ++k) {
      const int64_t i = p + 32 * k + lane;
      id[k] = i < p1 ? __ldg(ids + i) : kNoToken;
    }
#pragma unroll
    for (int k = 0; k < kSortBatch; ++k) {
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

template <typename TW, bool ALIGNED, bool ADD>
__device__ __forceinline__ void finish(TW* row, int h, int col, float scale, float (&x)[8]) {
  const bool whole = ALIGNED || (col >= 0 && col + 8 <= h);
  if (whole) {
    float old[8];
    if (ADD) {
      load8<true>(row + col, old);  // (chunks are cut at dW's own boundaries)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], scale, old[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= scale;
    }
    store8(row + col, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e >= 0 && col + e < h) put(row + col + e, ADD ? fmaf(x[e], scale, to_f32(row[col + e])) : x[e] * scale);
  }
}

constexpr int kZeroRows = 8;    // of a warp of the zeros' blocks
constexpr int kTokenBatch = 8;  // rows of dy in flight
static_assert(kTile == 32, "a lane holds one of a tile's tokens");

// Parts are rows of 8 cpr fp32: element c of the row at c + lead (see lead_of), so that every
// chunk is aligned.  Tile t has two: 2 t of a row that starts before it, 2 t + 1 of one that
// starts in it and goes on.
//   Blocks below `tile_blocks` take tiles, the others the rows without a token.
template <typename T, typename TW, bool ALIGNED, bool ADD>
__global__ void __launch_bounds__(256) embed_tiles_kernel(int n, int h, int v, float scale, int64_t tile_blocks,
                                                          const int32_t* __restrict__ start,
                                                          const int32_t* __restrict__ order,
                                                          const int32_t* __restrict__ sorted_id,
                                                          const T* __restrict__ dy, float* __restrict__ part,
                                                          TW* __restrict__ dw, int cpr, int* status) {
  griddep_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x >= tile_blocks) {
    const int64_t first = ((static_cast<int64_t>(blockIdx.x) - tile_blocks) * 8 + warp) * kZeroRows;
    const int at = first + lane <= v ? start[first + lane] : 0;  // (lane 8: where the last one ends)
    const int to = __shfl_down_sync(kFull, at, 1);
    const uint32_t none = __ballot_sync(kFull, lane < kZeroRows && first + lane < v && at == to);
    for (uint32_t left = none; left; left &= left - 1) {
      TW* row = dw + (first + __ffs(left) - 1) * h;
      for (int chunk = lane; chunk < cpr; chunk += 32) {
        const int col = chunk * 8 - lead_of<TW, ALIGNED>(row);
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (col < h) finish<TW, ALIGNED, false>(row, h, col, 0.f, x);
      }
    }
    return;
  }
  const int groups = (cpr + 31) / 32;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  const int64_t t = u / groups;
  const int chunk = static_cast<int>(u % groups) * 32 + lane;
  const int total = start[v];
  if (t * kTile >= total) return;
  const int s0 = static_cast<int>(t) * kTile, tokens = min(kTile, total - s0);
  const int my_id = lane < tokens ? sorted_id[s0 + lane] : -1;
  const int my_at = lane < tokens ? order[s0 + lane] : 0;
  const int before = s0 > 0 ? sorted_id[s0 - 1] : -1, after = s0 + tokens < total ? sorted_id[s0 + tokens] : -1;
  const bool live = chunk < cpr;
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll 1
  for (int b = 0; b < tokens; b += kTokenBatch) {
    float y[kTokenBatch][8];
    int id[kTokenBatch], col[kTokenBatch];
#pragma unroll
    for (int k = 0; k < kTokenBatch; ++k) {
      id[k] = __shfl_sync(kFull, my_id, b + k);
      const int64_t at = static_cast<int64_t>(__shfl_sync(kFull, my_at, b + k)) * h;
      col[k] = chunk * 8 - lead_of<TW, ALIGNED>(dw + static_cast<int64_t>(id[k]) * h);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[k][e] = 0.f;
      if (b + k >= tokens || !live || !in_bounds(at, static_cast<int64_t>(n) * h, status)) continue;
      if (ALIGNED || (col[k] >= 0 && col[k] + 8 <= h)) {
        load8<ALIGNED>(dy + at + col[k], y[k]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col[k] + e >= 0 && col[k] + e < h) y[k][e] = to_f32(dy[at + col[k] + e]);
      }
    }
#pragma unroll
    for (int k = 0; k < kTokenBatch; ++k) {
      const int i = b + k;
      if (i >= tokens) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += y[k][e];
      const int next = i + 1 < tokens ? __shfl_sync(kFull, my_id, i + 1) : after;
      if (next == id[k] && i + 1 < tokens) continue;
      // the row's last token in this tile; it began here unless the token before the tile is its own
      const bool began = before != id[k];
      if (began && next != id[k]) {
        if (live && col[k] < h) finish<TW, ALIGNED, ADD>(dw + static_cast<int64_t>(id[k]) * h, h, col[k], scale, x);
      } else if (live) {
        const int64_t to = (2 * t + (began ? 1 : 0)) * cpr * 8 + chunk * 8;
        if (in_bounds(to + 7, embed_part_floats(n, cpr * 8), status)) {
          *reinterpret_cast<float4*>(part + to) = make_float4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<float4*>(part + to + 4) = make_float4(x[4], x[5], x[6], x[7]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
  }
}

constexpr int kJoinAlone = 16;  // parts that a warp adds up by itself; more are cut into a run for each warp

// Block (t, g): 8 times 32 chunks of the row that starts in tile t and goes on, if there is one.
template <typename TW, bool ALIGNED, bool ADD>
__global__ void __launch_bounds__(256) embed_join_kernel(int h, int v, float scale, const int32_t* __restrict__ start,
                                                         const int32_t* __restrict__ sorted_id,
                                                         const float* __restrict__ part, TW* __restrict__ dw, int cpr) {
  griddep_begin();
  __shared__ float run[8][32][9];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (cpr + 31) / 32, wide = (groups + 7) / 8;
  const int64_t t = blockIdx.x / wide;
  const int g0 = static_cast<int>(blockIdx.x % wide) * 8;
  const int total = start[v];
  const int64_t s0 = t * kTile, s1 = s0 + kTile;
  if (s1 >= total) return;
  const int id = sorted_id[s1 - 1];
  const int a = start[id], b = start[id + 1];
  if (a < s0 || b <= s1) return;
  const int parts = static_cast<int>((b - 1) / kTile - t) + 1;  // part 0 is 2 t + 1, part i is 2 (t + i)
  const int64_t pitch = static_cast<int64_t>(cpr) * 8;
  TW* row = dw + static_cast<int64_t>(id) * h;
  const int lead = lead_of<TW, ALIGNED>(row);
  auto sum = [&](int chunk, int from, int to, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    if (chunk >= cpr) return;
#pragma unroll 4
    for (int i = from; i < to; ++i) {
      float q[8];
      load8<true>(part + (2 * (t + i) + (i == 0)) * pitch + chunk * 8, q);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += q[e];
    }
  };
  if (parts <= kJoinAlone) {
    const int chunk = (g0 + warp) * 32 + lane, col = chunk * 8 - lead;
    float x[8];
    sum(chunk, 0, parts, x);
    if (chunk < cpr && col < h) finish<TW, ALIGNED, ADD>(row, h, col, scale, x);
    return;
  }
  const int each = (parts + 7) / 8;
  for (int g = g0; g < min(g0 + 8, groups); ++g) {
    const int chunk = g * 32 + lane, col = chunk * 8 - lead;
    float x[8];
    sum(chunk, warp * each, min(parts, (warp + 1) * each), x);
    __syncthreads();  // (the runs of the group before have been read)
#pragma unroll
    for (int e = 0; e < 8; ++e) run[warp][lane][e] = x[e];
    __syncthreads();
    if (warp == 0 && chunk < cpr && col < h) {
      for (int k = 1; k < 8; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += run[k][lane][e];
      finish<TW, ALIGNED, ADD>(row, h, col, scale, x);
    }
  }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename T>
cudaError_t forward_of(const EmbedParams& q, const int32_t* ids, const void* w, void* y, int* status, cudaStream_t s) {
  const bool al = q.h % 8 == 0 && aligned16(w) && aligned16(y);
  const int cpr = chunks_of(q.h, al);
  const int64_t per_block = kFwdThreads * kFwdChunks;
  const int64_t blocks = (q.n * cpr + per_block - 1) / per_block + 1;
  if (blocks > INT_MAX) return cudaErrorInvalidValue;
  auto* k = al ? embed_forward_kernel<T, true> : embed_forward_kernel<T, false>;
  return launch_k(k, dim3(static_cast<unsigned>(blocks)), dim3(kFwdThreads), 0, s, q.n, q.h, q.v, q.scale, ids,
                  static_cast<const T*>(w), static_cast<T*>(y), cpr, status);
}

template <typename T, typename TW, bool ALIGNED, bool ADD>
cudaError_t backward_as(const EmbedParams& q, const void* dy, const EmbedSorted& o, void* dw, cudaStream_t s) {
  const int cpr = chunks_of(q.h, ALIGNED), groups = (cpr + 31) / 32;
  const int n = static_cast<int>(q.n), v = static_cast<int>(q.v);
  const int64_t tiles = (q.n + kTile - 1) / kTile, tile_blocks = (tiles * groups + 7) / 8;
  const int64_t zero_blocks = ADD ? 0 : (q.v + 8 * kZeroRows - 1) / (8 * kZeroRows);
  const int64_t join_blocks = (tiles - 1) * ((groups + 7) / 8);
  if (tile_blocks + zero_blocks > INT_MAX || join_blocks > INT_MAX) return cudaErrorInvalidValue;
  TW* out = static_cast<TW*>(dw);
  cudaError_t e = launch_k(embed_tiles_kernel<T, TW, ALIGNED, ADD>, dim3(static_cast<unsigned>(tile_blocks + zero_blocks)),
                           dim3(256), 0, s, n, q.h, v, q.scale, tile_blocks, o.start, o.order, o.sorted_id,
                           static_cast<const T*>(dy), o.part, out, cpr, o.status);
  if (e != cudaSuccess || join_blocks == 0) return e;
  return launch_k(embed_join_kernel<TW, ALIGNED, ADD>, dim3(static_cast<unsigned>(join_blocks)), dim3(256), 0, s, q.h, v,
                  q.scale, o.start, o.sorted_id, o.part, out, cpr);
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

cudaError_t launch_embed_sort(const EmbedParams& q, int pad, const int32_t* ids, const EmbedSorted& o, int sms,
                              cudaStream_t s) {
  // a range for each SM, or as many as keep a block's counts within its shared memory
  constexpr int kMostPer = 1536;
  const int64_t blocks0 = std::max<int64_t>(std::min<int64_t>(sms, q.v), (q.v + kMostPer - 1) / kMostPer);
  const int per = static_cast<int>((q.v + blocks0 - 1) / blocks0);
  const int64_t blocks = (q.v + per - 1) / per;
  const int seg = static_cast<int>((q.n + kSortThreads - 1) / kSortThreads) * 32;
  const size_t smem = sizeof(int32_t) * kSortWarps * static_cast<size_t>(per);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(embed_sort_kernel, sizeof(int32_t) * kSortWarps * kMostPer, done);
  if (e != cudaSuccess) return e;
  return launch_k(embed_sort_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kSortThreads), smem, s,
                  static_cast<int>(q.n), static_cast<int>(q.v), per, seg, pad, ids, o.start, o.order, o.sorted_id,
                  o.status);
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
