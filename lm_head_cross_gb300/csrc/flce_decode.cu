// Token log probabilities of a few rows (n <= 128): the decoding step of a serving batch.
//
// W is read once and that is the whole cost: its V x H bf16 at the HBM rate.  One CTA on
// each SM owns a contiguous range of vocabulary rows (cut at multiples of 16, so that all
// SMs read the same amount to within 16 rows), streams it tile by tile (256 rows, K in
// blocks of 64) through a TMA ring of 128 KiB, multiplies it with X on tcgen05 (M = 128
// token rows, N = up to 256 vocabulary rows, fp32 in TMEM) and keeps each token's softmax
// statistics and best logits.  The MMA's 128 rows cost 36% of the time that the tile's
// bytes take at H = 2048, whatever n is, so a smaller M would gain nothing.
//
// Warp roles: warp 0 loads, warp 1 issues the MMAs, warps 2-5 drain the other of two TMEM
// accumulators, a token a lane.  With n <= 32 X is staged four times, at rows 0, 32, 64
// and 96: every warp then finds all tokens in the TMEM quarter it can read, and takes a
// quarter of the tile's columns, which shortens what is exposed after the last tile.
//
// A second kernel, one block per token, joins the ranges' partial results.
#include <algorithm>

#include "flce_device.cuh"
#include "flce_internal.h"
#include "flce_launch.cuh"
#include "flce_rows.cuh"

namespace flce {

namespace {

constexpr int kTileV = 256;                       // vocabulary rows of a tile
constexpr int kSub = 16;                          // rows of the smallest box, and the ranges' grain
constexpr int kAStageBytes = 128 * kBK * 2;       // X rows: 16 KiB
constexpr int kBStageBytes = kTileV * kBK * 2;    // W rows: 32 KiB
constexpr int kRingStages = 4;
constexpr int kCandOff = kRingStages * (kAStageBytes + kBStageBytes);
constexpr int kCandBytes = kTopkCand * 32 * 8;    // one warp's candidates
constexpr int kBarOff = kCandOff + 4 * kCandBytes;
constexpr int kDecodeSmem = kBarOff + 256 + 1024;  // barriers; 1 KiB to align the ring
static_assert(kDecodeSmem <= 232448, "shared memory budget");
constexpr uint32_t kDecodeTmem = 2 * kTileV;

__device__ __forceinline__ void tmem_alloc_one(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_one(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void umma_bf16_one(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit_one(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// (value, id) as one number that grows with the value and, among equal ones, as the id falls; 0: none.
__device__ __forceinline__ uint64_t candidate_key(float v, int id) {
  return (static_cast<uint64_t>(topk_key(v + 0.f)) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
}

struct Range {
  int v0, v1;  // vocabulary rows [v0, v1)
};
__device__ __forceinline__ Range my_range(const DecodeParams& p) {
  const int64_t units = (p.v + kSub - 1) / kSub;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  const int64_t end = u1 * kSub;
  return Range{static_cast<int>(u0 * kSub), static_cast<int>(end < p.v ? end : p.v)};
}

__device__ void decode_producer(const DecodeMaps& maps, const DecodeParams& p, Range r, uint8_t* ring, uint64_t* full,
                                uint64_t* empty, volatile int* abort_flag, int* err) {
  const int kblocks = (p.h + kBK - 1) / kBK;
  const int copies = p.n <= 32 ? 4 : 1;
  const uint32_t a_bytes = static_cast<uint32_t>(copies * p.a_rows * kBK * 2);
  int stage = 0;
  uint32_t phase = 0;
  for (int n0 = r.v0; n0 < r.v1; n0 += kTileV) {
    const int rows = min(kTileV, r.v1 - n0);
    const int loaded = (rows + kSub - 1) / kSub * kSub;  // (past V: zeros)
    const uint32_t bytes = a_bytes + loaded * kBK * 2;
    for (int kb = 0; kb < kblocks; ++kb) {
      if (!mbar_wait(&empty[stage], phase ^ 1u, p.timeout_ns, abort_flag)) {
        *abort_flag = 1;
        *err = kErrTimeout;
        return;
      }
      uint8_t* sa = ring + stage * (kAStageBytes + kBStageBytes);
      uint8_t* sb = sa + kAStageBytes;
      mbar_arrive_expect_tx(&full[stage], bytes);
      const int k0 = kb * kBK;  // a multiple of 64 elements: the copies' 16-byte rule
      // the tile's rows as boxes of 256, 128, ... 16, one of each at most
      for (int i = 0, at = 0; i < kDecodeBoxes; ++i) {
        const int box = kTileV >> i;
        if (loaded - at < box) continue;
        tma_load_2d(sb + at * kBK * 2, &maps.w[i], &full[stage], k0, n0 + at);
        at += box;
      }
      for (int c = 0; c < copies; ++c) tma_load_2d(sa + c * 32 * kBK * 2, &maps.x, &full[stage], k0, 0);
      if (++stage == kRingStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
}

__device__ void decode_mma(const DecodeParams& p, Range r, uint8_t* ring, uint64_t* full, uint64_t* empty,
                           uint64_t* tfull, uint64_t* tempty, uint32_t tmem_base, volatile int* abort_flag, int* err) {
  const int kblocks = (p.h + kBK - 1) / kBK;
  int stage = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0;
  for (int n0 = r.v0; n0 < r.v1; n0 += kTileV) {
    const int cols = (min(kTileV, r.v1 - n0) + 15) / 16 * 16;
    const uint32_t idesc = instr_desc_bf16(128, cols, false, false);
    if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, p.timeout_ns, abort_flag)) {
      *abort_flag = 1;
      *err = kErrTimeout;
      return;
    }
    tc_fence_after_sync();
    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kTileV);
    for (int kb = 0; kb < kblocks; ++kb) {
      if (!mbar_wait(&full[stage], phase, p.timeout_ns, abort_flag)) {
        *abort_flag = 1;
        *err = kErrTimeout;
        return;
      }
      tc_fence_after_sync();
      const uint32_t sa = smem_u32(ring + stage * (kAStageBytes + kBStageBytes));
      const uint32_t sb = sa + kAStageBytes;
#pragma unroll
      for (int k = 0; k < kBK / 16; ++k)
        umma_bf16_one(d_tmem, smem_desc_sw128(sa + k * 32, 16, 1024), smem_desc_sw128(sb + k * 32, 16, 1024), idesc,
                      (kb | k) != 0 ? 1u : 0u);
      umma_commit_one(&empty[stage]);
      if (++stage == kRingStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    umma_commit_one(&tfull[acc]);
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
}

// TOP: also the best k logits.
template <bool TOP>
__device__ void decode_epilogue(const DecodeParams& p, Range r, uint8_t* cand, uint64_t* tfull, uint64_t* tempty,
                                uint32_t tmem_base, volatile int* abort_flag, int* err) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;  // the TMEM lanes this warp may read
  const bool narrow = p.n <= 32;
  const int row = narrow ? lane : quarter * 32 + lane;       // token
  const int c0 = narrow ? 2 * quarter : 0;                   // 32-column chunks of a tile this warp takes
  const int c1 = narrow ? c0 + 2 : kTileV / 32;
  const bool idle = !narrow && quarter * 32 >= p.n;          // a warp without a token only frees accumulators
  const int y = (row < p.n) ? label_at(p.tokens, row, p.shift, p.seq_len, p.ignore_index) : p.ignore_index;

  TopkBuf tk;
  tk.val = reinterpret_cast<float*>(cand + (warp - 2) * kCandBytes);
  tk.idx = reinterpret_cast<int*>(cand + (warp - 2) * kCandBytes + kTopkCand * 32 * sizeof(float));
  tk.count = 0;
  tk.thr = -INFINITY;
  tk.shared_thr = nullptr;
  float floor_thr = -INFINITY;  // nothing below it is among the row's best
  float m = -INFINITY, l = 0.f, es = 0.f;
  int acc = 0;
  uint32_t acc_phase = 0;
  for (int n0 = r.v0; n0 < r.v1; n0 += kTileV) {
    const int cols = min(kTileV, r.v1 - n0);
    // (the whole warp goes on or gives up)
    if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], acc_phase, p.timeout_ns, abort_flag))) {
      *abort_flag = 1;
      *err = kErrTimeout;
      return;
    }
    tc_fence_after_sync();
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * kTileV);
    if (TOP && !idle && n0 == r.v0 && cols >= c1 * 32) {
      // Before the first tile fills the buffer from nothing: each of 16 disjoint column groups
      // holds its maximum, so nothing below the least of those is among the best 16.
      float t0 = INFINITY;
#pragma unroll 1
      for (int c = c0; c < c1; ++c) {
        __syncwarp();
        uint32_t v[32];
        tmem_ld_32x32(tbase + c * 32, v);
        if (narrow) {  // groups of 4
#pragma unroll
          for (int g = 0; g < 8; ++g)
            t0 = fminf(t0, fmaxf(fmaxf(__uint_as_float(v[4 * g]), __uint_as_float(v[4 * g + 1])),
                                 fmaxf(__uint_as_float(v[4 * g + 2]), __uint_as_float(v[4 * g + 3]))));
        } else {  // groups of 16
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float mx = __uint_as_float(v[16 * g]);
#pragma unroll
            for (int j = 1; j < 16; ++j) mx = fmaxf(mx, __uint_as_float(v[16 * g + j]));
            t0 = fminf(t0, mx);
          }
        }
      }
      floor_thr = t0;
    }
#pragma unroll 1
    for (int c = c0; c < c1 && !idle; ++c) {
      if (c * 32 >= cols) break;  // the same for the whole warp
      __syncwarp();
      uint32_t v[32];
      tmem_ld_32x32(tbase + c * 32, v);
      const int col0 = n0 + c * 32;
      const int yi = y - col0;
      if (static_cast<unsigned>(yi) < 32u && y != p.ignore_index && row < p.n && yi < cols - c * 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == yi) p.tgt[row] = __uint_as_float(v[j]);
      }
      const int nv = cols - c * 32;
      if (nv < 32) {  // columns past the range (not loaded)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j >= nv) v[j] = __float_as_uint(-INFINITY);
      }
      float gmax[4];  // maxima of the chunk's 8-column blocks
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        gmax[g] = __uint_as_float(v[8 * g]);
#pragma unroll
        for (int j = 8 * g + 1; j < 8 * g + 8; ++j) gmax[g] = fmaxf(gmax[g], __uint_as_float(v[j]));
      }
      const float cmax = fmaxf(fmaxf(gmax[0], gmax[1]), fmaxf(gmax[2], gmax[3]));
      const float new_m = fmaxf(m, cmax * p.zscale);
      float s4[4] = {0.f, 0.f, 0.f, 0.f}, e4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float u = max_nan(fmaf(__uint_as_float(v[j]), p.zscale, -new_m), kNoLogit);
        const float w = fast_exp2(u);
        s4[j & 3] += w;
        e4[j & 3] = fmaf(w, u, e4[j & 3]);
      }
      const float d = max_nan(m - new_m, kNoLogit);
      const float f = fast_exp2(d);
      es = f * fmaf(l, d, es) + ((e4[0] + e4[1]) + (e4[2] + e4[3]));
      l = l * f + ((s4[0] + s4[1]) + (s4[2] + s4[3]));
      m = new_m;
      if (TOP && __any_sync(0xffffffffu, row < p.n && cmax > tk.thr && cmax >= floor_thr)) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (!__any_sync(0xffffffffu, row < p.n && gmax[g] > tk.thr && gmax[g] >= floor_thr)) continue;
#pragma unroll
          for (int j = 8 * g; j < 8 * g + 8; ++j) {
            const float x = __uint_as_float(v[j]);
            // ids grow along the range: an equal later value ranks after the kept one
            const bool keep = row < p.n && x > tk.thr && x >= floor_thr;
            const int at = topk_slot(tk.count, lane);
            if (keep) {
              tk.val[at] = x;
              tk.idx[at] = col0 + j;
            }
            tk.count += keep ? 1 : 0;
          }
          topk_compact_lanes(tk, lane, __ballot_sync(0xffffffffu, tk.count > kTopkCand - 8), p.k);
        }
      }
    }
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(&tempty[acc]);
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
  if (TOP) topk_compact_lanes(tk, lane, __ballot_sync(0xffffffffu, tk.count > p.k), p.k);
  if (row >= p.n) return;
  const int part = narrow ? blockIdx.x * 4 + quarter : blockIdx.x;
  const int64_t at = static_cast<int64_t>(row) * p.parts + part;
  if (!in_bounds(at, p.part_count, err)) return;
  p.part_m[at] = m;
  p.part_l[at] = l;
  p.part_s[at] = es;
  if (TOP)
    for (int e = 0; e < p.k; ++e)
      p.cand[at * p.k + e] = e < tk.count ? candidate_key(tk.val[topk_slot(e, lane)], tk.idx[topk_slot(e, lane)]) : 0;
}

template <bool TOP>
__global__ void __launch_bounds__(192, 1) decode_kernel(const __grid_constant__ DecodeMaps maps, const DecodeParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOff);
  uint64_t* empty = full + kRingStages;
  uint64_t* tfull = empty + kRingStages;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  int* flags = reinterpret_cast<int*>(tempty + 3);  // [0] abort, [1] error code
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRingStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4);  // one arrival per epilogue warp
    }
    flags[0] = flags[1] = 0;
    mbar_fence_init();
    fence_proxy_async_smem();
    tma_prefetch_map(&maps.x);
    for (int i = 0; i < kDecodeBoxes; ++i) tma_prefetch_map(&maps.w[i]);
  }
  if (warp == 1) tmem_alloc_one(tmem_slot, kDecodeTmem);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  griddep_begin();  // X and W may come from the kernels before
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;  // every call's word starts clear; only the join adds to it
  const Range r = my_range(p);
  if (warp == 0) {
    if (lane == 0) decode_producer(maps, p, r, smem, full, empty, flags, flags + 1);
  } else if (warp == 1) {
    if (lane == 0) decode_mma(p, r, smem, full, empty, tfull, tempty, tmem_base, flags, flags + 1);
  } else {
    decode_epilogue<TOP>(p, r, smem + kCandOff, tfull, tempty, tmem_base, flags, flags + 1);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (*static_cast<volatile int*>(flags)) {
    // a wait gave up: copies and MMAs in flight land before their memory is released
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) {
    }
  }
  if (threadIdx.x == 0) p.err[blockIdx.x] = flags[1];
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_one(tmem_base, kDecodeTmem);
  }
}

// ----------------------------------------------------------------------------- joining the ranges

constexpr int kJoinThreads = 128;

// One block per token: lse, entropy and the given token's log probability from the ranges'
// (max, sum, entropy sum), and the best k of their candidates.  For those, each thread takes
// every 128th range's list; the k-th largest of the threads' maxima is a bound that at least
// k candidates reach and few pass (at most k threads' lists hold any that do); those few are
// ranked by counting.
template <bool TOP>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const DecodeParams p, int ctas, float* logprob,
                                                                   float* entropy, float* lse, int32_t* top_ids,
                                                                   float* top_logprobs) {
  griddep_begin();
  constexpr int kMostParts = (4 * kDecodeCtas + kJoinThreads - 1) / kJoinThreads;
  __shared__ float red[3][kJoinThreads / 32];
  __shared__ __align__(16) uint64_t maxima[kJoinThreads];
  __shared__ uint64_t kept[TOP ? kTopkMax * kMostParts * kTopkMax : 1];
  __shared__ uint64_t bound;
  __shared__ int kept_count;
  const int row = blockIdx.x, t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int64_t base = static_cast<int64_t>(row) * p.parts;
  uint64_t best = 0;
  float m = -INFINITY;
  for (int s = t; s < p.parts; s += kJoinThreads) {
    m = fmaxf(m, p.part_m[base + s]);
    if (TOP)
      for (int e = 0; e < p.k; ++e) best = max(best, p.cand[(base + s) * p.k + e]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[0][warp] = m;
  if (TOP) {
    maxima[t] = best;
    if (t == 0) {
      bound = 0;
      kept_count = 0;
    }
  }
  __syncthreads();
  for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, red[0][w]);
  float l = 0.f, es = 0.f;
  for (int s = t; s < p.parts; s += kJoinThreads) {
    const float d = max_nan(p.part_m[base + s] - m, kNoLogit), pl = p.part_l[base + s];
    const float f = exp2f(d);
    l += pl * f;
    es += f * fmaf(pl, d, p.part_s[base + s]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, o);
    es += __shfl_xor_sync(0xffffffffu, es, o);
  }
  if (lane == 0) {
    red[1][warp] = l;
    red[2][warp] = es;
  }
  if (TOP && best != 0) {  // distinct non-zero numbers: one thread has this rank, if that many are non-zero
    int rank = 0;
#pragma unroll 8
    for (int q = 0; q < kJoinThreads; q += 2) {
      const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&maxima[q]);
      rank += (o.x > best) + (o.y > best);
    }
    if (rank == p.k - 1) bound = best;
  }
  __syncthreads();
  l = es = 0.f;
  for (int w = 0; w < kJoinThreads / 32; ++w) {
    l += red[1][w];
    es += red[2][w];
  }
  const float log2l = log2f(l);
  if (t == 0) {
    lse[row] = (m + log2l) * kLn2;
    if (entropy) entropy[row] = (log2l - es / l) * kLn2;
  }
  int code = 0;
  if (t == 0 && p.tokens) {
    const int y = label_at(p.tokens, row, p.shift, p.seq_len, p.ignore_index);
    float lp = 0.f;
    if (y != p.ignore_index) {
      if (y >= 0 && y < p.v) lp = (fmaf(p.tgt[row], p.zscale, -m) - log2l) * kLn2;
      else code = kErrLabel;
    }
    if (logprob) logprob[row] = lp;
  }
  if (code) atomicCAS(p.status, 0, code);
  if (row == 0)
    for (int c = t; c < ctas; c += kJoinThreads)
      if (p.err[c]) atomicCAS(p.status, 0, p.err[c]);
  if (!TOP) return;
  if (best >= bound && best != 0)
    for (int s = t; s < p.parts; s += kJoinThreads)
      for (int e = 0; e < p.k; ++e) {
        const uint64_t key = p.cand[(base + s) * p.k + e];
        if (key != 0 && key >= bound) kept[atomicAdd(&kept_count, 1)] = key;
      }
  __syncthreads();
  const int count = kept_count;
  for (int i = t; i < count; i += kJoinThreads) {
    const uint64_t key = kept[i];
    int rank = 0;
    for (int q = 0; q < count; ++q) rank += kept[q] > key;
    if (rank < p.k) {
      const float z = topk_unkey(static_cast<unsigned>(key >> 32));
      top_ids[static_cast<int64_t>(row) * p.k + rank] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key));
      top_logprobs[static_cast<int64_t>(row) * p.k + rank] = (fmaf(z, p.zscale, -m) - log2l) * kLn2;
    }
  }
  for (int i = count + t; i < p.k; i += kJoinThreads) {  // fewer than k ids
    top_ids[static_cast<int64_t>(row) * p.k + i] = -1;
    top_logprobs[static_cast<int64_t>(row) * p.k + i] = -INFINITY;
  }
}

template <bool TOP>
cudaError_t decode_launches(const DecodeMaps& maps, const DecodeParams& p, int ctas, float* logprob, float* entropy,
                            float* lse, int32_t* top_ids, float* top_logprobs, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(decode_kernel<TOP>, kDecodeSmem, done);
  if (e != cudaSuccess) return e;
  e = launch_k(decode_kernel<TOP>, dim3(ctas), dim3(192), kDecodeSmem, stream, maps, p);
  if (e != cudaSuccess) return e;
  return launch_k(decode_join_kernel<TOP>, dim3(p.n), dim3(kJoinThreads), 0, stream, p, ctas, logprob, entropy, lse,
                  top_ids, top_logprobs);
}

}  // namespace

cudaError_t launch_decode(const DecodeMaps& maps, const DecodeParams& p, int ctas, float* logprob, float* entropy,
                          float* lse, int32_t* top_ids, float* top_logprobs, cudaStream_t stream) {
  return p.k > 0 ? decode_launches<true>(maps, p, ctas, logprob, entropy, lse, top_ids, top_logprobs, stream)
                 : decode_launches<false>(maps, p, ctas, logprob, entropy, lse, top_ids, top_logprobs, stream);
}

}  // namespace flce
