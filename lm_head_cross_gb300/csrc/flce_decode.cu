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
// and 96 (n <= 64: twice): every warp then finds tokens in the TMEM quarter it can read,
// and takes a quarter (half) of the tile's columns for them, which shortens what is
// exposed after the last tile.
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
  const uint32_t a_bytes = static_cast<uint32_t>(p.copies * p.a_rows * kBK * 2);
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
      for (int c = 0; c < p.copies; ++c) tma_load_2d(sa + c * (128 / p.copies) * kBK * 2, &maps.x, &full[stage], k0, 0);
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
  const int copies = p.copies;
  const int share = quarter / (4 / copies);                  // which of the copies it reads
  const int row = quarter % (4 / copies) * 32 + lane;        // token
  const int c0 = share * (8 / copies);                       // 32-column chunks of a tile this warp takes
  const int c1 = c0 + 8 / copies;
  const bool idle = row - lane >= p.n;                       // a warp without a token only frees accumulators
  const int y = (row < p.n) ? label_at(p.tokens, row, p.shift, p.seq_len, p.ignore_index) : p.ignore_index;

  float* val = reinterpret_cast<float*>(cand + (warp - 2) * kCandBytes);
  int* idx = reinterpret_cast<int*>(cand + (warp - 2) * kCandBytes + kTopkCand * 32 * sizeof(float));
  int count = 0;
  float thr = -INFINITY;        // the range's own k-th best, once it is known: ids grow, so an equal later value is out
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
    if (TOP && !idle && n0 == r.v0)
      floor_thr = copies == 4   ? first_floor<1>(tbase + c0 * 32, cols - c0 * 32, p.k)
                  : copies == 2 ? first_floor<2>(tbase + c0 * 32, cols - c0 * 32, p.k)
                                : first_floor<4>(tbase, cols, p.k);
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
      if (TOP && __any_sync(0xffffffffu, row < p.n && cmax > thr && cmax >= floor_thr)) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (!__any_sync(0xffffffffu, row < p.n && gmax[g] > thr && gmax[g] >= floor_thr)) continue;
#pragma unroll
          for (int j = 8 * g; j < 8 * g + 8; ++j) {
            const float x = __uint_as_float(v[j]);
            // ids grow along the range: an equal later value ranks after the kept one
            const bool keep = row < p.n && x > thr && x >= floor_thr;
            const int at = topk_slot(count, lane);
            if (keep) {
              val[at] = x;
              idx[at] = col0 + j;
            }
            count += keep ? 1 : 0;
          }
          if (__any_sync(0xffffffffu, count > kTopkCand - 8)) {
            Trimmed t = topk_trim(val, idx, count, lane, p.k, floor_thr);
            floor_thr = t.thr;
            t = topk_cut(val, idx, t.count, thr, lane, p.k, kTopkCand - 8);  // (many equal values: ranked)
            count = t.count;
            thr = t.thr;
          }
        }
      }
    }
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(&tempty[acc]);
    // Room for the next tile's, made while that one loads.
    if (TOP && n0 + kTileV < r.v1 && __any_sync(0xffffffffu, count > p.k + 2)) {
      const Trimmed t = topk_trim(val, idx, count, lane, p.k, floor_thr);
      count = t.count;
      floor_thr = t.thr;
    }
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
  if (TOP && __any_sync(0xffffffffu, count > p.slots)) {
    count = topk_trim(val, idx, count, lane, p.k, floor_thr).count;
    count = topk_cut(val, idx, count, thr, lane, p.k, p.slots).count;
  }
  if (row >= p.n) return;
  const int part = blockIdx.x * copies + share;
  const int64_t at = static_cast<int64_t>(row) * p.parts + part;
  if (!in_bounds(at, p.part_count, err)) return;
  p.part_m[at] = m;
  p.part_l[at] = l;
  p.part_s[at] = es;
  if (TOP) {
#pragma unroll 4
    for (int e = 0; e < p.slots; ++e)
      p.cand[at * p.slots + e] = e < count ? candidate_key(val[topk_slot(e, lane)], idx[topk_slot(e, lane)]) : 0;
  }
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

constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;

// One block per token: lse, entropy and the given token's log probability from the ranges'
// (max, sum, entropy sum), and the best k of their candidates.  Those are a few thousand
// numbers that the threads hold in registers.  The k-th largest of the 16 warps' maxima is a
// bound that k candidates reach and few pass; where at most a block of them does, each is
// ranked by counting, else k rounds of a maximum over the block pick the best in order
// (0.7 us a round).
template <bool TOP>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const DecodeParams p, int ctas, float* logprob,
                                                                   float* entropy, float* lse, int32_t* top_ids,
                                                                   float* top_logprobs) {
  griddep_begin();
  constexpr int kMostParts = (4 * kDecodeCtas + kJoinThreads - 1) / kJoinThreads;
  constexpr int kMostCands = TOP ? (4 * kDecodeCtas * kDecodeSlots + kJoinThreads - 1) / kJoinThreads : 1;
  __shared__ float red[3][kJoinWarps];
  __shared__ __align__(16) uint64_t round_best[2][kJoinWarps];
  __shared__ uint64_t kept[TOP ? kJoinThreads : 1];
  __shared__ int kept_count;
  const int row = blockIdx.x, t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int64_t base = static_cast<int64_t>(row) * p.parts;
  // this thread's parts and candidates, loads first
  float pm[kMostParts], pl[kMostParts], ps[kMostParts];
#pragma unroll
  for (int i = 0; i < kMostParts; ++i) {
    const int s = t + i * kJoinThreads;
    const bool in = s < p.parts;
    pm[i] = in ? p.part_m[base + s] : -INFINITY;
    pl[i] = in ? p.part_l[base + s] : 0.f;
    ps[i] = in ? p.part_s[base + s] : 0.f;
  }
  uint64_t key[kMostCands], best = 0;
  if (TOP) {
    const uint64_t* cand = p.cand + base * p.slots;
    const int cands = p.parts * p.slots;
#pragma unroll
    for (int i = 0; i < kMostCands; ++i) {
      const int c = t + i * kJoinThreads;
      key[i] = c < cands ? cand[c] : 0;
    }
#pragma unroll
    for (int i = 0; i < kMostCands; ++i)
      if (key[i] > best) best = key[i];
  }
  float m = pm[0];
#pragma unroll
  for (int i = 1; i < kMostParts; ++i) m = fmaxf(m, pm[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, red[0][w]);
  float l = 0.f, es = 0.f;
#pragma unroll
  for (int i = 0; i < kMostParts; ++i) {
    const float d = max_nan(pm[i] - m, kNoLogit);
    const float f = exp2f(d);
    l += pl[i] * f;
    es += f * fmaf(pl[i], d, ps[i]);
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
  __syncthreads();
  l = es = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    l += red[1][w];
    es += red[2][w];
  }
  const float log2l = log2f(l);
  if (t == 0) {
    lse[row] = (m + log2l) * kLn2;
    if (entropy) entropy[row] = (log2l - es / l) * kLn2;
    if (p.tokens) {
      const int y = label_at(p.tokens, row, p.shift, p.seq_len, p.ignore_index);
      float lp = 0.f;
      if (y != p.ignore_index) {
        // relative to the same m as l: exact where the token holds the largest logit
        if (y >= 0 && y < p.v) lp = (fmaf(p.tgt[row], p.zscale, -m) - log2l) * kLn2;
        else atomicCAS(p.status, 0, kErrLabel);
      }
      if (logprob) logprob[row] = lp;
    }
  }
  if (row == 0 && t < ctas && p.err[t]) atomicCAS(p.status, 0, p.err[t]);
  if (!TOP) return;
  const auto put = [&](int rank, uint64_t won) {
    const float z = topk_unkey(static_cast<unsigned>(won >> 32));
    top_ids[static_cast<int64_t>(row) * p.k + rank] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(won));
    top_logprobs[static_cast<int64_t>(row) * p.k + rank] = (fmaf(z, p.zscale, -m) - log2l) * kLn2;
  };
  {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(best >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (best >> 32) == hi ? static_cast<uint32_t>(best) : 0u);
    if (lane == 0) round_best[0][warp] = (static_cast<uint64_t>(hi) << 32) | lo;
    if (t == 0) kept_count = 0;
    __syncthreads();
    uint64_t bound = 0;  // 0: fewer than k warps hold a candidate
    const uint64_t mine = lane < kJoinWarps ? round_best[0][lane] : 0;
    int rank = 0;
    for (int w = 0; w < kJoinWarps; ++w) rank += round_best[0][w] > mine;
    const unsigned at = __ballot_sync(0xffffffffu, mine != 0 && rank == p.k - 1);
    if (at) bound = round_best[0][__ffs(at) - 1];
    if (best >= bound) {
#pragma unroll
      for (int i = 0; i < kMostCands; ++i)
        if (key[i] != 0 && key[i] >= bound) {
          const int slot = atomicAdd(&kept_count, 1);
          if (slot < kJoinThreads) kept[slot] = key[i];
        }
    }
    __syncthreads();
    const int count = kept_count;
    if (count <= kJoinThreads) {
      if (t < count) {
        const uint64_t won = kept[t];
        int place = 0;
        for (int q = 0; q < count; ++q) place += kept[q] > won;
        if (place < p.k) put(place, won);
      } else if (t < p.k) {  // fewer than k ids
        top_ids[static_cast<int64_t>(row) * p.k + t] = -1;
        top_logprobs[static_cast<int64_t>(row) * p.k + t] = -INFINITY;
      }
      return;
    }
  }
  for (int r = 0; r < p.k; ++r) {
    __syncthreads();  // the words of two rounds ago, and the filter's, have been read
    // the warp's best: the largest value, then the largest id word among its holders
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(best >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (best >> 32) == hi ? static_cast<uint32_t>(best) : 0u);
    if (lane == 0) round_best[r & 1][warp] = (static_cast<uint64_t>(hi) << 32) | lo;
    __syncthreads();
    uint64_t win = 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; w += 2) {
      const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&round_best[r & 1][w]);
      if (o.x > win) win = o.x;
      if (o.y > win) win = o.y;
    }
    if (win == best && win != 0) {  // its holder (candidates are distinct)
      best = 0;
#pragma unroll
      for (int i = 0; i < kMostCands; ++i) {
        if (key[i] == win) key[i] = 0;
        if (key[i] > best) best = key[i];
      }
      put(r, win);
    }
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
