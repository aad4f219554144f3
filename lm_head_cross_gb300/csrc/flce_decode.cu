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
// exposed after the last tile, where that pays (decode_copies).  n <= 8: decode_epilogue_few.
//
// A second kernel, one block per token, joins the ranges' partial results.
//
// Measured (the two kernels, W at 2 V H bytes): 1 x 4096 x 128256 with 5 alternatives 165 us,
// 6.4 TB/s; 64 rows without alternatives 172 us, 6.1 TB/s, with 8 alternatives 184 us; 1 x
// 2048 x 32000 with 5 alternatives 29.5 us, of which W's bytes are 20 and the launch, the last
// tile's epilogue and the join the rest; 64 x 2048 x 32000, 8 alternatives, 38 us.
#include <algorithm>

#include "flce_device.cuh"
#include "flce_internal.h"
#include "flce_launch.cuh"
#include "flce_rows.cuh"

namespace flce {

namespace {

constexpr int kTileV = 256;                       // vocabulary rows of a tile, at most
constexpr int kSms = 152;                         // CTAs of a launch on a whole device
constexpr int kSub = 16;                          // rows of the smallest box, and the ranges' grain
constexpr int kAStageBytes = 128 * kBK * 2;       // X rows: 16 KiB
constexpr int kBStageBytes = kTileV * kBK * 2;    // W rows: 32 KiB
constexpr int kMostStages = 4;
constexpr int kCandBytes = kTopkCand * 32 * 8;    // one warp's candidates
constexpr int kDecodeSmem = 232448 - 512;         // what the kernel takes; barriers in its last 512 bytes
constexpr int kBarOff = kDecodeSmem - 1024 - 512; // (1 KiB aligns the ring)
constexpr uint32_t kDecodeTmem = 2 * kTileV;

// Shared memory, in order: W stages (32 KiB: a tile's block of K), X, then the warps'
// candidates or the few tokens' logits.
//   X streams beside W, 16 KiB a stage, or, for n <= 8 and as far as it fits, stays in shared
//   memory from the first tile on, 1 KiB (8 rows) for each block of K.  Every SM reads the
//   same X: streamed, its few lines were asked for by 152 SMs at a time, which held the whole
//   stream to 5.6 TB/s at H = 4096 (6.3 with X resident).  The MMA's rows 8 to 127 are then
//   the blocks that follow, and past the last one a margin: products in TMEM lanes nobody
//   reads.
constexpr int kFewRows = 8;
constexpr int kFewPitch = kTileV + 4;                    // floats of a token's logits
constexpr int kFewBytes = kFewRows * kFewPitch * 4;
constexpr int kResidentMargin = kAStageBytes - 1024;
struct SmemPlan {
  bool few;  // X resident, and the epilogue of few tokens
  int stages;
  int x_off, cand_off;
};
__host__ __device__ inline SmemPlan smem_plan(int n, int h) {
  const int x = (h + kBK - 1) / kBK * 1024 + kResidentMargin;
  const int left = (kBarOff - kFewBytes - x) / kBStageBytes;
  if (n <= kFewRows && left >= 3) {
    const int stages = left < 4 ? left : 4;
    return SmemPlan{true, stages, stages * kBStageBytes, stages * kBStageBytes + x};
  }
  return SmemPlan{false, 4, 4 * kBStageBytes, 4 * (kBStageBytes + kAStageBytes)};
}
static_assert(4 * (kBStageBytes + kAStageBytes) + 4 * kCandBytes <= kBarOff, "shared memory budget");

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

__device__ void decode_producer(const DecodeMaps& maps, const DecodeParams& p, const SmemPlan& plan, Range r,
                                uint8_t* smem, uint64_t* full, uint64_t* empty, volatile int* abort_flag,
                                int* err) {
  const int kblocks = (p.h + kBK - 1) / kBK;
  const uint32_t a_bytes = static_cast<uint32_t>(p.copies * p.a_rows * kBK * 2);
  uint8_t* const x = smem + plan.x_off;
  int stage = 0;
  uint32_t phase = 0;
  for (int n0 = r.v0; n0 < r.v1; n0 += kTileV) {
    const int rows = min(kTileV, r.v1 - n0);
    const int loaded = (rows + kSub - 1) / kSub * kSub;  // (past V: zeros)
    const bool load_x = !plan.few || n0 == r.v0;  // resident: with the first tile
    const uint32_t bytes = (load_x ? a_bytes : 0) + loaded * kBK * 2;
    for (int kb = 0; kb < kblocks; ++kb) {
      if (!mbar_wait(&empty[stage], phase ^ 1u, p.timeout_ns, abort_flag)) {
        *abort_flag = 1;
        *err = kErrTimeout;
        return;
      }
      uint8_t* sb = smem + stage * kTileV * kBK * 2;
      mbar_arrive_expect_tx(&full[stage], bytes);
      const int k0 = kb * kBK;  // a multiple of 64 elements: the copies' 16-byte rule
      // the tile's rows as boxes of 256, 128, ... 16, one of each at most
      for (int i = 0, at = 0; i < kDecodeBoxes; ++i) {
        const int box = kTileV >> i;
        if (loaded - at < box) continue;
        tma_load_2d(sb + at * kBK * 2, &maps.w[i], &full[stage], k0, n0 + at);
        at += box;
      }
      if (load_x) {
        uint8_t* sa = x + (plan.few ? kb * 1024 : stage * kAStageBytes);
        for (int c = 0; c < p.copies; ++c)
          tma_load_2d(sa + c * (128 / p.copies) * kBK * 2, &maps.x, &full[stage], k0, 0);
      }
      if (++stage == plan.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
}

__device__ void decode_mma(const DecodeParams& p, const SmemPlan& plan, Range r, uint8_t* smem, uint64_t* full,
                           uint64_t* empty, uint64_t* tfull, uint64_t* tempty, uint32_t tmem_base,
                           volatile int* abort_flag, int* err) {
  const int kblocks = (p.h + kBK - 1) / kBK;
  const uint32_t x = smem_u32(smem + plan.x_off);
  int stage = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0;
  bool ok = true;
  for (int n0 = r.v0; ok && n0 < r.v1; n0 += kTileV) {
    const int cols = (min(kTileV, r.v1 - n0) + 15) / 16 * 16;
    const uint32_t idesc = instr_desc_bf16(128, cols, false, false);
    ok = mbar_wait(&tempty[acc], acc_phase ^ 1u, p.timeout_ns, abort_flag);
    if (!ok) break;
    tc_fence_after_sync();
    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kTileV);
    for (int kb = 0; kb < kblocks; ++kb) {
      ok = mbar_wait(&full[stage], phase, p.timeout_ns, abort_flag);
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t sa = plan.few ? x + kb * 1024 : x + stage * kAStageBytes;
      const uint32_t sb = smem_u32(smem + stage * kTileV * kBK * 2);
#pragma unroll
      for (int k = 0; k < kBK / 16; ++k)
        umma_bf16_one(d_tmem, smem_desc_sw128(sa + k * 32, 16, 1024), smem_desc_sw128(sb + k * 32, 16, 1024), idesc,
                      (kb | k) != 0 ? 1u : 0u);
      umma_commit_one(&empty[stage]);
      if (++stage == plan.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) break;
    umma_commit_one(&tfull[acc]);
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
  if (!ok) {
    *abort_flag = 1;
    *err = kErrTimeout;
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
  const int chunks = kTileV / 32 / copies;                   // 32-column chunks of a tile this warp takes
  const int c0 = share * chunks, c1 = c0 + chunks;
  const bool idle = row - lane >= p.n;                       // a warp without a token only frees accumulators
  const int y = (row < p.n) ? label_at(p.tokens, row, p.shift, p.seq_len, p.ignore_index) : p.ignore_index;

  RowBest best;
  best.val = reinterpret_cast<float*>(cand + quarter * kCandBytes);
  best.idx = reinterpret_cast<int*>(best.val + kTopkCand * 32);
  best.at = best_slot(0, lane);
  best.thr = row < p.n ? -INFINITY : INFINITY;  // (a lane without a token keeps nothing)
  best.floor = -INFINITY;
  set_bar(best);
  RowSum sum{-INFINITY, 0.f, 0.f};
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
    if (TOP && !idle && n0 == r.v0) {
      const int valid = min(cols - c0 * 32, chunks * 32);
      best.floor = chunks <= 2   ? first_floor<1>(tbase + c0 * 32, valid, p.k)
                   : chunks == 4 ? first_floor<2>(tbase + c0 * 32, valid, p.k)
                                 : first_floor<4>(tbase, valid, p.k);
      set_bar(best);
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
      float gmax[4];
      const float cmax = block_maxima(v, gmax);
      add_chunk(sum, v, cmax, p.zscale);
      if (TOP) append_chunk(best, v, gmax, cmax, col0, lane, p.k);
    }
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(&tempty[acc]);
    // Room for the next tile's, made while that one loads.
    if (TOP && n0 + kTileV < r.v1 && __any_sync(0xffffffffu, best.at >= 32 * (p.k + 3)))
      trim_best(best, lane, p.k, kTopkCand - 8);
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
  if (TOP && __any_sync(0xffffffffu, best.at >= 32 * (p.slots + 1))) trim_best(best, lane, p.k, p.slots);
  if (row >= p.n) return;
  const int part = blockIdx.x * copies + share;
  const int64_t at = static_cast<int64_t>(row) * p.parts + part;
  if (!in_bounds(at, p.part_count, err)) return;
  p.part_m[at] = sum.m;
  p.part_l[at] = sum.l;
  p.part_s[at] = sum.es;
  if (TOP) {
    const int count = best.at >> 5;
#pragma unroll 4
    for (int e = 0; e < p.slots; ++e)
      p.cand[at * p.slots + e] =
          e < count ? candidate_key(best.val[best_slot(e, lane)], best.idx[best_slot(e, lane)]) : 0;
  }
}

// The epilogue of at most 8 tokens, which are 8 lanes of TMEM: the one warp that can read
// them copies the tile's logits to shared memory, and each token is a whole warp's, eight
// neighbouring columns a lane.  Its best k are rounds of a maximum over the warp: as many as
// k in the first tile, then only where a value beats the k-th so far.
template <bool TOP>
__device__ void decode_epilogue_few(const DecodeParams& p, Range r, float* logits, uint64_t* tfull, uint64_t* tempty,
                                    uint32_t tmem_base, volatile int* abort_flag, int* err, volatile int* go) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool reader = (warp & 3) == 0;  // TMEM lanes 0-31
  const auto sync = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };  // the four epilogue warps
  constexpr int kTokens = kFewRows / 4;  // of a warp: warp - 2, warp + 2
  float m[kTokens], l[kTokens], es[kTokens];
  uint64_t best[kTokens];      // lane i: the i-th kept
  uint64_t least[kTokens];     // the least of k kept (0: fewer)
  int kept[kTokens], y[kTokens];
#pragma unroll
  for (int q = 0; q < kTokens; ++q) {
    const int row = warp - 2 + 4 * q;
    m[q] = -INFINITY;
    l[q] = es[q] = 0.f;
    best[q] = least[q] = 0;
    kept[q] = 0;
    y[q] = (row < p.n) ? label_at(p.tokens, row, p.shift, p.seq_len, p.ignore_index) : p.ignore_index;
  }
  int acc = 0;
  uint32_t acc_phase = 0;
  for (int n0 = r.v0; n0 < r.v1; n0 += kTileV) {
    const int cols = min(kTileV, r.v1 - n0);
    if (reader) {
      // (the whole warp goes on or gives up, and with it the other three)
      const bool ok = __all_sync(0xffffffffu, mbar_wait(&tfull[acc], acc_phase, p.timeout_ns, abort_flag));
      if (ok) {
        tc_fence_after_sync();
#pragma unroll 1
        for (int c = 0; c * 32 < cols; ++c) {
          uint32_t v[32];
          __syncwarp();
          tmem_ld_32x32(tmem_base + static_cast<uint32_t>(acc * kTileV + c * 32), v);
          if (lane < p.n) {
            float4* o = reinterpret_cast<float4*>(logits + lane * kFewPitch + c * 32);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              o[j] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                 __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
          }
        }
        tc_fence_before_sync();
      } else {
        *abort_flag = 1;
        *err = kErrTimeout;
      }
      if (lane == 0) *go = ok;
    }
    sync();
    if (!*go) return;
    if (lane == 0) mbar_arrive(&tempty[acc]);
#pragma unroll
    for (int q = 0; q < kTokens; ++q) {
      const int row = warp - 2 + 4 * q;
      if (row >= p.n) break;
      const float4* in = reinterpret_cast<const float4*>(logits + row * kFewPitch + lane * 8);
      const float4 lo = in[0], hi = in[1];
      float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      const int yi = y[q] - n0 - lane * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (lane * 8 + j >= cols) v[j] = -INFINITY;  // past the range (not loaded)
        else if (j == yi && y[q] != p.ignore_index) p.tgt[row] = v[j];
      }
      float top = v[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) top = fmaxf(top, v[j]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float new_m = fmaxf(m[q], top * p.zscale);
      const float from = new_m == -INFINITY ? 0.f : new_m;  // nothing but minus infinity so far: adds 0
      float sl = 0.f, se = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = max_nan(fmaf(v[j], p.zscale, -from), kNoLogit);
        const float w = fast_exp2(u);
        sl += w;
        se = fmaf(w, u, se);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sl += __shfl_xor_sync(0xffffffffu, sl, o);
        se += __shfl_xor_sync(0xffffffffu, se, o);
      }
      const float d = fmaxf(m[q] - new_m, kNoLogit);  // (minus infinity twice: the sums are 0 or NaN)
      const float f = fast_exp2(d);
      es[q] = f * fmaf(l[q], d, es[q]) + se;
      l[q] = l[q] * f + sl;
      m[q] = new_m;
      if (!TOP) continue;
      uint32_t key[8], mine = 0;  // 0: none (a NaN, or minus infinity, which the join puts in)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        key[j] = v[j] > -INFINITY ? topk_key(v[j] + 0.f) : 0u;
        mine = max(mine, key[j]);
      }
      while (true) {
        const uint32_t won = __reduce_max_sync(0xffffffffu, mine);
        // ids grow along the range: an equal value ranks after those kept
        if (won == 0 || won <= static_cast<uint32_t>(least[q] >> 32)) break;
        const int owner = __ffs(__ballot_sync(0xffffffffu, mine == won)) - 1;
        int at = 8;
        if (lane == owner) {
          mine = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (at == 8 && key[j] == won) {
              at = j;
              key[j] = 0;
            }
            mine = max(mine, key[j]);
          }
        }
        const int id = n0 + owner * 8 + __shfl_sync(0xffffffffu, at, owner);
        const uint64_t entry = (static_cast<uint64_t>(won) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
        if (kept[q] < p.k) {
          if (lane == kept[q]) best[q] = entry;
          ++kept[q];
        } else if (best[q] == least[q]) {
          best[q] = entry;  // in the place of the least (one lane holds it: entries are distinct)
        }
        if (kept[q] == p.k) {
          const uint32_t vk = lane < p.k ? static_cast<uint32_t>(best[q] >> 32) : 0xffffffffu;
          const uint32_t vmin = __reduce_min_sync(0xffffffffu, vk);
          const uint32_t ik = lane < p.k && vk == vmin ? static_cast<uint32_t>(best[q]) : 0xffffffffu;
          least[q] = (static_cast<uint64_t>(vmin) << 32) | __reduce_min_sync(0xffffffffu, ik);
        }
      }
    }
    sync();  // the logits have been read
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
#pragma unroll
  for (int q = 0; q < kTokens; ++q) {
    const int row = warp - 2 + 4 * q;
    if (row >= p.n) break;
    const int64_t at = static_cast<int64_t>(row) * p.parts + blockIdx.x;
    if (!in_bounds(at, p.part_count, err)) return;
    if (lane == 0) {
      p.part_m[at] = m[q];
      p.part_l[at] = l[q];
      p.part_s[at] = es[q];
    }
    if (TOP && lane < p.slots) p.cand[at * p.slots + lane] = best[q];
  }
}

template <bool TOP>
__global__ void __launch_bounds__(192, 1) decode_kernel(const __grid_constant__ DecodeMaps maps, const DecodeParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOff);
  uint64_t* empty = full + kMostStages;
  uint64_t* tfull = empty + kMostStages;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  int* flags = reinterpret_cast<int*>(tempty + 3);  // [0] abort, [1] error code, [2] go on
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMostStages; ++i) {
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
  const SmemPlan plan = smem_plan(p.n, p.h);
  if (warp == 0) {
    if (lane == 0) decode_producer(maps, p, plan, r, smem, full, empty, flags, flags + 1);
  } else if (warp == 1) {
    if (lane == 0)
      decode_mma(p, plan, r, smem, full, empty, tfull, tempty, tmem_base, flags, flags + 1);
  } else if (plan.few) {
    decode_epilogue_few<TOP>(p, r, reinterpret_cast<float*>(smem + plan.cand_off), tfull, tempty, tmem_base, flags,
                             flags + 1, flags + 2);
  } else {
    decode_epilogue<TOP>(p, r, smem + plan.cand_off, tfull, tempty, tmem_base, flags, flags + 1);
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
    if (entropy) entropy[row] = at_least_zero((log2l - es / l) * kLn2);
    if (p.tokens) {
      const int y = label_at(p.tokens, row, p.shift, p.seq_len, p.ignore_index);
      float lp = 0.f;
      if (y != p.ignore_index) {
        // relative to the same m as l: exact where the token holds the largest logit
        if (y >= 0 && y < p.v) lp = at_most_zero((fmaf(p.tgt[row], p.zscale, -m) - log2l) * kLn2);
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
    top_logprobs[static_cast<int64_t>(row) * p.k + rank] = at_most_zero((fmaf(z, p.zscale, -m) - log2l) * kLn2);
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
      } else if (t < p.k) {  // fewer than k logits above minus infinity
        const int id = nth_other_id(kept, count, t - count);
        if (id < p.v) {
          put(t, other_key(id));
        } else {  // fewer than k ids
          top_ids[static_cast<int64_t>(row) * p.k + t] = -1;
          top_logprobs[static_cast<int64_t>(row) * p.k + t] = -INFINITY;
        }
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

// Copies of X in a stage.  They shorten the epilogue, of which the last tile's is exposed,
// and cost the reads of X, the same lines for all SMs, with every tile.  So one copy where
// a CTA has several tiles and either the epilogue is short (no candidates) or a tile's
// K loop long enough to cover it.  One copy and four (us): 16 x 4096 x 128256, k = 0 and 8:
// 171 and 179, 181 and 189; 32 x 2048 x 64000, k = 0 and 16: 48 and 51, 69 and 68;
// 32 x 1024 x 100000, k = 16: 73 and 57; with a tile a CTA, 32 x 2048 x 32000, k = 16: 54 and 39.
int decode_copies(int64_t n, int64_t h, int64_t v, int k) {
  if (smem_plan(static_cast<int>(n), static_cast<int>(h)).few) return 1;
  if (v > kSms * kTileV && (k == 0 || h >= 4096)) return 1;
  return n <= 32 ? 4 : n <= 64 ? 2 : 1;
}

cudaError_t launch_decode(const DecodeMaps& maps, const DecodeParams& p, int ctas, float* logprob, float* entropy,
                          float* lse, int32_t* top_ids, float* top_logprobs, cudaStream_t stream) {
  return p.k > 0 ? decode_launches<true>(maps, p, ctas, logprob, entropy, lse, top_ids, top_logprobs, stream)
                 : decode_launches<false>(maps, p, ctas, logprob, entropy, lse, top_ids, top_logprobs, stream);
}

}  // namespace flce
