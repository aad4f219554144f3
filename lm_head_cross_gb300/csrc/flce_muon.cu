// Muon: an update's matrix orthogonalised by Newton-Schulz products, alone or as a step.
//
//   m <- mu m + (1 - mu) g,   u = mu m + (1 - mu) g (Nesterov) or m         (a step's first part)
//   X = u / (|u|_F + eps), on the side where it has fewer rows than columns [r, c]
//   steps times:  A = X X^T,   P = a I + b A + c A^2,   X <- P X
//   w <- w (1 - lr wd) - lr scale X                                         (a step's last part)
//
// An odd polynomial of X's singular values: with the usual coefficients five steps bring those
// above about 1e-3 of the norm to between 0.7 and 1.2.
//
// Products: tcgen05 on CTA pairs, 256 x 256 tiles of fp16 operands with fp32 accumulators, three
// launches a step (kGram, kPoly, kApply), each over every matrix of the call.  A and P are
// symmetric: tiles on and above the diagonal are computed and written to both sides, half the
// operations of two of the three products.
//
// fp16, not bf16: singular values stay below 2 whatever the input, so that every scale is a power
// of two known beforehand (X 2^14, A 2^14, P by its polynomial's largest value) and the 3 bits
// more are free: rounding errors, which the steps amplify, leave 1e-3 of the result's norm, less
// than its own rounding to bf16 (1.7e-3); bf16 operands would leave 1e-2.
//
// A rounded X also carries noise of 2^-12 of its strong directions into its weak ones, which then
// grow faster, by up to a in each step (|u| of rank 8 with 2% of noise: 1.4e-2 of the result).
// So the first kMuonPairSteps iterates are kept as a pair hi + lo of fp16, 22 bits.  The products use
// hi alone and the epilogue adds a lo: what P lo - a lo would add lies along the strong directions
// themselves, where it does no harm (1.0e-3 of the result then).
//
// Matrices of at most kMuonExactRows rows average few rounding errors (8 x 8: 4e-3) and cost little:
// all of X, A and P are pairs there, each product hi hi + hi lo + lo hi.
#include <cuda_fp16.h>

#include "flce_device.cuh"
#include "flce_internal.h"
#include "flce_launch.cuh"

namespace flce {

namespace {

constexpr int kPairM = 2 * kBM;
constexpr int kHalfN = kBN / 2;
constexpr int kAStage = kBM * kBK * 2;
constexpr int kBStage = kHalfN * kBK * 2;
constexpr int kStageBytes = kAStage + kBStage;
constexpr int kMnBlock = 64 * kBK * 2;  // 64 columns of 64 K rows
constexpr int kStagingBuf = 32 * 128;
constexpr int kStagingPerWarp = 2 * kStagingBuf;
constexpr int kEpiWarps = 4;
constexpr int kProductThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kTmemCols = 2 * kBN;
constexpr uint16_t kPairMask = 0x3;
constexpr int kSmemStagingOff = kStages * kStageBytes;
constexpr int kSmemBarOff = kSmemStagingOff + kEpiWarps * kStagingPerWarp;
constexpr int kSmemBytes = kSmemBarOff + 256 + 1024;
static_assert(kSmemBytes <= 232448 && (2 * kStages + 6) * 8 <= 256, "shared memory budget");

// fp16 operands: formats 0 (see instr_desc_bf16).
__host__ __device__ constexpr uint32_t instr_desc_f16(int m, int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t mbar_cluster, int32_t x,
                                                 int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar_cluster), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// ----------------------------------------------------------------------------- products

// A tile of the launch: which group, which of its matrices, this CTA's first row, the tile's first
// column, and whether it is written to the other side of the diagonal as well.
struct Tile {
  const MuonGroup* g;
  int matrix, m0, n0;
  bool mirror;
};

template <int MODE>
__device__ __forceinline__ bool find_tile(const MuonArgs& a, int t, uint32_t rank, Tile& o) {
  if (t >= a.tiles) return false;
  int gi = 0;
  while (gi + 1 < a.groups && a.g[gi + 1].tile0 <= t) ++gi;
  const MuonGroup& g = a.g[gi];
  t -= g.tile0;
  o.g = &g;
  o.matrix = t / g.tiles_each;
  t -= o.matrix * g.tiles_each;
  int ti, tj;
  if (MODE == kMuonGram || MODE == kMuonPoly) {  // (ti, tj) with ti <= tj, tj (tj + 1) / 2 + ti = t
    tj = static_cast<int>((sqrtf(8.f * static_cast<float>(t) + 1.f) - 1.f) * 0.5f);
    while (tj * (tj + 1) / 2 > t) --tj;
    while ((tj + 1) * (tj + 2) / 2 <= t) ++tj;
    ti = t - tj * (tj + 1) / 2;
    o.mirror = ti != tj;
  } else {  // a column of tiles shares its part of X
    ti = t % g.row_tiles;
    tj = t / g.row_tiles;
    o.mirror = false;
  }
  o.m0 = ti * kPairM + static_cast<int>(rank) * kBM;
  o.n0 = tj * kBN;
  return true;
}

struct Bars {
  uint64_t *full, *empty, *tfull, *tempty;
  volatile int* abort_flag;
};

__device__ __forceinline__ void record_timeout(const MuonArgs& a, uint32_t rank, volatile int* abort_flag) {
  *abort_flag = 1;
  st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u), 1u);
  atomicCAS(a.status, 0, kErrTimeout);
}

template <int MODE>
__device__ void run_producer(const MuonArgs& a, uint32_t rank, int pair, int pairs, uint8_t* smem, const Bars& b) {
  const uint32_t full_even = mapa_shared(smem_u32(b.full), 0);
  const int bhalf = static_cast<int>(rank) * kHalfN;
  int stage = 0;
  uint32_t phase = 0;
  Tile t;
  for (int i = pair; find_tile<MODE>(a, i, rank, t); i += pairs) {
    const MuonGroup& g = *t.g;
    for (int seg = 0; seg < g.segments; ++seg) {  // hi hi, hi lo, lo hi
      const CUtensorMap* ma = seg == 2 ? &g.a_lo : &g.a;
      const CUtensorMap* mb = seg == 1 ? &g.b_lo : &g.b;
      for (int kb = 0; kb < g.kblocks; ++kb) {
        if (!mbar_wait(&b.empty[stage], phase ^ 1u, a.timeout_ns, b.abort_flag)) {
          record_timeout(a, rank, b.abort_flag);
          return;
        }
        uint8_t* sa = smem + stage * kStageBytes;
        uint8_t* sb = sa + kAStage;
        const uint32_t bar = full_even + 8u * stage;
        if (rank == 0) mbar_arrive_expect_tx(&b.full[stage], 2 * kStageBytes);
        const int k0 = kb * kBK;  // (64-element steps, so every inner coordinate is on a 128-byte boundary)
        tma_load_3d_pair(sa, ma, bar, k0, t.m0, t.matrix);
        if (MODE == kMuonGram || MODE == kMuonPoly) {
          tma_load_3d_pair(sb, mb, bar, k0, t.n0 + bhalf, t.matrix);
        } else {
#pragma unroll
          for (int j = 0; j < kHalfN / 64; ++j)
            tma_load_3d_pair(sb + j * kMnBlock, mb, bar, t.n0 + bhalf + 64 * j, k0, t.matrix);
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  }
}

template <int MODE>
__device__ void run_mma(const MuonArgs& a, int pair, int pairs, uint8_t* smem, uint32_t tmem_base, const Bars& b) {
  constexpr bool b_mn = MODE == kMuonApply || MODE == kMuonFinal;
  constexpr uint32_t idesc = instr_desc_f16(kPairM, kBN, b_mn);
  int stage = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0;
  Tile t;
  for (int i = pair; find_tile<MODE>(a, i, 0, t); i += pairs) {
    if (!mbar_wait(&b.tempty[acc], acc_phase ^ 1u, a.timeout_ns, b.abort_flag)) {
      record_timeout(a, 0, b.abort_flag);
      return;
    }
    tc_fence_after_sync();
    const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kBN);
    const int steps = t.g->segments * t.g->kblocks;
    for (int kb = 0; kb < steps; ++kb) {
      if (!mbar_wait(&b.full[stage], phase, a.timeout_ns, b.abort_flag)) {
        record_timeout(a, 0, b.abort_flag);
        return;
      }
      tc_fence_after_sync();
      const uint32_t sa = smem_u32(smem + stage * kStageBytes);
      const uint32_t sb = sa + kAStage;
#pragma unroll
      for (int k = 0; k < kBK / 16; ++k) {
        const uint64_t ad = smem_desc_sw128(sa + k * 32, 16, 1024);
        const uint64_t bd = b_mn ? smem_desc_sw128(sb + k * 2048, kMnBlock, 1024) : smem_desc_sw128(sb + k * 32, 16, 1024);
        umma_bf16_pair(d, ad, bd, idesc, (kb | k) != 0 ? 1u : 0u);  // (kind::f16: idesc names the type)
      }
      umma_commit_pair(&b.empty[stage], kPairMask);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    umma_commit_pair(&b.tfull[acc], kPairMask);
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
}

// 32 rows x 64 fp16 of this warp to the tensor of `map`.
__device__ __forceinline__ void stage_and_store(const CUtensorMap* map, uint8_t* stg, int& sbuf, int lane,
                                                const uint32_t (&w)[32], int x, int y, int z) {
  uint8_t* buf = stg + sbuf * kStagingBuf;
  if (lane == 0) bulk_wait_group_read<1>();
  __syncwarp();
  uint8_t* row = buf + lane * 128;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(row + ((c ^ (lane & 7)) << 4)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(map, buf, x, y, z);
    bulk_commit_group();
  }
  sbuf ^= 1;
}

// 64 fp16 of one row, as fp32; zeros where the row or a chunk of 8 lies outside.
__device__ __forceinline__ void load_row64(const __half* p, int valid, float (&x)[64]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (8 * c < valid) v = *reinterpret_cast<const uint4*>(p + 8 * c);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_half2(u[e]);
      x[8 * c + 2 * e] = f.x;
      x[8 * c + 2 * e + 1] = f.y;
    }
  }
}

// The last product's 32 columns of 32 rows (row `i0 + lane` in v): written as bf16, or taken off
// the weights.  x is the internal matrix's element (i, j): the tensor's (j, i) where it is tall.
__device__ __forceinline__ void emit(const MuonMatrix& m, float* buf, int lane, int i0, int j0, int r, int c,
                                     const float (&v)[32]) {
  const bool tall = m.flags & kMuonTall;
  if (!tall) {  // through shared memory, so that a warp's lanes hold one row's consecutive elements
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; ++j) buf[lane * 33 + j] = v[j];
    __syncwarp();
  }
  const int64_t pitch = tall ? r : c;
#pragma unroll 1
  for (int q = 0; q < 32; q += 8) {
    int64_t at[8];
    float x[8], p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = tall ? i0 + lane : i0 + q + e, j = tall ? j0 + q + e : j0 + lane;
      x[e] = 0.f;
      if (!tall) x[e] = buf[(q + e) * 33 + lane];
      at[e] = i < r && j < c ? (tall ? j * pitch + i : i * pitch + j) : -1;
    }
    if (tall) {
#pragma unroll
      for (int k = 0; k < 32; k += 8)
        if (k == q)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = v[k + e];
    }
    if (m.out) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at[e] >= 0) static_cast<__nv_bfloat16*>(m.out)[at[e]] = __float2bfloat16_rn(x[e]);
      continue;
    }
    const bool f32 = m.flags & kMuonParamF32;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p[e] = 0.f;
      if (at[e] < 0) continue;
      p[e] = m.master ? m.master[at[e]]
             : f32    ? static_cast<const float*>(m.param)[at[e]]
                      : __bfloat162float(static_cast<const __nv_bfloat16*>(m.param)[at[e]]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (at[e] < 0) continue;
      const float w = fmaf(-m.rate, x[e], p[e] * m.decay);
      if (m.master) m.master[at[e]] = w;
      if (f32) static_cast<float*>(m.param)[at[e]] = w;
      else static_cast<__nv_bfloat16*>(m.param)[at[e]] = __float2bfloat16_rn(w);
    }
  }
}

template <int MODE>
__device__ void run_epilogue(const MuonArgs& a, const MuonMatrix* mats, uint32_t rank, int pair, int pairs,
                             uint8_t* staging, uint32_t tmem_base, const Bars& b) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;  // TMEM lanes that this warp may read
  uint8_t* stg = staging + (warp - 2) * kStagingPerWarp;
  const uint32_t tempty_even = mapa_shared(smem_u32(b.tempty), 0);
  int sbuf = 0, acc = 0;
  uint32_t acc_phase = 0;
  Tile t;
  for (int i = pair; find_tile<MODE>(a, i, rank, t); i += pairs) {
    const MuonGroup& g = *t.g;
    if (!mbar_wait(&b.tfull[acc], acc_phase, a.timeout_ns, b.abort_flag)) {
      record_timeout(a, rank, b.abort_flag);
      break;
    }
    tc_fence_after_sync();
    const uint32_t tbase = tmem_base + static_cast<uint32_t>(acc * kBN) + (static_cast<uint32_t>(quarter * 32) << 16);
    const int i0 = t.m0 + quarter * 32;
    const int row = i0 + lane;
    if (i0 < g.r) {
      if (MODE == kMuonFinal) {
        const MuonMatrix& m = mats[g.matrix0 + t.matrix];
#pragma unroll 1
        for (int h = 0; h < kBN / 32; ++h) {
          const int j0 = t.n0 + h * 32;
          if (j0 >= g.n) break;
          __syncwarp();
          uint32_t d[32];
          tmem_ld_32x32(tbase + h * 32, d);
          float v[32];
          if (g.in_lo) {  // (at most kMuonPairSteps steps)
            const __half* src = g.in_lo + t.matrix * g.in_size + static_cast<int64_t>(row) * g.in_pitch + j0;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[j] = fmaf(__uint_as_float(d[j]), g.alpha, row < g.r && j0 + j < g.n ? g.beta * __half2float(src[j]) : 0.f);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(d[j]) * g.alpha;
          }
          emit(m, reinterpret_cast<float*>(stg), lane, i0, j0, g.r, g.n, v);
        }
      } else {
#pragma unroll 1
        for (int h = 0; h < kBN / 64; ++h) {
          const int j0 = t.n0 + h * 64;
          if (j0 >= g.n) break;
          __syncwarp();
          uint32_t d[64];
          tmem_ld_32x64(tbase + h * 64, d);
          float v[64];
#pragma unroll
          for (int j = 0; j < 64; ++j) v[j] = __uint_as_float(d[j]) * g.alpha;
          const int valid = row < g.r ? g.n - j0 : 0;
          const int64_t at = t.matrix * g.in_size + static_cast<int64_t>(row) * g.in_pitch + j0;
          if (MODE == kMuonPoly || (MODE == kMuonApply && g.in_lo)) {
            float x[64];
            if (MODE == kMuonPoly) {
              load_row64(g.in_hi + at, valid, x);
#pragma unroll
              for (int j = 0; j < 64; ++j) v[j] = fmaf(x[j], g.beta, v[j]);
            }
            if (g.in_lo) {
              load_row64(g.in_lo + at, valid, x);
#pragma unroll
              for (int j = 0; j < 64; ++j) v[j] = fmaf(x[j], g.beta, v[j]);
            }
            if (MODE == kMuonPoly) {
              const int diag = row - j0;
#pragma unroll
              for (int j = 0; j < 64; ++j)
                if (j == diag) v[j] += g.gamma;
            }
          }
          uint32_t w[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) w[j] = pack_half2(v[2 * j], v[2 * j + 1]);
          stage_and_store(&g.out, stg, sbuf, lane, w, j0, i0, t.matrix);
          const int64_t mir = t.matrix * g.mir_size + static_cast<int64_t>(j0) * g.mir_pitch + row;
          if (t.mirror && row < g.r) {
#pragma unroll
            for (int j = 0; j < 64; ++j) {
              const uint32_t u = (j & 1) ? w[j >> 1] >> 16 : w[j >> 1];
              if (j0 + j < g.n)
                reinterpret_cast<uint16_t*>(g.mir_hi)[mir + static_cast<int64_t>(j) * g.mir_pitch] = static_cast<uint16_t>(u);
            }
          }
          if (g.write_lo) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float2 f = unpack_half2(w[j]);
              w[j] = pack_half2(v[2 * j] - f.x, v[2 * j + 1] - f.y);
            }
            stage_and_store(&g.out_lo, stg, sbuf, lane, w, j0, i0, t.matrix);
            if (t.mirror && row < g.r) {
#pragma unroll
              for (int j = 0; j < 64; ++j) {
                const uint32_t u = (j & 1) ? w[j >> 1] >> 16 : w[j >> 1];
                if (j0 + j < g.n)
                  reinterpret_cast<uint16_t*>(g.mir_lo)[mir + static_cast<int64_t>(j) * g.mir_pitch] = static_cast<uint16_t>(u);
              }
            }
          }
        }
      }
    }
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(tempty_even + 8u * acc);
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
  if (lane == 0) bulk_wait_group_all();
  __syncwarp();
}

template <int MODE>
__device__ __forceinline__ void product_body(const MuonArgs& a, const MuonMatrix* mats) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kSmemBarOff);
  Bars b{bars, bars + kStages, bars + 2 * kStages, bars + 2 * kStages + 2,
         reinterpret_cast<volatile int*>(bars + 2 * kStages + 4)};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 5);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&b.full[i], 1);
      mbar_init(&b.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.tfull[i], 1);
      mbar_init(&b.tempty[i], 2 * kEpiWarps);
    }
    *b.abort_flag = 0;
    mbar_fence_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch();
  if (warp == 0) {
    if (lane == 0) run_producer<MODE>(a, rank, pair, pairs, smem, b);
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) run_mma<MODE>(a, pair, pairs, smem, tmem_base, b);
  } else {
    run_epilogue<MODE>(a, mats, rank, pair, pairs, smem + kSmemStagingOff, tmem_base, b);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (*b.abort_flag) {  // let copies and MMAs in flight land before shared memory and TMEM go
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) {
    }
  }
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kProductThreads, 1)
    muon_product_kernel(const __grid_constant__ MuonArgs a) {
  product_body<MODE>(a, nullptr);
}
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kProductThreads, 1)
    muon_final_kernel(const __grid_constant__ MuonArgs a, const __grid_constant__ MuonMatrices m) {
  product_body<kMuonFinal>(a, m.m);
}

// ----------------------------------------------------------------------------- momentum and norm

__device__ __forceinline__ float load_g(const MuonSource& s, int64_t i) {
  return (s.flags & kMuonGradF32) ? static_cast<const float*>(s.grad)[i]
                                  : __bfloat162float(static_cast<const __nv_bfloat16*>(s.grad)[i]);
}

// The source that holds chunk or strip c of the launch.
template <typename F>
__device__ __forceinline__ int find_source(int count, uint32_t c, F first) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first(mid) <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

constexpr int kNormThreads = 256;

// One chunk of kMuonChunk elements: the momentum moves, and the squares of u are added up.
__global__ void __launch_bounds__(kNormThreads) muon_momentum_kernel(const __grid_constant__ MuonSources a) {
  griddep_begin();
  const uint32_t c = blockIdx.x;
  if (c == 0 && threadIdx.x == 0 && a.status) *a.status = kOk;
  const int si = find_source(a.count, c, [&](int i) { return a.s[i].chunk0; });
  const MuonSource& s = a.s[si];
  const int64_t begin = static_cast<int64_t>(c - s.chunk0) * kMuonChunk;
  const int64_t end = min(begin + kMuonChunk, static_cast<int64_t>(s.rows) * s.cols);
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  float sum = 0.f;
#pragma unroll 4
  for (int64_t i = begin + threadIdx.x; i < end; i += kNormThreads) {
    float u = load_g(s, i) * gs;
    if (s.momentum) {
      const float m = s.momentum[i] * a.mu + u * a.omm;
      s.momentum[i] = m;
      u = a.nesterov ? m * a.mu + u * a.omm : m;
    }
    sum = fmaf(u, u, sum);
  }
  __shared__ float part[kNormThreads / 32];
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kNormThreads / 32; ++k) sum += part[k];
    a.part[c] = sum;
  }
}

constexpr int kStripR = 64, kStripC = 64;

// A 64 x 64 tile of one source: u / (|u| + eps) as a pair of fp16, turned where the matrix is tall.
__global__ void __launch_bounds__(kNormThreads) muon_scale_kernel(const __grid_constant__ MuonSources a) {
  griddep_begin();
  __shared__ float tile[kStripR][kStripC + 1];
  __shared__ double red[kNormThreads / 32];
  const uint32_t q = blockIdx.x;
  const int si = find_source(a.count, q, [&](int i) { return a.s[i].strip0; });
  const MuonSource& s = a.s[si];
  const int tid = threadIdx.x;
  const int64_t chunks = (static_cast<int64_t>(s.rows) * s.cols + kMuonChunk - 1) / kMuonChunk;
  double sum = 0.0;
  for (int64_t i = tid; i < chunks; i += kNormThreads) sum += static_cast<double>(a.part[s.chunk0 + i]);
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if ((tid & 31) == 0) red[tid >> 5] = sum;
  const int across = (s.cols + kStripC - 1) / kStripC;
  const int r0 = static_cast<int>(q - s.strip0) / across * kStripR, c0 = static_cast<int>(q - s.strip0) % across * kStripC;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
#pragma unroll 4
  for (int k = tid; k < kStripR * kStripC; k += kNormThreads) {
    const int i = k / kStripC, j = k % kStripC;
    float u = 0.f;
    if (r0 + i < s.rows && c0 + j < s.cols) {
      const int64_t at = static_cast<int64_t>(r0 + i) * s.cols + c0 + j;
      if (!s.momentum || a.nesterov) u = load_g(s, at) * gs;
      if (s.momentum) {
        const float m = s.momentum[at];
        u = a.nesterov ? m * a.mu + u * a.omm : m;
      }
    }
    tile[i][j] = u;
  }
  __syncthreads();
  sum = red[0];
#pragma unroll
  for (int k = 1; k < kNormThreads / 32; ++k) sum += red[k];
  // a sum of squares past fp32's range, or a non-finite element, makes the whole matrix NaN
  const float total = static_cast<float>(sum);
  const float inv = isfinite(total) ? kMuonXScale / (sqrtf(total) + a.eps) : NAN;
  const bool tall = s.flags & kMuonTall;
  const int rr = tall ? c0 : r0, cc = tall ? r0 : c0;  // the tile in the internal matrix
  const int nr = tall ? s.cols : s.rows, nc = tall ? s.rows : s.cols;
  for (int k = tid; k < kStripR * kStripC / 2; k += kNormThreads) {
    const int i = k / (kStripC / 2), j = k % (kStripC / 2) * 2;
    if (rr + i >= nr || cc + j >= nc) continue;
    const float x0 = (tall ? tile[j][i] : tile[i][j]) * inv;
    const float x1 = cc + j + 1 < nc ? (tall ? tile[j + 1][i] : tile[i][j + 1]) * inv : 0.f;  // (the pitch is even)
    const uint32_t hi = pack_half2(x0, x1);
    const float2 f = unpack_half2(hi);
    const int64_t at = static_cast<int64_t>(rr + i) * s.pitch + cc + j;
    *reinterpret_cast<uint32_t*>(s.hi + at) = hi;
    *reinterpret_cast<uint32_t*>(s.lo + at) = pack_half2(x0 - f.x, x1 - f.y);
  }
}

template <int MODE>
cudaError_t launch_mode(const MuonArgs& a, int grid, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(muon_product_kernel<MODE>, kSmemBytes, done);
  if (e != cudaSuccess) return e;
  return launch_k(muon_product_kernel<MODE>, dim3(grid), dim3(kProductThreads), kSmemBytes, s, a);
}

}  // namespace

cudaError_t launch_muon_momentum(const MuonSources& a, uint32_t chunks, cudaStream_t s) {
  return launch_k(muon_momentum_kernel, dim3(chunks), dim3(kNormThreads), 0, s, a);
}
cudaError_t launch_muon_scale(const MuonSources& a, uint32_t strips, cudaStream_t s) {
  return launch_k(muon_scale_kernel, dim3(strips), dim3(kNormThreads), 0, s, a);
}
int64_t muon_strips(int64_t rows, int64_t cols) {
  return (rows + kStripR - 1) / kStripR * ((cols + kStripC - 1) / kStripC);
}
cudaError_t launch_muon_product(int mode, const MuonArgs& a, const MuonMatrices& m, int sms, cudaStream_t s) {
  const int grid = pair_grid(sms, a.tiles);
  switch (mode) {
    case kMuonGram: return launch_mode<kMuonGram>(a, grid, s);
    case kMuonPoly: return launch_mode<kMuonPoly>(a, grid, s);
    case kMuonApply: return launch_mode<kMuonApply>(a, grid, s);
    default: break;
  }
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(muon_final_kernel, kSmemBytes, done);
  if (e != cudaSuccess) return e;
  return launch_k(muon_final_kernel, dim3(grid), dim3(kProductThreads), kSmemBytes, s, a, m);
}

}  // namespace flce
