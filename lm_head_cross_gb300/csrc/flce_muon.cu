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
// launches a step (kGram, kPoly, kApply), each over every matrix of the call.
//
// A and P are symmetric: half the operations of two of the three products are done, the tiles on
// and above the diagonal, and only they are stored.  A step of a contraction that needs a block
// below it loads the block above as the transposed operand it is (MN-major), so nothing is written
// twice.
//
// kGram stores A + (b / 2c) I, whose square gives P without another look at A:
//   P = c (A + (b / 2c) I)^2 + (a - b^2 / 4c) I   (c = 0: kGram stores P = a I + b A itself).
// What rounding the diagonal to fp16 leaves, up to 2^-11 of b / 2c where A's own is far smaller, is
// kept in fp32 for P's diagonal.
//
// fp16, not bf16: singular values stay below 2 whatever the input, so that every scale is a power
// of two known beforehand (X 2^14, A 2^13, P by its polynomial's largest value) and the 3 bits
// more are free: rounding errors, which the steps amplify, leave 1e-3 of the result's norm, less
// than its own rounding to bf16 (1.7e-3); bf16 operands would leave 1e-2.
//
// A rounded X also carries noise of 2^-12 of its strong directions into its weak ones, which then
// grow faster, by up to a in each step (|u| of rank 8 with 2% of noise: 1.4e-2 of the result).
// So the first kMuonPairSteps iterates are kept as a pair hi + lo of fp16, 22 bits.  The products
// use hi alone and the epilogue adds a lo: what P lo - a lo would add lies along the strong
// directions themselves, where it does no harm (1.0e-3 of the result then).
//
// Matrices of at most kMuonExactRows rows average few rounding errors (8 x 8: 4e-3) and cost
// little: all of X, A and P are pairs there, each product hi hi + hi lo + lo hi.
#include <cuda_fp16.h>

#include "flce_device.cuh"
#include "flce_internal.h"
#include "flce_launch.cuh"

namespace flce {

namespace {

constexpr int kPairM = 2 * kBM;
constexpr int kAStage = kBM * kBK * 2;
constexpr int kMnBlock = 64 * kBK * 2;  // 64 columns of 64 K rows
constexpr int kStagingBuf = 32 * 128;
constexpr int kStagingPerWarp = 2 * kStagingBuf;
constexpr int kEpiWarps = 8;  // two for each quarter of the TMEM lanes, each half of a tile's columns
constexpr int kProductThreads = 64 + 32 * kEpiWarps;
constexpr uint16_t kPairMask = 0x3;

// Tiles of 256 x BN.  BN = 128 where 256 x 256 tiles are fewer than the CTA pairs.
template <int BN>
struct Shape {
  static constexpr int kHalfN = BN / 2;  // B rows that each CTA stages
  static constexpr int kStageBytes = kAStage + kHalfN * kBK * 2;
  static constexpr int kStages = BN == 256 ? 5 : 6;
  static constexpr int kSmemStagingOff = kStages * kStageBytes;
  static constexpr int kSmemBarOff = kSmemStagingOff + kEpiWarps * kStagingPerWarp;
  static constexpr int kSmemBytes = kSmemBarOff + 256 + 1024;
  static_assert(kSmemBytes <= 232448 && (2 * kStages + 6 + kEpiWarps) * 8 <= 256, "shared memory budget");
};

// fp16 operands: formats 0 (see instr_desc_bf16).
__host__ __device__ constexpr uint32_t instr_desc_f16(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
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
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
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

// A tile of the launch: its group, which of its matrices, this CTA's first row, the first column.
struct Tile {
  const MuonGroup* g;
  int matrix, m0, n0;
};

template <int MODE, int BN>
__device__ __forceinline__ bool find_tile(const MuonArgs& a, int t, uint32_t rank, Tile& o) {
  if (t >= a.tiles) return false;
  int gi = 0;
  while (gi + 1 < a.groups && a.g[gi + 1].tile0 <= t) ++gi;
  const MuonGroup& g = a.g[gi];
  t -= g.tile0;
  o.g = &g;
  o.matrix = t / g.tiles_each;
  t -= o.matrix * g.tiles_each;
  int ti = 0, tj;
  if (MODE == kMuonApply) {  // a column of tiles shares its part of X
    ti = t % g.row_tiles;
    tj = t / g.row_tiles;
  } else {  // the tiles of row ti from the diagonal on
    constexpr int kPer = kPairM / BN;
    const int cols = (g.r + BN - 1) / BN;
    while (t >= cols - kPer * ti) t -= cols - kPer * ti++;
    tj = kPer * ti + t;
  }
  o.m0 = ti * kPairM + static_cast<int>(rank) * kBM;
  o.n0 = tj * BN;
  return true;
}

// Whether rows of the 256-row block that holds `row` are stored at column k0 of a symmetric
// matrix; else the block's transpose is.
__device__ __forceinline__ bool stored(int row, int k0) { return k0 >= (row & ~(kPairM - 1)); }

struct Bars {
  uint64_t *full, *empty, *tfull, *tempty, *ebar;
  volatile int* abort_flag;
};

__device__ __forceinline__ void record_timeout(const MuonArgs& a, uint32_t rank, volatile int* abort_flag) {
  *abort_flag = 1;
  st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u), 1u);
  atomicCAS(a.status, 0, kErrTimeout);
}

// Inner coordinates are multiples of 64 elements: every copy starts on a 128-byte boundary.
template <int MODE, int BN>
__device__ void run_producer(const MuonArgs& a, uint32_t rank, int pair, int pairs, uint8_t* smem, const Bars& b) {
  using S = Shape<BN>;
  const uint32_t full_even = mapa_shared(smem_u32(b.full), 0);
  const int bhalf = static_cast<int>(rank) * S::kHalfN;
  int stage = 0;
  uint32_t phase = 0;
  Tile t;
  for (int i = pair; find_tile<MODE, BN>(a, i, rank, t); i += pairs) {
    const MuonGroup& g = *t.g;
    const int n0 = t.n0 + bhalf;
    for (int seg = 0; seg < g.segments; ++seg) {  // hi hi, hi lo, lo hi
      const CUtensorMap* a128 = seg == 2 ? &g.a_lo128 : &g.a128;
      const CUtensorMap* a64 = seg == 2 ? &g.a_lo64 : &g.a64;
      const CUtensorMap* b128 = seg == 1 ? &g.b_lo128 : &g.b128;
      const CUtensorMap* b64 = seg == 1 ? &g.b_lo64 : &g.b64;
      for (int kb = 0; kb < g.kblocks; ++kb) {
        if (!mbar_wait(&b.empty[stage], phase ^ 1u, a.timeout_ns, b.abort_flag)) {
          record_timeout(a, rank, b.abort_flag);
          return;
        }
        uint8_t* sa = smem + stage * S::kStageBytes;
        uint8_t* sb = sa + kAStage;
        const uint32_t bar = full_even + 8u * stage;
        if (rank == 0) mbar_arrive_expect_tx(&b.full[stage], 2 * S::kStageBytes);
        const int k0 = kb * kBK;
        if (MODE == kMuonGram || stored(t.m0, k0)) {
          tma_load_3d_pair(sa, a128, bar, k0, t.m0, t.matrix);
        } else {
          tma_load_3d_pair(sa, a64, bar, t.m0, k0, t.matrix);
          tma_load_3d_pair(sa + kMnBlock, a64, bar, t.m0 + 64, k0, t.matrix);
        }
        if (MODE == kMuonGram || (MODE == kMuonPoly && stored(t.n0, k0))) {
          tma_load_3d_pair(sb, BN == 256 ? b128 : b64, bar, k0, n0, t.matrix);
        } else {
#pragma unroll
          for (int j = 0; j < S::kHalfN / 64; ++j)
            tma_load_3d_pair(sb + j * kMnBlock, b64, bar, n0 + 64 * j, k0, t.matrix);
        }
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  }
}

template <int MODE, int BN>
__device__ void run_mma(const MuonArgs& a, int pair, int pairs, uint8_t* smem, uint32_t tmem_base, const Bars& b) {
  using S = Shape<BN>;
  int stage = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0;
  Tile t;
  for (int i = pair; find_tile<MODE, BN>(a, i, 0, t); i += pairs) {
    if (!mbar_wait(&b.tempty[acc], acc_phase ^ 1u, a.timeout_ns, b.abort_flag)) {
      record_timeout(a, 0, b.abort_flag);
      return;
    }
    tc_fence_after_sync();
    const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
    uint32_t more = 0;
    for (int seg = 0; seg < t.g->segments; ++seg) {
      for (int kb = 0; kb < t.g->kblocks; ++kb) {
        const bool a_mn = MODE != kMuonGram && !stored(t.m0, kb * kBK);
        const bool b_mn = MODE == kMuonApply || (MODE == kMuonPoly && !stored(t.n0, kb * kBK));
        const uint32_t idesc = instr_desc_f16(kPairM, BN, a_mn, b_mn);
        if (!mbar_wait(&b.full[stage], phase, a.timeout_ns, b.abort_flag)) {
          record_timeout(a, 0, b.abort_flag);
          return;
        }
        tc_fence_after_sync();
        const uint32_t sa = smem_u32(smem + stage * S::kStageBytes);
        const uint32_t sb = sa + kAStage;
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k) {
          const uint64_t ad = a_mn ? smem_desc_sw128(sa + k * 2048, kMnBlock, 1024) : smem_desc_sw128(sa + k * 32, 16, 1024);
          const uint64_t bd = b_mn ? smem_desc_sw128(sb + k * 2048, kMnBlock, 1024) : smem_desc_sw128(sb + k * 32, 16, 1024);
          umma_bf16_pair(d, ad, bd, idesc, more);  // (kind::f16: idesc names the type)
          more = 1;
        }
        umma_commit_pair(&b.empty[stage], kPairMask);
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    umma_commit_pair(&b.tfull[acc], kPairMask);
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
}

// A lane's row of 64 fp16 in a staging buffer of 32, laid out as a 128-byte-swizzled box.
__device__ __forceinline__ uint4* staged(uint8_t* buf, int lane, int c) {
  return reinterpret_cast<uint4*>(buf + lane * 128 + ((c ^ (lane & 7)) << 4));
}
__device__ __forceinline__ void stage_and_store(const CUtensorMap* map, uint8_t* buf, int lane, const uint32_t (&w)[32],
                                                int x, int y, int z) {
#pragma unroll
  for (int c = 0; c < 8; ++c) *staged(buf, lane, c) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(map, buf, x, y, z);
    bulk_commit_group();
  }
}

template <int MODE, int BN>
__device__ void run_epilogue(const MuonArgs& a, uint32_t rank, int pair, int pairs, uint8_t* staging,
                             uint32_t tmem_base, const Bars& b) {
  constexpr int kCols = BN / 2;  // of a warp
  const int warp = (threadIdx.x >> 5) - 2, lane = threadIdx.x & 31;
  const int quarter = (warp + 2) & 3;  // TMEM lanes that this warp may read
  const int half = warp >> 2;
  uint8_t* stg = staging + warp * kStagingPerWarp;
  uint64_t* ebar = b.ebar + warp;
  const uint32_t tempty_even = mapa_shared(smem_u32(b.tempty), 0);
  int acc = 0, sbuf = 0;
  uint32_t acc_phase = 0, ephase = 0;
  Tile t;
  for (int i = pair; find_tile<MODE, BN>(a, i, rank, t); i += pairs) {
    const MuonGroup& g = *t.g;
    const int i0 = t.m0 + quarter * 32, row = i0 + lane;
    const int first = t.n0 + half * kCols;
    const bool lo_in = MODE == kMuonApply && g.lo_in;
    const bool pairs_out = g.write_lo;
    // the second buffer takes the old lo and then the new one
    auto fetch = [&](int j0) {
      if (lane == 0) {
        bulk_wait_group_read<0>();
        mbar_arrive_expect_tx(ebar, kStagingBuf);
        tma_load_3d(stg + kStagingBuf, &g.out_lo, ebar, j0, i0, t.matrix);
      }
    };
    if (lo_in && i0 < g.r && first < g.n) fetch(first);
    if (!mbar_wait(&b.tfull[acc], acc_phase, a.timeout_ns, b.abort_flag)) {
      record_timeout(a, rank, b.abort_flag);
      break;
    }
    tc_fence_after_sync();
    const uint32_t tbase = tmem_base + static_cast<uint32_t>(acc * BN + half * kCols) + (static_cast<uint32_t>(quarter * 32) << 16);
    bool gave_up = false;
#pragma unroll 1
    for (int h = 0; h < kCols / 64; ++h) {
      const int j0 = first + h * 64;
      if (i0 >= g.r || j0 >= g.n) break;
      __syncwarp();
      uint32_t d[64];
      tmem_ld_32x64(tbase + h * 64, d);
      float v[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) v[j] = __uint_as_float(d[j]) * g.alpha;
      if (MODE != kMuonApply) {
        const int diag = row - j0;  // in this chunk, for the lanes of one row block alone
        if (static_cast<unsigned>(i0 - j0 + 31) < 95u) {
          float* keep = g.diag ? g.diag + static_cast<int64_t>(t.matrix) * g.r + row : nullptr;
          float plus = g.gamma;
          if (MODE == kMuonPoly && keep && row < g.r) plus = fmaf(g.alpha, *keep, plus);
          float at = 0.f;
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            if (j == diag) {
              v[j] += plus;
              at = v[j];
            }
          }
          if (MODE == kMuonGram && keep && diag >= 0 && diag < 64 && row < g.r) {
            const float hi = __half2float(__float2half_rn(at)), left = at - hi;
            *keep = fmaf(2.f, hi, left) * left;  // of the square
          }
        }
      }
      if (lo_in) {
        if (!mbar_wait(ebar, ephase, a.timeout_ns, b.abort_flag)) {
          record_timeout(a, rank, b.abort_flag);
          gave_up = true;
          break;
        }
        ephase ^= 1u;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 q = *staged(stg + kStagingBuf, lane, c);
          const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack_half2(u[e]);
            v[8 * c + 2 * e] = fmaf(f.x, g.beta, v[8 * c + 2 * e]);
            v[8 * c + 2 * e + 1] = fmaf(f.y, g.beta, v[8 * c + 2 * e + 1]);
          }
        }
      }
      uint32_t w[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) w[j] = pack_half2(v[2 * j], v[2 * j + 1]);
      const bool alternate = !lo_in && !pairs_out;
      if (lane == 0) {
        if (alternate) bulk_wait_group_read<1>();
        else bulk_wait_group_read<0>();
      }
      __syncwarp();  // the old lo has been read, and the buffers' earlier stores are done with them
      stage_and_store(&g.out, stg + (alternate ? sbuf * kStagingBuf : 0), lane, w, j0, i0, t.matrix);
      sbuf ^= 1;
      if (pairs_out) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float2 f = unpack_half2(w[j]);
          w[j] = pack_half2(v[2 * j] - f.x, v[2 * j + 1] - f.y);
        }
        stage_and_store(&g.out_lo, stg + kStagingBuf, lane, w, j0, i0, t.matrix);
      }
      if (lo_in && h + 1 < kCols / 64 && j0 + 64 < g.n) fetch(j0 + 64);
    }
    if (gave_up) break;
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(tempty_even + 8u * acc);
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
  if (lane == 0) bulk_wait_group_all();
  __syncwarp();
}

template <int MODE, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kProductThreads, 1)
    muon_product_kernel(const __grid_constant__ MuonArgs a) {
  using S = Shape<BN>;
  constexpr uint32_t kTmemCols = 2 * BN;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kSmemBarOff);
  Bars b;
  b.full = bars;
  b.empty = b.full + S::kStages;
  b.tfull = b.empty + S::kStages;
  b.tempty = b.tfull + 2;
  b.ebar = b.tempty + 2;
  b.abort_flag = reinterpret_cast<volatile int*>(b.ebar + kEpiWarps);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(b.ebar + kEpiWarps + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&b.full[i], 1);
      mbar_init(&b.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.tfull[i], 1);
      mbar_init(&b.tempty[i], 2 * kEpiWarps);
    }
    for (int i = 0; i < kEpiWarps; ++i) mbar_init(&b.ebar[i], 1);
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
    if (lane == 0) run_producer<MODE, BN>(a, rank, pair, pairs, smem, b);
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) run_mma<MODE, BN>(a, pair, pairs, smem, tmem_base, b);
  } else {
    run_epilogue<MODE, BN>(a, rank, pair, pairs, smem + S::kSmemStagingOff, tmem_base, b);
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

// ----------------------------------------------------------------------------- momentum, norm, weights

template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  return F32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
// Four from an element that is a multiple of four.
__device__ __forceinline__ float4 load4(const void* p, int64_t i, bool f32) {
  if (f32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float load_g(const MuonSource& s, int64_t i) {
  return (s.flags & kMuonGradF32) ? load1<true>(s.grad, i) : load1<false>(s.grad, i);
}

// The source that holds block c of the launch.
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
static_assert(kMuonChunk == kNormThreads * 4 * 8, "eight vectors a thread");

struct Momentum {
  float mu, omm, gs;
  int nesterov;
  __device__ __forceinline__ float move(float m, float g) const { return m * mu + g * gs * omm; }
  // u, from the gradient and the momentum that has moved
  __device__ __forceinline__ float u(float m, float g) const { return nesterov ? m * mu + g * gs * omm : m; }
};
__device__ __forceinline__ Momentum momentum_of(const MuonSources& a) {
  return Momentum{a.mu, a.omm, a.grad_scale ? *a.grad_scale : 1.f, a.nesterov};
}

// One chunk of kMuonChunk elements: the momentum moves, and the squares of u are added up.
__global__ void __launch_bounds__(kNormThreads) muon_momentum_kernel(const __grid_constant__ MuonSources a) {
  griddep_begin();
  const uint32_t c = blockIdx.x;
  if (c == 0 && threadIdx.x == 0 && a.status) *a.status = kOk;
  const int si = find_source(a.count, c, [&](int i) { return a.s[i].chunk0; });
  const MuonSource& s = a.s[si];
  const int64_t begin = static_cast<int64_t>(c - s.chunk0) * kMuonChunk;
  const int64_t end = min(begin + kMuonChunk, static_cast<int64_t>(s.rows) * s.cols);
  const Momentum q = momentum_of(a);
  float sum = 0.f;
  if ((s.flags & kMuonAligned) && end - begin == kMuonChunk) {
    const bool f32 = s.flags & kMuonGradF32;
#pragma unroll
    for (int k0 = 0; k0 < 8; k0 += 4) {
      float4 g[4], m[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = begin + ((k0 + k) * kNormThreads + threadIdx.x) * 4;
        g[k] = load4(s.grad, i, f32);
        m[k] = s.momentum ? *reinterpret_cast<const float4*>(s.momentum + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float4 u = make_float4(g[k].x * q.gs, g[k].y * q.gs, g[k].z * q.gs, g[k].w * q.gs);
        if (s.momentum) {
          const float4 n = make_float4(q.move(m[k].x, g[k].x), q.move(m[k].y, g[k].y), q.move(m[k].z, g[k].z),
                                       q.move(m[k].w, g[k].w));
          *reinterpret_cast<float4*>(s.momentum + begin + ((k0 + k) * kNormThreads + threadIdx.x) * 4) = n;
          u = make_float4(q.u(n.x, g[k].x), q.u(n.y, g[k].y), q.u(n.z, g[k].z), q.u(n.w, g[k].w));
        }
        sum = fmaf(u.x, u.x, fmaf(u.y, u.y, fmaf(u.z, u.z, fmaf(u.w, u.w, sum))));
      }
    }
  } else {
#pragma unroll 4
    for (int64_t i = begin + threadIdx.x; i < end; i += kNormThreads) {
      const float g = load_g(s, i);
      float u = g * q.gs;
      if (s.momentum) {
        const float m = q.move(s.momentum[i], g);
        s.momentum[i] = m;
        u = q.u(m, g);
      }
      sum = fmaf(u, u, sum);
    }
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

constexpr int kStrip = 64;  // tiles of kStrip x kStrip go through shared memory, to be turned where the matrix is tall

struct Strip {
  int r0, c0;    // in the tensor
  int rr, cc;    // in the internal matrix
  int nr, nc;    // its size
  bool tall;
};
__device__ __forceinline__ Strip strip_of(const MuonSource& s, uint32_t q) {
  Strip t;
  const int across = (s.cols + kStrip - 1) / kStrip, k = static_cast<int>(q - s.strip0);
  t.r0 = k / across * kStrip;
  t.c0 = k % across * kStrip;
  t.tall = s.flags & kMuonTall;
  t.rr = t.tall ? t.c0 : t.r0;
  t.cc = t.tall ? t.r0 : t.c0;
  t.nr = t.tall ? s.cols : s.rows;
  t.nc = t.tall ? s.rows : s.cols;
  return t;
}

// One tile of one source: u / (|u| + eps) as a pair of fp16.  The launch runs through the sources
// backwards: what the momentum's pass left in L2 is read first.
__global__ void __launch_bounds__(kNormThreads) muon_scale_kernel(const __grid_constant__ MuonSources a) {
  griddep_begin();
  __shared__ float tile[kStrip][kStrip + 1];
  __shared__ double red[kNormThreads / 32];
  const uint32_t q = gridDim.x - 1 - blockIdx.x;
  const int si = find_source(a.count, q, [&](int i) { return a.s[i].strip0; });
  const MuonSource& s = a.s[si];
  const int tid = threadIdx.x;
  const Strip t = strip_of(s, q);
  const Momentum mo = momentum_of(a);
  const bool f32 = s.flags & kMuonGradF32;
  const bool need_g = !s.momentum || a.nesterov;
  if (s.flags & kMuonAlignedRows) {  // four columns a thread; rows are whole numbers of them
    float4 g[4], m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = (k * kNormThreads + tid) / (kStrip / 4), j = (k * kNormThreads + tid) % (kStrip / 4) * 4;
      g[k] = m[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t.r0 + i < s.rows && t.c0 + j < s.cols) {
        const int64_t at = static_cast<int64_t>(t.r0 + i) * s.cols + t.c0 + j;
        if (need_g) g[k] = load4(s.grad, at, f32);
        if (s.momentum) m[k] = *reinterpret_cast<const float4*>(s.momentum + at);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = (k * kNormThreads + tid) / (kStrip / 4), j = (k * kNormThreads + tid) % (kStrip / 4) * 4;
      float* o = &tile[i][j];
      const bool mom = s.momentum;
      o[0] = mom ? mo.u(m[k].x, g[k].x) : g[k].x * mo.gs;
      o[1] = mom ? mo.u(m[k].y, g[k].y) : g[k].y * mo.gs;
      o[2] = mom ? mo.u(m[k].z, g[k].z) : g[k].z * mo.gs;
      o[3] = mom ? mo.u(m[k].w, g[k].w) : g[k].w * mo.gs;
    }
  } else {
#pragma unroll 8
    for (int k = tid; k < kStrip * kStrip; k += kNormThreads) {
      const int i = k / kStrip, j = k % kStrip;
      float u = 0.f;
      if (t.r0 + i < s.rows && t.c0 + j < s.cols) {
        const int64_t at = static_cast<int64_t>(t.r0 + i) * s.cols + t.c0 + j;
        const float g = need_g ? load_g(s, at) : 0.f;
        u = s.momentum ? mo.u(s.momentum[at], g) : g * mo.gs;
      }
      tile[i][j] = u;
    }
  }
  const int64_t chunks = (static_cast<int64_t>(s.rows) * s.cols + kMuonChunk - 1) / kMuonChunk;
  double sum = 0.0;
  for (int64_t i = tid; i < chunks; i += kNormThreads) sum += static_cast<double>(a.part[s.chunk0 + i]);
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if ((tid & 31) == 0) red[tid >> 5] = sum;
  __syncthreads();
  sum = red[0];
#pragma unroll
  for (int k = 1; k < kNormThreads / 32; ++k) sum += red[k];
  // a sum of squares past fp32's range, or a non-finite element, makes the whole matrix NaN
  const float total = static_cast<float>(sum);
  const float inv = isfinite(total) ? kMuonXScale / (sqrtf(total) + a.eps) : NAN;
#pragma unroll
  for (int k = tid; k < kStrip * kStrip / 4; k += kNormThreads) {
    const int i = k / (kStrip / 4), j = k % (kStrip / 4) * 4;
    if (t.rr + i >= t.nr || t.cc + j >= t.nc) continue;  // (the pitch is a multiple of 8: four always fit)
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (t.tall ? tile[j + e][i] : tile[i][j + e]) * inv;
    uint2 hi, lo;
    hi.x = pack_half2(x[0], x[1]);
    hi.y = pack_half2(x[2], x[3]);
    const float2 f0 = unpack_half2(hi.x), f1 = unpack_half2(hi.y);
    lo.x = pack_half2(x[0] - f0.x, x[1] - f0.y);
    lo.y = pack_half2(x[2] - f1.x, x[3] - f1.y);
    const int64_t at = static_cast<int64_t>(t.rr + i) * s.pitch + t.cc + j;
    *reinterpret_cast<uint2*>(s.hi + at) = hi;
    *reinterpret_cast<uint2*>(s.lo + at) = lo;
  }
}

// One tile of one matrix: X, from the internal matrix, to out as bf16, or taken off the weights.
__global__ void __launch_bounds__(kNormThreads) muon_weights_kernel(const __grid_constant__ MuonTargets a) {
  griddep_begin();
  __shared__ float tile[kStrip][kStrip + 1];
  const uint32_t q = blockIdx.x;
  const int si = find_source(a.count, q, [&](int i) { return a.t[i].strip0; });
  const MuonTarget& s = a.t[si];
  const int tid = threadIdx.x;
  MuonSource shape{};
  shape.rows = s.rows;
  shape.cols = s.cols;
  shape.flags = s.flags;
  shape.strip0 = s.strip0;
  const Strip t = strip_of(shape, q);
  const bool f32 = s.flags & kMuonParamF32, vec = s.flags & kMuonAlignedRows;
  float4 w[4];
  if (!s.out && vec) {  // under way while X is turned
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = (k * kNormThreads + tid) / (kStrip / 4), j = (k * kNormThreads + tid) % (kStrip / 4) * 4;
      w[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t.r0 + i < s.rows && t.c0 + j < s.cols) {
        const int64_t at = static_cast<int64_t>(t.r0 + i) * s.cols + t.c0 + j;
        w[k] = s.master ? *reinterpret_cast<const float4*>(s.master + at) : load4(s.param, at, f32);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = (k * kNormThreads + tid) / (kStrip / 8), j = (k * kNormThreads + tid) % (kStrip / 8) * 8;
    uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
    if (t.rr + i < t.nr && t.cc + j < t.nc) {
      const int64_t at = static_cast<int64_t>(t.rr + i) * s.pitch + t.cc + j;
      hi = *reinterpret_cast<const uint4*>(s.hi + at);
      if (s.lo) lo = *reinterpret_cast<const uint4*>(s.lo + at);
    }
    const uint32_t uh[4] = {hi.x, hi.y, hi.z, hi.w}, ul[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_half2(uh[e]), g = unpack_half2(ul[e]);
      const float x0 = (f.x + g.x) * (1.f / kMuonXScale), x1 = (f.y + g.y) * (1.f / kMuonXScale);
      if (t.tall) {
        tile[j + 2 * e][i] = x0;
        tile[j + 2 * e + 1][i] = x1;
      } else {
        tile[i][j + 2 * e] = x0;
        tile[i][j + 2 * e + 1] = x1;
      }
    }
  }
  __syncthreads();
  if (vec) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = (k * kNormThreads + tid) / (kStrip / 4), j = (k * kNormThreads + tid) % (kStrip / 4) * 4;
      if (t.r0 + i >= s.rows || t.c0 + j >= s.cols) continue;
      const int64_t at = static_cast<int64_t>(t.r0 + i) * s.cols + t.c0 + j;
      float4 x = make_float4(tile[i][j], tile[i][j + 1], tile[i][j + 2], tile[i][j + 3]);
      void* to = s.out;
      if (!s.out) {
        x = make_float4(fmaf(-s.rate, x.x, w[k].x * s.decay), fmaf(-s.rate, x.y, w[k].y * s.decay),
                        fmaf(-s.rate, x.z, w[k].z * s.decay), fmaf(-s.rate, x.w, w[k].w * s.decay));
        if (s.master) *reinterpret_cast<float4*>(s.master + at) = x;
        to = s.param;
      }
      if (!s.out && f32) *reinterpret_cast<float4*>(static_cast<float*>(to) + at) = x;
      else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(to) + at) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
    }
  } else {
#pragma unroll 4
    for (int k = tid; k < kStrip * kStrip; k += kNormThreads) {
      const int i = k / kStrip, j = k % kStrip;
      if (t.r0 + i >= s.rows || t.c0 + j >= s.cols) continue;
      const int64_t at = static_cast<int64_t>(t.r0 + i) * s.cols + t.c0 + j;
      float x = tile[i][j];
      if (s.out) {
        static_cast<__nv_bfloat16*>(s.out)[at] = __float2bfloat16_rn(x);
        continue;
      }
      const float p = s.master ? s.master[at] : f32 ? load1<true>(s.param, at) : load1<false>(s.param, at);
      x = fmaf(-s.rate, x, p * s.decay);
      if (s.master) s.master[at] = x;
      if (f32) static_cast<float*>(s.param)[at] = x;
      else static_cast<__nv_bfloat16*>(s.param)[at] = __float2bfloat16_rn(x);
    }
  }
}

template <int MODE, int BN>
cudaError_t launch_mode(const MuonArgs& a, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(muon_product_kernel<MODE, BN>, Shape<BN>::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  return launch_k(muon_product_kernel<MODE, BN>, dim3(pair_grid(sms, a.tiles)), dim3(kProductThreads),
                  Shape<BN>::kSmemBytes, s, a);
}

template <int BN>
cudaError_t launch_width(int mode, const MuonArgs& a, int sms, cudaStream_t s) {
  return mode == kMuonGram   ? launch_mode<kMuonGram, BN>(a, sms, s)
         : mode == kMuonPoly ? launch_mode<kMuonPoly, BN>(a, sms, s)
                             : launch_mode<kMuonApply, BN>(a, sms, s);
}

}  // namespace

cudaError_t launch_muon_momentum(const MuonSources& a, uint32_t chunks, cudaStream_t s) {
  return launch_k(muon_momentum_kernel, dim3(chunks), dim3(kNormThreads), 0, s, a);
}
cudaError_t launch_muon_scale(const MuonSources& a, uint32_t strips, cudaStream_t s) {
  return launch_k(muon_scale_kernel, dim3(strips), dim3(kNormThreads), 0, s, a);
}
cudaError_t launch_muon_weights(const MuonTargets& a, uint32_t strips, cudaStream_t s) {
  return launch_k(muon_weights_kernel, dim3(strips), dim3(kNormThreads), 0, s, a);
}
int64_t muon_strips(int64_t rows, int64_t cols) {
  return (rows + kStrip - 1) / kStrip * ((cols + kStrip - 1) / kStrip);
}
cudaError_t launch_muon_product(int mode, int bn, const MuonArgs& a, int sms, cudaStream_t s) {
  return bn == 256 ? launch_width<256>(mode, a, sms, s) : launch_width<128>(mode, a, sms, s);
}

}  // namespace flce
