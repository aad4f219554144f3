// Muon: an update's matrix orthogonalised by Newton-Schulz products, alone or as a step.
//
//   m <- mu m + (1 - mu) g,   u = mu m + (1 - mu) g (Nesterov) or m         (a step's first part)
//   X = u / (|u|_F + eps)
//   steps times:  A = X X^T,   P = a I + b A + c A^2,   X <- P X     (rows <= columns)
//                 A = X^T X,   P the same,              X <- X P     (rows > columns)
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
// fp16, not bf16: singular values stay below 2.1 whatever the input, so that every scale is a power
// of two known beforehand (X 2^14, A 2^13, P by its polynomial's largest value) and the 3 bits
// more are free: rounding errors, which the steps amplify, leave 1e-3 of the result's norm, less
// than its own rounding to bf16 (1.7e-3); bf16 operands would leave 1e-2.
//
// A rounded X also carries noise of 2^-12 of its strong directions into its weak ones, which then
// grow faster, by up to a in each step (|u| of rank 8 with 2% of noise: 1.4e-2 of the result).
// So the iterates are kept as a pair hi + lo of fp16, 22 bits, but for the last ones, whose noise few
// steps are left to raise (kMuonPairGrowth).  The products
// use hi alone and the epilogue adds a lo: what P lo - a lo would add lies along the strong
// directions themselves, where it does no harm (1.0e-3 of the result then).
//
// Matrices of at most kMuonExactRows rows (or columns) average few rounding errors (8 x 8: 4e-3),
// and one block holds all of A, P and the product Q of the P: there every operand is a pair, each
// product hi hi + hi lo + lo hi, and the steps run on A alone,
//   P = a I + b A + c A^2,   Q <- P Q,   A <- P A P,
// X being read twice, for X X^T and for Q X: 1e-5 to 5e-4 of the result, 2e-3 where one direction
// holds nearly all of it.  A's rounding hides the squares of weak singular
// values, so after as many steps as that bears (kMuonReadGrowth; the usual coefficients' five)
// X <- Q X and the next steps start from a new X X^T.
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
constexpr int kEpiWarps = 8;  // two for each quarter of the TMEM lanes, each half of a tile's columns
constexpr int kProductThreads = 64 + 32 * kEpiWarps;
constexpr uint16_t kPairMask = 0x3;

// Tiles of 256 x BN.  With BN = 256 a warp of the epilogue has two staging buffers for its two
// groups of 64 columns; with 128 it has one of each, and three stages more hide the latency of
// loads that few tiles are bound by.
template <int BN>
struct Shape {
  static constexpr int kHalfN = BN / 2;  // B rows that each CTA stages
  static constexpr int kStageBytes = kAStage + kHalfN * kBK * 2;
  static constexpr int kStages = BN == 256 ? 5 : 8;
  static constexpr int kBuffers = BN == 256 ? 2 : 1;
  static constexpr int kStagingPerWarp = kBuffers * kStagingBuf;
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

// What bounds them.  At 4096 x 4096 X X^T and the square, 136 tiles on 76 pairs, take 50 us, P X, 256
// tiles, 95 and with the old lo 99: two and four waves.  Without the epilogue 44 and 84, so that a
// wave's main loop runs at 1.9 PFLOP/s, the library's rate; the last wave's idle pairs and the last
// tile's epilogue are the rest.  Four stages cost 7%, a sixth gives nothing.  28 matrices in one
// launch fill their waves: 128 to 450 us, 1.4 to 1.5 PFLOP/s, with the power cap.  Three
// of 777 x 1544 have one or two tiles for a pair: 13 to 23 us, of which the loop is 13 or 25 steps.

// A tile of the launch: its group, which of its matrices, this CTA's first row, the first column.
struct Tile {
  const MuonGroup* g;
  int matrix, m0, n0;
  int kb0, kb1;  // steps of the contraction
  int split;
};

template <int MODE, int BN, int G>
__device__ __forceinline__ bool find_tile(const MuonArgs<G>& a, int t, uint32_t rank, Tile& o) {
  if (t >= a.tiles) return false;
  int gi = 0;
  while (gi + 1 < a.groups && a.g[gi + 1].tile0 <= t) ++gi;
  const MuonGroup& g = a.g[gi];
  t -= g.tile0;
  o.g = &g;
  o.matrix = t / g.tiles_each;
  t -= o.matrix * g.tiles_each;
  int ti = 0, tj = 0;
  o.kb0 = o.split = 0;
  o.kb1 = g.kblocks;
  if (MODE == kMuonGram && g.part) {
    o.split = t;
    o.kb0 = t * g.split_blocks;
    o.kb1 = min(o.kb0 + g.split_blocks, g.kblocks);
  } else if (MODE == kMuonApply) {  // the tiles that share their part of X follow one another
    const int inner = g.tall ? g.col_tiles : g.row_tiles;
    ti = g.tall ? t / inner : t % inner;
    tj = g.tall ? t % inner : t / inner;
  } else {  // the tiles of row ti from the diagonal on
    constexpr int kPer = kPairM / BN;
    const int cols = g.col_tiles;
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

// Whether an operand's rows run along the contraction: X does in X X^T and as the left operand of
// X P, a symmetric matrix where the block is stored.
template <int MODE>
__device__ __forceinline__ bool a_k_major(const MuonGroup& g, const Tile& t, int k0) {
  return MODE == kMuonGram ? !g.tall : (MODE == kMuonApply && g.tall) || stored(t.m0, k0);
}
template <int MODE>
__device__ __forceinline__ bool b_k_major(const MuonGroup& g, const Tile& t, int k0) {
  return MODE == kMuonGram ? !g.tall : !(MODE == kMuonApply && !g.tall) && stored(t.n0, k0);
}

struct Bars {
  uint64_t *full, *empty, *tfull, *tempty, *ebar;
  volatile int* abort_flag;
};

template <int G>
__device__ __forceinline__ void record_timeout(const MuonArgs<G>& a, uint32_t rank, volatile int* abort_flag) {
  *abort_flag = 1;
  st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u), 1u);
  atomicCAS(a.status, 0, kErrTimeout);
}

// Inner coordinates are multiples of 64 elements: every copy starts on a 128-byte boundary.
template <int MODE, int BN, int G>
__device__ void run_producer(const MuonArgs<G>& a, uint32_t rank, int pair, int pairs, uint8_t* smem, const Bars& b) {
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
      for (int kb = t.kb0; kb < t.kb1; ++kb) {
        if (!mbar_wait(&b.empty[stage], phase ^ 1u, a.timeout_ns, b.abort_flag)) {
          record_timeout(a, rank, b.abort_flag);
          return;
        }
        uint8_t* sa = smem + stage * S::kStageBytes;
        uint8_t* sb = sa + kAStage;
        const uint32_t bar = full_even + 8u * stage;
        if (rank == 0) mbar_arrive_expect_tx(&b.full[stage], 2 * S::kStageBytes);
        const int k0 = kb * kBK;
        if (a_k_major<MODE>(g, t, k0)) {
          tma_load_3d_pair(sa, a128, bar, k0, t.m0, t.matrix);
        } else {
          tma_load_3d_pair(sa, a64, bar, t.m0, k0, t.matrix);
          tma_load_3d_pair(sa + kMnBlock, a64, bar, t.m0 + 64, k0, t.matrix);
        }
        if (b_k_major<MODE>(g, t, k0)) {
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

template <int MODE, int BN, int G>
__device__ void run_mma(const MuonArgs<G>& a, int pair, int pairs, uint8_t* smem, uint32_t tmem_base, const Bars& b) {
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
      for (int kb = t.kb0; kb < t.kb1; ++kb) {
        const bool a_mn = !a_k_major<MODE>(*t.g, t, kb * kBK);
        const bool b_mn = !b_k_major<MODE>(*t.g, t, kb * kBK);
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

template <int MODE, int BN, int G>
__device__ void run_epilogue(const MuonArgs<G>& a, uint32_t rank, int pair, int pairs, uint8_t* staging,
                             uint32_t tmem_base, const Bars& b) {
  constexpr int kCols = BN / 2;  // of a warp
  const int warp = (threadIdx.x >> 5) - 2, lane = threadIdx.x & 31;
  const int quarter = (warp + 2) & 3;  // TMEM lanes that this warp may read
  const int half = warp >> 2;
  using S = Shape<BN>;
  uint8_t* stg = staging + warp * S::kStagingPerWarp;
  uint64_t* ebar = b.ebar + warp;
  const uint32_t tempty_even = mapa_shared(smem_u32(b.tempty), 0);
  int acc = 0;
  uint32_t acc_phase = 0, ephase = 0;
  Tile t;
  for (int i = pair; find_tile<MODE, BN>(a, i, rank, t); i += pairs) {
    const MuonGroup& g = *t.g;
    const int i0 = t.m0 + quarter * 32, row = i0 + lane;
    const int first = t.n0 + half * kCols;
    const bool lo_in = MODE == kMuonApply && g.lo_in;
    const bool pairs_out = g.write_lo;
    // of 64 columns, one in each staging buffer
    const int chunks = i0 < g.m && first < g.n ? min(S::kBuffers, (g.n - first + 63) / 64) : 0;
    if (lo_in && chunks > 0 && lane == 0) {  // the old lo, while the tile is under way
      bulk_wait_group_read<0>();
      mbar_arrive_expect_tx(ebar, chunks * kStagingBuf);
      for (int h = 0; h < chunks; ++h)
        tma_load_3d(stg + h * kStagingBuf, &g.out_lo, ebar, first + 64 * h, i0, t.matrix);
    }
    float* keep = MODE != kMuonApply && g.diag ? g.diag + static_cast<int64_t>(t.matrix) * g.m + row : nullptr;
    const float kept = MODE == kMuonPoly && keep && row < g.m ? *keep : 0.f;  // (under way while the tile is)
    if (!mbar_wait(&b.tfull[acc], acc_phase, a.timeout_ns, b.abort_flag)) {
      record_timeout(a, rank, b.abort_flag);
      break;
    }
    tc_fence_after_sync();
    const uint32_t tbase = tmem_base + static_cast<uint32_t>(acc * BN + half * kCols) + (static_cast<uint32_t>(quarter * 32) << 16);
    if (lo_in && chunks > 0) {
      if (!mbar_wait(ebar, ephase, a.timeout_ns, b.abort_flag)) {
        record_timeout(a, rank, b.abort_flag);
        break;
      }
      ephase ^= 1u;
    }
#pragma unroll 1
    for (int h = 0; h < chunks; ++h) {
      const int j0 = first + h * 64;
      uint8_t* buf = stg + h * kStagingBuf;
      __syncwarp();
      uint32_t d[64];
      tmem_ld_32x64(tbase + h * 64, d);
      float v[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) v[j] = __uint_as_float(d[j]) * g.alpha;
      if (MODE == kMuonGram && g.part) {
        const int splits = g.tiles_each;
        float* to = g.part + ((static_cast<int64_t>(t.matrix) * splits + t.split) * kMuonExactRows + row) * kMuonExactRows + j0;
        if (row < g.m) {
#pragma unroll
          for (int j = 0; j < 64; j += 4) *reinterpret_cast<float4*>(to + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
        continue;
      }
      if (MODE != kMuonApply) {
        const int diag = row - j0;  // in this chunk, for the lanes of one row block alone
        if (static_cast<unsigned>(i0 - j0 + 31) < 95u) {
          const float plus = fmaf(g.alpha, kept, g.gamma);
          float at = 0.f;
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            if (j == diag) {
              v[j] += plus;
              at = v[j];
            }
          }
          if (MODE == kMuonGram && keep && diag >= 0 && diag < 64 && row < g.m) {
            const float hi = __half2float(__float2half_rn(at)), left = at - hi;
            *keep = fmaf(2.f, hi, left) * left;  // of the square
          }
        }
      }
      if (lo_in) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 q = *staged(buf, lane, c);
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
      // the last tile's stores are done with the buffers (the wait before the old lo's copies was the same)
      if (lane == 0 && h == 0 && !lo_in) bulk_wait_group_read<0>();
      __syncwarp();
      stage_and_store(&g.out, buf, lane, w, j0, i0, t.matrix);
      if (pairs_out) {
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float2 f = unpack_half2(w[j]);
          w[j] = pack_half2(v[2 * j] - f.x, v[2 * j + 1] - f.y);
        }
        stage_and_store(&g.out_lo, buf, lane, w, j0, i0, t.matrix);
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

template <int MODE, int BN, int G>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kProductThreads, 1)
    muon_product_kernel(const __grid_constant__ MuonArgs<G> a) {
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
    Tile t;  // what the first tile needs of the arguments, before the wait for the launch before
    if (find_tile<MODE, BN>(a, pair, rank, t)) {
      tma_prefetch_map(&t.g->a128);
      tma_prefetch_map(&t.g->a64);
      tma_prefetch_map(&t.g->b128);
      tma_prefetch_map(&t.g->b64);
      if (!t.g->part) tma_prefetch_map(&t.g->out);
      if (t.g->write_lo || t.g->lo_in) tma_prefetch_map(&t.g->out_lo);
    }
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

// ----------------------------------------------------------------------------- the steps of small matrices

constexpr int kChainThreads = 256;
constexpr int kChainHalf = kMuonExactRows * kMuonExactRows * 2;  // one fp16 matrix: two blocks of 64 columns
constexpr int kChainBlock = kChainHalf / 2;
constexpr int kChainBarOff = 6 * kChainHalf;                      // A (then P A), P, Q, each hi and lo
constexpr int kChainSmem = kChainBarOff + 64 + 1024;
static_assert(kChainSmem <= 232448, "shared memory budget");

__device__ __forceinline__ void umma_one(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t more) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(more)
      : "memory");
}

// mbar_wait without suspending the thread.
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity)
          : "memory");
      if (ok) return true;
    }
    if (global_timer_ns() - t0 > limit_ns) return false;
  }
}

// 8 fp16 of (row, columns 8 c .. 8 c + 7) of a matrix of the block.
__device__ __forceinline__ uint4* chain_at(uint8_t* m, int row, int c) {
  return reinterpret_cast<uint4*>(m + (c >> 3) * kChainBlock + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}
__device__ __forceinline__ void chain_store(uint8_t* m, int row, int c0, const float (&v)[64]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = v[8 * c + 2 * e], y = v[8 * c + 2 * e + 1];
      hi[e] = pack_half2(x, y);
      const float2 f = unpack_half2(hi[e]);
      lo[e] = pack_half2(x - f.x, y - f.y);
    }
    *chain_at(m, row, c0 + c) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *chain_at(m + kChainHalf, row, c0 + c) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// All of a matrix's steps on one X X^T in one block: operands in shared memory, one thread issues the products,
// a thread of the eight warps holds half a row of their results.  Symmetric operands are K-major
// on either side.
//   128 x 128, five steps: 48 us, of which 14 rounds of products (30 of 128 x 128 x 128, three each)
// take 18 and the results' way through registers to operands, 255 registers a thread, the others.
// One launch in the place of 13, which took 10 us each.
__global__ void __launch_bounds__(kChainThreads, 1) muon_chain_kernel(const __grid_constant__ MuonChain a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *ma = smem, *mp = smem + 2 * kChainHalf, *mq = smem + 4 * kChainHalf;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + kChainBarOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar + 1);
  uint32_t* slot = reinterpret_cast<uint32_t*>(bar + 2);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(256) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *slot;
  griddep_begin();
  int gi = 0;
  while (gi + 1 < a.groups && a.g[gi + 1].block0 <= blockIdx.x) ++gi;
  const MuonChainGroup& g = a.g[gi];
  const int64_t matrix = blockIdx.x - g.block0;
  const int r = g.r;
  const int row = (warp & 3) * 32 + lane, c0 = (warp >> 2) * 8;  // of the thread: columns 8 c0 .. 8 c0 + 63
  const bool live = 8 * c0 < r;
  const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + static_cast<uint32_t>(8 * c0);
  {
    float v[64];
#pragma unroll
    for (int j = 0; j < 64; ++j) v[j] = 0.f;
    if (row < r && live) {
      const float* from = g.part + (matrix * g.splits * kMuonExactRows + row) * kMuonExactRows + 8 * c0;
      for (int k = 0; k < g.splits; ++k, from += kMuonExactRows * kMuonExactRows) {
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          const float4 q = *reinterpret_cast<const float4*>(from + j);
          v[j] += q.x, v[j + 1] += q.y, v[j + 2] += q.z, v[j + 3] += q.w;
        }
      }
    }
    chain_store(ma, row, c0, v);
    if (!live) {  // columns that no product writes
#pragma unroll
      for (int j = 0; j < 64; ++j) v[j] = 0.f;
      chain_store(mp, row, c0, v);
      chain_store(mq, row, c0, v);
    }
  }
  uint32_t phase = 0;
  const uint32_t idesc = instr_desc_f16(kMuonExactRows, (r + 15) / 16 * 16, false, false);
  const int ksteps = (r + 15) / 16;
  auto multiply = [&](uint32_t d, uint8_t* x, uint8_t* y) {  // one thread
    const uint64_t dx = smem_desc_sw128(smem_u32(x), 16, 1024), dy = smem_desc_sw128(smem_u32(y), 16, 1024);
#pragma unroll
    for (int seg = 0; seg < 3; ++seg) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= ksteps) break;
        const int at = ((k >> 2) * kChainBlock + (k & 3) * 32) >> 4;  // (addresses are in units of 16 bytes)
        umma_one(d, dx + (at + (seg == 2 ? kChainHalf >> 4 : 0)), dy + (at + (seg == 1 ? kChainHalf >> 4 : 0)), idesc,
                 (seg | k) != 0 ? 1u : 0u);
      }
    }
  };
  // operands written by all threads; up to two products; their results ready for all threads
  auto products = [&](uint8_t* x, uint8_t* y, uint8_t* z) {
    fence_proxy_async_smem();
    tc_fence_before_sync();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after_sync();
      if (y) multiply(tmem, x, y);
      if (z) multiply(tmem + kMuonExactRows, x, z);
      asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
    }
    // one answer for all.  The products take about a microsecond: asking again finds their end
    // sooner than sleeping on it does.
    const bool done = __syncthreads_and(warp != 0 || mbar_poll(bar, phase, a.timeout_ns));
    phase ^= 1u;
    tc_fence_after_sync();
    return done;
  };
  auto result = [&](uint32_t at, float (&v)[64]) {
    uint32_t d[64];
    __syncwarp();
    tmem_ld_32x64(at, d);
#pragma unroll
    for (int j = 0; j < 64; ++j) v[j] = __uint_as_float(d[j]);
  };
  bool ok = true;
  for (int k = 0; k < a.steps && ok; ++k) {
    const bool last = k + 1 == a.steps;
    const float ps = a.p_scale;
    // P = a I + b A + c A^2
    if (a.c[k] != 0.f) ok = products(ma, ma, nullptr);
    if (live) {
      float v[64];
      if (a.c[k] != 0.f) {
        result(mine, v);
      } else {
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] = 0.f;
      }
      const float alpha = a.c[k] * ps / (kMuonAScale * kMuonAScale), beta = a.b[k] * ps / kMuonAScale;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 h = *chain_at(ma, row, c0 + c), l = *chain_at(ma + kChainHalf, row, c0 + c);
        const uint32_t uh[4] = {h.x, h.y, h.z, h.w}, ul[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_half2(uh[e]), q = unpack_half2(ul[e]);
          const int j = 8 * c + 2 * e, col = 8 * c0 + j;
          v[j] = fmaf(v[j], alpha, fmaf(f.x + q.x, beta, col == row && row < r ? a.a[k] * ps : 0.f));
          v[j + 1] = fmaf(v[j + 1], alpha, fmaf(f.y + q.y, beta, col + 1 == row && row < r ? a.a[k] * ps : 0.f));
        }
      }
      chain_store(mp, row, c0, v);
      if (k == 0) {
        const float to_q = a.q_scale[0] / ps;
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] *= to_q;
        chain_store(mq, row, c0, v);
      }
    }
    if (last && k == 0) break;
    // P A and P Q, then (P A) P
    if (ok) ok = products(mp, last ? nullptr : ma, k == 0 ? nullptr : mq);
    if (live) {
      float v[64];
      if (!last) {
        result(mine, v);
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] *= 1.f / ps;
        chain_store(ma, row, c0, v);
      }
      if (k > 0) {
        result(mine + kMuonExactRows, v);
        const float to_q = a.q_scale[k] / (ps * a.q_scale[k - 1]);
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] *= to_q;
        chain_store(mq, row, c0, v);
      }
    }
    if (last) break;
    if (ok) ok = products(ma, mp, nullptr);
    if (live) {
      float v[64];
      result(mine, v);
#pragma unroll
      for (int j = 0; j < 64; ++j) v[j] *= 1.f / ps;
      chain_store(ma, row, c0, v);
    }
  }
  if (!ok && tid == 0) {
    *abort_flag = 1;
    atomicCAS(a.status, 0, kErrTimeout);
  }
  if (live && row < r) {
    const int64_t to = (matrix * r + row) * g.pitch;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (8 * (c0 + c) >= g.pitch) continue;  // (rows end at a multiple of 8)
      *reinterpret_cast<uint4*>(g.q + to + 8 * (c0 + c)) = *chain_at(mq, row, c0 + c);
      *reinterpret_cast<uint4*>(g.q_lo + to + 8 * (c0 + c)) = *chain_at(mq + kChainHalf, row, c0 + c);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (*abort_flag) {  // products that are still under way land before shared memory and TMEM go
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) {
    }
  }
  if (warp == 0) {
    tc_fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(256) : "memory");
  }
}

// ----------------------------------------------------------------------------- momentum, norm, weights

// V (4, 2 or 1) consecutive elements from a multiple of V on, as they lie in memory: loads are
// issued together, and their words are taken apart after the last.
template <int V>
struct Words {
  uint32_t u[4];
  __device__ __forceinline__ void load(const void* p, int64_t i, bool f32) {
    if (f32) {
      const float* q = static_cast<const float*>(p) + i;
      if (V == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(q);
        u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
      } else if (V == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(q);
        u[0] = v.x, u[1] = v.y;
      } else {
        u[0] = *reinterpret_cast<const uint32_t*>(q);
      }
    } else {
      load16(static_cast<const uint16_t*>(p) + i);
    }
  }
  // of a two-byte type
  __device__ __forceinline__ void load16(const uint16_t* q) {
    if (V == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(q);
      u[0] = v.x, u[1] = v.y;
    } else if (V == 2) {
      u[0] = *reinterpret_cast<const uint32_t*>(q);
    } else {
      u[0] = *q;
    }
  }
  __device__ __forceinline__ void zero() { u[0] = u[1] = u[2] = u[3] = 0; }
  __device__ __forceinline__ float value(int e, bool f32) const {  // fp32 or bf16
    return f32 ? __uint_as_float(u[e]) : __uint_as_float((e & 1) ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
  }
  __device__ __forceinline__ float half(int e) const {
    const float2 f = unpack_half2(u[e >> 1]);
    return (e & 1) ? f.y : f.x;
  }
};

// The source that holds block c of the launch.
__device__ __forceinline__ int find_source(const uint32_t* first, int count, uint32_t c) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= c) lo = mid;
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
template <int N>
__device__ __forceinline__ Momentum momentum_of(const MuonSources<N>& a) {
  return Momentum{a.mu, a.omm, a.grad_scale ? *a.grad_scale : 1.f, a.nesterov};
}

// One chunk of kMuonChunk elements: the momentum moves, and the squares of u are added up.  Bound by
// memory: 112 matrices of 40M elements in 60 us, 73% of DRAM's nominal rate.
template <int N>
__global__ void __launch_bounds__(kNormThreads) muon_momentum_kernel(const __grid_constant__ MuonSources<N> a) {
  griddep_begin();
  const uint32_t c = blockIdx.x;
  if (c == 0 && threadIdx.x == 0 && a.first) *a.status = kOk;
  const int si = find_source(a.chunk0, a.count, c);
  const MuonSource& s = a.s[si];
  const int64_t size = static_cast<int64_t>(s.rows) * s.cols;
  const int64_t begin = static_cast<int64_t>(c - a.chunk0[si]) * kMuonChunk, end = min(begin + kMuonChunk, size);
  const Momentum q = momentum_of(a);
  const bool f32 = s.flags & kMuonGradF32, mom = s.momentum != nullptr;
  float sum = 0.f;
  if ((s.flags & kMuonAligned) && end - begin == kMuonChunk) {
#pragma unroll
    for (int k0 = 0; k0 < 8; k0 += 4) {
      const int64_t i0 = begin + (k0 * kNormThreads + static_cast<int>(threadIdx.x)) * 4;
      Words<4> g[4], m[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = i0 + k * (4 * kNormThreads);
        g[k].zero();
        m[k].zero();
        if (!in_bounds(i + 3, size, a.status)) continue;
        g[k].load(s.grad, i, f32);
        if (mom) m[k].load(s.momentum, i, true);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = i0 + k * (4 * kNormThreads);
        float n[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float gv = g[k].value(e, f32);
          n[e] = q.move(m[k].value(e, true), gv);
          const float u = mom ? q.u(n[e], gv) : gv * q.gs;
          sum = fmaf(u, u, sum);
        }
        if (mom && in_bounds(i + 3, size, a.status))
          *reinterpret_cast<float4*>(s.momentum + i) = make_float4(n[0], n[1], n[2], n[3]);
      }
    }
  } else {
    for (int64_t i = begin + threadIdx.x; i < end; i += kNormThreads) {
      if (!in_bounds(i, size, a.status)) continue;
      Words<1> g;
      g.load(s.grad, i, f32);
      const float gv = g.value(0, f32);
      float u = gv * q.gs;
      if (mom) {
        const float m = q.move(s.momentum[i], gv);
        s.momentum[i] = m;
        u = q.u(m, gv);
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

// The passes between a tensor and its X take blocks of kMuonStrip elements: a warp's lanes hold V
// (4, 2 or 1, as the rows' alignment allows) consecutive columns each, a thread 16 / V rows.
static_assert(kMuonStrip == kNormThreads * 16, "16 elements a thread (32 leave too few warps: 401 us for 319)");

template <int V>
struct Strip {
  int row, col, rows, cols;
  __device__ __forceinline__ Strip(int rows_, int cols_, uint32_t k) : rows(rows_), cols(cols_) {
    const uint32_t across = (static_cast<uint32_t>(cols) + 32 * V - 1) / (32 * V);
    row = static_cast<int>(k / across) * (128 / V) + static_cast<int>(threadIdx.x >> 5);
    col = static_cast<int>(k % across) * (32 * V) + static_cast<int>(threadIdx.x & 31) * V;
  }
  __device__ __forceinline__ bool in(int k) const { return row + 8 * k < rows && col < cols; }
  __device__ __forceinline__ int64_t at(int k, int pitch) const { return static_cast<int64_t>(row + 8 * k) * pitch + col; }
};

template <int V>
__device__ __forceinline__ void store_v(void* p, int64_t i, bool f32, const float (&x)[V]) {
  if (f32) {
    float* q = static_cast<float*>(p) + i;
    if (V == 4) *reinterpret_cast<float4*>(q) = make_float4(x[0], x[1 % V], x[2 % V], x[3 % V]);
    else if (V == 2) *reinterpret_cast<float2*>(q) = make_float2(x[0], x[1 % V]);
    else *q = x[0];
  } else {
    __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p) + i;
    if (V == 4) *reinterpret_cast<uint2*>(q) = make_uint2(pack_bf16x2(x[0], x[1 % V]), pack_bf16x2(x[2 % V], x[3 % V]));
    else if (V == 2) *reinterpret_cast<uint32_t*>(q) = pack_bf16x2(x[0], x[1 % V]);
    else *q = __float2bfloat16_rn(x[0]);
  }
}
template <int V>
__device__ __forceinline__ void store_h(__half* p, const float (&x)[V]) {
  if (V == 4) *reinterpret_cast<uint2*>(p) = make_uint2(pack_half2(x[0], x[1 % V]), pack_half2(x[2 % V], x[3 % V]));
  else if (V == 2) *reinterpret_cast<uint32_t*>(p) = pack_half2(x[0], x[1 % V]);
  else *p = __float2half_rn(x[0]);
}

// X = u / (|u| + eps) as a pair of fp16.
template <int V, int N>
__device__ __forceinline__ void scale_strip(const MuonSources<N>& a, const MuonSource& s, uint32_t k0, const Momentum& mo,
                                            float inv) {
  constexpr int kRows = 16 / V;
  constexpr int kBatch = kRows < 8 ? kRows : 8;
  const Strip<V> t(s.rows, s.cols, k0);
  const int64_t size = static_cast<int64_t>(s.rows) * s.cols, room = static_cast<int64_t>(s.rows) * s.pitch;
  const bool f32 = s.flags & kMuonGradF32, mom = s.momentum != nullptr, need_g = !mom || a.nesterov;
#pragma unroll
  for (int b = 0; b < kRows; b += kBatch) {
    Words<V> g[kBatch], m[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      g[k].zero();
      m[k].zero();
      const int64_t at = t.at(b + k, s.cols);
      if (!t.in(b + k) || !in_bounds(at + V - 1, size, a.status)) continue;
      if (need_g) g[k].load(s.grad, at, f32);
      if (mom) m[k].load(s.momentum, at, true);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      float hi[V], lo[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float gv = g[k].value(e, f32);
        hi[e] = (mom ? mo.u(m[k].value(e, true), gv) : gv * mo.gs) * inv;
        lo[e] = hi[e] - __half2float(__float2half_rn(hi[e]));
      }
      const int64_t at = t.at(b + k, s.pitch);
      if (!t.in(b + k) || !in_bounds(at + V - 1, room, a.status)) continue;
      store_h<V>(s.hi + at, hi);
      store_h<V>(s.lo + at, lo);
    }
  }
}

// 1 / (|u| + eps), times X's scale.  A sum of squares past fp32's range, or a non-finite element,
// makes the whole matrix NaN.
template <int N>
__device__ __forceinline__ float norm_factor(const MuonSources<N>& a, int si, float* red) {
  float sum = 0.f;
  for (uint32_t i = a.chunk0[si] + threadIdx.x; i < a.chunk0[si + 1]; i += kNormThreads) sum += a.part[i];
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  __syncthreads();  // (the last factor has been read)
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = red[0];
#pragma unroll
  for (int k = 1; k < kNormThreads / 32; ++k) sum += red[k];
  return isfinite(sum) ? kMuonXScale / (sqrtf(sum) + a.eps) : NAN;
}

// Blocks take runs of consecutive strips, from the last source to the first: what the momentum's
// pass left in L2 is read first.  The same 40M elements in 80 us: 359 MB through DRAM, and the
// issue slots half busy with roundings to the pair.
template <int N>
__global__ void __launch_bounds__(kNormThreads, 5) muon_scale_kernel(const __grid_constant__ MuonSources<N> a, uint32_t run) {
  griddep_begin();
  __shared__ float red[kNormThreads / 32];
  const uint32_t begin = (gridDim.x - 1 - blockIdx.x) * run, end = min(begin + run, a.strip0[a.count]);
  if (begin >= end) return;
  int si = find_source(a.strip0, a.count, begin);
  const Momentum mo = momentum_of(a);
  float inv = norm_factor(a, si, red);
  for (uint32_t q = begin; q < end; ++q) {
    if (q >= a.strip0[si + 1]) inv = norm_factor(a, ++si, red);
    const MuonSource& s = a.s[si];
    const uint32_t k = q - a.strip0[si];
    if (s.vec == 4) scale_strip<4>(a, s, k, mo, inv);
    else if (s.vec == 2) scale_strip<2>(a, s, k, mo, inv);
    else scale_strip<1>(a, s, k, mo, inv);
  }
}

template <int V>
__device__ __forceinline__ void weights_strip(const MuonTarget& s, uint32_t k0, int* status) {
  constexpr int kRows = 16 / V;
  constexpr int kBatch = kRows < 8 ? kRows : 8;
  const Strip<V> t(s.rows, s.cols, k0);
  const int64_t size = static_cast<int64_t>(s.rows) * s.cols, room = static_cast<int64_t>(s.rows) * s.pitch;
  const bool f32 = s.flags & kMuonParamF32, master = s.master != nullptr;
  const void* old = master ? s.master : s.param;  // null: X itself is the result
#pragma unroll
  for (int b = 0; b < kRows; b += kBatch) {
    Words<V> x[kBatch], l[kBatch], w[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      x[k].zero();
      l[k].zero();
      w[k].zero();
      const int64_t from = t.at(b + k, s.pitch), at = t.at(b + k, s.cols);
      if (!t.in(b + k) || !in_bounds(from + V - 1, room, status) || !in_bounds(at + V - 1, size, status)) continue;
      x[k].load16(reinterpret_cast<const uint16_t*>(s.hi) + from);
      if (s.lo) l[k].load16(reinterpret_cast<const uint16_t*>(s.lo) + from);
      if (old) w[k].load(old, at, f32 || master);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      float y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        y[e] = (x[k].half(e) + l[k].half(e)) * (1.f / kMuonXScale);
        if (old) y[e] = fmaf(-s.rate, y[e], w[k].value(e, f32 || master) * s.decay);
      }
      const int64_t at = t.at(b + k, s.cols);
      if (!t.in(b + k) || !in_bounds(at + V - 1, size, status)) continue;
      if (master) store_v<V>(s.master, at, true, y);
      if (old) store_v<V>(s.param, at, f32, y);
      else store_v<V>(s.out, at, false, y);
    }
  }
}

// X to out as bf16, or taken off the weights.  Bound by memory: 40M bf16 weights in 55 us, 193 MB of
// them through DRAM and the rest, X, from L2.
template <int N>
__global__ void __launch_bounds__(kNormThreads, 4) muon_weights_kernel(const __grid_constant__ MuonTargets<N> a, uint32_t run) {
  griddep_begin();
  const uint32_t begin = blockIdx.x * run, end = min(begin + run, a.strip0[a.count]);
  if (begin >= end) return;
  int si = find_source(a.strip0, a.count, begin);
  for (uint32_t q = begin; q < end; ++q) {
    if (q >= a.strip0[si + 1]) ++si;
    const MuonTarget& s = a.t[si];
    const uint32_t k = q - a.strip0[si];
    if (s.vec == 4) weights_strip<4>(s, k, a.status);
    else if (s.vec == 2) weights_strip<2>(s, k, a.status);
    else weights_strip<1>(s, k, a.status);
  }
}

// Strips of a block's run, so that a launch has up to `blocks` blocks for each SM: 32 for the scale's
// pass (135M elements in 314 us, with 16 in 323, with one strip a block in 463), 64 for the
// weights' (178 us; with 16 203).
uint32_t run_length(uint32_t strips, int sms, int blocks) {
  return std::max<uint32_t>(1, strips / static_cast<uint32_t>(sms * blocks));
}

template <int MODE, int BN, int G>
cudaError_t launch_mode(const MuonArgs<G>& a, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(muon_product_kernel<MODE, BN, G>, Shape<BN>::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  return launch_k(muon_product_kernel<MODE, BN, G>, dim3(pair_grid(sms, a.tiles)), dim3(kProductThreads),
                  Shape<BN>::kSmemBytes, s, a);
}

template <int BN, int G>
cudaError_t launch_width(int mode, const MuonArgs<G>& a, int sms, cudaStream_t s) {
  return mode == kMuonGram   ? launch_mode<kMuonGram, BN, G>(a, sms, s)
         : mode == kMuonPoly ? launch_mode<kMuonPoly, BN, G>(a, sms, s)
                             : launch_mode<kMuonApply, BN, G>(a, sms, s);
}

}  // namespace

cudaError_t launch_muon_chain(const MuonChain& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(muon_chain_kernel, kChainSmem, done);
  if (e != cudaSuccess) return e;
  return launch_k(muon_chain_kernel, dim3(a.blocks), dim3(kChainThreads), kChainSmem, s, a);
}
template <int N>
cudaError_t launch_muon_momentum(const MuonSources<N>& a, cudaStream_t s) {
  return launch_k(muon_momentum_kernel<N>, dim3(a.chunk0[a.count]), dim3(kNormThreads), 0, s, a);
}
template <int N>
cudaError_t launch_muon_scale(const MuonSources<N>& a, int sms, cudaStream_t s) {
  const uint32_t n = a.strip0[a.count], run = run_length(n, sms, 32);
  return launch_k(muon_scale_kernel<N>, dim3((n + run - 1) / run), dim3(kNormThreads), 0, s, a, run);
}
template <int N>
cudaError_t launch_muon_weights(const MuonTargets<N>& a, int sms, cudaStream_t s) {
  const uint32_t n = a.strip0[a.count], run = run_length(n, sms, 64);
  return launch_k(muon_weights_kernel<N>, dim3((n + run - 1) / run), dim3(kNormThreads), 0, s, a, run);
}
template cudaError_t launch_muon_momentum<kMuonFewMatrices>(const MuonSources<kMuonFewMatrices>&, cudaStream_t);
template cudaError_t launch_muon_momentum<kMuonMatrices>(const MuonSources<kMuonMatrices>&, cudaStream_t);
template cudaError_t launch_muon_scale<kMuonFewMatrices>(const MuonSources<kMuonFewMatrices>&, int, cudaStream_t);
template cudaError_t launch_muon_scale<kMuonMatrices>(const MuonSources<kMuonMatrices>&, int, cudaStream_t);
template cudaError_t launch_muon_weights<kMuonFewMatrices>(const MuonTargets<kMuonFewMatrices>&, int, cudaStream_t);
template cudaError_t launch_muon_weights<kMuonMatrices>(const MuonTargets<kMuonMatrices>&, int, cudaStream_t);
int64_t muon_strips(int64_t rows, int64_t cols, int vec) {
  return (rows * vec + 127) / 128 * ((cols + 32 * vec - 1) / (32 * vec));
}
template <int G>
cudaError_t launch_muon_product(int mode, int bn, const MuonArgs<G>& a, int sms, cudaStream_t s) {
  return bn == 256 ? launch_width<256, G>(mode, a, sms, s) : launch_width<128, G>(mode, a, sms, s);
}
template cudaError_t launch_muon_product<kMuonFewGroups>(int, int, const MuonArgs<kMuonFewGroups>&, int, cudaStream_t);
template cudaError_t launch_muon_product<kMuonGroups>(int, int, const MuonArgs<kMuonGroups>&, int, cudaStream_t);

}  // namespace flce
