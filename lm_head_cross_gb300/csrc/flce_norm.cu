// Layer norm: forward, and backward with the reduction of the weight's and
// bias's gradients over the rows.
#include <algorithm>

#include "flce_device.cuh"
#include "flce_internal.h"
#include "flce_launch.cuh"

namespace flce {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormSms = 152;  // SMs of the GPU this is written for

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Sum of (a, b) over the block, in a fixed order; every thread gets it.
__device__ __forceinline__ float2 block_sum(float2 v, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  __syncthreads();  // the previous sum has been read
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float2 s = red[0];
  for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) {
    s.x += red[w].x;
    s.y += red[w].y;
  }
  return s;
}

// N elements of T as one access.
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

// Hides where a register's value came from.  Between two uses of a row held in bf16 it
// keeps the compiler from holding the row as fp32 instead, in twice the registers (162
// rather than 94 for 4096 elements a warp: 8 warps an SM, and 2.2 TB/s).
template <typename T, int N>
__device__ __forceinline__ void keep_packed(Pack<T, N>& p) {
  if (sizeof(Pack<T, N>) % 4 == 0 && sizeof(T) < 4) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&p);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(Pack<T, N>) / 4); ++i) asm("" : "+r"(w[i]));
  }
}

// Element e of a pack, as fp32.
template <typename T, int N>
__device__ __forceinline__ float element(const Pack<T, N>& p, int e) {
  if (sizeof(T) == 2 && N > 1) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(&p)[e >> 1];
    return __uint_as_float((e & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  return to_f32(p.v[e]);
}

// Elements 2e and 2e + 1.
template <typename T, int N>
__device__ __forceinline__ float2 element2(const Pack<T, N>& p, int e) {
  return make_float2(element(p, 2 * e), element(p, 2 * e + 1));
}

template <typename T, int N>
__device__ __forceinline__ void pack_f32(Pack<T, N>& p, const float (&o)[N]) {
  if (sizeof(T) == 2 && N > 1) {
#pragma unroll
    for (int e = 0; e + 1 < N; e += 2) reinterpret_cast<uint32_t*>(&p)[e >> 1] = pack_bf16x2(o[e], o[e + 1]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) p.v[e] = from_f32<T>(o[e]);
  }
}

// N elements of a vector of either type, as fp32 (f32 is the same for the whole grid).
template <int N>
__device__ __forceinline__ void load_w(const void* w, bool f32, int j, float (&o)[N]) {
  if (f32) {
    constexpr int kStep = N < 4 ? N : 4;  // 16 bytes at a time
#pragma unroll
    for (int e = 0; e < N; e += kStep) {
      const auto p = *reinterpret_cast<const Pack<float, kStep>*>(static_cast<const float*>(w) + j + e);
#pragma unroll
      for (int i = 0; i < kStep; ++i) o[e + i] = p.v[i];
    }
  } else {
    const auto p = *reinterpret_cast<const Pack<__nv_bfloat16, N>*>(static_cast<const __nv_bfloat16*>(w) + j);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = element(p, i);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the WARPS warps that share a row: the warp, or the block.
template <int WARPS>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (WARPS == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) s += red[w];
  return s;
}

// Forward: the row stays in registers between its three uses (mean, squares about the
// mean, y), so memory sees one read of x and one write of y: bound by their bytes, 131072 x
// 4096 bf16 in 307 us, 7.0 TB/s (with fp32 weights, whose loads fill the first-level cache's
// ports, 352).  WARPS warps share a row, VPL accesses of N elements a
// lane, all in flight at once; a row each with WARPS = 1, whose sums are shuffles alone, and
// then several rows a block where they are short (the device starts about one block a
// nanosecond).
template <int WARPS, int VPL>
constexpr int kFwdThreads = WARPS > 1 ? 32 * WARPS : VPL <= 4 ? 256 : 64;

template <typename T, int N, int WARPS, int VPL>
__global__ void __launch_bounds__(kFwdThreads<WARPS, VPL>) norm_fwd_rows_kernel(int64_t n, int h, int64_t pitch, float eps,
                                                                     const T* __restrict__ x,
                                                                     const void* __restrict__ weight,
                                                                     const void* __restrict__ bias, bool w_f32,
                                                                     T* __restrict__ y, float* __restrict__ mean,
                                                                     float* __restrict__ rstd) {
  griddep_begin();
  __shared__ float red[2][WARPS];
  constexpr int kLanes = 32 * WARPS;
  const int lane = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = WARPS == 1 ? blockIdx.x * int64_t{kFwdThreads<1, VPL> / 32} + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= n) return;  // whole warps (WARPS = 1), else never
  const T* xr = x + row * pitch;
  Pack<T, N> v[VPL];
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const int j = (lane + k * kLanes) * N;
    if (j < h) v[k] = *reinterpret_cast<const Pack<T, N>*>(xr + j);
  }
  float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < VPL; ++k)
    if ((lane + k * kLanes) * N < h) {
#pragma unroll
      for (int e = 0; e < N / 2; ++e) s2 = add2(s2, element2(v[k], e));
      if (N == 1) s2.x += element(v[k], 0);
    }
  const float s = s2.x + s2.y;
#pragma unroll
  for (int k = 0; k < VPL; ++k) keep_packed(v[k]);
  const float mu = row_sum<WARPS>(s, red[0]) / h;
  float2 q2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < VPL; ++k)
    if ((lane + k * kLanes) * N < h) {
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const float2 d = add2(element2(v[k], e), both(-mu));
        q2 = fma2(d, d, q2);
      }
      if (N == 1) q2.x = fmaf(element(v[k], 0) - mu, element(v[k], 0) - mu, q2.x);
    }
  const float q = q2.x + q2.y;
#pragma unroll
  for (int k = 0; k < VPL; ++k) keep_packed(v[k]);
  const float rs = 1.f / sqrtf(row_sum<WARPS>(q, red[1]) / h + eps);
  T* yr = y + row * h;
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const int j = (lane + k * kLanes) * N;
    if (j >= h) continue;
    float w[N], b[N];
    load_w<N>(weight, w_f32, j, w);
    if (bias) {
      load_w<N>(bias, w_f32, j, b);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) b[e] = 0.f;
    }
    if (N == 1) w[0] = fmaf((element(v[k], 0) - mu) * rs, w[0], b[0]);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const float2 o = fma2(mul2(add2(element2(v[k], e), both(-mu)), both(rs)), make_float2(w[2 * e], w[2 * e + 1]),
                            make_float2(b[2 * e], b[2 * e + 1]));
      w[2 * e] = o.x;
      w[2 * e + 1] = o.y;
    }
    pack_f32(v[k], w);
    *reinterpret_cast<Pack<T, N>*>(yr + j) = v[k];
  }
  if (lane == 0) {
    mean[row] = mu;
    rstd[row] = rs;
  }
}

template <int BYTES>
__device__ __forceinline__ void cp_async(void* smem, const void* gmem) {
  static_assert(BYTES == 16 || BYTES == 4, "sizes used");
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
}
// 16 bytes, of which the first `bytes` are read and the others are zeros.
__device__ __forceinline__ void cp_async_part(void* smem, const void* gmem, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem)), "l"(gmem), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ----------------------------------------------------------------------------- rows at any 16-byte phase

// Rows whose length no 16-byte access divides start at every phase of one, but row r + 8's
// is row r's.  So a block takes rows a multiple of 8 apart, and its lanes' accesses start
// where the 16-byte lines do: `phase` elements before each row, the same for all of the
// block's rows.  The lanes then own the same columns of every row as in the aligned
// kernels; only a row's first and last access are cut.
__device__ __forceinline__ int row_phase(int h, int n) {
  return static_cast<int>((blockIdx.x * static_cast<unsigned>(h)) & static_cast<unsigned>(n - 1));
}

// Blocks of a launch whose blocks keep to one phase: `most` is a multiple of 8.
int phase_blocks(int64_t blocks, int most) {
  return static_cast<int>(std::min<int64_t>((blocks + 7) / 8 * 8, most));
}

// Copies an access that starts at column c of its row (column 0 at `row`), zeros past h.
template <typename T, int N>
__device__ __forceinline__ void cp_async_row(void* smem, const T* row, int c, int h) {
  cp_async_part(smem, row + c, (h - c < N ? h - c : N) * static_cast<int>(sizeof(T)));
}

// Columns [c, c + N) of a row, of which those in [0, h) exist.
template <typename T, int N>
__device__ __forceinline__ void store_row(T* row, int c, int h, const Pack<T, N>& p) {
  if (c >= 0 && c + N <= h) {
    *reinterpret_cast<Pack<T, N>*>(row + c) = p;
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e >= 0 && c + e < h) row[c + e] = p.v[e];
  }
}

template <int N>
__device__ __forceinline__ void load_w_row(const void* w, bool f32, int c, int h, float (&o)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    o[e] = 0.f;
    if (c + e < 0 || c + e >= h) continue;
    o[e] = f32 ? static_cast<const float*>(w)[c + e] : to_f32(static_cast<const __nv_bfloat16*>(w)[c + e]);
  }
}

template <typename T, int N, int GW, int VPL>
struct FwdPhaseShape {
  static constexpr int kWarps = 16;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kGroups = kWarps / GW;
  static constexpr int kColumns = 32 * GW * VPL * N;               // the widest row, with its phase
  static constexpr int kStages = VPL <= 1 ? 4 : VPL <= 2 ? 3 : 2;  // rows in flight for each group
  static constexpr int kStageBytes = kThreads * VPL * 16;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kSmemBytes = kRingBytes + 8 * kColumns;  // weight and bias in fp32
  static constexpr int kBlocks = kSmemBytes <= 112 * 1024 ? 2 : 1;  // on one SM
};

// Forward at any phase.  GW warps share a row, kGroups rows in a block at a time; blocks stay,
// because no vector access fits the weight and bias here: a block lays them out once, in
// fp32 and in the lanes' order, and its rows stream through a ring of asynchronous copies, of
// which a lane reads back only its own.  Bound by issue and the exchange of the row's two sums:
// bf16 65536 x 2049 in 126 us, 4.3 TB/s (246 by single elements), fp32 32768 x 2050 in 90 us,
// 6.0 TB/s.
template <typename T, int N, int GW, int VPL>
__global__ void __launch_bounds__(FwdPhaseShape<T, N, GW, VPL>::kThreads, FwdPhaseShape<T, N, GW, VPL>::kBlocks)
    norm_fwd_phase_kernel(int n, int h, int64_t pitch, float eps, const T* __restrict__ x,
                          const void* __restrict__ weight, const void* __restrict__ bias, bool w_f32,
                          T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  using S = FwdPhaseShape<T, N, GW, VPL>;
  static_assert(VPL * N <= 32 && N % 4 == 0, "a bit for each of a lane's columns");
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][S::kWarps];
  griddep_begin();
  const int group = static_cast<int>(threadIdx.x) / (32 * GW);
  const int lane = static_cast<int>(threadIdx.x) % (32 * GW);
  const int first = blockIdx.x + group * gridDim.x;
  const int step = gridDim.x * S::kGroups;  // (row + step fits 32 bits: see norm_forward)
  const int phase = row_phase(h, N);
  const auto column = [&](int k) { return (k * 32 * GW + lane) * N - phase; };
  const auto slot = [&](int stage, int k) { return ring + stage * S::kStageBytes + (k * S::kThreads + threadIdx.x) * 16; };
  const auto fetch = [&](int row, int stage) {
    if (row < n) {
      const T* xr = x + row * pitch;
#pragma unroll
      for (int k = 0; k < VPL; ++k)
        if (column(k) < h) cp_async_row<T, N>(slot(stage, k), xr, column(k), h);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < S::kStages; ++s) fetch(first + s * step, s);

  // Which of the lane's columns exist (bit k N + e), and for each access: whether the warp
  // has any (bit 2k), and whether some are missing (bit 2k + 1).
  constexpr uint32_t kFull = (1u << N) - 1;
  uint32_t valid = 0, uses = 0;
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) m |= (column(k) + e >= 0 && column(k) + e < h ? 1u : 0u) << e;
    valid |= m << (k * N);
    uses |= (__any_sync(0xffffffffu, m != 0) ? 1u : 0u) << (2 * k);
    uses |= (__any_sync(0xffffffffu, m != kFull) ? 2u : 0u) << (2 * k);
    if (column(k) >= h)  // zeros throughout
      for (int s = 0; s < S::kStages; ++s) *reinterpret_cast<uint4*>(slot(s, k)) = make_uint4(0, 0, 0, 0);
  }
  float4* const wb = reinterpret_cast<float4*>(ring + S::kRingBytes);
  constexpr int kBias = S::kColumns / 4;  // where the bias starts
  if (group == 0) {
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      float w[N], b[N] = {};
      load_w_row<N>(weight, w_f32, column(k), h, w);
      if (bias) load_w_row<N>(bias, w_f32, column(k), h, b);
#pragma unroll
      for (int q = 0; q < N / 4; ++q) {
        const int at = (k * (N / 4) + q) * 32 * GW + lane;
        wb[at] = make_float4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        wb[kBias + at] = make_float4(b[4 * q], b[4 * q + 1], b[4 * q + 2], b[4 * q + 3]);
      }
    }
  }
  __syncthreads();
  const auto group_sum = [&](float v, float* at) {
    v = warp_sum(v);
    if constexpr (GW > 1) {
      // (either half of red[] is rewritten only after the other's next barrier)
      if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = v;
      if constexpr (S::kGroups == 1) __syncthreads();
      else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * GW) : "memory");
      v = 0.f;
#pragma unroll
      for (int q = 0; q < GW; ++q) v += at[group * GW + q];
    }
    return v;
  };
  int stage = 0;
  for (int row = first; row < n; row += step) {
    cp_async_wait<S::kStages - 1>();
    Pack<T, N> v[VPL];
#pragma unroll
    for (int k = 0; k < VPL; ++k) v[k] = *reinterpret_cast<const Pack<T, N>*>(slot(stage, k));
    __syncwarp();
    fetch(row + S::kStages * step, stage);
    if (++stage == S::kStages) stage = 0;
    if (lane == 0 && phase > 0) {  // the row before
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < phase) v[0].v[e] = from_f32<T>(0.f);
    }
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
#pragma unroll
      for (int e = 0; e < N / 2; ++e) s2 = add2(s2, element2(v[k], e));
    }
#pragma unroll
    for (int k = 0; k < VPL; ++k) keep_packed(v[k]);
    const float mu = group_sum(s2.x + s2.y, red[0]) / h;
    float2 q2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      if ((uses >> (2 * k) & 2u) == 0) {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          const float2 d = add2(element2(v[k], e), both(-mu));
          q2 = fma2(d, d, q2);
        }
      } else if (uses >> (2 * k) & 1u) {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          float2 d = add2(element2(v[k], e), both(-mu));
          if (!(valid >> (k * N + 2 * e) & 1u)) d.x = 0.f;
          if (!(valid >> (k * N + 2 * e + 1) & 1u)) d.y = 0.f;
          q2 = fma2(d, d, q2);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < VPL; ++k) keep_packed(v[k]);
    const float rs = 1.f / sqrtf(group_sum(q2.x + q2.y, red[1]) / h + eps);
    T* yr = y + static_cast<int64_t>(row) * h;
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      if (!(uses >> (2 * k) & 1u)) continue;
      float o[N];
#pragma unroll
      for (int q = 0; q < N / 4; ++q) {
        const int at = (k * (N / 4) + q) * 32 * GW + lane;
        const float4 w = wb[at], b = wb[kBias + at];
        const float2 t0 = fma2(mul2(add2(element2(v[k], 2 * q), both(-mu)), both(rs)), make_float2(w.x, w.y),
                               make_float2(b.x, b.y));
        const float2 t1 = fma2(mul2(add2(element2(v[k], 2 * q + 1), both(-mu)), both(rs)), make_float2(w.z, w.w),
                               make_float2(b.z, b.w));
        o[4 * q] = t0.x;
        o[4 * q + 1] = t0.y;
        o[4 * q + 2] = t1.x;
        o[4 * q + 3] = t1.y;
      }
      pack_f32(v[k], o);
      if ((valid >> (k * N) & kFull) == kFull) {
        *reinterpret_cast<Pack<T, N>*>(yr + column(k)) = v[k];
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (valid >> (k * N + e) & 1u) yr[column(k) + e] = v[k].v[e];
      }
    }
    if (lane == 0) {
      mean[row] = mu;
      rstd[row] = rs;
    }
  }
}

// Rows too wide for registers (past 65536 columns in bf16, 32768 in fp32; that no 16-byte
// access divides, past 16384 and 8192): one block per row, the row read three times (the
// second and third time from L2) in single elements, whose issue bounds it: 2048 x 80000 bf16
// 347 us, 1.9 TB/s, fp32 484 us, 2.7 TB/s; 8192 x 20001 bf16 236 us, 2.8 TB/s.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(int64_t n, int h, int64_t pitch, float eps,
                                                                const T* __restrict__ x,
                                                                const void* __restrict__ weight,
                                                                const void* __restrict__ bias, bool w_f32,
                                                                T* __restrict__ y, float* __restrict__ mean,
                                                                float* __restrict__ rstd) {
  griddep_begin();
  __shared__ float2 red[kNormThreads / 32];
  for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
    const T* xr = x + row * pitch;
    T* yr = y + row * h;
    float s = 0.f;
    for (int j = threadIdx.x; j < h; j += kNormThreads) s += to_f32(xr[j]);
    const float mu = block_sum(make_float2(s, 0.f), red).x / h;
    float q = 0.f;
    for (int j = threadIdx.x; j < h; j += kNormThreads) {
      const float d = to_f32(xr[j]) - mu;
      q += d * d;
    }
    const float rs = 1.f / sqrtf(block_sum(make_float2(q, 0.f), red).x / h + eps);
    for (int j = threadIdx.x; j < h; j += kNormThreads) {
      float w[1], b[1] = {0.f};
      load_w<1>(weight, w_f32, j, w);
      if (bias) load_w<1>(bias, w_f32, j, b);
      yr[j] = from_f32<T>(fmaf((to_f32(xr[j]) - mu) * rs, w[0], b[0]));
    }
    if (threadIdx.x == 0) {
      mean[row] = mu;
      rstd[row] = rs;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_dx_kernel(int64_t n, int h, int64_t pitch,
                                                               const T* __restrict__ dy, const T* __restrict__ x,
                                                               const void* __restrict__ weight, bool w_f32,
                                                               const float* __restrict__ mean,
                                                               const float* __restrict__ rstd, T* __restrict__ dx) {
  griddep_begin();
  __shared__ float2 red[kNormThreads / 32];
  for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
    const T* xr = x + row * pitch;
    const T* dr = dy + row * h;
    T* or_ = dx + row * h;
    const float mu = mean[row], rs = rstd[row];
    float2 s = make_float2(0.f, 0.f);
    for (int j = threadIdx.x; j < h; j += kNormThreads) {
      float w[1];
      load_w<1>(weight, w_f32, j, w);
      const float u = to_f32(dr[j]) * w[0];
      s.x += u;
      s.y += u * ((to_f32(xr[j]) - mu) * rs);
    }
    s = block_sum(s, red);
    const float a = s.x / h, b = s.y / h;
    for (int j = threadIdx.x; j < h; j += kNormThreads) {
      float w[1];
      load_w<1>(weight, w_f32, j, w);
      const float u = to_f32(dr[j]) * w[0];
      or_[j] = from_f32<T>(rs * (u - a - (to_f32(xr[j]) - mu) * rs * b));
    }
  }
}

// Partial sums over a slice of rows: part[slice][0][j] = sum dy xhat, part[slice][1][j] = sum dy.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_dw_partial_kernel(int64_t n, int h, int64_t pitch, int64_t rows,
                                                                       const T* __restrict__ dy,
                                                                       const T* __restrict__ x,
                                                                       const float* __restrict__ mean,
                                                                       const float* __restrict__ rstd,
                                                                       float* __restrict__ part) {
  griddep_begin();
  const int j = blockIdx.x * kNormThreads + threadIdx.x;
  if (j >= h) return;
  const int64_t r0 = blockIdx.y * rows;
  const int64_t r1 = r0 + rows < n ? r0 + rows : n;
  float a = 0.f, b = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float d = to_f32(dy[r * h + j]);
    a += d * ((to_f32(x[r * pitch + j]) - mean[r]) * rstd[r]);
    b += d;
  }
  float* out = part + static_cast<int64_t>(blockIdx.y) * 2 * h;
  out[j] = a;
  out[h + j] = b;
}

// dweight, dbias: sums of `slices` rows of 2 `half` partial sums each.  32 sums a block, the
// rows dealt over its 32 warps (about ten loads each, all in flight) and joined in warp
// order.  Sum p of a half belongs to column (p / (n lanes)) n lanes + (p % lanes) n + (p /
// lanes) % n: value p / lanes of lane p % lanes, n columns an access.
constexpr int kFinalWarps = 32;
template <typename W>
__global__ void __launch_bounds__(32 * kFinalWarps) norm_dw_final_kernel(int h, int slices, int half, int lanes, int n,
                                                                         const float* __restrict__ part,
                                                                         W* __restrict__ dweight,
                                                                         W* __restrict__ dbias) {
  griddep_begin();
  __shared__ float red[kFinalWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t j = blockIdx.x * int64_t{32} + lane;  // of [dweight | dbias]
  const bool in = j < 2 * static_cast<int64_t>(half);
  float a = 0.f;
  if (in) {
#pragma unroll 10
    for (int s = warp; s < slices; s += kFinalWarps) a += part[static_cast<int64_t>(s) * 2 * half + j];
  }
  red[warp][lane] = a;
  __syncthreads();
  if (warp != 0 || !in) return;
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < kFinalWarps; ++w) t += red[w][lane];
  const int p = static_cast<int>(j < half ? j : j - half);
  const int column = lanes == 1 ? p : p / (n * lanes) * n * lanes + p % lanes * n + p / lanes % n;
  if (column >= h) return;
  if (j < half) dweight[column] = from_f32<W>(t);
  else if (dbias) dbias[column] = from_f32<W>(t);
}

// ----------------------------------------------------------------------------- backward in one pass

// Shape of the one-pass backward: GW warps share a row, VPL accesses of N elements a lane,
// kGroups rows in a block at a time.
template <typename T, int N, int GW, int VPL>
struct BwdShape {
  static constexpr int kAccess = sizeof(T) * N;             // bytes of an access
  static constexpr bool kRing = kAccess >= 4;               // what an asynchronous copy can move
  static constexpr int kWarps = N == 1 && GW <= 8 ? 8 : GW % 3 == 0 ? 12 : 16;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kGroups = kWarps / GW;
  static constexpr int kColumns = 32 * GW * VPL * N;  // the widest row
  static constexpr int kPairs = N * VPL / 2;          // column pairs of a lane
  static constexpr int kBlocks = N == 1 ? (GW <= 8 ? 3 : 1) : kPairs <= 4 ? 2 : 1;  // on one SM
  static constexpr int kStages = N == 1 ? 4 : VPL == 1 ? 5 : VPL == 2 && N == 8 ? 3 : 2;  // rows in flight for each group
  static constexpr int kStageBytes = kThreads * VPL * 2 * kAccess;  // x and dy
  static constexpr int kRingBytes = kRing ? kStages * kStageBytes : 0;
  static constexpr int kStatsBytes = kStages * kWarps * 8;  // mean and rstd of the rows in flight, for each warp
  static constexpr int kWeightBytes = N == 1 ? 0 : 4 * kColumns;  // fp32, in the lanes' order
  static constexpr int kJoinBytes = kRing ? 8 * kColumns : kGroups > 1 ? 8 * kColumns : 0;
  static constexpr int kSmemBytes = std::max(kRingBytes + kStatsBytes + kWeightBytes, kJoinBytes);
};

// dx, and the rows' share of dweight and dbias, in one pass over x and dy.  A lane owns the
// same columns of every row, so the column sums are registers; the two sums over a row
// (u and u xhat) are shuffles and, with GW > 1, one exchange through shared memory.  Blocks
// stay for the whole grid's rows: each ends with one row of partial sums.
//   Rows stream through shared memory by asynchronous copies, kStages of them in flight; a
//   lane reads back only what it copied (a warp its row's mean and rstd), so no barrier
//   guards the ring.  Single bf16 elements (rows that no 16-byte access fits) are too small
//   to copy: there the next row waits in registers.
// Columns past h are zeros throughout.  Bound by its three streams: 131072 x 2048 bf16 in
// 244 us, 6.6 TB/s; its instructions, 58% of the issue slots, come next.  At 8192 x 2048 (24
// us, 4.2 TB/s) the start, the partial sums and the launch that adds them show.
template <typename T, int N, int GW, int VPL, bool PHASE>
__global__ void __launch_bounds__(BwdShape<T, N, GW, VPL>::kThreads, BwdShape<T, N, GW, VPL>::kBlocks)
    norm_bwd_rows_kernel(int n, int h, int64_t pitch, const T* __restrict__ dy, const T* __restrict__ x,
                         const void* __restrict__ weight, bool w_f32, const float* __restrict__ mean,
                         const float* __restrict__ rstd, T* __restrict__ dx, float* __restrict__ part) {
  using S = BwdShape<T, N, GW, VPL>;
  constexpr int kPairs = S::kPairs;
  static_assert(N > 1 || VPL % 2 == 0, "columns come in pairs");
  static_assert(N > 1 || !PHASE, "single elements have no phase");
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float2 red[2][S::kWarps];
  griddep_begin();
  const int group = static_cast<int>(threadIdx.x) / (32 * GW);
  const int lane = static_cast<int>(threadIdx.x) % (32 * GW);
  const int first = blockIdx.x + group * gridDim.x;
  const int step = gridDim.x * S::kGroups;  // (row + step fits 32 bits: see norm_backward)
  constexpr int kAcross = 32 * GW * N;  // columns one access of the group covers
  const int phase = PHASE ? row_phase(h, N) : 0;
  const auto column = [&](int k) { return k * kAcross + lane * N - phase; };

  const auto slot = [&](int stage, int k, int which) {  // this lane's x or dy of one access
    return ring + stage * S::kStageBytes + ((2 * k + which) * S::kThreads + threadIdx.x) * S::kAccess;
  };
  float2* const stats = reinterpret_cast<float2*>(ring + S::kRingBytes) + (threadIdx.x >> 5);  // + stage * kWarps
  Pack<T, N> px[VPL], pd[VPL];  // without a ring: the prefetched row
  const auto fetch = [&](int row, int stage) {
    if (row < n) {
      const T* xr = x + static_cast<int64_t>(row) * pitch + lane * N;
      const T* dr = dy + static_cast<int64_t>(row) * h + lane * N;
#pragma unroll
      for (int k = 0; k < VPL; ++k) {
        if (column(k) >= h) continue;
        if constexpr (PHASE) {
          cp_async_row<T, N>(slot(stage, k, 0), xr - lane * N, column(k), h);
          cp_async_row<T, N>(slot(stage, k, 1), dr - lane * N, column(k), h);
        } else if constexpr (S::kRing) {
          cp_async<S::kAccess>(slot(stage, k, 0), xr + k * kAcross);
          cp_async<S::kAccess>(slot(stage, k, 1), dr + k * kAcross);
        } else {
          px[k].v[0] = xr[k * kAcross];
          pd[k].v[0] = dr[k * kAcross];
        }
      }
    }
  };
  const auto fetch_stats = [&](int row, int stage) {
    if (row < n && (threadIdx.x & 31) == 0) {
      cp_async<4>(&stats[stage * S::kWarps].x, mean + row);
      cp_async<4>(&stats[stage * S::kWarps].y, rstd + row);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    if constexpr (S::kRing) {
      if (column(k) >= h)
        for (int s = 0; s < 2 * S::kStages; ++s)
          *reinterpret_cast<Pack<T, N>*>(slot(s >> 1, k, s & 1)) = Pack<T, N>{};
    } else {
      px[k].v[0] = pd[k].v[0] = from_f32<T>(0.f);
    }
  }
  // the rows start on their way before anything else is asked for
#pragma unroll
  for (int s = 0; s < S::kStages; ++s) {
    if (S::kRing || s == 0) fetch(first + s * step, s);
    fetch_stats(first + s * step, s);
  }

  // The weight: registers, or in fp32 behind the ring, where every group finds it in the
  // lanes' order (16 bytes a lane).
  float2 w[N == 1 ? kPairs : 1], aw[kPairs], ab[kPairs];
  float4* const ws = reinterpret_cast<float4*>(ring + S::kRingBytes + S::kStatsBytes);
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    float t[N] = {};
    if constexpr (PHASE) load_w_row<N>(weight, w_f32, column(k), h, t);
    else if (column(k) < h) load_w<N>(weight, w_f32, column(k), t);
    if constexpr (N == 1) {
      reinterpret_cast<float*>(w)[k] = t[0];
    } else if (group == 0) {
#pragma unroll
      for (int q = 0; q < N / 4; ++q)
        ws[(k * (N / 4) + q) * 32 * GW + lane] = make_float4(t[4 * q], t[4 * q + 1], t[4 * q + 2], t[4 * q + 3]);
    }
  }
  if constexpr (N > 1) __syncthreads();
#pragma unroll
  for (int i = 0; i < kPairs; ++i) aw[i] = ab[i] = make_float2(0.f, 0.f);

  const float inv_h = 1.f / h;
  int stage = 0, parity = 0;
  for (int row = first; row < n; row += step) {
    float2 xh[kPairs], u[kPairs];  // x then xhat; dy then u
    cp_async_wait<S::kStages - 1>();
    __syncwarp();
    const float2 stat = stats[stage * S::kWarps];
    const float mu = stat.x, rs = stat.y;
    if constexpr (S::kRing && N > 1) {
#pragma unroll
      for (int k = 0; k < VPL; ++k) {
        const auto vx = *reinterpret_cast<const Pack<T, N>*>(slot(stage, k, 0));
        const auto vd = *reinterpret_cast<const Pack<T, N>*>(slot(stage, k, 1));
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          xh[k * (N / 2) + e] = make_float2(element(vx, 2 * e), element(vx, 2 * e + 1));
          u[k * (N / 2) + e] = make_float2(element(vd, 2 * e), element(vd, 2 * e + 1));
        }
      }
      if (PHASE && lane == 0) {  // the row before
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (e < phase) reinterpret_cast<float*>(xh)[e] = reinterpret_cast<float*>(u)[e] = 0.f;
      }
    } else {
#pragma unroll
      for (int k = 0; k < VPL; k += 2) {
        if constexpr (S::kRing) {
          xh[k / 2] = make_float2(*reinterpret_cast<const float*>(slot(stage, k, 0)),
                                  *reinterpret_cast<const float*>(slot(stage, k + 1, 0)));
          u[k / 2] = make_float2(*reinterpret_cast<const float*>(slot(stage, k, 1)),
                                 *reinterpret_cast<const float*>(slot(stage, k + 1, 1)));
        } else {
          xh[k / 2] = make_float2(to_f32(px[k].v[0]), to_f32(px[k + 1].v[0]));
          u[k / 2] = make_float2(to_f32(pd[k].v[0]), to_f32(pd[k + 1].v[0]));
        }
      }
    }
    __syncwarp();  // the warp has read its mean and rstd
    // into the slots just read
    fetch(row + (S::kRing ? S::kStages : 1) * step, stage);
    fetch_stats(row + S::kStages * step, stage);
    if (++stage == S::kStages) stage = 0;
    float2 s1 = make_float2(0.f, 0.f), s2 = s1;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      xh[i] = mul2(add2(xh[i], both(-mu)), both(rs));
      aw[i] = fma2(u[i], xh[i], aw[i]);
      ab[i] = add2(ab[i], u[i]);
      if constexpr (N == 1) {
        u[i] = mul2(u[i], w[i]);
      } else {
        const float4 wq = ws[(i / 2) * 32 * GW + lane];
        u[i] = mul2(u[i], (i & 1) ? make_float2(wq.z, wq.w) : make_float2(wq.x, wq.y));
      }
      s1 = add2(s1, u[i]);
      s2 = fma2(u[i], xh[i], s2);
    }
    float2 sum = make_float2(s1.x + s1.y, s2.x + s2.y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      sum = add2(sum, make_float2(__shfl_xor_sync(0xffffffffu, sum.x, o), __shfl_xor_sync(0xffffffffu, sum.y, o)));
    if constexpr (GW > 1) {
      // the other half of red[] is rewritten only after the next row's barrier
      if ((threadIdx.x & 31) == 0) red[parity][threadIdx.x >> 5] = sum;
      if constexpr (S::kGroups == 1) __syncthreads();
      else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * GW) : "memory");
      sum = make_float2(0.f, 0.f);
      if constexpr (GW % 2 == 0) {
#pragma unroll
        for (int q = 0; q < GW; q += 2) {
          const float4 t = *reinterpret_cast<const float4*>(&red[parity][group * GW + q]);
          sum = add2(sum, add2(make_float2(t.x, t.y), make_float2(t.z, t.w)));
        }
      } else {
#pragma unroll
        for (int q = 0; q < GW; ++q) sum = add2(sum, red[parity][group * GW + q]);
      }
      parity ^= 1;
    }
    // dx = rstd (u - mean u - xhat mean(u xhat))
    const float2 c0 = both(-rs * (sum.x * inv_h)), c1 = both(-rs * (sum.y * inv_h));
    T* or_ = dx + static_cast<int64_t>(row) * h + lane * N;
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      if constexpr (N > 1) {
        float o[N];
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          const int i = k * (N / 2) + e;
          const float2 d = fma2(xh[i], c1, fma2(u[i], both(rs), c0));
          o[2 * e] = d.x;
          o[2 * e + 1] = d.y;
        }
        Pack<T, N> out;
        pack_f32(out, o);
        if constexpr (PHASE) {
          if (column(k) < h) store_row<T, N>(or_ - lane * N, column(k), h, out);
        } else {
          if (column(k) < h) *reinterpret_cast<Pack<T, N>*>(or_ + k * kAcross) = out;
        }
      } else if (k % 2 == 0) {
        const float2 d = fma2(xh[k / 2], c1, fma2(u[k / 2], both(rs), c0));
        if (column(k) < h) or_[k * kAcross] = from_f32<T>(d.x);
        if (column(k + 1) < h) or_[(k + 1) * kAcross] = from_f32<T>(d.y);
      }
    }
  }

  // one row of partial sums a block, in the lanes' order (value i of lane l at i * 32 GW + l),
  // or with a phase, which differs by block, in the columns'; its groups join in order
  constexpr int kHalf = S::kColumns;
  constexpr bool kJoin = PHASE || S::kGroups > 1;
  float* out = part + static_cast<int64_t>(blockIdx.x) * 2 * (PHASE ? h : kHalf);
  float* to = out;
  if constexpr (kJoin) {
    cp_async_wait<0>();
    to = reinterpret_cast<float*>(ring);
  }
#pragma unroll 1
  for (int g = 0; g < S::kGroups; ++g) {
    if constexpr (kJoin) __syncthreads();
    if (g != group) continue;
#pragma unroll
    for (int i = 0; i < VPL * N; ++i) {
      const int j = i * 32 * GW + lane;
      to[j] = (g ? to[j] : 0.f) + reinterpret_cast<const float*>(aw)[i];
      to[kHalf + j] = (g ? to[kHalf + j] : 0.f) + reinterpret_cast<const float*>(ab)[i];
    }
  }
  if constexpr (kJoin) {
    __syncthreads();
    if constexpr (PHASE) {
      for (int j = threadIdx.x; j < h; j += S::kThreads) {
        const int p = j + phase;
        const int at = (p / kAcross * N + p % N) * 32 * GW + p % kAcross / N;
        out[j] = to[at];
        out[h + j] = to[kHalf + at];
      }
    } else {
      for (int j = threadIdx.x; j < 2 * kHalf; j += S::kThreads) out[j] = to[j];
    }
  }
}

struct NormForwardArgs {
  NormParams q;
  const void *x, *weight, *bias;
  void* y;
  float *mean, *rstd;
  cudaStream_t stream;
};

template <typename T, int N, int WARPS, int VPL>
cudaError_t norm_forward_rows(const NormForwardArgs& a) {
  const int64_t rows = WARPS == 1 ? kFwdThreads<1, VPL> / 32 : 1;
  return launch_k(norm_fwd_rows_kernel<T, N, WARPS, VPL>, dim3(static_cast<unsigned>((a.q.n + rows - 1) / rows)),
                  dim3(kFwdThreads<WARPS, VPL>), 0, a.stream, a.q.n, a.q.h, a.q.x_pitch, a.q.eps, static_cast<const T*>(a.x),
                  a.weight, a.bias, a.q.w_f32, static_cast<T*>(a.y), a.mean, a.rstd);
}

// Accesses of a lane that a row of many is dealt in: 64 or 128 bytes, single elements 16.
template <typename T, int N>
constexpr int kFwdWant = sizeof(T) * N == 16 ? 8 : 16;

// The narrowest VPL whose WARPS warps hold a row of `accesses` accesses, of those that
// norm_forward_warps asks for (two warps or more hold over half of kFwdWant, or one).
template <typename T, int N, int WARPS>
cudaError_t norm_forward_vpl(const NormForwardArgs& a, int accesses) {
  const int per = (accesses + 32 * WARPS - 1) / (32 * WARPS);
  constexpr bool kAny = WARPS == 1 || WARPS == 16;
  constexpr int kWant = kFwdWant<T, N>;
  if (per <= 1) return norm_forward_rows<T, N, WARPS, 1>(a);
  if constexpr (kAny) {
    if (per <= 2) return norm_forward_rows<T, N, WARPS, 2>(a);
    if (per <= 4) return norm_forward_rows<T, N, WARPS, 4>(a);
  }
  if constexpr (kAny || kWant == 8) {
    if (per <= 6) return norm_forward_rows<T, N, WARPS, 6>(a);
    if (per <= 8) return norm_forward_rows<T, N, WARPS, 8>(a);
  }
  if constexpr (WARPS == 16 || kWant == 16) {
    if (per <= 12) return norm_forward_rows<T, N, WARPS, 12>(a);
    return norm_forward_rows<T, N, WARPS, 16>(a);
  }
  return cudaErrorInvalidValue;
}

template <typename T, int N>
cudaError_t norm_forward_warps(const NormForwardArgs& a) {
  const int accesses = (a.q.h + N - 1) / N;
  // Warps on a row.  Many rows: the fewest that leave a lane 8 accesses of 16 bytes (bf16,
  // GB/s with 1 / 2 / 4 / 8 warps: h 2048 6554 / 6317 / 5527 / 3702, h 4096 5757 / 6853 / 6512 /
  // 5341, h 8192 5793 / 5709 / 6836 / 5781), or 16 of a single element (fp32, h 1031, 4 warps
  // 4870, 8 warps 3731).  Few rows leave SMs idle, and a row is done sooner by more warps (4 x
  // 4096 as timed with its launch, 1 / 4 / 16 warps: 21 / 10 / 7 us).
  const int want = a.q.n < 1024 ? 1 : kFwdWant<T, N>;
  if (accesses <= 32 * want) return norm_forward_vpl<T, N, 1>(a, accesses);
  if (accesses <= 64 * want) return norm_forward_vpl<T, N, 2>(a, accesses);
  if (accesses <= 128 * want) return norm_forward_vpl<T, N, 4>(a, accesses);
  if (accesses <= 256 * want) return norm_forward_vpl<T, N, 8>(a, accesses);
  return norm_forward_vpl<T, N, 16>(a, accesses);
}

template <typename T, int N, int GW, int VPL>
cudaError_t norm_forward_phase(const NormForwardArgs& a) {
  using S = FwdPhaseShape<T, N, GW, VPL>;
  auto* kernel = norm_fwd_phase_kernel<T, N, GW, VPL>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = S::kSmemBytes > 40 * 1024 ? allow_smem(kernel, S::kSmemBytes, done) : cudaSuccess;
  if (e != cudaSuccess) return e;
  const int blocks = phase_blocks((a.q.n + S::kGroups - 1) / S::kGroups, S::kBlocks * kNormSms);
  return launch_k(kernel, dim3(blocks), dim3(S::kThreads), S::kSmemBytes, a.stream, static_cast<int>(a.q.n), a.q.h,
                  a.q.x_pitch, a.q.eps, static_cast<const T*>(a.x), a.weight, a.bias, a.q.w_f32,
                  static_cast<T*>(a.y), a.mean, a.rstd);
}

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool at16(const void* p) { return aligned(p, 16); }

// Rows of x and of the contiguous tensors start at the same phase of a 16-byte access.
template <int N>
bool same_phase(const NormParams& q) {
  return (q.x_pitch - q.h) % N == 0;
}

template <typename T>
cudaError_t norm_forward(const NormForwardArgs& a) {
  constexpr int kVec = 16 / sizeof(T);
  constexpr int kMost = 32 * 16 * 16;  // accesses of the widest row held in registers
  const auto fits = [&](int n) {       // rows, weight and bias in accesses of n elements
    const int size = n * static_cast<int>(sizeof(T)), w_size = a.q.w_f32 ? 16 : 2 * n;
    return a.q.h % n == 0 && a.q.x_pitch % n == 0 && aligned(a.x, size) && aligned(a.y, size) &&
           aligned(a.weight, w_size) && aligned(a.bias, w_size) && a.q.n <= 0x7fffffff && a.q.h <= kMost * n;
  };
  // bf16 rows with fp32 weights go by 4 elements: a warp's weights are then 512 consecutive
  // bytes, where 8 would be every other 16 of 1024, and the first-level cache's rate bounds
  // (65536 x 768 38 us, by 8 41; 65536 x 5120 228 and 234).
  if constexpr (kVec == 8)
    if ((a.q.w_f32 || !fits(8)) && fits(4)) return norm_forward_warps<T, 4>(a);
  if (fits(kVec)) return norm_forward_warps<T, kVec>(a);
  if (at16(a.x) && at16(a.y)) {
    // Accesses at a phase against single elements (us): bf16 65536 x 2049 126 and 246, 65536 x
    // 999 49 and 74, 131072 x 250 43 and 66, but 131072 x 100 35 and 31, where a row is less than
    // a warp's worth; fp32 65536 x 1031 92 and 111, 32768 x 2050 90 and 130, but 65536 x 501 48
    // and 41, where single elements need no barrier.  Laying out the weight takes 2 us, which
    // smaller calls do not earn back (bf16 2048 x 1001 4.8 and 4.0, 2048 x 1501 5.7 and 6.1).
    const bool earns = a.q.n * a.q.h >= (3 << 20) && a.q.h > (sizeof(T) == 2 ? 128 : 1024);
    if (same_phase<kVec>(a.q) && a.q.n <= (1 << 30) && (earns || a.q.h > kMost)) {
      const int accesses = (a.q.h + 2 * kVec - 2) / kVec;
      if constexpr (kVec == 8) {  // (fp32 rows are wider)
        if (accesses <= 32) return norm_forward_phase<T, kVec, 1, 1>(a);
        if (accesses <= 64) return norm_forward_phase<T, kVec, 1, 2>(a);
        if (accesses <= 96) return norm_forward_phase<T, kVec, 1, 3>(a);
        if (accesses <= 128) return norm_forward_phase<T, kVec, 1, 4>(a);
        if (accesses <= 192) return norm_forward_phase<T, kVec, 2, 3>(a);
        if (accesses <= 256) return norm_forward_phase<T, kVec, 2, 4>(a);
      }
      if (accesses <= 384) return norm_forward_phase<T, kVec, 4, 3>(a);
      if (accesses <= 512) return norm_forward_phase<T, kVec, 4, 4>(a);
      if (accesses <= 768) return norm_forward_phase<T, kVec, 8, 3>(a);
      if (accesses <= 1024) return norm_forward_phase<T, kVec, 8, 4>(a);
      if (accesses <= 1536) return norm_forward_phase<T, kVec, 16, 3>(a);
      if (accesses <= 2048) return norm_forward_phase<T, kVec, 16, 4>(a);
    }
  }
  if (a.q.n <= 0x7fffffff && a.q.h <= kMost) return norm_forward_warps<T, 1>(a);
  const int grid = static_cast<int>(std::min<int64_t>(a.q.n, 1 << 20));
  return launch_k(norm_fwd_kernel<T>, dim3(grid), dim3(kNormThreads), 0, a.stream, a.q.n, a.q.h, a.q.x_pitch, a.q.eps,
                  static_cast<const T*>(a.x), a.weight, a.bias, a.q.w_f32, static_cast<T*>(a.y), a.mean, a.rstd);
}

struct NormBackwardArgs {
  NormParams q;
  const void *dy, *x, *weight;
  const float *mean, *rstd;
  void* dx;
  float* part;
  cudaStream_t stream;
};

// The partial sums that a backward pass leaves (see norm_dw_final_kernel).
struct PartialLayout {
  int slices, half;
  int lanes, n;
};

template <typename T, int N, int GW, int VPL, bool PHASE>
cudaError_t norm_backward_rows(const NormBackwardArgs& a, PartialLayout* left) {
  using S = BwdShape<T, N, GW, VPL>;
  static_assert(S::kSmemBytes <= 227 * 1024 / S::kBlocks - 1536, "shared memory budget");
  auto* kernel = norm_bwd_rows_kernel<T, N, GW, VPL, PHASE>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = S::kSmemBytes > 40 * 1024 ? allow_smem(kernel, S::kSmemBytes, done) : cudaSuccess;
  if (e != cudaSuccess) return e;
  const int64_t blocks = (a.q.n + S::kGroups - 1) / S::kGroups;
  if (PHASE) *left = PartialLayout{phase_blocks(blocks, S::kBlocks * kNormSms), a.q.h, 1, 1};
  else *left = PartialLayout{static_cast<int>(std::min<int64_t>(blocks, S::kBlocks * kNormSms)), S::kColumns, 32 * GW, N};
  return launch_k(kernel, dim3(left->slices), dim3(S::kThreads), S::kSmemBytes, a.stream, static_cast<int>(a.q.n),
                  a.q.h, a.q.x_pitch, static_cast<const T*>(a.dy), static_cast<const T*>(a.x), a.weight, a.q.w_f32,
                  a.mean, a.rstd, static_cast<T*>(a.dx), a.part);
}

// Two passes for rows past every one-pass shape (16384 columns in bf16, 8192 in fp32, 4096 of
// single elements): dx row by row, then the column sums over slices of rows.  x and dy are read
// three times by single elements, whose issue bounds it: 8192 x 20000 bf16 852 us, 1.15 TB/s
// of the three streams a single pass would move, 8192 x 12000 fp32 557 us, 2.1 TB/s.
template <typename T>
cudaError_t norm_backward_wide(const NormBackwardArgs& a, PartialLayout* left) {
  const int grid = static_cast<int>(std::min<int64_t>(a.q.n, 1 << 20));
  cudaError_t e = launch_k(norm_dx_kernel<T>, dim3(grid), dim3(kNormThreads), 0, a.stream, a.q.n, a.q.h, a.q.x_pitch,
                           static_cast<const T*>(a.dy), static_cast<const T*>(a.x), a.weight, a.q.w_f32, a.mean,
                           a.rstd, static_cast<T*>(a.dx));
  if (e != cudaSuccess) return e;
  const int slices = static_cast<int>(std::min<int64_t>(a.q.n, 128));
  *left = PartialLayout{slices, a.q.h, 1, 1};
  const int64_t rows = (a.q.n + slices - 1) / slices;
  const int cols = (a.q.h + kNormThreads - 1) / kNormThreads;
  return launch_k(norm_dw_partial_kernel<T>, dim3(cols, slices), dim3(kNormThreads), 0, a.stream, a.q.n, a.q.h,
                  a.q.x_pitch, rows, static_cast<const T*>(a.dy), static_cast<const T*>(a.x), a.mean, a.rstd, a.part);
}

// The narrowest shape that holds `accesses` accesses of 16 bytes (2048 at most).
template <typename T, bool PHASE>
cudaError_t norm_backward_vec(const NormBackwardArgs& a, PartialLayout* left, int accesses) {
  constexpr int kVec = 16 / sizeof(T);
  if (accesses <= 32) return norm_backward_rows<T, kVec, 1, 1, PHASE>(a, left);
  if (accesses <= 64) return norm_backward_rows<T, kVec, 2, 1, PHASE>(a, left);
  if (accesses <= 96) return norm_backward_rows<T, kVec, 3, 1, PHASE>(a, left);
  if (accesses <= 128) return norm_backward_rows<T, kVec, 4, 1, PHASE>(a, left);
  if (accesses <= 192) return norm_backward_rows<T, kVec, 6, 1, PHASE>(a, left);
  if (accesses <= 256) return norm_backward_rows<T, kVec, 8, 1, PHASE>(a, left);
  if (accesses <= 384) return norm_backward_rows<T, kVec, 12, 1, PHASE>(a, left);
  if (accesses <= 512) return norm_backward_rows<T, kVec, 16, 1, PHASE>(a, left);
  if (accesses <= 768) return norm_backward_rows<T, kVec, 12, 2, PHASE>(a, left);
  if (accesses <= 1024) return norm_backward_rows<T, kVec, 16, 2, PHASE>(a, left);
  return norm_backward_rows<T, kVec, 16, 4, PHASE>(a, left);
}

template <typename T>
cudaError_t norm_backward(const NormBackwardArgs& a, PartialLayout* left) {
  constexpr int kVec = 16 / sizeof(T);
  const int h = a.q.h;
  if (a.q.n > (1 << 30)) return norm_backward_wide<T>(a, left);  // 32-bit row numbers in one pass
  const int most = 2048 * kVec;  // columns of the widest vector shape
  if (at16(a.x) && at16(a.dy) && at16(a.dx)) {
    if (h % kVec == 0 && a.q.x_pitch % kVec == 0 && at16(a.weight) && h <= most)
      return norm_backward_vec<T, false>(a, left, h / kVec);
    // Accesses at a phase against single elements (us): bf16 65536 x 2049 206 and 350, 32768 x
    // 8001 256 and 1289, 131072 x 250 72 and 123, but 131072 x 100 46 and 33; fp32 65536 x 501 69
    // and 104.  The weight's and the partial sums' own order take 1 to 2 us more (bf16 2048 x
    // 1501 12.8 and 11.0, 8192 x 1501 23.1 and 22.4; fp32 8192 x 1001 23.9 and 30.5), so only for
    // many rows, or rows for which single elements are slow (bf16 2048 x 2049 15.1 and 16.6).
    const bool earns = h > 4096 || (h > 2048 && a.q.n >= 1024) || (h > 16 * kVec && a.q.n >= 8192);
    if (same_phase<kVec>(a.q) && h + kVec - 1 <= most && earns)
      return norm_backward_vec<T, true>(a, left, (h + 2 * kVec - 2) / kVec);
  }
  if (h <= 128) return norm_backward_rows<T, 1, 1, 4, false>(a, left);
  if (h <= 512) return norm_backward_rows<T, 1, 4, 4, false>(a, left);
  if (h <= 1024) return norm_backward_rows<T, 1, 8, 4, false>(a, left);
  if (h <= 1536) return norm_backward_rows<T, 1, 8, 6, false>(a, left);
  if (h <= 2048) return norm_backward_rows<T, 1, 8, 8, false>(a, left);
  if (h <= 4096) return norm_backward_rows<T, 1, 16, 8, false>(a, left);
  return norm_backward_wide<T>(a, left);
}

}  // namespace

// Every shape: at most 512 or twice h columns, and blocks for three on an SM only for single
// elements of narrow rows.
size_t norm_partial_floats(int64_t n, int64_t h) {
  const int64_t slices = phase_blocks(std::max<int64_t>(n, 1), (h <= 2048 ? 3 : 2) * kNormSms);
  return static_cast<size_t>(slices) * 2 * static_cast<size_t>(std::max<int64_t>(512, 2 * h));
}

cudaError_t launch_norm_forward(const NormParams& q, const void* x, const void* weight, const void* bias, void* y,
                                float* mean, float* rstd, cudaStream_t stream) {
  const NormForwardArgs a{q, x, weight, bias, y, mean, rstd, stream};
  return q.x_f32 ? norm_forward<float>(a) : norm_forward<__nv_bfloat16>(a);
}

cudaError_t launch_norm_backward(const NormParams& q, const void* dy, const void* x, const void* weight,
                                 const float* mean, const float* rstd, void* dx, void* dweight, void* dbias,
                                 float* part, cudaStream_t stream) {
  const NormBackwardArgs a{q, dy, x, weight, mean, rstd, dx, part, stream};
  PartialLayout left{};
  cudaError_t e = q.x_f32 ? norm_backward<float>(a, &left) : norm_backward<__nv_bfloat16>(a, &left);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((2 * static_cast<int64_t>(left.half) + 31) / 32));
  if (q.w_f32)
    return launch_k(norm_dw_final_kernel<float>, grid, dim3(32 * kFinalWarps), 0, stream, q.h, left.slices, left.half,
                    left.lanes, left.n, part, static_cast<float*>(dweight), static_cast<float*>(dbias));
  return launch_k(norm_dw_final_kernel<__nv_bfloat16>, grid, dim3(32 * kFinalWarps), 0, stream, q.h, left.slices,
                  left.half, left.lanes, left.n, part, static_cast<__nv_bfloat16*>(dweight),
                  static_cast<__nv_bfloat16*>(dbias));
}

}  // namespace flce
