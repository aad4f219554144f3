// Layer norm: forward, and backward with the reduction of the weight's and
// bias's gradients over the rows.
#include <algorithm>

#include "flce_device.cuh"
#include "flce_internal.h"
#include "flce_launch.cuh"

namespace flce {

namespace {

constexpr int kNormThreads = 256;

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
// 4096 bf16 in 313 us, 6.85 TB/s.  WARPS warps share a row, VPL accesses of N elements a
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
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < VPL; ++k)
    if ((lane + k * kLanes) * N < h) {
#pragma unroll
      for (int e = 0; e < N; ++e) s += element(v[k], e);
    }
#pragma unroll
  for (int k = 0; k < VPL; ++k) keep_packed(v[k]);
  const float mu = row_sum<WARPS>(s, red[0]) / h;
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < VPL; ++k)
    if ((lane + k * kLanes) * N < h) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float d = element(v[k], e) - mu;
        q = fmaf(d, d, q);
      }
    }
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
    if (bias) load_w<N>(bias, w_f32, j, b);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float o = (element(v[k], e) - mu) * rs;
      w[e] = bias ? fmaf(o, w[e], b[e]) : o * w[e];
    }
    pack_f32(v[k], w);
    *reinterpret_cast<Pack<T, N>*>(yr + j) = v[k];
  }
  if (lane == 0) {
    mean[row] = mu;
    rstd[row] = rs;
  }
}

// Rows too wide for registers: one block per row, the row read three times (the second
// and third time from L2).
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

template <typename T, typename W>
__global__ void __launch_bounds__(kNormThreads) norm_dx_kernel(int64_t n, int h, int64_t pitch,
                                                               const T* __restrict__ dy, const T* __restrict__ x,
                                                               const W* __restrict__ weight,
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
      const float u = to_f32(dr[j]) * to_f32(weight[j]);
      s.x += u;
      s.y += u * ((to_f32(xr[j]) - mu) * rs);
    }
    s = block_sum(s, red);
    const float a = s.x / h, b = s.y / h;
    for (int j = threadIdx.x; j < h; j += kNormThreads) {
      const float u = to_f32(dr[j]) * to_f32(weight[j]);
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

template <typename W>
__global__ void __launch_bounds__(kNormThreads) norm_dw_final_kernel(int h, int slices, const float* __restrict__ part,
                                                                     W* __restrict__ dweight, W* __restrict__ dbias) {
  griddep_begin();
  const int j = blockIdx.x * kNormThreads + threadIdx.x;
  if (j >= h) return;
  float a = 0.f, b = 0.f;
  for (int s = 0; s < slices; ++s) {
    const float* p = part + static_cast<int64_t>(s) * 2 * h;
    a += p[j];
    b += p[h + j];
  }
  dweight[j] = from_f32<W>(a);
  if (dbias) dbias[j] = from_f32<W>(b);
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

// The narrowest VPL whose WARPS warps hold a row of `accesses` accesses.
template <typename T, int N, int WARPS>
cudaError_t norm_forward_vpl(const NormForwardArgs& a, int accesses) {
  const int per = (accesses + 32 * WARPS - 1) / (32 * WARPS);
  if (per <= 1) return norm_forward_rows<T, N, WARPS, 1>(a);
  if (per <= 2) return norm_forward_rows<T, N, WARPS, 2>(a);
  if (per <= 4) return norm_forward_rows<T, N, WARPS, 4>(a);
  if (per <= 8) return norm_forward_rows<T, N, WARPS, 8>(a);
  return norm_forward_rows<T, N, WARPS, 16>(a);
}

template <typename T, int N>
cudaError_t norm_forward_warps(const NormForwardArgs& a) {
  const int accesses = (a.q.h + N - 1) / N;
  // Warps on a row.  Many rows: the fewest that leave a lane 8 accesses of 16 bytes (bf16,
  // GB/s with 1 / 2 / 4 / 8 warps: h 2048 6554 / 6317 / 5527 / 3702, h 4096 5757 / 6853 / 6512 /
  // 5341, h 8192 5793 / 5709 / 6836 / 5781), or 16 of a single element (fp32, h 1031, 4 warps
  // 4870, 8 warps 3731).  Few rows leave SMs idle, and a row is done sooner by more warps (4 x
  // 4096 as timed with its launch, 1 / 4 / 16 warps: 21 / 10 / 7 us).
  const int want = a.q.n < 1024 ? 1 : N == 1 ? 16 : 8;
  if (accesses <= 32 * want) return norm_forward_vpl<T, N, 1>(a, accesses);
  if (accesses <= 64 * want) return norm_forward_vpl<T, N, 2>(a, accesses);
  if (accesses <= 128 * want) return norm_forward_vpl<T, N, 4>(a, accesses);
  if (accesses <= 256 * want) return norm_forward_vpl<T, N, 8>(a, accesses);
  return norm_forward_vpl<T, N, 16>(a, accesses);
}

template <typename T>
cudaError_t norm_forward(const NormForwardArgs& a) {
  constexpr int kVec = 16 / sizeof(T);
  const size_t row = sizeof(T) * static_cast<size_t>(a.q.x_pitch);
  const auto at16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool vec = a.q.h % kVec == 0 && row % 16 == 0 && at16(a.x) && at16(a.y) && at16(a.weight) && at16(a.bias);
  constexpr int kMost = 32 * 16 * 16;  // accesses of the widest row held in registers
  if (a.q.n <= 0x7fffffff) {
    if (vec && a.q.h <= kMost * kVec) return norm_forward_warps<T, kVec>(a);
    if (!vec && a.q.h <= kMost) return norm_forward_warps<T, 1>(a);
  }
  const int grid = static_cast<int>(std::min<int64_t>(a.q.n, 1 << 20));
  return launch_k(norm_fwd_kernel<T>, dim3(grid), dim3(kNormThreads), 0, a.stream, a.q.n, a.q.h, a.q.x_pitch, a.q.eps,
                  static_cast<const T*>(a.x), a.weight, a.bias, a.q.w_f32, static_cast<T*>(a.y), a.mean, a.rstd);
}

template <typename T, typename W>
cudaError_t norm_backward(const NormParams& q, const void* dy, const void* x, const void* weight, const float* mean,
                          const float* rstd, void* dx, void* dweight, void* dbias, float* part, cudaStream_t stream) {
  const int grid = static_cast<int>(std::min<int64_t>(q.n, 1 << 20));
  cudaError_t e = launch_k(norm_dx_kernel<T, W>, dim3(grid), dim3(kNormThreads), 0, stream, q.n, q.h, q.x_pitch,
                           static_cast<const T*>(dy), static_cast<const T*>(x), static_cast<const W*>(weight), mean,
                           rstd, static_cast<T*>(dx));
  if (e != cudaSuccess) return e;
  const int slices = norm_slices(q.n);
  const int64_t rows = (q.n + slices - 1) / slices;
  const int cols = (q.h + kNormThreads - 1) / kNormThreads;
  e = launch_k(norm_dw_partial_kernel<T>, dim3(cols, slices), dim3(kNormThreads), 0, stream, q.n, q.h, q.x_pitch, rows,
               static_cast<const T*>(dy), static_cast<const T*>(x), mean, rstd, part);
  if (e != cudaSuccess) return e;
  return launch_k(norm_dw_final_kernel<W>, dim3(cols), dim3(kNormThreads), 0, stream, q.h, slices, part,
                  static_cast<W*>(dweight), static_cast<W*>(dbias));
}

}  // namespace

int norm_slices(int64_t n) { return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(128, n / 32))); }

cudaError_t launch_norm_forward(const NormParams& q, const void* x, const void* weight, const void* bias, void* y,
                                float* mean, float* rstd, cudaStream_t stream) {
  const NormForwardArgs a{q, x, weight, bias, y, mean, rstd, stream};
  return q.x_f32 ? norm_forward<float>(a) : norm_forward<__nv_bfloat16>(a);
}

cudaError_t launch_norm_backward(const NormParams& q, const void* dy, const void* x, const void* weight,
                                 const float* mean, const float* rstd, void* dx, void* dweight, void* dbias,
                                 float* part, cudaStream_t stream) {
  if (q.x_f32)
    return q.w_f32
               ? norm_backward<float, float>(q, dy, x, weight, mean, rstd, dx, dweight, dbias, part, stream)
               : norm_backward<float, __nv_bfloat16>(q, dy, x, weight, mean, rstd, dx, dweight, dbias, part, stream);
  return q.w_f32 ? norm_backward<__nv_bfloat16, float>(q, dy, x, weight, mean, rstd, dx, dweight, dbias, part, stream)
                 : norm_backward<__nv_bfloat16, __nv_bfloat16>(q, dy, x, weight, mean, rstd, dx, dweight, dbias, part,
                                                               stream);
}

}  // namespace flce
