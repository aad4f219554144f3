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

// One block per row; the row is read three times (mean, squares about it, y).
template <typename T, typename W>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(int64_t n, int h, int64_t pitch, float eps,
                                                                const T* __restrict__ x, const W* __restrict__ weight,
                                                                const W* __restrict__ bias, T* __restrict__ y,
                                                                float* __restrict__ mean, float* __restrict__ rstd) {
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
      const float v = (to_f32(xr[j]) - mu) * rs * to_f32(weight[j]);
      yr[j] = from_f32<T>(bias ? v + to_f32(bias[j]) : v);
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

template <typename T, typename W>
cudaError_t norm_forward(const NormParams& q, const void* x, const void* weight, const void* bias, void* y, float* mean,
                         float* rstd, cudaStream_t stream) {
  const int grid = static_cast<int>(std::min<int64_t>(q.n, 1 << 20));
  return launch_k(norm_fwd_kernel<T, W>, dim3(grid), dim3(kNormThreads), 0, stream, q.n, q.h, q.x_pitch, q.eps,
                  static_cast<const T*>(x), static_cast<const W*>(weight), static_cast<const W*>(bias),
                  static_cast<T*>(y), mean, rstd);
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
  if (q.x_f32)
    return q.w_f32 ? norm_forward<float, float>(q, x, weight, bias, y, mean, rstd, stream)
                   : norm_forward<float, __nv_bfloat16>(q, x, weight, bias, y, mean, rstd, stream);
  return q.w_f32 ? norm_forward<__nv_bfloat16, float>(q, x, weight, bias, y, mean, rstd, stream)
                 : norm_forward<__nv_bfloat16, __nv_bfloat16>(q, x, weight, bias, y, mean, rstd, stream);
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
