// AdamW over many tensors, moments in 32 or in 8 bits.
#include <cuda_fp8.h>

#include "flce_device.cuh"
#include "flce_internal.h"
#include "flce_launch.cuh"

namespace flce {

namespace {

// What the 8-bit codes depend on (m, v, r, the scales and the scaled values) is computed
// in separately rounded IEEE operations, so that a code never depends on how a compiler
// contracts or approximates: a moment next to a rounding threshold would otherwise come
// out a whole 8-bit step apart.  The parameter's update, which nothing rounds to 8 bits,
// is free of that.

constexpr int kAdamwThreads = 256;
constexpr float kFp8Max = 448.f;  // largest e4m3 value
// A block whose largest magnitude is below this is stored as zeros: 448 over it would
// pass fp32's range (a root of a non-zero fp32 v is above 3e-23).
constexpr float kTiny = 1e-35f;

// The tensor that holds chunk c: the last one whose first chunk is not past it.
template <int N>
__device__ __forceinline__ int find_tensor(const AdamwArgs<N>& a, uint32_t c) {
  int lo = 0, hi = a.tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.t[mid].chunk0 <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// 32 bits for elements 4q .. 4q + 3 (one byte each) of this step: two rounds of
// multiply and xor-shift over a Weyl sequence.
__device__ __forceinline__ uint32_t rounding_bits(uint32_t q, uint32_t step_key) {
  constexpr uint32_t k = 0x9E3779B1u;
  uint32_t h = q * k + step_key;
  h = (h ^ (h >> 16)) * k;
  h = (h ^ (h >> 13)) * k;
  return h ^ (h >> 16);
}

// e4m3 byte of q in [0, 448], rounded up where the fraction of the step passed plus
// rnd / 256 reaches 1.  Below 2^-6 the grid's steps are equal, as they are in [2^-6, 2^-5).
__device__ __forceinline__ uint32_t e4m3_dithered(float q, uint32_t rnd) {
  const bool low = q < 0.015625f;
  const uint32_t bits = __float_as_uint(low ? q + 0.015625f : q);
  const uint32_t code = ((bits + (rnd << 12)) >> 20) - (120u << 3) - (low ? 8u : 0u);
  return q > 0.f ? max(code, 1u) : 0u;
}

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  __nv_fp8_e4m3 v;
  v.__x = c;
  return static_cast<float>(v);
}

// One block per chunk, one element per thread and round (256 elements: one 8-bit block).
template <int N, int BITS>
__global__ void __launch_bounds__(kAdamwThreads) adamw_kernel(const __grid_constant__ AdamwArgs<N> a) {
  griddep_begin();
  __shared__ float red[2][kAdamwThreads / 32];
  const int ti = find_tensor(a, blockIdx.x);
  const AdamwTensor& t = a.t[ti];
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const int64_t base = static_cast<int64_t>(blockIdx.x - t.chunk0) * kAdamwChunk;
  for (int64_t b = base; b < base + kAdamwChunk && b < t.count; b += kAdamwThreads) {
    const int64_t i = b + threadIdx.x;
    const bool live = i < t.count;
    float g = 0.f, p = 0.f, m = 0.f, v = 0.f;
    if (live) {
      g = gs * ((t.flags & kAdamwGradF32) ? static_cast<const float*>(t.grad)[i]
                                          : __bfloat162float(static_cast<const __nv_bfloat16*>(t.grad)[i]));
      p = t.master ? t.master[i]
                   : ((t.flags & kAdamwParamF32) ? static_cast<const float*>(t.param)[i]
                                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(t.param)[i]));
      if (BITS == 32) {
        m = static_cast<const float*>(t.m)[i];
        v = static_cast<const float*>(t.v)[i];
      } else {
        m = e4m3_value(static_cast<const uint8_t*>(t.m)[i]) * t.m_scale[b / kAdamwBlock];
        const float r = e4m3_value(static_cast<const uint8_t*>(t.v)[i]) * t.v_scale[b / kAdamwBlock];
        v = r * r;
      }
    }
    m = __fadd_rn(__fmul_rn(m, a.beta1), __fmul_rn(g, a.omb1));
    v = __fadd_rn(__fmul_rn(v, a.beta2), __fmul_rn(__fmul_rn(g, g), a.omb2));
    const float r = __fsqrt_rn(v);
    p = p * t.decay - t.rate * m / (r * a.inv_root_bc2 + a.eps);
    if (live) {
      if (t.master) t.master[i] = p;
      if (t.flags & kAdamwParamF32) static_cast<float*>(t.param)[i] = p;
      else static_cast<__nv_bfloat16*>(t.param)[i] = __float2bfloat16_rn(p);
    }
    if (BITS == 32) {
      if (live) {
        static_cast<float*>(t.m)[i] = m;
        static_cast<float*>(t.v)[i] = v;
      }
      continue;
    }
    // largest magnitudes of the block; a NaN must not vanish in fmaxf, so it is carried as infinity
    float mm = live ? (fabsf(m) <= 3.402823466e38f ? fabsf(m) : INFINITY) : 0.f;
    float mr = live ? (r <= 3.402823466e38f ? r : INFINITY) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
      mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, o));
    }
    __syncthreads();  // the last round's maxima and scales have been read
    if ((threadIdx.x & 31) == 0) {
      red[0][threadIdx.x >> 5] = mm;
      red[1][threadIdx.x >> 5] = mr;
    }
    __syncthreads();
    for (int w = 0; w < kAdamwThreads / 32; ++w) {
      mm = fmaxf(mm, red[0][w]);
      mr = fmaxf(mr, red[1][w]);
    }
    if (threadIdx.x == 0) {
      t.m_scale[b / kAdamwBlock] = mm < kTiny ? 0.f : mm < INFINITY ? mm * (1.f / kFp8Max) : NAN;
      t.v_scale[b / kAdamwBlock] = mr < kTiny ? 0.f : mr < INFINITY ? mr * (1.f / kFp8Max) : NAN;
    }
    if (live) {
      const float im = mm >= kTiny && mm < INFINITY ? __fmul_rn(__frcp_rn(mm), kFp8Max) : 0.f;
      const float ir = mr >= kTiny && mr < INFINITY ? __fmul_rn(__frcp_rn(mr), kFp8Max) : 0.f;
      const uint32_t h = rounding_bits(static_cast<uint32_t>(i >> 2), a.step_key);
      const float qr = fminf(r * ir, kFp8Max);
      static_cast<uint8_t*>(t.m)[i] = __nv_cvt_float_to_fp8(im > 0.f ? m * im : 0.f, __NV_SATFINITE, __NV_E4M3);
      static_cast<uint8_t*>(t.v)[i] =
          static_cast<uint8_t>(e4m3_dithered(ir > 0.f ? qr : 0.f, (h >> (8 * (static_cast<uint32_t>(i) & 3))) & 0xffu));
    }
  }
}

}  // namespace

template <int N>
cudaError_t launch_adamw(const AdamwArgs<N>& a, int state_bits, cudaStream_t stream) {
  return state_bits == 8 ? launch_k(adamw_kernel<N, 8>, dim3(a.chunks), dim3(kAdamwThreads), 0, stream, a)
                         : launch_k(adamw_kernel<N, 32>, dim3(a.chunks), dim3(kAdamwThreads), 0, stream, a);
}

template cudaError_t launch_adamw<kAdamwFewTensors>(const AdamwArgs<kAdamwFewTensors>&, int, cudaStream_t);
template cudaError_t launch_adamw<kAdamwManyTensors>(const AdamwArgs<kAdamwManyTensors>&, int, cudaStream_t);

}  // namespace flce
