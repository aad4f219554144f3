// AdamW over many tensors, moments in 32 or in 8 bits.
#include <cuda_fp16.h>
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

__device__ __forceinline__ float2 e4m3x2_values(uint32_t pair) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair & 0xffffu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// What one step needs besides the elements.
struct StepScalars {
  float beta1, omb1, beta2, omb2, inv_root_bc2, eps, decay, rate;
};

// One element: m, v and the parameter (or its master) move; r = sqrt(v).
__device__ __forceinline__ void adamw_element(const StepScalars& s, float g, float& p, float& m, float& v, float& r) {
  m = __fadd_rn(__fmul_rn(m, s.beta1), __fmul_rn(g, s.omb1));
  v = __fadd_rn(__fmul_rn(v, s.beta2), __fmul_rn(__fmul_rn(g, g), s.omb2));
  r = __fsqrt_rn(v);
  p = fmaf(p, s.decay, -__fdividef(s.rate * m, fmaf(r, s.inv_root_bc2, s.eps)));
}

// Scale and 1 / scale of a block whose largest magnitude has these bits.  Non-negative
// floats order like their bits, with infinity and NaN on top.
__device__ __forceinline__ void block_scale(uint32_t top_bits, float* scale, float* inv) {
  const float top = __uint_as_float(top_bits);
  const bool finite = top_bits < 0x7f800000u, zero = top < kTiny;
  *scale = !finite ? NAN : zero ? 0.f : top * (1.f / kFp8Max);
  *inv = !finite || zero ? 0.f : __fmul_rn(__frcp_rn(top), kFp8Max);
}

__device__ __forceinline__ void unpack8(const uint4& a, const uint4& b, bool f32, float (&x)[8]) {
  const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (f32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(u[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(u[e] << 16);
      x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ void store8(void* base, int64_t i, bool f32, const float (&x)[8]) {
  if (f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    __stcs(o, make_float4(x[0], x[1], x[2], x[3]));
    __stcs(o + 1, make_float4(x[4], x[5], x[6], x[7]));
  } else {
    __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i),
           make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7])));
  }
}

__device__ __forceinline__ void load8(const void* base, int64_t i, bool f32, uint4& a, uint4& b) {
  const uint4* o = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + i * (f32 ? 4 : 2));
  a = __ldcs(o);
  if (f32) b = __ldcs(o + 1);
}

// The raw words of one unit (256 elements, 8 consecutive ones a lane).
struct UnitWords {
  uint4 g[2], p[2], m[2], v[2];
  float ms, vs;
};

template <int BITS>
__device__ __forceinline__ void load_unit(const AdamwTensor& t, int64_t i, UnitWords& w) {
  load8(t.grad, i, t.flags & kAdamwGradF32, w.g[0], w.g[1]);
  if (t.master) load8(t.master, i, true, w.p[0], w.p[1]);
  else load8(t.param, i, t.flags & kAdamwParamF32, w.p[0], w.p[1]);
  if (BITS == 32) {
    load8(t.m, i, true, w.m[0], w.m[1]);
    load8(t.v, i, true, w.v[0], w.v[1]);
  } else {
    const uint2 m = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + i));
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + i));
    w.m[0] = make_uint4(m.x, m.y, 0, 0);
    w.v[0] = make_uint4(v.x, v.y, 0, 0);
    w.ms = t.m_scale[i / kAdamwBlock];
    w.vs = t.v_scale[i / kAdamwBlock];
  }
}

template <int BITS>
__device__ __forceinline__ void step_unit(const AdamwTensor& t, const StepScalars& s, float gs, uint32_t step_key,
                                          int64_t i, int lane, const UnitWords& w) {
  float g[8], p[8], m[8], v[8], r[8];
  unpack8(w.g[0], w.g[1], t.flags & kAdamwGradF32, g);
  unpack8(w.p[0], w.p[1], t.master || (t.flags & kAdamwParamF32), p);
  if (BITS == 32) {
    unpack8(w.m[0], w.m[1], true, m);
    unpack8(w.v[0], w.v[1], true, v);
  } else {
    const uint32_t mu[2] = {w.m[0].x, w.m[0].y}, vu[2] = {w.v[0].x, w.v[0].y};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = e4m3x2_values(mu[e >> 1] >> (16 * (e & 1)));
      const float2 b = e4m3x2_values(vu[e >> 1] >> (16 * (e & 1)));
      m[2 * e] = __fmul_rn(a.x, w.ms);
      m[2 * e + 1] = __fmul_rn(a.y, w.ms);
      const float r0 = __fmul_rn(b.x, w.vs), r1 = __fmul_rn(b.y, w.vs);
      v[2 * e] = __fmul_rn(r0, r0);
      v[2 * e + 1] = __fmul_rn(r1, r1);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) adamw_element(s, __fmul_rn(g[e], gs), p[e], m[e], v[e], r[e]);
  if (t.master) store8(t.master, i, true, p);
  store8(t.param, i, t.flags & kAdamwParamF32, p);
  if (BITS == 32) {
    store8(t.m, i, true, m);
    store8(t.v, i, true, v);
    return;
  }
  uint32_t mm = 0, mr = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    mm = max(mm, __float_as_uint(fabsf(m[e])));
    mr = max(mr, __float_as_uint(r[e]) & 0x7fffffffu);  // (a NaN root may carry a sign)
  }
  mm = __reduce_max_sync(0xffffffffu, mm);
  mr = __reduce_max_sync(0xffffffffu, mr);
  float sm, sr, im, ir;
  block_scale(mm, &sm, &im);
  block_scale(mr, &sr, &ir);
  if (lane == 0) {
    t.m_scale[i / kAdamwBlock] = sm;
    t.v_scale[i / kAdamwBlock] = sr;
  }
  uint32_t mo[2], vo[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t h = rounding_bits(static_cast<uint32_t>(i >> 2) + q, step_key);
    const float* a = m + 4 * q;
    const __nv_fp8x2_storage_t lo =
        __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(a[0], im), __fmul_rn(a[1], im)), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi =
        __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(a[2], im), __fmul_rn(a[3], im)), __NV_SATFINITE, __NV_E4M3);
    mo[q] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    vo[q] = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      vo[q] |= e4m3_dithered(fminf(__fmul_rn(r[4 * q + e], ir), kFp8Max), (h >> (8 * e)) & 0xffu) << (8 * e);
  }
  __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + i), make_uint2(mo[0], mo[1]));
  __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + i), make_uint2(vo[0], vo[1]));
}

// The last unit of a tensor, and every unit of a tensor that no vector access fits:
// element by element, 32 apart in a lane.  2^27 parameters (bf16, fp32 masters) whose tensors
// all start off 16 bytes: 1240 us with 32-bit moments, 3.0 TB/s (552 aligned), 1037 us with 8-bit
// ones, 2.1 TB/s (328 aligned).
template <int BITS>
__device__ __noinline__ void step_unit_scalar(const AdamwTensor& t, const StepScalars& s, float gs, uint32_t step_key,
                                              int64_t base, int lane) {
  float m[8], r[8];
  uint32_t mm = 0, mr = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t i = base + lane + 32 * e;
    m[e] = r[e] = 0.f;
    if (i >= t.count) continue;
    const float g = (t.flags & kAdamwGradF32) ? static_cast<const float*>(t.grad)[i]
                                              : __bfloat162float(static_cast<const __nv_bfloat16*>(t.grad)[i]);
    float p = t.master ? t.master[i]
                       : ((t.flags & kAdamwParamF32) ? static_cast<const float*>(t.param)[i]
                                                     : __bfloat162float(static_cast<const __nv_bfloat16*>(t.param)[i]));
    float v;
    if (BITS == 32) {
      m[e] = static_cast<const float*>(t.m)[i];
      v = static_cast<const float*>(t.v)[i];
    } else {
      const float2 c = e4m3x2_values(static_cast<const uint8_t*>(t.m)[i] |
                                     (static_cast<uint32_t>(static_cast<const uint8_t*>(t.v)[i]) << 8));
      m[e] = __fmul_rn(c.x, t.m_scale[i / kAdamwBlock]);
      const float q = __fmul_rn(c.y, t.v_scale[i / kAdamwBlock]);
      v = __fmul_rn(q, q);
    }
    adamw_element(s, __fmul_rn(g, gs), p, m[e], v, r[e]);
    if (t.master) t.master[i] = p;
    if (t.flags & kAdamwParamF32) static_cast<float*>(t.param)[i] = p;
    else static_cast<__nv_bfloat16*>(t.param)[i] = __float2bfloat16_rn(p);
    if (BITS == 32) {
      static_cast<float*>(t.m)[i] = m[e];
      static_cast<float*>(t.v)[i] = v;
    }
    mm = max(mm, __float_as_uint(fabsf(m[e])));
    mr = max(mr, __float_as_uint(r[e]) & 0x7fffffffu);
  }
  if (BITS == 32) return;
  mm = __reduce_max_sync(0xffffffffu, mm);
  mr = __reduce_max_sync(0xffffffffu, mr);
  float sm, sr, im, ir;
  block_scale(mm, &sm, &im);
  block_scale(mr, &sr, &ir);
  __syncwarp();  // every lane has read the old scales
  if (lane == 0) {
    t.m_scale[base / kAdamwBlock] = sm;
    t.v_scale[base / kAdamwBlock] = sr;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t i = base + lane + 32 * e;
    if (i >= t.count) continue;
    const uint32_t h = rounding_bits(static_cast<uint32_t>(i >> 2), step_key);
    static_cast<uint8_t*>(t.m)[i] = __nv_cvt_float_to_fp8(__fmul_rn(m[e], im), __NV_SATFINITE, __NV_E4M3);
    static_cast<uint8_t*>(t.v)[i] = static_cast<uint8_t>(
        e4m3_dithered(fminf(__fmul_rn(r[e], ir), kFp8Max), (h >> (8 * (static_cast<uint32_t>(i) & 3))) & 0xffu));
  }
}

// One block per chunk of 16 units, two units a warp; a unit is 256 elements, the block of
// one 8-bit scale, so its largest magnitudes are two warp reductions.  All of a warp's loads
// (two units: 96 to 160 bytes a lane) go out before its first operation.  Bound by its
// streams, each byte once: 525 M parameters in bf16 with fp32 masters and 8-bit moments (16
// bytes each) in 1257 us, 6.7 TB/s; 149 tensors of 56 M parameters with 32-bit moments (28
// bytes each) in 227 us, 6.9 TB/s.  With 8-bit moments the arithmetic takes 85% of the issue
// slots, with 32-bit ones 27%.
template <int N, int BITS>
__global__ void __launch_bounds__(kAdamwThreads) adamw_kernel(const __grid_constant__ AdamwArgs<N> a) {
  griddep_begin();
  const AdamwTensor& t = a.t[find_tensor(a, blockIdx.x)];
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const StepScalars s{a.beta1, a.omb1, a.beta2, a.omb2, a.inv_root_bc2, a.eps, t.decay, t.rate};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kUnits = kAdamwChunk / kAdamwBlock / (kAdamwThreads / 32);
  const int64_t base = static_cast<int64_t>(blockIdx.x - t.chunk0) * kAdamwChunk + warp * kAdamwBlock;
  constexpr int64_t kApart = kAdamwBlock * (kAdamwThreads / 32);
  if ((t.flags & kAdamwAligned) && base + (kUnits - 1) * kApart + kAdamwBlock <= t.count) {
    UnitWords w[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) load_unit<BITS>(t, base + u * kApart + lane * 8, w[u]);
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
      step_unit<BITS>(t, s, gs, a.step_key, base + u * kApart + lane * 8, lane, w[u]);
    return;
  }
  for (int u = 0; u < kUnits; ++u) {
    const int64_t b = base + u * kApart;
    if (b >= t.count) return;
    if ((t.flags & kAdamwAligned) && b + kAdamwBlock <= t.count) {
      UnitWords w;
      load_unit<BITS>(t, b + lane * 8, w);
      step_unit<BITS>(t, s, gs, a.step_key, b + lane * 8, lane, w);
    } else {
      step_unit_scalar<BITS>(t, s, gs, a.step_key, b, lane);
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
