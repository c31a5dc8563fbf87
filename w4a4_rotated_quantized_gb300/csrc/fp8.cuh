// Shared pieces of the 8-bit operators: 16-bit inputs of either type, and the
// block quantizer to e4m3.
//
// The block quantizer ([S] Stage 2b's symmetric abs-max quantizer on the e4m3
// grid, one scale for each block): with m = max(max |v|, 1e-12),
//   scale = m / 448,   code = e4m3(v * 448 / m)   (nearest, ties to even).
// The quotient is formed so that an exact tie stays one: with f the power of
// two that brings m into [2, 4), t = v * 448 f and b = m f, the quotient
// t / b is q0 = t * rn(1 / b) corrected once by its residual, q0 +
// (t - q0 b) rn(1 / b) (P. Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990).  A tie of the e4m3 grid has 5
// significant bits; when t / b is one, the residual is exact and the
// correction lands on it.  A plain v * (448 / m) in fp32 breaks a quarter of
// a percent of such ties the wrong way for bf16 inputs, whose few significant
// bits make exact ties common.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace quarot {
namespace fp8 {

constexpr int BLK = 128;                 // columns (and weight rows) that share a scale
constexpr float kMaxCode = 448.0f;       // largest e4m3 value
constexpr float kAmaxFloor = 1e-12f;     // smallest abs-max a scale is made from

template <typename T>
__device__ __forceinline__ float2 to_f2(uint32_t v);
template <>
__device__ __forceinline__ float2 to_f2<__half>(uint32_t v) {
  return h2_to_f2(v);
}
template <>
__device__ __forceinline__ float2 to_f2<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t from_f2(float2 v);
template <>
__device__ __forceinline__ uint32_t from_f2<__half>(float2 v) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t from_f2<__nv_bfloat16>(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Maximum in which a NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The abs-max a block is quantized with: floored, and NaN where the block
// holds an infinity or a NaN (its scale and all its codes are then NaN).
__device__ __forceinline__ float block_amax(float m) {
  return __float_as_uint(m) >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(m, kAmaxFloor);
}
__device__ __forceinline__ float block_scale(float m) { return __fdiv_rn(m, kMaxCode); }

struct Quotient {  // v -> v * 448 / m
  float2 p, nb, inv;
  __device__ __forceinline__ explicit Quotient(float m) {
    const uint32_t mb = __float_as_uint(m);
    // m finite: 2^(128 - e) for m's biased exponent e, so m f is in [2, 4)
    const float f = __uint_as_float((255u << 23) - (mb & 0x7F800000u));
    const float b = m * f;  // exact; NaN stays NaN
    const float r = __frcp_rn(b);
    p = make_float2(kMaxCode * f, kMaxCode * f);
    nb = make_float2(-b, -b);
    inv = make_float2(r, r);
  }
  __device__ __forceinline__ float2 operator()(float2 v) const {
    const float2 t = __fmul2_rn(v, p);
    const float2 q0 = __fmul2_rn(t, inv);
    return __ffma2_rn(__ffma2_rn(q0, nb, t), inv, q0);
  }
};

// Two e4m3 codes, the first in the low byte (round to nearest even).
__device__ __forceinline__ uint32_t cvt_e4m3x2(float2 v) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(v.y), "f"(v.x));
  return d;
}
__device__ __forceinline__ uint32_t cvt_e4m3x4(float2 a, float2 b) { return cvt_e4m3x2(a) | (cvt_e4m3x2(b) << 16); }

// The 8-bit calls follow one another in a layer, most of them hardly longer
// than a launch and its set-up, so they are launched as programmatic
// dependents: the next kernel of the stream may start when every CTA of this
// one has called next_may_start() or ended, and it waits in
// wait_for_previous() until this one is over and its writes are visible.
// Every thread waits there before its first access to global memory, reads and
// writes alike, so a kernel ends after all that came before it in the stream.
// A CTA that needs tensor memory takes it before it lets the next kernel
// start, which therefore never holds what an earlier one still waits for.  One
// after another, without and with it: quantizer, 1 x 4096: 1.85 and 1.43 us;
// weights, 12288 x 4096: 27.7 and 26.5 us; product, 1 x 4096 x 4096: 8.3 and
// 6.9 us; gated, 4 x 12288 x 4096: 20.1 and 18.8 us (and 20.1 us where the
// product lets the next one start before its main loop).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The status is that of this launch alone.
template <typename... P, typename... A>
inline int launch_dependent(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster,
                            cudaStream_t st, A... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, kern, P(args)...)) ? QUAROT_OK : QUAROT_ERR_LAUNCH;
}

}  // namespace fp8
}  // namespace quarot
