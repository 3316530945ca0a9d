// gated_device.cuh -- device helpers of the per-channel gated recurrence
// (gated_scan.cu): typed loads and stores and the gate.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace kdn {
namespace gated {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The gate alpha = exp(z), z = -A d, as alpha = a + e: a the rounded value, e
// what the rounding lost, and w = 1 - alpha.  A long memory has alpha next to
// 1, where a float's step is 6e-8 whatever 1 - alpha is; a scan that used the
// rounded alpha alone would drift by that much per token of its memory
// (7e-6 of the state at a memory of a thousand tokens; with e, 1e-7).
//
// |z| <= 0.35: expm1(z) = z p(z), p the degree-5 Chebyshev interpolant of
// (e^z - 1)/z on [-0.35, 0.35] (1.3e-7 relative with its roundings).  Beyond,
// memories are three tokens and 2^(z log2 e) of the hardware serves.
struct Gate {
    float a, e, w;
};

__device__ __forceinline__ Gate gate(float z) {
    float p = 0.0013934532f;
    p = fmaf(p, z, 0.008369861f);
    p = fmaf(p, z, 0.041666456f);
    p = fmaf(p, z, 0.16666499f);
    p = fmaf(p, z, 0.5f);
    p = fmaf(p, z, 1.0f);
    float big;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(big) : "f"(z * 1.4426950408889634f));
    const bool small = fabsf(z) <= 0.35f;
    const float m = small ? z * p : big - 1.f;   // expm1(z)
    Gate g;
    g.a = small ? 1.f + m : big;
    g.e = small ? m - (g.a - 1.f) : 0.f;
    g.w = -m;
    return g;
}

// a * s + b with a = the gate
__device__ __forceinline__ float decay_add(const Gate& g, float s, float b) {
    return fmaf(g.a, s, fmaf(g.e, s, b));
}

}  // namespace gated
}  // namespace kdn
