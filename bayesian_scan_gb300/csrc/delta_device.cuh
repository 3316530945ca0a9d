// delta_device.cuh -- what the kernels of the gated delta rule share: the
// arguments, which tokens a state row's sequence has, where its chunks lie in
// the scratch, and 16-byte asynchronous copies into shared memory.
//
// The rule, per head with a d_v x d_k state S:
//     S_t = a_t S_{t-1} + u_t k_t^T,   u_t = beta_t r_t,
//     r_t = v_t - a_t S_{t-1} k_t,     o_t = S_t q_t,      a_t = exp(-A d_t).
// The gate and the layouts are the diagonal scan's ("Learning to Remember,
// Learn, and Forget in Attention-Based Models", Metodologia 1); the update
// writes what the decayed state does not yet answer for the key.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kdn_internal.h"

namespace kdn {
namespace delta {
namespace {

constexpr int CHUNK = 64;   // tokens between the states that the backward keeps

template <typename T>
__device__ __forceinline__ float to_f32(T x) { return static_cast<float>(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Four consecutive elements, 16-byte (fp32) or 8-byte (bf16) aligned.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The tokens of one sequence: of state row n, the rows lo .. hi - 1 of every
// head, and its first chunk in the scratch.  A packed sequence's chunks begin
// at lo / CHUNK + n: sequences that follow one another never share a chunk,
// and all of them fit in T / CHUNK + nseq + 1 (decreasing offsets may share
// some, which spoils their values alone).
struct Span {
    int lo, hi;
    long long row;      // batch row: token t of head h is element (row * H + h) * T + t
    long long slot;     // the first chunk: chunk c of head h is number (slot + c) * H + h
};

__device__ __forceinline__ int clamped(int x, int T) { return min(max(x, 0), T); }

__device__ __forceinline__ Span span_of(const DeltaArgs& a, long long n) {
    Span s;
    if (a.offsets) {
        s.lo = clamped(a.offsets[n], a.T);
        s.hi = clamped(a.offsets[n + 1], a.T);
        s.row = 0;
        s.slot = s.lo / CHUNK + n;
    } else {
        s.lo = 0;
        s.hi = a.T;
        s.row = n;
        s.slot = n * ((a.T + CHUNK - 1) / CHUNK);
    }
    return s;
}

// The chunk of slot `slot`: its sequence and first token; false where none is.
__device__ __forceinline__ bool chunk_of(const DeltaArgs& a, long long slot, long long* n, int* t0, int* m, long long* row) {
    if (!a.offsets) {
        const int per = (a.T + CHUNK - 1) / CHUNK;
        *n = *row = slot / per;
        *t0 = static_cast<int>(slot % per) * CHUNK;
        *m = min(CHUNK, a.T - *t0);
        return true;
    }
    int low = 0, high = a.nseq - 1;   // the last sequence that begins at or before the slot
    while (low < high) {
        const int mid = (low + high + 1) / 2;
        if (clamped(a.offsets[mid], a.T) / CHUNK + mid <= slot) low = mid;
        else high = mid - 1;
    }
    const int lo = clamped(a.offsets[low], a.T), hi = clamped(a.offsets[low + 1], a.T);
    const long long c = slot - (lo / CHUNK + low);
    if (c < 0 || c * CHUNK >= hi - lo) return false;
    *n = low;
    *row = 0;
    *t0 = lo + static_cast<int>(c) * CHUNK;
    *m = min(CHUNK, hi - *t0);
    return true;
}

}  // namespace

// Chunks that the scratch has room for.
inline long long slots_of(int B, int T, int nseq) {
    const long long per = (static_cast<long long>(T) + CHUNK - 1) / CHUNK;
    return nseq > 0 ? per + nseq + 1 : B * per;
}

}  // namespace delta
}  // namespace kdn
