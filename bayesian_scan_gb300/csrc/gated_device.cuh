// gated_device.cuh -- device helpers of the per-channel gated recurrence
// (gated_scan.cu): typed loads and stores, packed fp32 pairs and the gate.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

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

// Two fp32 values per instruction (sm_100 and later).
struct F2 {
    float x, y;
};

__device__ __forceinline__ uint64_t pk(F2 a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ F2 unpk(uint64_t r) {
    F2 a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
    return a;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)), "l"(pk(c)));
    return unpk(r);
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)));
    return unpk(r);
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)));
    return unpk(r);
}
__device__ __forceinline__ F2 both(float v) { return F2{v, v}; }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

constexpr float LOG2E = 1.4426950408889634f;

// The gate alpha = exp(-A d) = 2^y, y = -A log2(e) d, of two elements, and
// w = 1 - alpha where that is wanted (W).
//
// Near 0, 2^y - 1 = y p(y), p a Chebyshev interpolant of (2^y - 1)/y of degree
// 4 on [-0.36, 0.36] (1.9e-7 of it with its roundings; alpha to half a step
// and a little).  Beyond, memories are four tokens and the hardware's 2^y
// (2^-22) serves.  w = 1 - alpha is then within 7 half steps (measured, next
// to -0.36), which fp32 results show: for them (FINE) w has degree 6 on [-1,
// 0.5], and is within 3.5 everywhere (in every call: convex 65536 x 2048 bf16
// 228 us, against 213).
struct Gate2 {
    F2 a, w;
};

__device__ __forceinline__ bool is_near(float y) { return fabsf(y + 0.25f) <= 0.75f; }

template <bool W, bool FINE>
__device__ __forceinline__ Gate2 gate2(F2 y) {
    F2 p;
    if (W && FINE) {
        p = both(1.319523016718449e-05f);
        p = fma2(p, y, both(0.00015371742483694106f));
        p = fma2(p, y, both(0.0013341674348339438f));
        p = fma2(p, y, both(0.009618356823921204f));
        p = fma2(p, y, both(0.05550402030348778f));
        p = fma2(p, y, both(0.24022649228572845f));
    } else {
        p = both(0.0013358289143070579f);
        p = fma2(p, y, both(0.009643110446631908f));
        p = fma2(p, y, both(0.055504027754068375f));
        p = fma2(p, y, both(0.24022570252418518f));
    }
    p = fma2(p, y, both(0.6931471824645996f));
    const F2 big{ex2(y.x), ex2(y.y)}, near = fma2(p, y, both(1.f));
    const bool bx = W && FINE ? is_near(y.x) : fabsf(y.x) <= 0.36f,
               by = W && FINE ? is_near(y.y) : fabsf(y.y) <= 0.36f;
    Gate2 g;
    g.a = F2{bx ? near.x : big.x, by ? near.y : big.y};
    if (W) {
        const F2 m = mul2(p, F2{-y.x, -y.y}), f = fma2(big, both(-1.f), both(1.f));
        g.w = F2{bx ? m.x : f.x, by ? m.y : f.y};
    }
    return g;
}

// The same as alpha = a + e: a the value rounded down, e what the rounding lost.
// A long memory has alpha next to 1, where a float's step is 6e-8 whatever
// 1 - alpha is: a state carried through a thousand rounded decays would be
// off by 7e-6.  So a span's decay is 2^y of its summed exponents, in this
// form, and only the at most 16 tokens that a warp composes itself multiply
// rounded alphas.
//
// On [-1, 0.5] 2^y - 1 is the interpolant of degree 6; beyond, a - 1 and m are
// the same rounding, and e is what TINY makes of zero.
//
// An infinite state goes through a s + (e s + b) as it is: a and e have one
// sign and neither is 0 (a alone where y = -infinity, a decay of nothing: 0
// times infinity is NaN) -- also of a span whose decay underflows where no
// token's does.
constexpr float TINY = 1.4e-45f;   // 2^-149

struct Gate {
    float a, e, w;
};

__device__ __forceinline__ Gate gate(float y) {
    float p = 1.319523016718449e-05f;
    p = fmaf(p, y, 0.00015371742483694106f);
    p = fmaf(p, y, 0.0013341674348339438f);
    p = fmaf(p, y, 0.009618356823921204f);
    p = fmaf(p, y, 0.05550402030348778f);
    p = fmaf(p, y, 0.24022649228572845f);
    p = fmaf(p, y, 0.6931471824645996f);
    const float big = ex2(y);
    const bool small = is_near(y);
    const float m = small ? y * p : big - 1.f;   // 2^y - 1
    Gate g;
    g.a = max_nan(small ? __fadd_rd(1.f, m) : big, y > -INFINITY ? TINY : 0.f);
    g.e = max_nan(m - (g.a - 1.f), TINY);
    g.w = -m;
    return g;
}

// alpha s + b
__device__ __forceinline__ float decay_add(float a, float e, float s, float b) {
    return fmaf(a, s, fmaf(e, s, b));
}
__device__ __forceinline__ float decay_add(const Gate& g, float s, float b) {
    return decay_add(g.a, g.e, s, b);
}

// V adjacent elements of a type, as loaded and stored by one lane.
template <typename T, int V>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 1> {
    uint16_t r;
    __device__ __forceinline__ float get(int) const { return __uint_as_float(static_cast<uint32_t>(r) << 16); }
    __device__ __forceinline__ void set(const float* f) { r = __bfloat16_as_ushort(__float2bfloat16_rn(f[0])); }
};
template <>
struct Vec<__nv_bfloat16, 2> {
    uint32_t r;
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i == 0 ? r << 16 : r & 0xffff0000u);
    }
    __device__ __forceinline__ void set(const float* f) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[0], f[1]);
        r = *reinterpret_cast<const uint32_t*>(&b);
    }
};
template <>
struct Vec<float, 1> {
    float r;
    __device__ __forceinline__ float get(int) const { return r; }
    __device__ __forceinline__ void set(const float* f) { r = f[0]; }
};
template <>
struct Vec<float, 2> {
    float2 r;
    __device__ __forceinline__ float get(int i) const { return i == 0 ? r.x : r.y; }
    __device__ __forceinline__ void set(const float* f) { r = make_float2(f[0], f[1]); }
};

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> peek(const char* p) {
    Vec<T, V> v;
    v.r = *reinterpret_cast<const decltype(v.r)*>(p);
    return v;
}
template <typename T, int V>
__device__ __forceinline__ void poke(char* p, const Vec<T, V>& v) {
    *reinterpret_cast<std::remove_const_t<decltype(v.r)>*>(p) = v.r;
}
// N adjacent elements as fp32; N = 4 takes aligned addresses.
template <int N, typename T>
__device__ __forceinline__ void load_n(const T* p, float* v) {
    if constexpr (N == 1) {
        v[0] = to_f32(*p);
    } else if constexpr (sizeof(T) == 4) {
        const float4 q = *reinterpret_cast<const float4*>(p);
        v[0] = q.x;
        v[1] = q.y;
        v[2] = q.z;
        v[3] = q.w;
    } else {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        v[0] = __uint_as_float(q.x << 16);
        v[1] = __uint_as_float(q.x & 0xffff0000u);
        v[2] = __uint_as_float(q.y << 16);
        v[3] = __uint_as_float(q.y & 0xffff0000u);
    }
}
template <int N, typename T>
__device__ __forceinline__ void store_n(T* p, const float* v) {
    if constexpr (N == 1) {
        *p = from_f32<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        uint2 q;
        q.x = *reinterpret_cast<const uint32_t*>(&a);
        q.y = *reinterpret_cast<const uint32_t*>(&b);
        *reinterpret_cast<uint2*>(p) = q;
    }
}

// Asynchronous copies global -> shared memory; `bytes` < SIZE fills the rest
// with zeros (0: nothing is read).
template <int SIZE>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int bytes) {
    if (SIZE == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A warp's K x ROWB block of rows `ld` bytes apart: rows first <= j < last,
// columns below `width` bytes; the rest of the block becomes zeros (`safe`:
// any valid address, named where nothing is read).  SIZE 16: lanes take
// 16-byte pieces in order; SIZE 4: a lane takes 4-byte words 32 apart; SIZE 2:
// 2-byte elements 32 apart, by plain loads.
template <int SIZE, int ROWB, int K>
struct Rows {
    static constexpr int SIZE_ = SIZE;
    static constexpr int PER = ROWB  / SIZE;                    // pieces per row
    static constexpr int RPI = PER >= 32 ? 1 : 32 / PER;       // rows per instruction
    static constexpr int CPR = PER >= 32 ? PER / 32 : 1;       // instructions per row
};

template <int SIZE, int ROWB, int K>
__device__ __forceinline__ void rows_in(char* to, const void* safe, const char* src, long long ld, int first,
                                        int last, int width, int lane) {
    using R = Rows<SIZE < 4 ? 4 : SIZE, ROWB, K>;
    if constexpr (SIZE == 2) {
        // by element, in two batches of loads
#pragma unroll
        for (int h = 0; h < K; h += K / 2) {
            uint16_t v[K / 2][ROWB / 64];
#pragma unroll
            for (int i = 0; i < K / 2; ++i)
#pragma unroll
                for (int q = 0; q < ROWB / 64; ++q) {
                    const int j = h + i, col = (q * 32 + lane) * 2;
                    const bool ok = j >= first && j < last && col < width;
                    v[i][q] = ok ? *reinterpret_cast<const uint16_t*>(src + j * ld + col) : uint16_t(0);
                }
#pragma unroll
            for (int i = 0; i < K / 2; ++i)
#pragma unroll
                for (int q = 0; q < ROWB / 64; ++q)
                    *reinterpret_cast<uint16_t*>(to + (h + i) * ROWB + (q * 32 + lane) * 2) = v[i][q];
        }
        return;
    }
    uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    const int j0 = R::PER >= 32 ? 0 : lane / R::PER, col = (R::PER >= 32 ? lane : lane % R::PER) * R::SIZE_;
    const char* p = src + j0 * ld + col;
    dst += j0 * ROWB + col;
    if (first <= 0 && last >= K && width >= ROWB) {            // (the warp as one)
#pragma unroll
        for (int i = 0; i < K / R::RPI; ++i) {
#pragma unroll
            for (int q = 0; q < R::CPR; ++q)
                copy_async<SIZE < 4 ? 4 : SIZE>(dst + i * R::RPI * ROWB + q * 32 * R::SIZE_, p + q * 32 * R::SIZE_, R::SIZE_);
            p += R::RPI * ld;
        }
    } else {
#pragma unroll
        for (int i = 0; i < K / R::RPI; ++i) {
            const int j = j0 + i * R::RPI;
#pragma unroll
            for (int q = 0; q < R::CPR; ++q) {
                const bool ok = j >= first && j < last && col + q * 32 * R::SIZE_ < width;
                copy_async<SIZE < 4 ? 4 : SIZE>(dst + i * R::RPI * ROWB + q * 32 * R::SIZE_, ok ? p + q * 32 * R::SIZE_ : safe, ok ? R::SIZE_ : 0);
            }
            p += R::RPI * ld;
        }
    }
}

// The other way, 16-byte pieces from shared memory.
template <int ROWB, int K>
__device__ __forceinline__ void rows_out(char* dst, long long ld, const char* src, int first, int last, int width,
                                         int lane) {
    using R = Rows<16, ROWB, K>;
    const int j0 = lane / R::PER, col = lane % R::PER * 16;
    char* p = dst + j0 * ld + col;
    src += j0 * ROWB + col;
    const bool full = first <= 0 && last >= K && width >= ROWB;
#pragma unroll
    for (int i = 0; i < K / R::RPI; ++i) {
        const int j = j0 + i * R::RPI;
        if (full || (j >= first && j < last && col < width))
            __stcs(reinterpret_cast<float4*>(p), *reinterpret_cast<const float4*>(src + i * R::RPI * ROWB));
        p += R::RPI * ld;
    }
}

}  // namespace gated
}  // namespace kdn
