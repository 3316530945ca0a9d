// add_norm.cu -- the residual's addition and its root-mean-square norm, what
// stands before a mixer's projection: per row of C channels
//     s = x + residual (rounded to the residual's type),
//     y = w . s / sqrt(mean(s^2) + eps),
// y in bf16, fp32 or e4m3 with a scale for each group of 128 channels, and the
// gradients of both.  One pass: a row's elements stay in registers between its
// sum of squares and its outputs, so x and the residual are read and s and y
// written once (8 bytes an element in bf16, bound by HBM).
//
// Forward: a warp to a row of up to 512 channels, a CTA of G warps to a longer
// one (or to few rows: a decode batch waits for latency), 64 bytes a thread.  A
// warp's elements are whole groups of 128, so a group's largest value is a matter
// of shuffles.
//
// Backward: n = s rstd, t = w . grad_y;
//     grad = rstd (t - n mean(t . n)) + grad_sum,   grad_w = sum_rows grad_y . n.
// A thread keeps its columns for all rows that its CTA takes, and with them
// their share of grad_w; several rows are in flight at a time, and the sums of
// ROWS rows are one exchange.  The CTAs' shares are added in a fixed order (sum_rows.cuh).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kdn.h"
#include "kdn_internal.h"
#include "kernel_setup.h"
#include "sum_rows.cuh"

namespace kdn {
namespace {

constexpr int GROUP = 128;               // channels to a scale
constexpr float TOP = 448.f;             // the largest e4m3 value
constexpr int WARPS = 8;                 // of a CTA whose warps have rows of their own

struct E4m3 {
    unsigned char bits;
};

// VEC consecutive elements as fp32.
template <int VEC, typename T>
__device__ __forceinline__ void load(const T* p, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = static_cast<float>(*p);
    } else if constexpr (sizeof(T) == 2) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
}
template <int VEC, typename T>
__device__ __forceinline__ void store(T* p, const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        if constexpr (std::is_same<T, E4m3>::value) p->bits = __nv_cvt_float_to_fp8(f[0], __NV_SATFINITE, __NV_E4M3);
        else if constexpr (sizeof(T) == 2) *p = __float2bfloat16_rn(f[0]);
        else *p = f[0];
    } else if constexpr (std::is_same<T, E4m3>::value) {
        uint32_t u[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i], f[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2], f[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
            u[i] = lo | hi << 16;
        }
        *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
    } else if constexpr (sizeof(T) == 2) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// What fp32 becomes in T and back.
template <typename T>
__device__ __forceinline__ float as(float x) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(__float2bfloat16_rn(x));
    else return x;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// A warp's NV vectors a lane of the row (from element `first`): rounded sums
// into s (written to memory too where there is a residual) and their squares.
template <int VEC, int NV, typename TX, typename TR>
__device__ __forceinline__ float sum_part(const TX* x, const TR* res, TR* sum, int first, int C, float (&s)[NV][VEC]) {
    const int lane = threadIdx.x & 31;
    float r[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = first + (j * 32 + lane) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[j][e] = r[j][e] = 0.f;
        if (c < C) {
            load<VEC>(x + c, s[j]);
            if (res) load<VEC>(res + c, r[j]);
        }
    }
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = first + (j * 32 + lane) * VEC;
        if (res) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[j][e] = as<TR>(s[j][e] + r[j][e]);
            if (c < C) store<VEC>(sum + c, s[j]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) q = fmaf(s[j][e], s[j][e], q);
    }
    return q;
}

template <int VEC, int NV, typename TY>
__device__ __forceinline__ void norm_part(float (&s)[NV][VEC], float rstd, const float* w, TY* y, float* scale, int first,
                                          int C) {
    const int lane = threadIdx.x & 31;
    float top[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = first + (j * 32 + lane) * VEC;
        float f[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = 1.f;
        if (w && c < C) load<VEC>(w + c, f);
        top[j] = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            s[j][e] = s[j][e] * rstd * f[e];
            top[j] = fmaxf(top[j], fabsf(s[j][e]));
        }
        if constexpr (!std::is_same<TY, E4m3>::value)
            if (c < C) store<VEC>(y + c, s[j]);
    }
    if constexpr (std::is_same<TY, E4m3>::value) {
        // a group is 16 lanes of one vector of 8, or the whole warp in 4 strips of single elements
        if constexpr (VEC == 1) {
#pragma unroll
            for (int j = 0; j < NV; j += 4) {
                const float t = fmaxf(fmaxf(top[j], top[j + 1]), fmaxf(top[j + 2], top[j + 3]));
                top[j] = top[j + 1] = top[j + 2] = top[j + 3] = t;
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = first + (j * 32 + lane) * VEC;
#pragma unroll
            for (int o = VEC == 1 ? 16 : 8; o > 0; o >>= 1) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
            // a group whose largest is 0 or rounds to it here (up to 224 x 2^-149) has scale 1
            const float part = top[j] / TOP, sc = part > 0.f ? part : 1.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[j][e] = s[j][e] / sc;
            if (c < C) {
                store<VEC>(y + c, s[j]);
                if (c % GROUP == 0) scale[c / GROUP] = sc;
            }
        }
    }
}

// G = 1: a warp to a row, no exchange.  G > 1: a CTA of G warps to a row.
template <int VEC, int NV, typename TX, typename TR, typename TY, bool ALONE>
__global__ void __launch_bounds__(ALONE ? WARPS * 32 : 1024) add_norm_kernel(const NormArgs a) {
    __shared__ float share[32];
    constexpr int PER = 32 * NV * VEC;       // elements of a warp
    const int warp = threadIdx.x >> 5, G = ALONE ? 1 : blockDim.x >> 5;
    const long long row = ALONE ? static_cast<long long>(blockIdx.x) * WARPS + warp : blockIdx.x;
    if (ALONE && row >= a.rows) return;
    const int C = a.C, first = ALONE ? 0 : warp * PER;
    const TX* x = static_cast<const TX*>(a.x) + row * a.x_ld;
    const TR* res = a.residual ? static_cast<const TR*>(a.residual) + row * C : nullptr;
    TR* sum = static_cast<TR*>(a.sum) + row * C;
    TY* y = static_cast<TY*>(a.y) + row * C;
    float* scale = a.scale + row * ((C + GROUP - 1) / GROUP);
    float s[NV][VEC];
    float q = sum_part<VEC, NV>(x, res, sum, first, C, s);
    for (int c = first + G * PER; c < C; c += G * PER) {     // rows that the registers do not hold
        float more[NV][VEC];
        q += sum_part<VEC, NV>(x, res, sum, c, C, more);
    }
    q = warp_sum(q);
    if constexpr (!ALONE) {
        if ((threadIdx.x & 31) == 0) share[warp] = q;
        __syncthreads();
        q = warp_sum((threadIdx.x & 31) < G ? share[threadIdx.x & 31] : 0.f);
    }
    const float rstd = rsqrtf(q / static_cast<float>(C) + a.eps);
    norm_part<VEC, NV, TY>(s, rstd, a.weight, y, scale, first, C);
    for (int c = first + G * PER; c < C; c += G * PER) {
        // each thread reads back what it has written itself (or x)
        float more[NV][VEC];
        if (res) sum_part<VEC, NV>(sum, static_cast<const TR*>(nullptr), static_cast<TR*>(nullptr), c, C, more);
        else sum_part<VEC, NV>(x, static_cast<const TR*>(nullptr), static_cast<TR*>(nullptr), c, C, more);
        norm_part<VEC, NV, TY>(more, rstd, a.weight, y, scale, c, C);
    }
}

// ---- backward ----------------------------------------------------------------

constexpr int BACK_CTAS = 8;                 // CTAs to an SM at most (their shares of grad_w are read once more)

// VEC consecutive elements as they lie in memory.
template <int VEC, typename T>
struct Raw {
    uint4 w[VEC * sizeof(T) / 16];
    __device__ __forceinline__ void get(const T* p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(VEC * sizeof(T) / 16); ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void to(float (&f)[VEC]) const {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t u = i == 0 ? w[0].x : i == 1 ? w[0].y : i == 2 ? w[0].z : w[0].w;
                f[2 * i] = __uint_as_float(u << 16);
                f[2 * i + 1] = __uint_as_float(u & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[4 * i] = __uint_as_float(w[i].x);
                f[4 * i + 1] = __uint_as_float(w[i].y);
                f[4 * i + 2] = __uint_as_float(w[i].z);
                f[4 * i + 3] = __uint_as_float(w[i].w);
            }
        }
    }
};
template <typename T>
struct Raw<1, T> {
    T v;
    __device__ __forceinline__ void get(const T* p) { v = *p; }
    __device__ __forceinline__ void to(float (&f)[1]) const { f[0] = static_cast<float>(v); }
};

// blockDim.x threads have VEC columns each of one slice of blockDim.x * VEC
// columns at a time; a row of one slice stays in registers, as it came, and the
// next rows' loads are under way meanwhile; a longer one is read twice.
// MOST threads: 256 with four rows of 16-bit types in flight or two of others
// (two and three CTAs to an SM gain 8 % at 2048 bf16 channels and lose a third at
// 1000 of fp32), 1024 (registers for one row) where a row is longer.
template <int VEC, int MOST, typename TX, typename TR, typename TY>
__global__ void __launch_bounds__(MOST) add_norm_back_kernel(const NormArgs a, float* shares, int slices) {
    constexpr int ROWS = MOST > 256 ? 1 : sizeof(TR) + sizeof(TY) == 4 ? 4 : 2;
    __shared__ float part[2][32][2 * ROWS];
    const int C = a.C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int step = blockDim.x * VEC, mine = threadIdx.x * VEC;
    const bool in = mine < C;
    const TR* sum = static_cast<const TR*>(a.residual);
    const TY* gy = static_cast<const TY*>(a.grad_y);
    const TR* gs = static_cast<const TR*>(a.grad_sum);
    float acc[VEC], w[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        acc[e] = 0.f;
        w[e] = 1.f;
    }
    if (a.weight && in) load<VEC>(a.weight + mine, w);
    Raw<VEC, TR> rs[ROWS], ro[ROWS];
    Raw<VEC, TY> rg[ROWS];
    const long long first = static_cast<long long>(blockIdx.x) * ROWS, stride = static_cast<long long>(gridDim.x) * ROWS;
    auto fetch = [&](long long r0) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (in && r0 + i < a.rows) {
                const long long at = (r0 + i) * C + mine;
                rs[i].get(sum + at);
                rg[i].get(gy + at);
                if (gs) ro[i].get(gs + at);
            }
    };
    fetch(first);
    int turn = 0;
    for (long long r0 = first; r0 < a.rows; r0 += stride, turn ^= 1) {
        float sums[2 * ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            float q = 0.f, d = 0.f;
            if (in && r0 + i < a.rows) {
                float s[VEC], g[VEC];
                rs[i].to(s);
                rg[i].to(g);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    q = fmaf(s[e], s[e], q);
                    d = fmaf(g[e] * w[e], s[e], d);
                }
            }
            for (int k = 1; k < slices; ++k) {               // columns that the registers do not hold
                const int c = k * step + mine;
                if (r0 + i < a.rows && c < C) {
                    float sv[VEC], gv[VEC], wv[VEC];
                    load<VEC>(sum + (r0 + i) * C + c, sv);
                    load<VEC>(gy + (r0 + i) * C + c, gv);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) wv[e] = 1.f;
                    if (a.weight) load<VEC>(a.weight + c, wv);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        q = fmaf(sv[e], sv[e], q);
                        d = fmaf(gv[e] * wv[e], sv[e], d);
                    }
                }
            }
            sums[2 * i] = warp_sum(q);
            sums[2 * i + 1] = warp_sum(d);
        }
        if (warps > 1) {   // (two arrays in turn: the last rows' readers are past it when it is written again)
            if (lane == 0)
#pragma unroll
                for (int i = 0; i < 2 * ROWS; ++i) part[turn][warp][i] = sums[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2 * ROWS; ++i) sums[i] = warp_sum(lane < warps ? part[turn][lane][i] : 0.f);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (r0 + i >= a.rows) break;
            const float rstd = rsqrtf(sums[2 * i] / static_cast<float>(C) + a.eps);
            const float mean = sums[2 * i + 1] * rstd / static_cast<float>(C);       // of t . n
            if (in) {
                const long long at = (r0 + i) * C + mine;
                float s[VEC], g[VEC], out[VEC];
                rs[i].to(s);
                rg[i].to(g);
                if (gs) {
                    ro[i].to(out);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) out[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float n = s[e] * rstd;
                    acc[e] = fmaf(g[e], n, acc[e]);
                    out[e] = fmaf(rstd, g[e] * w[e] - n * mean, out[e]);
                }
                if (a.grad_residual) store<VEC>(static_cast<TR*>(a.grad_residual) + at, out);
                if (a.grad_x) store<VEC>(static_cast<TX*>(a.grad_x) + at, out);
                const long long next = r0 + stride + i;      // this row's registers are free
                if (next < a.rows) {
                    rs[i].get(sum + next * C + mine);
                    rg[i].get(gy + next * C + mine);
                    if (gs) ro[i].get(gs + next * C + mine);
                }
            }
            for (int k = 1; k < slices; ++k) {
                const int c = k * step + mine;
                if (c >= C) break;
                const long long more = (r0 + i) * C + c;
                float sv[VEC], gv[VEC], wv[VEC], ov[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    wv[e] = 1.f;
                    ov[e] = 0.f;
                }
                load<VEC>(sum + more, sv);
                load<VEC>(gy + more, gv);
                if (a.weight) load<VEC>(a.weight + c, wv);
                if (gs) load<VEC>(gs + more, ov);
                float* share = shares ? shares + static_cast<long long>(blockIdx.x) * C + c : nullptr;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float n = sv[e] * rstd;
                    // (the CTA's first row sets the share, its later ones add to it)
                    if (share) share[e] = r0 == first && i == 0 ? gv[e] * n : fmaf(gv[e], n, share[e]);
                    ov[e] = fmaf(rstd, gv[e] * wv[e] - n * mean, ov[e]);
                }
                if (a.grad_residual) store<VEC>(static_cast<TR*>(a.grad_residual) + more, ov);
                if (a.grad_x) store<VEC>(static_cast<TX*>(a.grad_x) + more, ov);
            }
        }
    }
    if (shares && in) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) shares[static_cast<long long>(blockIdx.x) * C + mine + e] = acc[e];
    }
}

// The same for rows of 16-bit types that up to 256 threads hold (C <= 2048):
// coming rows lie in a ring in shared memory, a thread's own bytes, which only it
// writes and reads (no barrier): GROUPS groups of ROWS rows, all but one on their
// way.  (us in registers and through the ring: 32768 x 2048 145 and 112, 65536 x
// 512 73 and 58.  Of wider types or rows fewer fit: 32768 x 1000 fp32 104 and 139,
// 8192 x 8192 bf16 199 and 248.)
constexpr int RING_ROWS = 2, RING_GROUPS = 4, RING_BYTES = RING_GROUPS * RING_ROWS * 3 * 16;   // a thread's

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}

template <typename TX>
__global__ void __launch_bounds__(256) add_norm_back_ring_kernel(const NormArgs a, float* shares) {
    using T = __nv_bfloat16;
    constexpr int ROWS = RING_ROWS, GROUPS = RING_GROUPS;
    __shared__ float part[2][8][2 * ROWS];
    extern __shared__ __align__(16) unsigned char ring[];
    const int C = a.C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, mine = threadIdx.x * 8;
    const bool in = mine < C;
    const T* from[3] = {static_cast<const T*>(a.residual), static_cast<const T*>(a.grad_y), static_cast<const T*>(a.grad_sum)};
    float acc[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        acc[e] = 0.f;
        w[e] = 1.f;
    }
    if (a.weight && in) load<8>(a.weight + mine, w);
    const long long first = static_cast<long long>(blockIdx.x) * ROWS, stride = static_cast<long long>(gridDim.x) * ROWS;
    auto place = [&](int group, int i, int which) {
        return ring + (((group * ROWS + i) * 3 + which) * blockDim.x + threadIdx.x) * 16;
    };
    auto fetch = [&](long long r0, int group) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (in && r0 + i < a.rows)
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (k < 2 || from[2]) copy16(place(group, i, k), from[k] + (r0 + i) * C + mine);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int g = 0; g < GROUPS - 1; ++g) fetch(first + g * stride, g);
    int now = 0, turn = 0;
    for (long long r0 = first; r0 < a.rows; r0 += stride, turn ^= 1) {
        fetch(r0 + (GROUPS - 1) * stride, (now + GROUPS - 1) % GROUPS);
        asm volatile("cp.async.wait_group %0;" ::"n"(GROUPS - 1) : "memory");
        float s[ROWS][8], g[ROWS][8], sums[2 * ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            float q = 0.f, d = 0.f;
            if (in && r0 + i < a.rows) {
                load<8>(reinterpret_cast<const T*>(place(now, i, 0)), s[i]);
                load<8>(reinterpret_cast<const T*>(place(now, i, 1)), g[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    q = fmaf(s[i][e], s[i][e], q);
                    d = fmaf(g[i][e] * w[e], s[i][e], d);
                }
            }
            sums[2 * i] = warp_sum(q);
            sums[2 * i + 1] = warp_sum(d);
        }
        if (warps > 1) {   // (two arrays in turn: the last rows' readers are past it when it is written again)
            if (lane == 0)
#pragma unroll
                for (int i = 0; i < 2 * ROWS; ++i) part[turn][warp][i] = sums[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2 * ROWS; ++i) sums[i] = warp_sum(lane < warps ? part[turn][lane][i] : 0.f);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (in && r0 + i < a.rows) {
                const float rstd = rsqrtf(sums[2 * i] / static_cast<float>(C) + a.eps);
                const float mean = sums[2 * i + 1] * rstd / static_cast<float>(C);   // of t . n
                const long long at = (r0 + i) * C + mine;
                float out[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) out[e] = 0.f;
                if (from[2]) load<8>(reinterpret_cast<const T*>(place(now, i, 2)), out);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = s[i][e] * rstd;
                    acc[e] = fmaf(g[i][e], n, acc[e]);
                    out[e] = fmaf(rstd, g[i][e] * w[e] - n * mean, out[e]);
                }
                if (a.grad_residual) store<8>(static_cast<T*>(a.grad_residual) + at, out);
                if (a.grad_x) store<8>(static_cast<TX*>(a.grad_x) + at, out);
            }
        now = (now + 1) % GROUPS;
    }
    if (shares && in) {
#pragma unroll
        for (int e = 0; e < 8; ++e) shares[static_cast<long long>(blockIdx.x) * C + mine + e] = acc[e];
    }
}

// ---- host --------------------------------------------------------------------

template <typename F>
kdn_status by_dtype(kdn_dtype t, F f) {
    return t == KDN_BF16 ? f(__nv_bfloat16()) : f(float());
}

bool vectors(const NormArgs& a) {
    const void* p[] = {a.x, a.residual, a.weight, a.sum, a.y, a.grad_y, a.grad_sum, a.grad_residual, a.grad_x};
    for (const void* q : p)
        if (reinterpret_cast<uintptr_t>(q) % 16 != 0) return false;
    return a.C % 8 == 0 && a.x_ld % 8 == 0;
}

constexpr long long kMostBlocks = 0x7fffffffLL;

template <int VEC, int NV, typename TX, typename TR, typename TY>
kdn_status launch_fwd(const NormArgs& a, bool alone, int warps, cudaStream_t stream) {
    if (alone) {
        const long long blocks = (a.rows + WARPS - 1) / WARPS;
        if (blocks > kMostBlocks) return KDN_ERR_INVALID_ARG;
        add_norm_kernel<VEC, NV, TX, TR, TY, true><<<static_cast<unsigned>(blocks), WARPS * 32, 0, stream>>>(a);
    } else {
        if (a.rows > kMostBlocks) return KDN_ERR_INVALID_ARG;
        add_norm_kernel<VEC, NV, TX, TR, TY, false><<<static_cast<unsigned>(a.rows), warps * 32, 0, stream>>>(a);
    }
    return from_cuda(cudaGetLastError());
}

// CTAs of the backward: enough to fill the device, each with rows enough.
long long back_blocks(long long rows) {
    const long long want = (rows + 3) / 4, most = static_cast<long long>(sm_count()) * BACK_CTAS;
    return want < most ? want : most;
}

}  // namespace

kdn_status norm_fwd_launch(const NormArgs& a, cudaStream_t stream) {
    if (a.rows == 0) return KDN_OK;
    return by_dtype(a.x_dtype, [&](auto tx) {
        return by_dtype(a.res_dtype, [&](auto tr) {
            using TX = decltype(tx);
            using TR = decltype(tr);
            auto go = [&](auto ty) {
                using TY = decltype(ty);
                if (!vectors(a)) {
                    constexpr int PER = 32 * 16;
                    const int warps = (a.C + PER - 1) / PER;
                    return launch_fwd<1, 16, TX, TR, TY>(a, warps == 1, warps < 32 ? warps : 32, stream);
                }
                // a warp to a row of up to 512, CTAs beyond with 64 bytes a thread (two vectors
                // of 16-bit x, one of fp32): many small CTAs keep the memory busy while others sum (32768 x
                // 2048 bf16: a warp to a row 205 us, eight warps 111 us, four with two vectors 94 us)
                constexpr int PER = 32 * 8;
                const int one = (a.C + PER - 1) / PER, two = (one + 1) / 2;
                if (one == 1) return launch_fwd<8, 1, TX, TR, TY>(a, true, 1, stream);
                if (one == 2 && a.rows >= static_cast<long long>(sm_count()) * WARPS)
                    return launch_fwd<8, 2, TX, TR, TY>(a, true, 1, stream);
                if (one <= 16 && sizeof(TX) == 4) return launch_fwd<8, 1, TX, TR, TY>(a, false, one, stream);
                return launch_fwd<8, 2, TX, TR, TY>(a, false, two < 32 ? two : 32, stream);
            };
            if (a.y_dtype == KDN_E4M3) return go(E4m3());
            return a.y_dtype == KDN_BF16 ? go(__nv_bfloat16()) : go(float());
        });
    });
}

long long norm_bwd_workspace_bytes(long long rows, int C) { return back_blocks(rows) * C * 4; }

kdn_status norm_bwd_launch(const NormArgs& a, cudaStream_t stream) {
    if (a.rows == 0)
        return a.grad_weight ? from_cuda(cudaMemsetAsync(a.grad_weight, 0, sizeof(float) * a.C, stream)) : KDN_OK;
    const long long blocks = back_blocks(a.rows);
    void* mine = nullptr;
    float* shares = nullptr;
    if (a.grad_weight) {
        shares = static_cast<float*>(a.workspace);
        if (!shares) {
            const kdn_status s = from_cuda(cudaMallocAsync(&mine, static_cast<size_t>(norm_bwd_workspace_bytes(a.rows, a.C)), stream));
            if (s != KDN_OK) return s;
            shares = static_cast<float*>(mine);
        }
    }
    kdn_status s = by_dtype(a.x_dtype, [&](auto tx) {
        return by_dtype(a.res_dtype, [&](auto tr) {
            return by_dtype(a.y_dtype, [&](auto ty) {
                using TX = decltype(tx);
                using TR = decltype(tr);
                using TY = decltype(ty);
                if constexpr (sizeof(TR) == 2 && sizeof(TY) == 2) {
                    if (vectors(a) && a.C <= 256 * 8) {
                        const int threads = (a.C / 8 + 31) / 32 * 32;
                        auto kernel = add_norm_back_ring_kernel<TX>;
                        const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), 256 * RING_BYTES);
                        if (e != cudaSuccess) return from_cuda(e);
                        kernel<<<static_cast<unsigned>(blocks), threads, threads * RING_BYTES, stream>>>(a, shares);
                        return from_cuda(cudaGetLastError());
                    }
                }
                auto go = [&](auto vec) {
                    constexpr int VEC = decltype(vec)::value;
                    const int want = (a.C + VEC - 1) / VEC, threads = want < 1024 ? (want + 31) / 32 * 32 : 1024;
                    const int slices = (want + threads - 1) / threads;
                    auto kernel = threads <= 256 ? add_norm_back_kernel<VEC, 256, TX, TR, TY> : add_norm_back_kernel<VEC, 1024, TX, TR, TY>;
                    kernel<<<static_cast<unsigned>(blocks), threads, 0, stream>>>(a, shares, slices);
                    return from_cuda(cudaGetLastError());
                };
                return vectors(a) ? go(std::integral_constant<int, 8>()) : go(std::integral_constant<int, 1>());
            });
        });
    });
    if (s == KDN_OK && shares) s = from_cuda(sum_rows(shares, blocks, a.C, a.grad_weight, nullptr, a.C, stream));
    if (mine) cudaFreeAsync(mine, stream);
    return s;
}

}  // namespace kdn
