// qk_norm_rope.cu -- queries and keys for the scans from the rows of a
// projection: norm of every head, weight, position rotation, and the scans'
// [B,H,T,dk] layout, in one pass; and the backward pass.
//
//     r = (sum x^2 / n + eps)^(-1/2)   (n = dk: rms, 1: l2; no norm: r = 1)
//     y = r x w;   (o1, o2) = (y1 cos - y2 sin, y1 sin + y2 cos)
// with theta = pos inv_freq of the pair's axis.  Backward, g the transposed
// rotation of the incoming gradient and t = g w:
//     grad x = r t - r^3 x (sum t x) / n,   grad w = sum over rows of r x g.
//
// A warp takes one head of one token at a time.
#include <cuda_bf16.h>

#include <cstdint>

#include "gated_device.cuh"
#include "kdn_internal.h"

namespace kdn {
namespace {

using gated::from_f32;
using gated::to_f32;

constexpr int WARPS = 8;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// cos and sin of pos * f, in 64-bit fixed-point turns: f / (2 pi) keeps 53
// bits, the product with an integer position is exact modulo a turn, so the
// angle is right to 2^-24 turns at the farthest position.
__device__ __forceinline__ unsigned long long turns_per_position(float f) {
    double t = static_cast<double>(f) * 0.15915494309189533577;
    t -= floor(t);
    return static_cast<unsigned long long>(t * 18446744073709551616.0);
}

__device__ __forceinline__ float2 cos_sin(int pos, unsigned long long per) {
    const unsigned long long ph = static_cast<unsigned long long>(static_cast<long long>(pos)) * per;
    const int half = static_cast<int>(ph >> 32);   // in 2^-32 turns, [-1/2, 1/2)
    float s, c;
    sincospif(static_cast<float>(half) * 4.656612873077392578125e-10f, &s, &c);   // 2^-31: half turns
    return make_float2(c, s);
}

struct Row {
    int which, h;          // q or k, head
    long long b;
    int t;
    long long token;
};

__device__ __forceinline__ Row row_of(const QkArgs& p, long long r) {
    const int heads = p.heads[0] + p.heads[1];
    Row w;
    w.token = r / heads;
    w.h = static_cast<int>(r - w.token * heads);
    w.which = w.h >= p.heads[0];
    if (w.which) w.h -= p.heads[0];
    w.b = w.token / p.T;
    w.t = static_cast<int>(w.token - w.b * p.T);
    return w;
}

__device__ __forceinline__ float2 rotation(const QkArgs& p, const Row& w, int pair) {
    int ax = p.axis ? p.axis[pair] : 0;
    ax = min(max(ax, 0), p.axes - 1);
    const int pos = p.pos ? p.pos[(static_cast<long long>(ax) * p.B + w.b) * p.T + w.t] : w.t;
    return cos_sin(pos, turns_per_position(p.inv_freq[pair]));
}

// The partner of element j and the sign its sine takes in the forward.
__device__ __forceinline__ void partner(const QkArgs& p, int j, int* other, int* pair, float* sign) {
    const int half = p.rot / 2;
    if (p.interleaved) {
        *other = j ^ 1;
        *pair = j >> 1;
        *sign = j & 1 ? 1.f : -1.f;
    } else {
        *other = j < half ? j + half : j - half;
        *pair = j < half ? j : j - half;
        *sign = j < half ? -1.f : 1.f;
    }
}

template <typename TI, typename TO, int DK>
__global__ void __launch_bounds__(WARPS * 32) qk_fwd_kernel(QkArgs p) {
    __shared__ float y[WARPS][DK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long rows = static_cast<long long>(p.B) * p.T * (p.heads[0] + p.heads[1]);
    for (long long r = static_cast<long long>(blockIdx.x) * WARPS + warp; r < rows;
         r += static_cast<long long>(gridDim.x) * WARPS) {
        const Row w = row_of(p, r);
        const TI* x = static_cast<const TI*>(p.x[w.which]) + w.token * p.ld[w.which] + w.h * DK;
        const float* wt = p.w[w.which];
        float ss = 0.f;
        for (int j = lane; j < DK; j += 32) {
            const float v = to_f32(x[j]);
            ss = fmaf(v, v, ss);
        }
        ss = warp_sum(ss);
        const float rn = p.norm == KDN_NORM_NONE ? 1.f
                         : rsqrtf((p.norm == KDN_NORM_RMS ? ss / DK : ss) + p.eps);
        for (int j = lane; j < DK; j += 32) y[warp][j] = to_f32(x[j]) * rn * (wt ? wt[j] : 1.f);
        __syncwarp();
        TO* o = static_cast<TO*>(p.y[w.which]) +
                ((w.b * p.heads[w.which] + w.h) * p.T + w.t) * DK;
        for (int j = lane; j < DK; j += 32) {
            float v = y[warp][j];
            if (j < p.rot) {
                int other, pair;
                float sign;
                partner(p, j, &other, &pair, &sign);
                const float2 cs = rotation(p, w, pair);
                v = fmaf(sign * cs.y, y[warp][other], v * cs.x);
            }
            o[j] = from_f32<TO>(v);
        }
        __syncwarp();
    }
}

template <typename TI, typename TO, int DK>
__global__ void __launch_bounds__(WARPS * 32) qk_bwd_kernel(QkArgs p, float* part) {
    constexpr int PER = (DK + 31) / 32;
    __shared__ float y[WARPS][DK];
    __shared__ float acc[WARPS][2][DK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long rows = static_cast<long long>(p.B) * p.T * (p.heads[0] + p.heads[1]);
    for (int j = lane; j < DK; j += 32) acc[warp][0][j] = acc[warp][1][j] = 0.f;
    for (long long r = static_cast<long long>(blockIdx.x) * WARPS + warp; r < rows;
         r += static_cast<long long>(gridDim.x) * WARPS) {
        const Row w = row_of(p, r);
        const TI* x = static_cast<const TI*>(p.x[w.which]) + w.token * p.ld[w.which] + w.h * DK;
        const TO* go = static_cast<const TO*>(p.grad_y[w.which]) +
                       ((w.b * p.heads[w.which] + w.h) * p.T + w.t) * DK;
        const float* wt = p.w[w.which];
        for (int j = lane; j < DK; j += 32) y[warp][j] = to_f32(go[j]);
        __syncwarp();
        float g[PER], xs[PER], ss = 0.f, tx = 0.f;
        for (int j = lane, i = 0; j < DK; j += 32, ++i) {
            float v = y[warp][j];
            if (j < p.rot) {
                int other, pair;
                float sign;
                partner(p, j, &other, &pair, &sign);
                const float2 cs = rotation(p, w, pair);
                v = fmaf(-sign * cs.y, y[warp][other], v * cs.x);
            }
            g[i] = v;
            xs[i] = to_f32(x[j]);
            ss = fmaf(xs[i], xs[i], ss);
            tx = fmaf(xs[i], v * (wt ? wt[j] : 1.f), tx);
        }
        ss = warp_sum(ss);
        tx = warp_sum(tx);
        const float n = p.norm == KDN_NORM_RMS ? 1.f / DK : 1.f;
        const float rn = p.norm == KDN_NORM_NONE ? 1.f : rsqrtf(ss * n + p.eps);
        const float back = p.norm == KDN_NORM_NONE ? 0.f : rn * rn * rn * tx * n;
        TI* gx = static_cast<TI*>(p.grad_x[w.which]) + w.token * p.grad_ld[w.which] + w.h * DK;
        for (int j = lane, i = 0; j < DK; j += 32, ++i) {
            gx[j] = from_f32<TI>(rn * g[i] * (wt ? wt[j] : 1.f) - xs[i] * back);
            acc[warp][w.which][j] += rn * xs[i] * g[i];
        }
        __syncwarp();
    }
    __syncthreads();
    if (part)
        for (int j = threadIdx.x; j < 2 * DK; j += WARPS * 32) {
            float s = 0.f;
            for (int k = 0; k < WARPS; ++k) s += acc[k][j / DK][j % DK];
            part[static_cast<long long>(blockIdx.x) * 2 * DK + j] = s;
        }
}

__global__ void qk_dw_kernel(const float* __restrict__ part, int blocks, int dk, float* gwq, float* gwk) {
    const int j = threadIdx.x;
    float s = 0.f;
    for (int b = 0; b < blocks; ++b) s += part[static_cast<long long>(b) * 2 * dk + j];
    if (j < dk) {
        if (gwq) gwq[j] = s;
    } else if (gwk) {
        gwk[j - dk] = s;
    }
}

int qk_blocks(int B, int T, int Hq, int Hk) {
    const long long rows = static_cast<long long>(B) * T * (Hq + Hk);
    const long long blocks = (rows + WARPS - 1) / WARPS, cap = static_cast<long long>(sm_count()) * 8;
    return static_cast<int>(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
}

template <typename F>
kdn_status by_type(const QkArgs& a, F f) {
    if (a.in_dtype == KDN_BF16)
        return a.out_dtype == KDN_BF16 ? f(__nv_bfloat16(), __nv_bfloat16()) : f(__nv_bfloat16(), float());
    return a.out_dtype == KDN_BF16 ? f(float(), __nv_bfloat16()) : f(float(), float());
}

template <int N>
struct Int {
    static constexpr int value = N;
};

template <typename F>
kdn_status by_dk(int dk, F f) {
    switch (dk) {
        case 16: return f(Int<16>());
        case 32: return f(Int<32>());
        case 64: return f(Int<64>());
        default: return f(Int<128>());
    }
}

}  // namespace

long long qk_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int dk) {
    return static_cast<long long>(qk_blocks(B, T, Hq, Hk)) * 2 * dk * 4;
}

kdn_status qk_fwd_launch(const QkArgs& a, cudaStream_t stream) {
    const int blocks = qk_blocks(a.B, a.T, a.heads[0], a.heads[1]);
    return by_type(a, [&](auto ti, auto to) {
        return by_dk(a.dk, [&](auto n) {
            qk_fwd_kernel<decltype(ti), decltype(to), decltype(n)::value>
                <<<blocks, WARPS * 32, 0, stream>>>(a);
            return from_cuda(cudaGetLastError());
        });
    });
}

kdn_status qk_bwd_launch(const QkArgs& a, cudaStream_t stream) {
    const int blocks = qk_blocks(a.B, a.T, a.heads[0], a.heads[1]);
    const bool dw = a.grad_w[0] || a.grad_w[1];
    float* part = dw ? static_cast<float*>(a.workspace) : nullptr;
    if (dw && !part) {
        const kdn_status s = from_cuda(cudaMallocAsync(
            &part, qk_bwd_workspace_bytes(a.B, a.T, a.heads[0], a.heads[1], a.dk), stream));
        if (s != KDN_OK) return s;
    }
    kdn_status s = by_type(a, [&](auto ti, auto to) {
        return by_dk(a.dk, [&](auto n) {
            qk_bwd_kernel<decltype(ti), decltype(to), decltype(n)::value>
                <<<blocks, WARPS * 32, 0, stream>>>(a, part);
            return from_cuda(cudaGetLastError());
        });
    });
    if (s == KDN_OK && dw) {
        qk_dw_kernel<<<1, 2 * a.dk, 0, stream>>>(part, blocks, a.dk, a.grad_w[0], a.grad_w[1]);
        s = from_cuda(cudaGetLastError());
    }
    if (part && part != a.workspace) {
        const kdn_status f = from_cuda(cudaFreeAsync(part, stream));
        if (s == KDN_OK) s = f;
    }
    return s;
}

}  // namespace kdn
