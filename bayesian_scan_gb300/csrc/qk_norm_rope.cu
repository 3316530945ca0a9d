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
// HBM bounds both (4 bytes per element forward, 8 backward, bf16 in and
// fp32 gradients).  A lane holds 4 pairs of a head, whichever elements those
// are, so the rotation needs no other lane; dk / 8 lanes hold a head, and a
// warp 32 / (dk / 8) heads side by side, all of one token where there are so
// many.  It keeps the token's cos and sin in registers and walks the heads,
// UNROLL rows' loads in flight; the angles, too dear to take per head, cost
// a tenth of the instructions at 32 heads.
#include <cuda_bf16.h>

#include <cstdint>

#include "gated_device.cuh"
#include "kdn_internal.h"
#include "sum_rows.cuh"

namespace kdn {
namespace {

using gated::from_f32;
using gated::to_f32;

constexpr int WARPS = 8;
constexpr int UNROLL = 4;

// The turns per position of a frequency, f / (2 pi) modulo 1, in 2^-64: the
// double's 53 bits in a 64-bit fraction, whose product with an integer
// position is exact modulo a turn.  The angle is right to 2^-24 turns at the
// farthest position.
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

// What a lane holds of a row: pairs 4l .. 4l + 3 of the dk/2, pair p < rot/2
// being elements (p, p + rot/2) or, interleaved, (2p, 2p + 1), the others
// (2p, 2p + 1).  Where its 8 elements are two aligned groups of 4 (always
// but for a rot that 8 does not divide) they move as vectors.
struct Place {
    int g0, g1;            // the groups' first elements
    bool vec;
    int p0, half;          // first pair, number of rotating pairs
    bool inter;
    __device__ __forceinline__ int first(int i) const {
        return inter || p0 + i >= half ? 2 * (p0 + i) : p0 + i;
    }
    __device__ __forceinline__ int second(int i) const {
        return inter || p0 + i >= half ? 2 * (p0 + i) + 1 : p0 + i + half;
    }
};

template <bool INTER>
__device__ __forceinline__ Place place_of(int l, int rot) {
    Place q;
    q.p0 = 4 * l;
    q.half = rot / 2;
    q.inter = INTER;
    q.vec = INTER || rot % 8 == 0;
    const bool side = INTER || 4 * l >= rot / 2;
    q.g0 = side ? 8 * l : 4 * l;
    q.g1 = side ? 8 * l + 4 : rot / 2 + 4 * l;
    return q;
}

__device__ __forceinline__ void get4(const float* p, float* v) {
    const float4 q = __ldcs(reinterpret_cast<const float4*>(p));
    v[0] = q.x;
    v[1] = q.y;
    v[2] = q.z;
    v[3] = q.w;
}
__device__ __forceinline__ void get4(const __nv_bfloat16* p, float* v) {
    const uint2 q = __ldcs(reinterpret_cast<const uint2*>(p));
    v[0] = __uint_as_float(q.x << 16);
    v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16);
    v[3] = __uint_as_float(q.y & 0xffff0000u);
}
__device__ __forceinline__ void put4(float* p, const float* v) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, const float* v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 q;
    q.x = *reinterpret_cast<const uint32_t*>(&a);
    q.y = *reinterpret_cast<const uint32_t*>(&b);
    __stcs(reinterpret_cast<uint2*>(p), q);
}

// A row's 8 elements, v[i] and v[i + 4] a pair (INTER: v[2i], v[2i + 1]).
template <bool INTER, typename T>
__device__ __forceinline__ void get_row(const T* p, const Place& q, float* v) {
    if (q.vec) {
        get4(p + q.g0, v);
        get4(p + q.g1, v + 4);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = to_f32(p[q.first(i)]);
            v[i + 4] = to_f32(p[q.second(i)]);
        }
    }
}
template <bool INTER, typename T>
__device__ __forceinline__ void put_row(T* p, const Place& q, const float* v) {
    if (q.vec) {
        put4(p + q.g0, v);
        put4(p + q.g1, v + 4);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[q.first(i)] = from_f32<T>(v[i]);
            p[q.second(i)] = from_f32<T>(v[i + 4]);
        }
    }
}
template <bool INTER>
__device__ __forceinline__ constexpr int one(int i) { return INTER ? 2 * i : i; }
template <bool INTER>
__device__ __forceinline__ constexpr int two(int i) { return INTER ? 2 * i + 1 : i + 4; }

// How one call's rows are dealt out: HS heads of a token side by side in a
// warp (TPW = tokens side by side), the heads of a token over `chunks` warps.
struct Deal {
    long long items;       // groups of TPW tokens x chunks
    int HS, chunks;
};

template <int LPR>
struct Lane {
    int l, head, token;    // lane in the row, head and token of the first row (token: in the group)
};

template <int LPR>
__device__ __forceinline__ Lane<LPR> lane_of(int HS) {
    const int lane = threadIdx.x & 31, sub = lane / LPR;
    return Lane<LPR>{lane % LPR, sub % HS, sub / HS};
}

// cos and sin of a lane's 4 pairs at its token.  The HS rows of a token need
// the same ones: with two of them each takes every second pair, with four or
// more each takes one, and the lanes exchange them.
template <int LPR, int M>
__device__ __forceinline__ void angles_shared(const QkArgs& p, const int* pos, long long stride, int l, int sub,
                                              int base, const unsigned long long* per, const int* ax, float2* cs) {
    float2 mine[4 / M];
#pragma unroll
    for (int k = 0; k < 4 / M; ++k) {
        const int i = sub % M + M * k;
        unsigned long long f = per[0];
        int a = ax[0];
#pragma unroll
        for (int j = 1; j < 4; ++j)
            if (i == j) {
                f = per[j];
                a = ax[j];
            }
        mine[k] = cos_sin(pos ? pos[a * stride] : static_cast<int>(stride), f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (M == 1) {
            cs[i] = mine[i];
        } else {
            const int src = (base + i % M) * LPR + l;
            cs[i].x = __shfl_sync(0xffffffffu, mine[i / M].x, src);
            cs[i].y = __shfl_sync(0xffffffffu, mine[i / M].y, src);
        }
    }
}

template <int LPR>
struct Angles {
    unsigned long long per[4];
    int ax[4], half, p0;

    __device__ __forceinline__ void begin(const QkArgs& p, const Place& q) {
        half = q.half;
        p0 = q.p0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            per[i] = 0;
            ax[i] = 0;
            if (p0 + i < half) {
                per[i] = turns_per_position(p.inv_freq[p0 + i]);
                if (p.axis) ax[i] = min(max(p.axis[p0 + i], 0), p.axes - 1);
            }
        }
    }
    // (the whole warp; a lane without a token passes any valid one)
    __device__ __forceinline__ void at(const QkArgs& p, long long token, int HS, int l, float2* cs) const {
        const int sub = (threadIdx.x & 31) / LPR, base = sub / HS * HS;
        const long long n = static_cast<long long>(p.B) * p.T;
        const int* pos = p.pos ? p.pos + token : nullptr;
        const long long stride = p.pos ? n : token % p.T;
        if (HS >= 4) angles_shared<LPR, 4>(p, pos, stride, l, sub, base, per, ax, cs);
        else if (HS == 2) angles_shared<LPR, 2>(p, pos, stride, l, sub, base, per, ax, cs);
        else angles_shared<LPR, 1>(p, pos, stride, l, sub, base, per, ax, cs);
        // pairs behind rot have no frequency: per = 0, cos = 1, sin = 0
    }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int DK>
__device__ __forceinline__ float inverse_norm(const QkArgs& p, float ss) {
    if (p.norm == KDN_NORM_NONE) return 1.f;
    return rsqrtf((p.norm == KDN_NORM_RMS ? ss * (1.f / DK) : ss) + p.eps);
}

template <typename TI, typename TO, int DK, bool INTER>
__global__ void __launch_bounds__(WARPS * 32) qk_fwd_kernel(const QkArgs p, const Deal deal) {
    constexpr int LPR = DK / 8, RPW = 32 / LPR;
    const long long item = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
    if (item >= deal.items) return;
    const int HS = deal.HS, tpw = RPW / HS;
    const Lane<LPR> ln = lane_of<LPR>(HS);
    const long long tokens = static_cast<long long>(p.B) * p.T;
    const long long group = item / deal.chunks;
    const int chunk = static_cast<int>(item - group * deal.chunks);
    long long token = group * tpw + ln.token;
    const bool here = token < tokens;
    if (!here) token = tokens - 1;
    const long long b = token / p.T;
    const int t = static_cast<int>(token - b * p.T);
    const Place q = place_of<INTER>(ln.l, p.rot);
    float2 cs[4];
    if (p.rot > 0) {
        Angles<LPR> an;
        an.begin(p, q);
        an.at(p, token, HS, ln.l, cs);
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const int H = p.heads[which];
        if (H == 0) continue;
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.f;
        if (p.w[which]) get_row<INTER>(p.w[which], q, w);
        // this warp's heads: every chunks-th group of HS
        const TI* x = static_cast<const TI*>(p.x[which]) + token * p.ld[which];
        TO* y = static_cast<TO*>(p.y[which]) + (b * H * p.T + t) * DK;
        const long long ystep = static_cast<long long>(p.T) * DK;
        const int step = HS * deal.chunks;
        for (int h0 = chunk * HS + ln.head; h0 - ln.head < H; h0 += UNROLL * step) {
            float v[UNROLL][8];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int h = h0 + u * step;
                if (here && h < H) {
                    get_row<INTER>(x + h * DK, q, v[u]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int h = h0 + u * step;
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(v[u][i], v[u][i], ss);
                const float r = inverse_norm<DK>(p, row_sum<LPR>(ss));
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= r * w[i];
                if (p.rot > 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float y1 = v[u][one<INTER>(i)], y2 = v[u][two<INTER>(i)];
                        v[u][one<INTER>(i)] = fmaf(y1, cs[i].x, -y2 * cs[i].y);
                        v[u][two<INTER>(i)] = fmaf(y1, cs[i].y, y2 * cs[i].x);
                    }
                }
                if (here && h < H) put_row<INTER>(y + h * ystep, q, v[u]);
            }
        }
    }
}

// Backward.  A persistent grid, so that few blocks' shares of the weights'
// gradients are left to add: part [block][2 dk], q's then k's.
template <typename TI, typename TO, int DK, bool INTER>
__global__ void __launch_bounds__(WARPS * 32) qk_bwd_kernel(const QkArgs p, const Deal deal, float* part) {
    constexpr int LPR = DK / 8, RPW = 32 / LPR, UNR = 2;
    __shared__ float share[WARPS][DK];
    const int warp = threadIdx.x >> 5;
    const int HS = deal.HS, tpw = RPW / HS;
    const Lane<LPR> ln = lane_of<LPR>(HS);
    const long long tokens = static_cast<long long>(p.B) * p.T;
    const Place q = place_of<INTER>(ln.l, p.rot);
    const float inv_n = p.norm == KDN_NORM_RMS ? 1.f / DK : 1.f;
    Angles<LPR> an;
    if (p.rot > 0) an.begin(p, q);
    float dw[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;

    for (long long item = static_cast<long long>(blockIdx.x) * WARPS + warp; item < deal.items;
         item += static_cast<long long>(gridDim.x) * WARPS) {
        const long long group = item / deal.chunks;
        const int chunk = static_cast<int>(item - group * deal.chunks);
        long long token = group * tpw + ln.token;
        const bool here = token < tokens;
        if (!here) token = tokens - 1;
        const long long b = token / p.T;
        const int t = static_cast<int>(token - b * p.T);
        float2 cs[4];
        if (p.rot > 0) an.at(p, token, HS, ln.l, cs);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int H = p.heads[which];
            if (H == 0) continue;
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 1.f;
            if (p.w[which]) get_row<INTER>(p.w[which], q, w);
            const TI* x = static_cast<const TI*>(p.x[which]) + token * p.ld[which];
            TI* gx = static_cast<TI*>(p.grad_x[which]) + token * p.grad_ld[which];
            const TO* gy = static_cast<const TO*>(p.grad_y[which]) + (b * H * p.T + t) * DK;
            const long long ystep = static_cast<long long>(p.T) * DK;
            const int step = HS * deal.chunks;
            for (int h0 = chunk * HS + ln.head; h0 - ln.head < H; h0 += UNR * step) {
                float v[UNR][8], g[UNR][8];
#pragma unroll
                for (int u = 0; u < UNR; ++u) {
                    const int h = h0 + u * step;
                    if (here && h < H) {
                        get_row<INTER>(x + h * DK, q, v[u]);
                        get_row<INTER>(gy + h * ystep, q, g[u]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[u][i] = g[u][i] = 0.f;
                    }
                }
#pragma unroll
                for (int u = 0; u < UNR; ++u) {
                    const int h = h0 + u * step;
                    if (p.rot > 0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float g1 = g[u][one<INTER>(i)], g2 = g[u][two<INTER>(i)];
                            g[u][one<INTER>(i)] = fmaf(g1, cs[i].x, g2 * cs[i].y);
                            g[u][two<INTER>(i)] = fmaf(g2, cs[i].x, -g1 * cs[i].y);
                        }
                    }
                    float ss = 0.f, tx = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        ss = fmaf(v[u][i], v[u][i], ss);
                        tx = fmaf(v[u][i], g[u][i] * w[i], tx);
                    }
                    const float r = inverse_norm<DK>(p, row_sum<LPR>(ss));
                    const float back = p.norm == KDN_NORM_NONE ? 0.f : r * r * r * row_sum<LPR>(tx) * inv_n;
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float rg = r * g[u][i];
                        dw[which][i] = fmaf(v[u][i], rg, dw[which][i]);
                        o[i] = fmaf(rg, w[i], -v[u][i] * back);
                    }
                    if (here && h < H) put_row<INTER>(gx + h * DK, q, o);
                }
            }
        }
    }
    if (!part) return;
    // the rows side by side in a warp, then the warps, in order
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s = dw[which][i];
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if ((threadIdx.x & 31) < LPR) {
                const int j = INTER ? 8 * ln.l + i : i < 4 ? q.first(i) : q.second(i - 4);
                // vectors' groups are elements in order
                share[warp][q.vec ? (i < 4 ? q.g0 + i : q.g1 + i - 4) : j] = s;
            }
        }
        __syncthreads();
        for (int j = threadIdx.x; j < DK; j += WARPS * 32) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) s += share[k][j];
            part[(static_cast<long long>(blockIdx.x) * 2 + which) * DK + j] = s;
        }
        __syncthreads();
    }
}

constexpr int BWD_BLOCKS_PER_SM = 2;

// Heads side by side: a power of two, as many as a warp takes and there are.
// Few tokens' heads are dealt to more warps, so that every SM has some.
Deal deal_of(long long tokens, int Hq, int Hk, int dk) {
    const int rpw = 32 / (dk / 8), heads = Hq > Hk ? Hq : Hk;
    Deal d{0, 1, 1};
    while (d.HS < rpw && d.HS < heads) d.HS *= 2;
    const int tpw = rpw / d.HS, groups = (heads + d.HS - 1) / d.HS;
    d.items = (tokens + tpw - 1) / tpw;
    const long long want = static_cast<long long>(sm_count()) * WARPS * 2;
    while (d.chunks < groups && d.items * d.chunks < want) d.chunks *= 2;
    d.items *= d.chunks;
    return d;
}

int bwd_blocks(int B, int T, int Hq, int Hk, int dk) {
    const long long items = deal_of(static_cast<long long>(B) * T, Hq, Hk, dk).items;
    const long long blocks = (items + WARPS - 1) / WARPS, cap = static_cast<long long>(sm_count()) * BWD_BLOCKS_PER_SM;
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
    return static_cast<long long>(bwd_blocks(B, T, Hq, Hk, dk)) * 2 * dk * 4;
}

kdn_status qk_fwd_launch(const QkArgs& a, cudaStream_t stream) {
    const Deal deal = deal_of(static_cast<long long>(a.B) * a.T, a.heads[0], a.heads[1], a.dk);
    const long long blocks = (deal.items + WARPS - 1) / WARPS;
    if (blocks > 0x7fffffffLL) return KDN_ERR_INVALID_ARG;
    return by_type(a, [&](auto ti, auto to) {
        return by_dk(a.dk, [&](auto n) {
            using TI = decltype(ti);
            using TO = decltype(to);
            constexpr int DK = decltype(n)::value;
            if (a.interleaved)
                qk_fwd_kernel<TI, TO, DK, true><<<static_cast<unsigned>(blocks), WARPS * 32, 0, stream>>>(a, deal);
            else
                qk_fwd_kernel<TI, TO, DK, false><<<static_cast<unsigned>(blocks), WARPS * 32, 0, stream>>>(a, deal);
            return from_cuda(cudaGetLastError());
        });
    });
}

kdn_status qk_bwd_launch(const QkArgs& a, cudaStream_t stream) {
    const int Hq = a.heads[0], Hk = a.heads[1];
    const Deal deal = deal_of(static_cast<long long>(a.B) * a.T, Hq, Hk, a.dk);
    const int blocks = bwd_blocks(a.B, a.T, Hq, Hk, a.dk);
    const bool dw = a.grad_w[0] || a.grad_w[1];
    float* part = dw ? static_cast<float*>(a.workspace) : nullptr;
    if (dw && !part) {
        const kdn_status s = from_cuda(cudaMallocAsync(&part, qk_bwd_workspace_bytes(a.B, a.T, Hq, Hk, a.dk), stream));
        if (s != KDN_OK) return s;
    }
    kdn_status s = by_type(a, [&](auto ti, auto to) {
        return by_dk(a.dk, [&](auto n) {
            using TI = decltype(ti);
            using TO = decltype(to);
            constexpr int DK = decltype(n)::value;
            if (a.interleaved) qk_bwd_kernel<TI, TO, DK, true><<<blocks, WARPS * 32, 0, stream>>>(a, deal, part);
            else qk_bwd_kernel<TI, TO, DK, false><<<blocks, WARPS * 32, 0, stream>>>(a, deal, part);
            return from_cuda(cudaGetLastError());
        });
    });
    if (s == KDN_OK && dw)
        s = from_cuda(sum_rows(part, blocks, 2 * a.dk, a.grad_w[0], a.grad_w[1], a.dk, stream));
    if (part && part != a.workspace) {
        const kdn_status f = from_cuda(cudaFreeAsync(part, stream));
        if (s == KDN_OK) s = f;
    }
    return s;
}

}  // namespace kdn
