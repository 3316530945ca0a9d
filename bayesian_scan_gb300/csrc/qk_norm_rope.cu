// qk_norm_rope.cu -- queries and keys for the scans from the rows of a
// projection: norm of every head, weight, position rotation, and the scans'
// [B,H,T,dk] layout, in one pass; and the backward pass.
//
//     r = (sum x^2 / n + eps)^(-1/2)   (n = dk: rms, 1: l2; no norm: r = 1)
//     y = r x w;   (o1, o2) = (y1 cos - y2 sin, y1 sin + y2 cos)
// with theta = pos inv_freq of the pair's axis.  Backward, g the transposed
// rotation of the incoming gradient and t = g w:
//     grad x = r (t - r x (r sum t x) / n),   grad w = sum over rows of r x g
// (r x is of order one; an r^3 would leave fp32 where rows are of 1e13 or 1e-13).
//
// HBM bounds both (4 bytes per element forward, 8 backward, bf16 in and
// fp32 gradients).  A lane holds 4 pairs of a head, whichever elements those
// are, so the rotation needs no other lane; dk / 8 lanes hold a head, and a
// warp 32 / (dk / 8) heads side by side, all of one token where there are so
// many.  It keeps the token's cos and sin in registers and walks the heads,
// a few rows' loads in flight.
#include <cuda_bf16.h>

#include <cfloat>
#include <cstdint>

#include "gated_device.cuh"
#include "kdn_device.cuh"
#include "kdn_internal.h"
#include "kernel_setup.h"
#include "sum_rows.cuh"

namespace kdn {
namespace {

using namespace gated;

constexpr int WARPS = 8;
constexpr int SEG = 4096, SEG_DEPTH = 2;   // bytes of a bulk copy, copies in flight per warp

__device__ int g_qk_error = 0;
constexpr int FWD_BLOCKS_PER_SM = 3, BWD_BLOCKS_PER_SM = 2, BWD_DEPTH = 4;

// The turns per position of a frequency, f / (2 pi) modulo 1, in 2^-64, and
// within two of them up to |f| = 2^40: f times 1 / (2 pi) as a double and what
// that leaves out, the first product's whole turns dropped before its rounding
// error is added.  The product with an integer position is exact modulo a
// turn, so the angle of the farthest position is within 2^-32 turns.
__device__ __forceinline__ unsigned long long turns_per_position(float f) {
    constexpr double HI = 0.15915494309189535, LO = -9.839338337591243e-18;
    const double g = fabsf(f), t = __dmul_rn(g, HI), rest = __fma_rn(g, LO, __fma_rn(g, HI, -t));
    const unsigned long long turns = static_cast<unsigned long long>((t - floor(t)) * 0x1p64) +   // (exact for t >= 0)
                                     static_cast<unsigned long long>(__double2ll_rn(rest * 0x1p64));
    return f < 0.f ? 0ull - turns : turns;
}

// Reduced to an eighth of a turn either side of the nearest quarter, all 64
// bits of it (a slow frequency's sine is its angle), x in [-1, 1] eighths:
// sin(x pi/4) = x S(x^2), cos(x pi/4) = C(x^2), S and C the Chebyshev
// interpolants of degree 3 and 4 on [0, 1] (both within 2^-23.5).  Both are
// within 6 half steps of themselves for the angle that they are given.
__device__ __forceinline__ float2 cos_sin(int pos, unsigned long long per) {
    const unsigned long long ph = static_cast<unsigned long long>(static_cast<long long>(pos)) * per;
    const unsigned int quarter = (static_cast<unsigned int>(ph >> 32) + 0x20000000u) >> 30;
    const float x = static_cast<float>(static_cast<long long>(ph - (static_cast<unsigned long long>(quarter) << 62))) * 0x1p-61f;
    const float u = x * x;
    float s = -3.595429006963968e-05f;
    s = fmaf(s, u, 0.0024900068528950214f);
    s = fmaf(s, u, -0.08074543625116348f);
    s = fmaf(s, u, 0.7853981852531433f);
    s *= x;
    float c = 3.5297971407999285e-06f;
    c = fmaf(c, u, -0.0003259385994169861f);
    c = fmaf(c, u, 0.015854325145483017f);
    c = fmaf(c, u, -0.3084251284599304f);
    c = fmaf(c, u, 1.f);
    const bool swap = quarter & 1;
    const float co = swap ? s : c, si = swap ? c : s;
    return make_float2(__uint_as_float(__float_as_uint(co) ^ ((quarter + 1) & 2) << 30),
                       __uint_as_float(__float_as_uint(si) ^ (quarter & 2) << 30));
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

// A row's 8 elements: the pairs' first elements in a, their second in b.
struct Row8 {
    F2 a[2], b[2];
};

// The same as loaded: one or two 4-element groups.
template <typename T>
struct Raw4;
template <>
struct Raw4<float> {
    float4 r;
    __device__ __forceinline__ float get(int i) const { return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w; }
    __device__ __forceinline__ void set(float a, float b, float c, float d) { r = make_float4(a, b, c, d); }
};
template <>
struct Raw4<__nv_bfloat16> {
    uint2 r;
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 2 ? r.x : r.y;
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
    __device__ __forceinline__ void set(float a, float b, float c, float d) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(a, b), q = __floats2bfloat162_rn(c, d);
        r.x = *reinterpret_cast<const uint32_t*>(&p);
        r.y = *reinterpret_cast<const uint32_t*>(&q);
    }
};
template <typename T>
struct RawRow {
    Raw4<T> u, v;
};

template <typename T>
__device__ __forceinline__ RawRow<T> get_raw(const T* p, const Place& q) {
    RawRow<T> r;
    if (q.vec) {
        r.u.r = __ldcs(reinterpret_cast<const decltype(r.u.r)*>(p + q.g0));
        r.v.r = __ldcs(reinterpret_cast<const decltype(r.v.r)*>(p + q.g1));
    } else {   // (never interleaved) pair by pair
        r.u.set(to_f32(p[q.first(0)]), to_f32(p[q.first(1)]), to_f32(p[q.first(2)]), to_f32(p[q.first(3)]));
        r.v.set(to_f32(p[q.second(0)]), to_f32(p[q.second(1)]), to_f32(p[q.second(2)]), to_f32(p[q.second(3)]));
    }
    return r;
}

template <bool INTER, typename T>
__device__ __forceinline__ Row8 row_of(const RawRow<T>& r) {
    Row8 o;
    if (INTER) {
        o.a[0] = F2{r.u.get(0), r.u.get(2)};
        o.b[0] = F2{r.u.get(1), r.u.get(3)};
        o.a[1] = F2{r.v.get(0), r.v.get(2)};
        o.b[1] = F2{r.v.get(1), r.v.get(3)};
    } else {
        o.a[0] = F2{r.u.get(0), r.u.get(1)};
        o.a[1] = F2{r.u.get(2), r.u.get(3)};
        o.b[0] = F2{r.v.get(0), r.v.get(1)};
        o.b[1] = F2{r.v.get(2), r.v.get(3)};
    }
    return o;
}

template <bool INTER, typename T>
__device__ __forceinline__ void put_row(T* p, const Place& q, const Row8& o) {
    RawRow<T> r;
    if (INTER) {
        r.u.set(o.a[0].x, o.b[0].x, o.a[0].y, o.b[0].y);
        r.v.set(o.a[1].x, o.b[1].x, o.a[1].y, o.b[1].y);
    } else {
        r.u.set(o.a[0].x, o.a[0].y, o.a[1].x, o.a[1].y);
        r.v.set(o.b[0].x, o.b[0].y, o.b[1].x, o.b[1].y);
    }
    if (q.vec) {
        __stcs(reinterpret_cast<decltype(r.u.r)*>(p + q.g0), r.u.r);
        __stcs(reinterpret_cast<decltype(r.v.r)*>(p + q.g1), r.v.r);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[q.first(i)] = from_f32<T>(r.u.get(i));
            p[q.second(i)] = from_f32<T>(r.v.get(i));
        }
    }
}

__device__ __forceinline__ Row8 times(const Row8& x, const Row8& y) {
    return Row8{{mul2(x.a[0], y.a[0]), mul2(x.a[1], y.a[1])}, {mul2(x.b[0], y.b[0]), mul2(x.b[1], y.b[1])}};
}

__device__ __forceinline__ F2 neg2(F2 v) { return F2{-v.x, -v.y}; }

// Rotation by the pairs' angles, c and s each (pair 0, pair 1), (pair 2, pair 3).
struct Turn {
    F2 c[2], s[2];
};
// Pairs behind rot have cos = 1 and sin = 0, whose product with an infinite or
// NaN element is NaN for its partner.  EXACT leaves those pairs as they are.
//
// Calls that rotate part of a head have kernels of their own (PART) that go
// over rows again, exactly, that turn out to hold other than numbers: in one
// kernel for all calls this cost the layer 90 -> 91 us and its backward 176 ->
// 183, selects in every row 94 and 182.
template <bool BACK, bool EXACT>
__device__ __forceinline__ void rotate(Row8& v, const Turn& t, const Place& q) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const F2 s = BACK ? neg2(t.s[i]) : t.s[i];
        const F2 a = fma2(v.a[i], t.c[i], neg2(mul2(v.b[i], s))), b = fma2(v.a[i], s, mul2(v.b[i], t.c[i]));
        const bool x = !EXACT || q.p0 + 2 * i < q.half, y = !EXACT || q.p0 + 2 * i + 1 < q.half;
        v.a[i] = F2{x ? a.x : v.a[i].x, y ? a.y : v.a[i].y};
        v.b[i] = F2{x ? b.x : v.b[i].x, y ? b.y : v.b[i].y};
    }
}

template <bool INTER>
__device__ __forceinline__ Row8 weight_of(const float* w, const Place& q) {
    if (!w) return Row8{{both(1.f), both(1.f)}, {both(1.f), both(1.f)}};
    return row_of<INTER>(get_raw(w, q));
}

// The sum of squares up to which a row's elements, each times its weight, are
// numbers: any (of less than 2^64, then) unless a weight is 2^63 or more.
template <bool INTER>
__device__ __forceinline__ float most_squares(const QkArgs& p, const Place& q) {
    float most = FLT_MAX;
    for (const float* w : p.w) {
        if (!w) continue;
        const Row8 r = weight_of<INTER>(w, q);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (!(fabsf(r.a[i].x) < 0x1p63f && fabsf(r.a[i].y) < 0x1p63f && fabsf(r.b[i].x) < 0x1p63f &&
                  fabsf(r.b[i].y) < 0x1p63f))
                most = -1.f;
    }
    return most;
}

// How one call's rows are dealt out: HS heads of a token side by side in a
// warp (TPW = tokens side by side), the heads of a token over `chunks` warps.
struct Deal {
    long long items;       // groups of TPW tokens x chunks
    int HS, chunks;
};

// The frequencies of a call in shared memory: turns per position and axis of
// every pair; pairs behind rot have neither (cos = 1, sin = 0).
template <int DK>
struct Freqs {
    unsigned long long per[DK / 2];
    int ax[DK / 2];

    __device__ __forceinline__ void fill(const QkArgs& p) {
        for (int i = threadIdx.x; i < DK / 2; i += blockDim.x) {
            per[i] = 0;
            ax[i] = 0;
            if (2 * i < p.rot) {
                per[i] = turns_per_position(p.inv_freq[i]);
                if (p.axis) ax[i] = min(max(p.axis[i], 0), p.axes - 1);
            }
        }
        __syncthreads();
    }
};

// cos and sin of a lane's 4 pairs at its token.  The HS rows of a token need
// the same ones: with two of them each takes every second pair, with four or
// more each takes one, and the lanes exchange them.
template <int DK, int M>
__device__ __forceinline__ Turn turn_shared(const Freqs<DK>& f, const int* pos, long long stride, int t, int l, int sub,
                                            int base) {
    constexpr int LPR = DK / 8;
    float2 mine[4 / M], cs[4];
#pragma unroll
    for (int k = 0; k < 4 / M; ++k) {
        const int i = 4 * l + sub % M + M * k;
        mine[k] = cos_sin(pos ? pos[f.ax[i] * stride] : t, f.per[i]);
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
    return Turn{{F2{cs[0].x, cs[1].x}, F2{cs[2].x, cs[3].x}}, {F2{cs[0].y, cs[1].y}, F2{cs[2].y, cs[3].y}}};
}

// (the whole warp; a lane without a token passes any valid one)
template <int DK>
__device__ __forceinline__ Turn turn_at(const Freqs<DK>& f, const QkArgs& p, long long token, int t, int HS, int l) {
    if (p.rot == 0) return Turn{{both(1.f), both(1.f)}, {both(0.f), both(0.f)}};
    const int sub = (threadIdx.x & 31) / (DK / 8), base = sub / HS * HS;
    const long long n = static_cast<long long>(p.B) * p.T;
    const int* pos = p.pos ? p.pos + token : nullptr;
    if (HS >= 4) return turn_shared<DK, 4>(f, pos, n, t, l, sub, base);
    if (HS == 2) return turn_shared<DK, 2>(f, pos, n, t, l, sub, base);
    return turn_shared<DK, 1>(f, pos, n, t, l, sub, base);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum of products of two rows' elements over the row's lanes.
template <int LPR>
__device__ __forceinline__ float row_dot(const Row8& x, const Row8& y) {
    const F2 s = fma2(x.a[0], y.a[0], fma2(x.a[1], y.a[1], fma2(x.b[0], y.b[0], mul2(x.b[1], y.b[1]))));
    return row_sum<LPR>(s.x + s.y);
}

template <int DK>
__device__ __forceinline__ float inverse_norm(const QkArgs& p, float ss) {
    if (p.norm == KDN_NORM_NONE) return 1.f;
    return rsqrtf((p.norm == KDN_NORM_RMS ? ss * (1.f / DK) : ss) + p.eps);
}

// A warp's place in a call: an item is a group of tokens and a share of their
// heads, every chunks-th step of HS heads, the queries' and then the keys'.
template <int DK>
struct Place2 {
    static constexpr int LPR = DK / 8, RPW = 32 / LPR;
    int l, sub, t, b, n0, n, h;   // steps of the queries' heads, of both; first head of the lane
    long long token;
    bool here;

    __device__ __forceinline__ Place2() : l(threadIdx.x % 32 % LPR), sub(threadIdx.x % 32 / LPR) {}
    __device__ __forceinline__ void at(const QkArgs& p, const Deal& d, long long item) {
        const long long group = item / d.chunks, tokens = static_cast<long long>(p.B) * p.T;
        const int first = static_cast<int>(item - group * d.chunks) * d.HS, step = d.HS * d.chunks;
        token = group * (RPW / d.HS) + sub / d.HS;
        here = token < tokens;
        if (!here) token = tokens - 1;
        b = static_cast<int>(token / p.T);
        t = static_cast<int>(token - static_cast<long long>(b) * p.T);
        n0 = p.heads[0] > first ? (p.heads[0] - first + step - 1) / step : 0;
        n = n0 + (p.heads[1] > first ? (p.heads[1] - first + step - 1) / step : 0);
        h = first + sub % d.HS;
    }
};

// A lane's rows on their way: a slot per step in shared memory that the lane
// alone fills and reads, DEPTH steps ahead, so that neither registers nor a
// barrier is needed for what is in flight.
template <typename T, int DEPTH>
struct Ring {
    Raw4<T> slot[DEPTH][2][WARPS * 32];      // 8 or 16 adjacent bytes a lane: no bank conflicts

    __device__ __forceinline__ void fetch(int i, const T* row, const Place& q) {
        const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(&slot[i % DEPTH][0][threadIdx.x])),
                       b = a + sizeof(Raw4<T>) * WARPS * 32;
        if (sizeof(T) == 2) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(a), "l"(row + q.g0) : "memory");
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(b), "l"(row + q.g1) : "memory");
        } else {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(a), "l"(row + q.g0) : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(b), "l"(row + q.g1) : "memory");
        }
    }
    __device__ __forceinline__ RawRow<T> take(int i) const {
        return RawRow<T>{slot[i % DEPTH][0][threadIdx.x], slot[i % DEPTH][1][threadIdx.x]};
    }
};

// One row from the loaded elements to the stored ones; returns its sum of
// squares.
template <typename TI, typename TO, int DK, bool INTER, bool EXACT = false>
__device__ __forceinline__ float qk_row(const QkArgs& p, const RawRow<TI>& raw, const Row8& w, const Turn& turn,
                                        const Place& q, TO* y, bool on) {
    Row8 v = row_of<INTER>(raw);
    const float ss = row_dot<DK / 8>(v, v);
    const F2 r = both(inverse_norm<DK>(p, ss));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        v.a[k] = mul2(v.a[k], mul2(r, w.a[k]));
        v.b[k] = mul2(v.b[k], mul2(r, w.b[k]));
    }
    rotate<false, EXACT>(v, turn, q);
    if (on) put_row<INTER>(y, q, v);
    return ss;
}

template <typename TI, typename TO, int DK, bool INTER, bool PART>
__global__ void __launch_bounds__(WARPS * 32, FWD_BLOCKS_PER_SM)
qk_fwd_kernel(const __grid_constant__ QkArgs p, const Deal deal) {
    constexpr int UNROLL = sizeof(TI) == 2 ? 4 : 2;
    __shared__ Freqs<DK> freqs;
    freqs.fill(p);
    Place2<DK> at;
    const Place q = place_of<INTER>(at.l, p.rot);
    const float most = PART ? most_squares<INTER>(p, q) : 0.f;
    const int step = deal.HS * deal.chunks;
    const long long xstep = static_cast<long long>(step) * DK, ystep = xstep * p.T;
    for (long long item = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5); item < deal.items;
         item += static_cast<long long>(gridDim.x) * WARPS) {
        at.at(p, deal, item);
        const Turn turn = turn_at<DK>(freqs, p, at.token, at.t, deal.HS, at.l);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int H = p.heads[which], steps = which ? at.n - at.n0 : at.n0;
            if (steps == 0) continue;
            const Row8 w = weight_of<INTER>(p.w[which], q);
            const TI* x = static_cast<const TI*>(p.x[which]) + at.token * p.ld[which] + at.h * DK;
            TO* y = static_cast<TO*>(p.y[which]) +
                    ((static_cast<long long>(at.b) * H + at.h) * p.T + at.t) * DK;
            // UNROLL rows' loads in flight; a batch whose rows are all there has no predicates
            float worst = 0.f;
            const int whole = !__all_sync(0xffffffffu, at.here) ? 0
                              : __all_sync(0xffffffffu, at.h + (steps - 1) * step < H) ? steps : steps - 1;
            for (int i = 0; i < steps; i += UNROLL) {
                RawRow<TI> raw[UNROLL];
                if (i + UNROLL <= whole) {
#pragma unroll
                    for (int u = 0; u < UNROLL; ++u) {
                        raw[u] = get_raw(x, q);
                        x += xstep;
                    }
#pragma unroll
                    for (int u = 0; u < UNROLL; ++u) {
                        worst = max_nan(worst, qk_row<TI, TO, DK, INTER>(p, raw[u], w, turn, q, y, true));
                        y += ystep;
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < UNROLL; ++u) {
                        raw[u] = RawRow<TI>{};
                        if (at.here && at.h + (i + u) * step < H) raw[u] = get_raw(x, q);
                        x += xstep;
                    }
#pragma unroll
                    for (int u = 0; u < UNROLL; ++u) {
                        if (i + u >= steps) break;             // (the warp as one)
                        worst = max_nan(worst, qk_row<TI, TO, DK, INTER>(p, raw[u], w, turn, q, y,
                                                                         at.here && at.h + (i + u) * step < H));
                        y += ystep;
                    }
                }
            }
            if (PART && __any_sync(0xffffffffu, !(worst <= most))) {
                x = static_cast<const TI*>(p.x[which]) + at.token * p.ld[which] + at.h * DK;
                y = static_cast<TO*>(p.y[which]) + ((static_cast<long long>(at.b) * H + at.h) * p.T + at.t) * DK;
#pragma unroll 1
                for (int i = 0; i < steps; ++i) {
                    const bool on = at.here && at.h + i * step < H;
                    RawRow<TI> raw{};
                    if (on) raw = get_raw(x, q);
                    qk_row<TI, TO, DK, INTER, true>(p, raw, w, turn, q, y, on);
                    x += xstep;
                    y += ystep;
                }
            }
        }
    }
}

// The forward of many tokens with a warp's worth of heads: a token's heads lie
// side by side in its row, so they come as bulk copies of up to SEG bytes into
// the warp's ring, SEG_DEPTH of them ahead, without a load instruction or a
// register.  The kernel above waits for its loads (half of all stalls), and
// rows ahead in registers cost more than they hide: 8 x 4096 tokens, 16 + 16
// heads of 128, bf16: 102 us there, 90 us here (87 % of the copy's rate;
// three copies ahead 92 us, six of half the size 101 us).
template <int DK>
struct BulkShared {
    char ring[WARPS][SEG_DEPTH][SEG];
    uint64_t full[WARPS][SEG_DEPTH];
    Freqs<DK> freqs;
};

template <typename TI, typename TO, int DK, bool INTER, bool PART>
__global__ void __launch_bounds__(WARPS * 32, 2)
qk_fwd_bulk_kernel(const __grid_constant__ QkArgs p, long long wait_ns) {
    constexpr int LPR = DK / 8, RPW = 32 / LPR, ROW = DK * static_cast<int>(sizeof(TI)), HEADS = SEG / ROW;
    extern __shared__ __align__(16) char smem[];
    BulkShared<DK>& sh = *reinterpret_cast<BulkShared<DK>*>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
    if (threadIdx.x == 0) {
        for (int i = 0; i < WARPS * SEG_DEPTH; ++i) mbar_init(&sh.full[0][0] + i, 1);
        mbar_init_fence();
    }
    sh.freqs.fill(p);                                          // (and a barrier)
    const Place q = place_of<INTER>(l, p.rot);
    const float most = PART ? most_squares<INTER>(p, q) : 0.f;
    const long long tokens = static_cast<long long>(p.B) * p.T, stride = static_cast<long long>(gridDim.x) * WARPS;
    const int segs[2] = {(p.heads[0] + HEADS - 1) / HEADS, (p.heads[1] + HEADS - 1) / HEADS}, per = segs[0] + segs[1];
    const long long first = static_cast<long long>(blockIdx.x) * WARPS + warp;
    const long long ystep = static_cast<long long>(p.T) * DK;

    // the copies run ahead: their token, segment and slot
    long long ct = first;
    int cs = 0, cslot = 0;
    auto copy = [&]() {
        if (ct >= tokens) return;
        const int which = cs >= segs[0], h = (cs - (which ? segs[0] : 0)) * HEADS;
        const int n = min(HEADS, p.heads[which] - h);
        if (lane == 0) {
            mbar_arrive_expect_tx(&sh.full[warp][cslot], n * ROW);
            bulk_g2s(sh.ring[warp][cslot], static_cast<const TI*>(p.x[which]) + ct * p.ld[which] + h * DK, n * ROW,
                     &sh.full[warp][cslot]);
        }
        if (++cs == per) {
            cs = 0;
            ct += stride;
        }
        if (++cslot == SEG_DEPTH) cslot = 0;
    };
    for (int i = 0; i < SEG_DEPTH; ++i) copy();

    int slot = 0;
    uint32_t parity = 0;
    bool ok = true;
    Row8 w{};
    for (long long token = first; token < tokens; token += stride) {
        const int b = static_cast<int>(token / p.T), t = static_cast<int>(token - static_cast<long long>(b) * p.T);
        const Turn turn = turn_at<DK>(sh.freqs, p, token, t, RPW, l);
        for (int seg = 0; seg < per; ++seg) {
            const int which = seg >= segs[0], h0 = (seg - (which ? segs[0] : 0)) * HEADS;
            const int H = p.heads[which], n = min(HEADS, H - h0);
            if (seg == 0 || seg == segs[0]) w = weight_of<INTER>(p.w[which], q);
            if (ok && !mbar_wait(&sh.full[warp][slot], parity, wait_ns)) {
                record_error(&g_qk_error, KDN_ERR_TIMEOUT);
                ok = false;
                ct = tokens;                                   // no more copies; those in flight get one more wait each
                int s = slot;
                uint32_t ph = parity;
                do {
                    mbar_wait(&sh.full[warp][s], ph, wait_ns);
                    if (++s == SEG_DEPTH) {
                        s = 0;
                        ph ^= 1;
                    }
                } while (s != cslot);
            }
            const TI* x0 = reinterpret_cast<const TI*>(sh.ring[warp][slot]) + sub * DK;
            TO* y0 = static_cast<TO*>(p.y[which]) + ((static_cast<long long>(b) * H + h0 + sub) * p.T + t) * DK;
            const TI* x = x0;
            TO* y = y0;
            float worst = 0.f;
            int i = 0;
#pragma unroll 4
            for (; i + RPW <= n; i += RPW) {
                RawRow<TI> raw;
                raw.u = *reinterpret_cast<const Raw4<TI>*>(x + q.g0);
                raw.v = *reinterpret_cast<const Raw4<TI>*>(x + q.g1);
                worst = max_nan(worst, qk_row<TI, TO, DK, INTER>(p, raw, w, turn, q, y, true));
                x += RPW * DK;
                y += RPW * ystep;
            }
            if (i < n) {
                RawRow<TI> raw{};
                if (i + sub < n) {
                    raw.u = *reinterpret_cast<const Raw4<TI>*>(x + q.g0);
                    raw.v = *reinterpret_cast<const Raw4<TI>*>(x + q.g1);
                }
                worst = max_nan(worst, qk_row<TI, TO, DK, INTER>(p, raw, w, turn, q, y, i + sub < n));
            }
            if (PART && __any_sync(0xffffffffu, !(worst <= most))) {
                x = x0;
                y = y0;
#pragma unroll 1
                for (i = 0; i < n; i += RPW) {
                    RawRow<TI> raw{};
                    if (i + sub < n) {
                        raw.u = *reinterpret_cast<const Raw4<TI>*>(x + q.g0);
                        raw.v = *reinterpret_cast<const Raw4<TI>*>(x + q.g1);
                    }
                    qk_row<TI, TO, DK, INTER, true>(p, raw, w, turn, q, y, i + sub < n);
                    x += RPW * DK;
                    y += RPW * ystep;
                }
            }
            __syncwarp();                                      // the slot has been read
            copy();
            if (++slot == SEG_DEPTH) {
                slot = 0;
                parity ^= 1;
            }
        }
    }
}

// Backward.  part [block][2 dk] takes each block's share of the weights'
// gradients, q's then k's.
template <typename TI, typename TO, int DEPTH>
struct BwdRing {
    Ring<TI, DEPTH> x;
    Ring<TO, DEPTH> g;
};

// (PART here also without a norm: its gradient has no term of x, not even 0 x.)
template <typename TI, typename TO, int DK, bool INTER, bool PART>
__global__ void __launch_bounds__(WARPS * 32, BWD_BLOCKS_PER_SM)
qk_bwd_kernel(const __grid_constant__ QkArgs p, const Deal deal, float* part) {
    constexpr int LPR = DK / 8, DEPTH = BWD_DEPTH;
    __shared__ Freqs<DK> freqs;
    __shared__ float share[WARPS][DK];
    extern __shared__ __align__(16) char smem[];
    BwdRing<TI, TO, DEPTH>& ring = *reinterpret_cast<BwdRing<TI, TO, DEPTH>*>(smem);
    freqs.fill(p);
    Place2<DK> at;
    const Place q = place_of<INTER>(at.l, p.rot);
    const float inv_n = p.norm == KDN_NORM_RMS ? 1.f / DK : 1.f;
    const int step = deal.HS * deal.chunks;
    const long long ystep = static_cast<long long>(p.T) * DK;
    Row8 dw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) dw[0].a[i] = dw[0].b[i] = dw[1].a[i] = dw[1].b[i] = both(0.f);

    for (long long item = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5); item < deal.items;
         item += static_cast<long long>(gridDim.x) * WARPS) {
        at.at(p, deal, item);
        const TI* x[2];
        const TO* gy[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            x[w] = static_cast<const TI*>(p.x[w]) + at.token * p.ld[w];
            gy[w] = static_cast<const TO*>(p.grad_y[w]) + (static_cast<long long>(at.b) * p.heads[w] * p.T + at.t) * DK;
        }
        auto fetch = [&](int i) {
            if (i < at.n) {
                const int which = i >= at.n0, h = at.h + (which ? i - at.n0 : i) * step;
                if (q.vec && at.here && h < p.heads[which]) {
                    ring.x.fetch(i, (which ? x[1] : x[0]) + h * DK, q);
                    ring.g.fetch(i, (which ? gy[1] : gy[0]) + h * ystep, q);
                }
            }
            copy_commit();
        };
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) fetch(i);
        const Turn turn = turn_at<DK>(freqs, p, at.token, at.t, deal.HS, at.l);
        int i = 0;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int H = p.heads[which], end = which ? at.n : at.n0;
            if (i >= end) continue;
            const Row8 w = weight_of<INTER>(p.w[which], q);
            int h = at.h;
            TI* gx = static_cast<TI*>(p.grad_x[which]) + at.token * p.grad_ld[which];
            for (; i < end; ++i, h += step) {
                const bool on = at.here && h < H;
                copy_wait<DEPTH - 1>();
                RawRow<TI> xr{};
                RawRow<TO> gr{};
                if (on) {
                    xr = q.vec ? ring.x.take(i) : get_raw(x[which] + h * DK, q);
                    gr = q.vec ? ring.g.take(i) : get_raw(gy[which] + h * ystep, q);
                }
                const Row8 v = row_of<INTER>(xr);
                Row8 g = row_of<INTER>(gr);
                rotate<true, false>(g, turn, q);
                // a row that is not there adds nothing, whatever 1 / sqrt(eps) is
                const float ss = row_dot<LPR>(v, v), r = on ? inverse_norm<DK>(p, ss) : 0.f;
                fetch(i + DEPTH);
                Row8 t = times(g, w);
                float dot = row_dot<LPR>(t, v);
                const bool odd = PART && __any_sync(0xffffffffu, !(fabsf(dot) <= FLT_MAX));
                if (odd) {                                     // x or g is not finite, or their product
                    g = row_of<INTER>(gr);
                    rotate<true, true>(g, turn, q);
                    t = times(g, w);
                    dot = row_dot<LPR>(t, v);
                }
                const float along = p.norm == KDN_NORM_NONE ? 0.f : -(r * dot) * inv_n;
                Row8 o;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const F2 na = mul2(both(r), v.a[k]), nb = mul2(both(r), v.b[k]);
                    o.a[k] = mul2(both(r), fma2(na, both(along), t.a[k]));
                    o.b[k] = mul2(both(r), fma2(nb, both(along), t.b[k]));
                    dw[which].a[k] = fma2(na, g.a[k], dw[which].a[k]);
                    dw[which].b[k] = fma2(nb, g.b[k], dw[which].b[k]);
                }
                if (odd && p.norm == KDN_NORM_NONE) o = t;
                if (on) put_row<INTER>(gx + h * DK, q, o);
            }
        }
    }
    if (!part) return;
    // the rows side by side in a warp, then the warps, in order
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const F2 f = i < 4 ? dw[which].a[i / 2] : dw[which].b[(i - 4) / 2];
            float s = i & 1 ? f.y : f.x;
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            // pair i & 3, its first element (i < 4) or its second; where a lane holds two
            // groups of a half-rotated head's rest, `a` is the first group
            int j;
            if (INTER) j = 2 * (q.p0 + (i & 3)) + (i >= 4);
            else if (q.vec) j = (i < 4 ? q.g0 : q.g1) + (i & 3);
            else j = i < 4 ? q.first(i) : q.second(i - 4);
            if ((threadIdx.x & 31) < LPR) share[threadIdx.x >> 5][j] = s;
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

// Heads side by side: a power of two, as many as a warp takes and there are.
// Few tokens' heads are dealt to more warps, so that every SM has some.  (Not
// to even out the last wave: the angles that each warp takes cost more, 3 x
// 1271 tokens of 32 + 8 heads 15.4 us, 19.4 us with the heads over 4 warps.)
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

// A persistent grid: the frequencies are taken once per block, and few
// blocks' shares of the weights' gradients are left to add.
int blocks_of(const Deal& d, int per_sm) {
    const long long blocks = (d.items + WARPS - 1) / WARPS, cap = static_cast<long long>(sm_count()) * per_sm;
    return static_cast<int>(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
}

int bwd_blocks(int B, int T, int Hq, int Hk, int dk) {
    return blocks_of(deal_of(static_cast<long long>(B) * T, Hq, Hk, dk), BWD_BLOCKS_PER_SM);
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

// Whether a forward call is one for bulk copies: vector places, heads for a
// whole warp in either tensor, and a token for half of the warps or more (3 x
// 1271 tokens of 32 + 8 heads 13.9 us, 15.4 by loads; 128 tokens are faster
// dealt out by heads).
bool bulk_ok(const QkArgs& a, int blocks) {
    const int rpw = 32 / (a.dk / 8);
    for (int H : a.heads)
        if (H != 0 && H < rpw) return false;
    return (a.interleaved || a.rot % 8 == 0) &&
           static_cast<long long>(a.B) * a.T >= WARPS * blocks / 2;
}

}  // namespace

long long qk_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int dk) {
    return static_cast<long long>(bwd_blocks(B, T, Hq, Hk, dk)) * 2 * dk * 4;
}

kdn_status qk_fwd_launch(const QkArgs& a, cudaStream_t stream, long long wait_ns) {
    const Deal deal = deal_of(static_cast<long long>(a.B) * a.T, a.heads[0], a.heads[1], a.dk);
    const int blocks = blocks_of(deal, FWD_BLOCKS_PER_SM);
    return by_type(a, [&](auto ti, auto to) {
        return by_dk(a.dk, [&](auto n) {
            using TI = decltype(ti);
            using TO = decltype(to);
            constexpr int DK = decltype(n)::value;
            const int form = 2 * a.interleaved + (a.rot < DK);
            if (bulk_ok(a, 2 * sm_count())) {
                const decltype(&qk_fwd_bulk_kernel<TI, TO, DK, false, false>) forms[] = {
                    qk_fwd_bulk_kernel<TI, TO, DK, false, false>, qk_fwd_bulk_kernel<TI, TO, DK, false, true>,
                    qk_fwd_bulk_kernel<TI, TO, DK, true, false>, qk_fwd_bulk_kernel<TI, TO, DK, true, true>};
                const auto kernel = forms[form];
                const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), sizeof(BulkShared<DK>));
                if (e != cudaSuccess) return from_cuda(e);
                kernel<<<2 * sm_count(), WARPS * 32, sizeof(BulkShared<DK>), stream>>>(a, wait_ns);
                return from_cuda(cudaGetLastError());
            }
            const decltype(&qk_fwd_kernel<TI, TO, DK, false, false>) forms[] = {
                qk_fwd_kernel<TI, TO, DK, false, false>, qk_fwd_kernel<TI, TO, DK, false, true>,
                qk_fwd_kernel<TI, TO, DK, true, false>, qk_fwd_kernel<TI, TO, DK, true, true>};
            forms[form]<<<blocks, WARPS * 32, 0, stream>>>(a, deal);
            return from_cuda(cudaGetLastError());
        });
    });
}

cudaError_t qk_take_device_error(int* status) {
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_qk_error, sizeof(int));
    if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(g_qk_error, &zero, sizeof(int));
    *status = v;
    return e;
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
            const decltype(&qk_bwd_kernel<TI, TO, DK, false, false>) forms[] = {
                qk_bwd_kernel<TI, TO, DK, false, false>, qk_bwd_kernel<TI, TO, DK, false, true>,
                qk_bwd_kernel<TI, TO, DK, true, false>, qk_bwd_kernel<TI, TO, DK, true, true>};
            const auto kernel = forms[2 * a.interleaved + (a.rot < DK || a.norm == KDN_NORM_NONE)];
            const size_t smem = sizeof(BwdRing<TI, TO, BWD_DEPTH>);
            const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem);
            if (e != cudaSuccess) return from_cuda(e);
            kernel<<<blocks, WARPS * 32, smem, stream>>>(a, deal, part);
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
