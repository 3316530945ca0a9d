// delta_scan.cu -- the gated delta rule token by token on the CUDA cores, in
// fp32 for every type and head size: forward, backward and one-token step.
// (delta_tc.cu has the chunked form on the tensor cores; delta_device.cuh the
// rule.)
//
// Forward and the reverse walk.  A state's rows do not touch one another: row
// i needs k_t, q_t and its own v_t[i].  LPR lanes hold a row (DK / LPR columns
// each, R rows a lane, so that a lane's loads of k and q serve R rows), the
// two dots S k and S q are sums over those lanes, and a CTA owns ROWS rows of
// one head.  k, q and v come in tiles of TT tokens by asynchronous copies, one
// tile ahead.  A token costs 6 d_k flops a row and one trip dot -> shuffles ->
// u -> update, about 345 cycles (d_k = 64, few heads): few heads are bound by
// that trip, many by the FMA rate.  The dot with q reads the state after the token, off that trip.
//
// Backward.  The adjoint D_t of S_t walks the other way with the same shape
// (rows apart, one dot a token), and needs no state:
//     D <- D + do_t q_t^T,  y_t = D k_t,  D <- a_t (D - beta_t y_t k_t^T).
// The forward walk keeps r_t and the state before each chunk of 64 tokens, the
// reverse walk y_t and the adjoint behind each chunk, and a third kernel makes
// the gradients of all chunks side by side from products of whole chunks: with
// g_t the log decay since the chunk began, E_ts = e^{g_t - g_s},
// u = beta r, l = beta y,
//     dP = (dO u^T) . E (s <= t),    dG = -(l u^T) . E (s < t),
//     dq = e^g dO S0 + dP k,
//     dk = [-e^g l S0 + dG k] + [dP^T q + dG^T k + e^{g_C - g} u D1],
//     dv = l,   dbeta_t = r_t . y_t,
// and the gradient of a token's log decay is all that is read from it on of what
// was written before it: with W_ts = dP_ts q_t.k_s + dG_ts k_t.k_s
//     sum_{r >= t, s < t} W_rs + sum_{r >= t} (e^g (do S0).q - e^g (l S0).k)_r
//     + sum_{s < t} (e^{g_C - g} (u D1).k)_s + e^{g_C} <D1, S0>,
// each term of which has that token's decay in it.  (As sum_{r >= t} (q.dq +
// k.dk_read - k.dk_write)_r + <D1, S1> the pairs that do not stand across the
// token cancel but for their roundings, which are larger than the gradient of a
// strong decay.)
#include <type_traits>

#include "delta_device.cuh"
#include "delta_tc.h"
#include "kdn.h"
#include "kdn_internal.h"
#include "kernel_setup.h"
#include "sum_rows.cuh"

namespace kdn {
namespace delta {
namespace {

// four warps walk, a fifth brings the tiles and their gates
constexpr int WALK_WARPS = 4, WALK_THREADS = WALK_WARPS * 32, WALK_ALL = WALK_THREADS + 32;

template <int DK>
struct Shape {
    static constexpr int LPR = DK >= 64 ? 8 : 4;             // lanes to a row
    static constexpr int CPL = DK / LPR;                     // columns a lane: 16, 8, 8, 4
    static constexpr int R = 2;                              // rows a lane
    static constexpr int ROWS = WALK_WARPS * (32 / LPR) * R; // rows a CTA: 32 or 64
};

// A tile of tokens as it lies in memory; TT so that two tiles leave room for
// several CTAs.
template <typename TI, typename TV, int DK>
struct WalkShared {
    static constexpr int ROWS = Shape<DK>::ROWS;
    static constexpr int TT = DK * sizeof(TI) > 256 ? 16 : 32;
    static constexpr int BYTES_K = TT * DK * sizeof(TI), BYTES_V = TT * ROWS * sizeof(TV);
    static constexpr int STAGE = 2 * BYTES_K + BYTES_V;      // k, q, v (or do)
    static constexpr int GATES = 2 * (4 * TT + 4) * 4 + TT * 4;   // of two tiles, and k.q of one
    static constexpr int BYTES = 2 * STAGE + GATES + TT * (ROWS + 1) * 4;
};

// What the backward keeps of a walk; null in a forward call.
struct Keep {
    float* states;      // [slots,H,dv,dk]
    float* rows;        // [B,H,T,dv]
};

// By one warp: n tokens of DK elements, and n rows of `width` from rows dv apart.
template <typename TI, typename TV, int DK>
__device__ __forceinline__ void tile_copies(unsigned char* stage, const TI* k, const TI* q, const TV* v, int n, int dv,
                                            int width) {
    using Sh = WalkShared<TI, TV, DK>;
    constexpr int PER = DK * sizeof(TI) / 16;
    const int lane = threadIdx.x & 31;
    for (int i = lane; i < n * PER; i += 32) {
        copy16(stage + i * 16, reinterpret_cast<const char*>(k) + i * 16);
        copy16(stage + Sh::BYTES_K + i * 16, reinterpret_cast<const char*>(q) + i * 16);
    }
    constexpr int PV = Sh::ROWS * sizeof(TV) / 16;
    const int pieces = width * static_cast<int>(sizeof(TV)) / 16;
    for (int i = lane; i < n * PV; i += 32) {
        const int t = i / PV, c = i % PV;
        if (c < pieces)
            copy16(stage + 2 * Sh::BYTES_K + i * 16,
                   reinterpret_cast<const char*>(v + static_cast<long long>(t) * dv) + c * 16);
    }
}

// Gates of a tile's tokens, by one warp.  The state (or adjoint) is kept
// as 2^-x times its value, x the log decay since the tile began, so that a
// token's update is one multiply-add an element and rounds each once: with a
// decay of its own each, a memory of n tokens would gather 2 n roundings and n
// of alpha (1.7e-6 of a state of 1000 tokens instead of 0.6e-6).  x is a sum in
// 64 bits; whole multiples of 8 are taken out of it as exact powers of two
// (`shift`, 1 for most tokens), so the factors stay within 2^-8 and 2^8.
// Forward: x of token t counts its own decay; backward the decays behind it.
template <int TT>
struct Gates {
    float f[TT], w[TT], beta[TT], shift[TT];   // 2^x, beta (back: 1) over 2^x, beta, shift before token t
    float end;                                 // what the tile leaves of the kept value
    float pad[3];
};

template <typename TI, int TT, bool BACK>
__device__ __forceinline__ void tile_gates(Gates<TT>* gates, const TI* d, const TI* beta, float A, int n) {
    const int t = threadIdx.x & 31;
    const bool on = t < n;                     // (n <= TT <= 32)
    const float be = on ? to_f32(beta[t]) : 0.f;
    double z = on ? -1.4426950408889634 * A * to_f32(d[t]) : 0.0;
    if (z < -1024.0) z = -1024.0;              // 0 in fp32 alike, and no difference of infinities
    double x = z;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = BACK ? __shfl_down_sync(0xffffffffu, x, o) : __shfl_up_sync(0xffffffffu, x, o);
        if (BACK ? t + o < 32 : t >= o) x += y;
    }
    const double all = x;
    if (BACK) x -= z;
    const double m = floor(-x * 0.125);
    double before = BACK ? __shfl_down_sync(0xffffffffu, m, 1) : __shfl_up_sync(0xffffffffu, m, 1);
    if (t == (BACK ? 31 : 0)) before = 0.0;
    const float f = exp2f(static_cast<float>(x + 8.0 * m));
    if (on) {
        gates->f[t] = f;
        gates->w[t] = (BACK ? 1.f : be) / f;
        gates->beta[t] = be;
        gates->shift[t] = m == before ? 1.f : exp2f(static_cast<float>(-8.0 * (m - before)));
    }
    if (BACK && t == 0) gates->end = exp2f(static_cast<float>(all + 8.0 * m));
    if (!BACK && t == n - 1) gates->end = f;
}

template <int LPR, int R>
__device__ __forceinline__ void row_sums(float (&p)[R]) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) p[r] += __shfl_xor_sync(0xffffffffu, p[r], o);
}

// A lane's columns of token row `x`: groups of 4, LPR groups apart.
template <int LPR, int CPL, typename T>
__device__ __forceinline__ void columns(const T* x, int sub, float (&c)[CPL]) {
#pragma unroll
    for (int j = 0; j < CPL / 4; ++j) {
        const float4 f = load4(x + (j * LPR + sub) * 4);
        c[4 * j] = f.x;
        c[4 * j + 1] = f.y;
        c[4 * j + 2] = f.z;
        c[4 * j + 3] = f.w;
    }
}

template <int CPL>
__device__ __forceinline__ float dot(const float (&a)[CPL], const float (&b)[CPL]) {
    float e = 0.f, f = 0.f;
#pragma unroll
    for (int c = 0; c < CPL; c += 2) {
        e = fmaf(a[c], b[c], e);
        f = fmaf(a[c + 1], b[c + 1], f);
    }
    return e + f;
}
template <int CPL, int R>
__device__ __forceinline__ void scaled(float (&S)[R][CPL], float by) {
    if (by == 1.f) return;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < CPL; ++c) S[r][c] *= by;
}

template <int LPR, int CPL, int R>
__device__ __forceinline__ void load_state(float (&S)[R][CPL], const float* src, int first, int sub, int dv, int DK) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < CPL / 4; ++j) {
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (src && first + r < dv) f = load4(src + static_cast<long long>(first + r) * DK + (j * LPR + sub) * 4);
            S[r][4 * j] = f.x;
            S[r][4 * j + 1] = f.y;
            S[r][4 * j + 2] = f.z;
            S[r][4 * j + 3] = f.w;
        }
}
template <int LPR, int CPL, int R>
__device__ __forceinline__ void store_state(const float (&S)[R][CPL], float* dst, int first, int sub, int dv, int DK) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < CPL / 4; ++j)
            if (first + r < dv)
                *reinterpret_cast<float4*>(dst + static_cast<long long>(first + r) * DK + (j * LPR + sub) * 4) =
                    make_float4(S[r][4 * j], S[r][4 * j + 1], S[r][4 * j + 2], S[r][4 * j + 3]);
}

// A tile's [n, width] results from shared rows into memory, dv apart.
template <typename TO, int ROWS>
__device__ __forceinline__ void tile_out(const float* so, TO* dst, int n, int dv, int width) {
    for (int i = threadIdx.x; i < n * ROWS; i += WALK_ALL) {
        const int t = i / ROWS, r = i % ROWS;
        if (r < width) dst[static_cast<long long>(t) * dv + r] = from_f32<TO>(so[t * (ROWS + 1) + r]);
    }
}

template <typename TI, typename TO, int DK, bool KEEP>
__global__ void __launch_bounds__(WALK_ALL) delta_walk_kernel(const DeltaArgs a, const Keep keep) {
    using Sp = Shape<DK>;
    using Sh = WalkShared<TI, TI, DK>;
    constexpr int LPR = Sp::LPR, CPL = Sp::CPL, R = Sp::R, ROWS = Sp::ROWS, TT = Sh::TT;
    extern __shared__ __align__(128) unsigned char smem[];
    Gates<TT>* gates = reinterpret_cast<Gates<TT>*>(smem + 2 * Sh::STAGE);
    float* so = reinterpret_cast<float*>(gates + 2) + TT;
    const int blocks = (a.dv + ROWS - 1) / ROWS;
    const long long sr = blockIdx.x / blocks;                // state row n * H + h
    const int i0 = (blockIdx.x % blocks) * ROWS, width = min(ROWS, a.dv - i0);
    const long long n = sr / a.H;
    const int h = static_cast<int>(sr % a.H);
    const Span sp = span_of(a, n);
    const long long tok = (sp.row * a.H + h) * a.T + sp.lo;
    const int len = sp.hi - sp.lo;
    const int lane = threadIdx.x & 31, sub = lane % LPR;
    const bool helper = threadIdx.x >= WALK_THREADS;
    const int mine = ((threadIdx.x >> 5) * (32 / LPR) + lane / LPR) * R;   // this lane's first row in the CTA
    const long long size = static_cast<long long>(a.dv) * DK;
    const TI* q = static_cast<const TI*>(a.q) + tok * DK;
    const TI* k = static_cast<const TI*>(a.k) + tok * DK;
    const TI* v = static_cast<const TI*>(a.v) + tok * a.dv + i0;
    const TI* d = static_cast<const TI*>(a.d) + tok;
    const TI* beta = static_cast<const TI*>(a.beta) + tok;

    float S[R][CPL];
    if (!helper)
        load_state<LPR, CPL, R>(S, a.S0 ? a.S0 + sr * size : nullptr, i0 + mine, sub, a.dv, DK);
    if (len > 0) {
        const float A = a.A[h];
        auto fetch = [&](int t0) {
            const int m = min(TT, len - t0), st = (t0 / TT) & 1;
            tile_copies<TI, TI, DK>(smem + st * Sh::STAGE, k + static_cast<long long>(t0) * DK,
                                    q + static_cast<long long>(t0) * DK, v + static_cast<long long>(t0) * a.dv, m,
                                    a.dv, width);
            tile_gates<TI, TT, false>(gates + st, d + t0, beta + t0, A, m);
        };
        if (helper) {
            fetch(0);
            copies_done();
        }
        __syncthreads();
        for (int t0 = 0; t0 < len; t0 += TT) {
            const int m = min(TT, len - t0), st = (t0 / TT) & 1;
            if (helper) {
                if (t0 + TT < len) {
                    fetch(t0 + TT);
                    copies_done();
                }
            } else {
                if (KEEP && t0 % CHUNK == 0)
                    store_state<LPR, CPL, R>(S, keep.states + ((sp.slot + t0 / CHUNK) * a.H + h) * size, i0 + mine, sub,
                                             a.dv, DK);
                const unsigned char* stage = smem + st * Sh::STAGE;
                const TI* sk = reinterpret_cast<const TI*>(stage);
                const TI* sq = reinterpret_cast<const TI*>(stage + Sh::BYTES_K);
                const TI* sv = reinterpret_cast<const TI*>(stage + 2 * Sh::BYTES_K);
                const Gates<TT>* sg = gates + st;
                // p: the state before token t times k_t.  The dots of the state after a token with its
                // own q and the next k share one round of shuffles.
                float kc[CPL], p[R];
                columns<LPR, CPL>(sk, sub, kc);
#pragma unroll
                for (int r = 0; r < R; ++r) p[r] = dot(S[r], kc);
                row_sums<LPR>(p);
                for (int t = 0; t < m; ++t) {
                    float qc[CPL], kn[CPL], both[2 * R];
                    columns<LPR, CPL>(sk + min(t + 1, m - 1) * DK, sub, kn);
                    if (!KEEP) columns<LPR, CPL>(sq + t * DK, sub, qc);
                    const float f = sg->f[t], w = sg->w[t], by = sg->shift[t];
                    if (by != 1.f) {
                        scaled(S, by);
#pragma unroll
                        for (int r = 0; r < R; ++r) p[r] *= by;
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float miss = to_f32(sv[t * ROWS + mine + r]) - f * p[r], u = w * miss;
                        if (KEEP && sub == 0) so[t * (ROWS + 1) + mine + r] = miss;
#pragma unroll
                        for (int c = 0; c < CPL; ++c) S[r][c] = fmaf(u, kc[c], S[r][c]);
                    }
                    if (KEEP) {
#pragma unroll
                        for (int r = 0; r < R; ++r) p[r] = dot(S[r], kn);
                        row_sums<LPR>(p);
                    } else {
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            both[r] = dot(S[r], kn);
                            both[R + r] = dot(S[r], qc);
                        }
                        row_sums<LPR>(both);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            p[r] = both[r];
                            if (sub == 0) so[t * (ROWS + 1) + mine + r] = f * both[R + r];
                        }
                    }
#pragma unroll
                    for (int c = 0; c < CPL; ++c) kc[c] = kn[c];
                }
                scaled(S, sg->end);
            }
            __syncthreads();   // every warp's results are in `so`, and the next tile is here
            if (KEEP)
                tile_out<float, ROWS>(so, keep.rows + (tok + t0) * a.dv + i0, m, a.dv, width);
            else
                tile_out<TO, ROWS>(so, static_cast<TO*>(a.out) + (tok + t0) * a.dv + i0, m, a.dv, width);
            __syncthreads();   // `so` is free
        }
    }
    if (helper) return;
    if (a.final_state) store_state<LPR, CPL, R>(S, a.final_state + sr * size, i0 + mine, sub, a.dv, DK);
}

// The adjoint's walk, last token first; keep.states: the adjoint behind each
// chunk, keep.rows: y.
template <typename TI, typename TO, int DK>
__global__ void __launch_bounds__(WALK_ALL) delta_back_kernel(const DeltaArgs a, const Keep keep) {
    using Sp = Shape<DK>;
    using Sh = WalkShared<TI, TO, DK>;
    constexpr int LPR = Sp::LPR, CPL = Sp::CPL, R = Sp::R, ROWS = Sp::ROWS, TT = Sh::TT;
    extern __shared__ __align__(128) unsigned char smem[];
    Gates<TT>* gates = reinterpret_cast<Gates<TT>*>(smem + 2 * Sh::STAGE);
    float* skq = reinterpret_cast<float*>(gates + 2);
    float* so = skq + TT;
    const int blocks = (a.dv + ROWS - 1) / ROWS;
    const long long sr = blockIdx.x / blocks;
    const int i0 = (blockIdx.x % blocks) * ROWS, width = min(ROWS, a.dv - i0);
    const long long n = sr / a.H;
    const int h = static_cast<int>(sr % a.H);
    const Span sp = span_of(a, n);
    const long long tok = (sp.row * a.H + h) * a.T + sp.lo;
    const int len = sp.hi - sp.lo;
    const int lane = threadIdx.x & 31, sub = lane % LPR;
    const bool helper = threadIdx.x >= WALK_THREADS;
    const int mine = ((threadIdx.x >> 5) * (32 / LPR) + lane / LPR) * R;
    const long long size = static_cast<long long>(a.dv) * DK;
    const TI* q = static_cast<const TI*>(a.q) + tok * DK;
    const TI* k = static_cast<const TI*>(a.k) + tok * DK;
    const TO* g = static_cast<const TO*>(a.grad_out) + tok * a.dv + i0;
    const TI* d = static_cast<const TI*>(a.d) + tok;
    const TI* beta = static_cast<const TI*>(a.beta) + tok;

    float D[R][CPL];
    if (!helper)
        load_state<LPR, CPL, R>(D, a.grad_final_state ? a.grad_final_state + sr * size : nullptr, i0 + mine, sub, a.dv,
                                DK);
    if (len > 0) {
        const float A = a.A[h];
        const int last = (len - 1) / TT * TT;
        auto fetch = [&](int t0) {
            const int m = min(TT, len - t0), st = (t0 / TT) & 1;
            tile_copies<TI, TO, DK>(smem + st * Sh::STAGE, k + static_cast<long long>(t0) * DK,
                                    q + static_cast<long long>(t0) * DK, g + static_cast<long long>(t0) * a.dv, m,
                                    a.dv, width);
            tile_gates<TI, TT, true>(gates + st, d + t0, beta + t0, A, m);
        };
        if (helper) {
            fetch(last);
            copies_done();
        }
        __syncthreads();
        for (int t0 = last; t0 >= 0; t0 -= TT) {
            const int m = min(TT, len - t0), st = (t0 / TT) & 1;
            if (helper) {
                if (t0 > 0) {
                    fetch(t0 - TT);
                    copies_done();
                }
            } else {
                const unsigned char* stage = smem + st * Sh::STAGE;
                const TI* sk = reinterpret_cast<const TI*>(stage);
                const TI* sq = reinterpret_cast<const TI*>(stage + Sh::BYTES_K);
                const TO* sg = reinterpret_cast<const TO*>(stage + 2 * Sh::BYTES_K);
                const Gates<TT>* sa = gates + st;
                {   // k.q of every token: D k after do q^T came in is D k + do (q.k)
                    constexpr int PER = WALK_THREADS / TT;   // threads to a token: 4 or 8
                    const int t = threadIdx.x / PER;
                    float e = 0.f;
                    if (t < m)
                        for (int c = threadIdx.x % PER; c < DK; c += PER)
                            e = fmaf(to_f32(sk[t * DK + c]), to_f32(sq[t * DK + c]), e);
#pragma unroll
                    for (int o = PER / 2; o > 0; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
                    if (threadIdx.x % PER == 0) skq[t] = e;
                }
                if (t0 == last || (t0 + TT) % CHUNK == 0)
                    store_state<LPR, CPL, R>(D, keep.states + ((sp.slot + t0 / CHUNK) * a.H + h) * size, i0 + mine,
                                             sub, a.dv, DK);
                asm volatile("bar.sync 1, %0;" ::"n"(WALK_THREADS) : "memory");   // k.q is here
                float kc[CPL], qc[CPL], kn[CPL], qn[CPL], p[R];
                columns<LPR, CPL>(sk + (m - 1) * DK, sub, kc);
                columns<LPR, CPL>(sq + (m - 1) * DK, sub, qc);
                for (int t = m - 1; t >= 0; --t) {
                    scaled(D, sa->shift[t]);
#pragma unroll
                    for (int r = 0; r < R; ++r) p[r] = dot(D[r], kc);
                    columns<LPR, CPL>(sk + max(t - 1, 0) * DK, sub, kn);
                    columns<LPR, CPL>(sq + max(t - 1, 0) * DK, sub, qn);
                    row_sums<LPR>(p);
                    const float f = sa->f[t], w = sa->w[t], be = sa->beta[t], kq = skq[t];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float gr = to_f32(sg[t * ROWS + mine + r]), y = fmaf(gr, kq, f * p[r]);
                        if (sub == 0) so[t * (ROWS + 1) + mine + r] = y;
                        const float wg = w * gr, wy = -w * (be * y);
#pragma unroll
                        for (int c = 0; c < CPL; ++c) D[r][c] = fmaf(wy, kc[c], fmaf(wg, qc[c], D[r][c]));
                    }
#pragma unroll
                    for (int c = 0; c < CPL; ++c) {
                        kc[c] = kn[c];
                        qc[c] = qn[c];
                    }
                }
                scaled(D, sa->end);
            }
            __syncthreads();
            tile_out<float, ROWS>(so, keep.rows + (tok + t0) * a.dv + i0, m, a.dv, width);
            __syncthreads();
        }
    }
    if (helper) return;
    if (a.grad_S0) store_state<LPR, CPL, R>(D, a.grad_S0 + sr * size, i0 + mine, sub, a.dv, DK);
}

// ---- the gradients of a chunk ----------------------------------------------

struct GradIn {
    const float* states;    // [slots,H,dv,dk] before each chunk
    const float* adjoints;  // behind each chunk
    const float* r;         // [B,H,T,dv]
    const float* y;
    float* sum_A;           // [slots,H]: each chunk's share of dA, or null
};

constexpr int GRAD_THREADS = 256;

template <int DK>
constexpr int grad_smem(int dv) {
    return (2 * CHUNK * (DK + 4) + 3 * CHUNK * (dv + 4) + 2 * CHUNK * (CHUNK + 4) + (8 + GRAD_THREADS / 32) * CHUNK +
            GRAD_THREADS / 32) * 4;
}

__device__ __forceinline__ float block_sum(float x, float* share) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) == 0) share[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < GRAD_THREADS / 32; ++w) s += share[w];
    return s;
}

// N consecutive floats (N of 1, 2, 4; aligned to N).
template <int N>
__device__ __forceinline__ void vec_of(const float* p, float (&x)[N]) {
    if constexpr (N == 4) {
        const float4 f = *reinterpret_cast<const float4*>(p);
        x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
    } else if constexpr (N == 2) {
        const float2 f = *reinterpret_cast<const float2*>(p);
        x[0] = f.x; x[1] = f.y;
    } else {
        x[0] = *p;
    }
}
// acc[t] += sum_r A[t][at + r] B[r] of 4 rows r: A's rows in shared memory, the
// same for the whole warp, one wide load each.
template <int CJ>
__device__ __forceinline__ void four_rows(float (&acc)[8][CJ], const float* A, int ld, const float (&B)[4][CJ]) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const float4 a = *reinterpret_cast<const float4*>(A + t * ld);
#pragma unroll
        for (int c = 0; c < CJ; ++c)
            acc[t][c] = fmaf(a.x, B[0][c], fmaf(a.y, B[1][c], fmaf(a.z, B[2][c], fmaf(a.w, B[3][c], acc[t][c]))));
    }
}

// A CTA makes one chunk's gradients of one head.  All operands but the states
// lie in shared memory as fp32; a warp owns 8 tokens and all d_k columns of
// dq, dk_read and dk_write, so that their dots with q and k stay in the warp.
template <typename TI, typename TO, int DK>
__global__ void __launch_bounds__(GRAD_THREADS) delta_grad_kernel(const DeltaArgs a, const GradIn in) {
    extern __shared__ __align__(16) float sm[];
    const int dv = a.dv, LDK = DK + 4, LDV = dv + 4;
    constexpr int LDC = CHUNK + 4;
    float* sq = sm;                          // [CHUNK][LDK]
    float* sk = sq + CHUNK * LDK;
    float* sg = sk + CHUNK * LDK;            // [CHUNK][LDV]: dO, then l = beta y, u = beta r
    float* sl = sg + CHUNK * LDV;
    float* su = sl + CHUNK * LDV;
    float* dP = su + CHUNK * LDV;            // [t][s]
    float* dG = dP + CHUNK * LDC;
    float* gh = dG + CHUNK * LDC;            // log decay since the chunk began, as a sum of two floats
    float* gl = gh + CHUNK;
    float* eg = gl + CHUNK;                  // e^g, e^{g_C - g}
    float* ew = eg + CHUNK;
    float* sb = ew + CHUNK;                  // beta, d
    float* sd = sb + CHUNK;
    float* sc = sd + CHUNK;                  // what each token reads of S0, q.(e^g dO S0) - k.(e^g l S0)
    float* si = sc + CHUNK;                  // and writes to D1, k.(e^{g_C - g} u D1)
    float* sw = si + CHUNK;                  // [GRAD_THREADS / 32][CHUNK]: shares of the sums of W across a token
    float* share = sw + GRAD_THREADS / 32 * CHUNK;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = static_cast<int>(blockIdx.x % a.H);
    const long long slot = blockIdx.x / a.H;
    long long n, row;
    int t0, m;
    if (!chunk_of(a, slot, &n, &t0, &m, &row)) {
        if (in.sum_A && tid == 0) in.sum_A[slot * a.H + h] = 0.f;
        return;
    }
    const long long tok = (row * a.H + h) * a.T + t0;
    const long long size = static_cast<long long>(dv) * DK, at = (slot * a.H + h) * size;
    const float* S0 = in.states + at;
    const float* D1 = in.adjoints + at;
    const float A = a.A[h];

    if (warp == 0) {
        // the running sum in 64 bits: its differences are small where it is large.  (A token's own
        // decay of e^-300 and e^-2000 is 0 alike.)
        double g[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            const float dt = t < m ? to_f32(static_cast<const TI*>(a.d)[tok + t]) : 0.f;
            sd[t] = dt;
            sb[t] = t < m ? to_f32(static_cast<const TI*>(a.beta)[tok + t]) : 0.f;
            g[e] = t < m ? fmaxf(-A * dt, -1000.f) : 0.f;
        }
        double s = g[0] + g[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += x;
        }
        const double end = __shfl_sync(0xffffffffu, s, 31), before = __shfl_up_sync(0xffffffffu, s, 1);
        if (lane > 0) g[0] += before;
        g[1] = s;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            gh[t] = static_cast<float>(g[e]);
            gl[t] = static_cast<float>(g[e] - gh[t]);
            eg[t] = expf(static_cast<float>(g[e]));
            ew[t] = expf(static_cast<float>(end - g[e]));
        }
    }
    for (int i = tid; i < CHUNK * (DK / 4); i += GRAD_THREADS) {
        const int t = i / (DK / 4), c = i % (DK / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), z = x;
        if (t < m) {
            x = load4(static_cast<const TI*>(a.q) + (tok + t) * DK + c);
            z = load4(static_cast<const TI*>(a.k) + (tok + t) * DK + c);
        }
        *reinterpret_cast<float4*>(sq + t * LDK + c) = x;
        *reinterpret_cast<float4*>(sk + t * LDK + c) = z;
    }
    __syncthreads();   // gates
    for (int i = tid; i < CHUNK * (dv / 4); i += GRAD_THREADS) {
        const int t = i / (dv / 4), c = i % (dv / 4) * 4;
        float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g, l = g;
        if (t < m) {
            const float b = sb[t];
            g = load4(static_cast<const TO*>(a.grad_out) + (tok + t) * dv + c);
            u = load4(in.r + (tok + t) * dv + c);
            l = load4(in.y + (tok + t) * dv + c);
            u = make_float4(b * u.x, b * u.y, b * u.z, b * u.w);
            l = make_float4(b * l.x, b * l.y, b * l.z, b * l.w);
            TI* gv = static_cast<TI*>(a.grad_v) + (tok + t) * dv + c;
            gv[0] = from_f32<TI>(l.x);
            gv[1] = from_f32<TI>(l.y);
            gv[2] = from_f32<TI>(l.z);
            gv[3] = from_f32<TI>(l.w);
        }
        *reinterpret_cast<float4*>(sg + t * LDV + c) = g;
        *reinterpret_cast<float4*>(su + t * LDV + c) = u;
        *reinterpret_cast<float4*>(sl + t * LDV + c) = l;
    }
    __syncthreads();
    // dbeta_t = r_t . y_t from the unscaled rows
    for (int t = warp; t < m; t += GRAD_THREADS / 32) {
        float s = 0.f;
        for (int i = lane; i < dv; i += 32) s = fmaf(in.r[(tok + t) * dv + i], in.y[(tok + t) * dv + i], s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) static_cast<TI*>(a.grad_beta)[tok + t] = from_f32<TI>(s);
    }
    {   // dP, dG: thread (ty, tx) has rows ty + 16 a, columns tx + 16 b
        const int tx = tid & 15, ty = tid >> 4;
        float p[4][4] = {}, w[4][4] = {}, pk[4][4] = {}, wk[4][4] = {};
        for (int i = 0; i < DK; i += 4) {    // q_t.k_s, k_t.k_s
            float4 u[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) u[b] = *reinterpret_cast<const float4*>(sk + (tx + 16 * b) * LDK + i);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 g = *reinterpret_cast<const float4*>(sq + (ty + 16 * r) * LDK + i);
                const float4 l = *reinterpret_cast<const float4*>(sk + (ty + 16 * r) * LDK + i);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    pk[r][b] += g.x * u[b].x + g.y * u[b].y + g.z * u[b].z + g.w * u[b].w;
                    wk[r][b] += l.x * u[b].x + l.y * u[b].y + l.z * u[b].z + l.w * u[b].w;
                }
            }
        }
        for (int i = 0; i < dv; i += 4) {
            float4 u[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) u[b] = *reinterpret_cast<const float4*>(su + (tx + 16 * b) * LDV + i);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 g = *reinterpret_cast<const float4*>(sg + (ty + 16 * r) * LDV + i);
                const float4 l = *reinterpret_cast<const float4*>(sl + (ty + 16 * r) * LDV + i);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    p[r][b] += g.x * u[b].x + g.y * u[b].y + g.z * u[b].z + g.w * u[b].w;
                    w[r][b] += l.x * u[b].x + l.y * u[b].y + l.z * u[b].z + l.w * u[b].w;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int t = ty + 16 * r, s = tx + 16 * b;
                const float e = s <= t ? expf((gh[t] - gh[s]) + (gl[t] - gl[s])) : 0.f;
                p[r][b] = s <= t ? p[r][b] * e : 0.f;
                w[r][b] = s < t ? -w[r][b] * e : 0.f;
                dP[t * LDC + s] = p[r][b];
                dG[t * LDC + s] = w[r][b];
                // W_ts: what t reads of what s wrote
                pk[r][b] = s < t ? fmaf(p[r][b], pk[r][b], w[r][b] * wk[r][b]) : 0.f;
            }
        // across token x: rows t >= x of W, in each the sum of the columns before x
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float before = 0.f;              // the columns of the blocks of 16 before this one
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float x = pk[r][b];
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) {
                    const float y = __shfl_up_sync(0xffffffffu, x, o, 16);
                    if (tx >= o) x += y;
                }
                const float y = __shfl_up_sync(0xffffffffu, x, 1, 16), all = __shfl_sync(0xffffffffu, x, 15, 16);
                pk[r][b] = tx + 16 * b <= ty + 16 * r ? (tx > 0 ? before + y : before) : 0.f;
                before += all;
            }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float x = (pk[0][b] + pk[1][b]) + (pk[2][b] + pk[3][b]);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            if (lane < 16) sw[warp * CHUNK + tx + 16 * b] = x;
        }
    }
    __syncthreads();
    constexpr int CJ = DK >= 32 ? DK / 32 : 1;               // columns a lane
    const int j = lane * CJ;
    const bool on = j < DK;
    const int tw = warp * 8;
    float c8[8], in8[8];
    {   // dq and dk_read of 8 tokens
        float dq[8][CJ] = {}, kr[8][CJ] = {};
#pragma unroll
        for (int t = 0; t < 8; ++t) c8[t] = 0.f;
        if (on) {
            for (int i = 0; i < dv; i += 4) {
                float s0[4][CJ];
#pragma unroll
                for (int r = 0; r < 4; ++r) vec_of<CJ>(S0 + static_cast<long long>(i + r) * DK + j, s0[r]);
                four_rows<CJ>(dq, sg + tw * LDV + i, LDV, s0);
                four_rows<CJ>(kr, sl + tw * LDV + i, LDV, s0);
            }
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int c = 0; c < CJ; ++c) {
                    dq[t][c] *= eg[tw + t];
                    kr[t][c] *= -eg[tw + t];
                    const float q = sq[(tw + t) * LDK + j + c], k = sk[(tw + t) * LDK + j + c];
                    c8[t] = fmaf(q, dq[t][c], fmaf(k, kr[t][c], c8[t]));
                }
            for (int s = 0; s < tw + 8; s += 4) {
                float kc[4][CJ];
#pragma unroll
                for (int r = 0; r < 4; ++r) vec_of<CJ>(sk + (s + r) * LDK + j, kc[r]);
                four_rows<CJ>(dq, dP + tw * LDC + s, LDC, kc);
                four_rows<CJ>(kr, dG + tw * LDC + s, LDC, kc);
            }
        }
        // dk_write, added to dk_read for dk
        float kw[8][CJ] = {}, fw[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) fw[t] = 0.f;
        if (on) {
            for (int i = 0; i < dv; i += 4) {
                float d1[4][CJ];
#pragma unroll
                for (int r = 0; r < 4; ++r) vec_of<CJ>(D1 + static_cast<long long>(i + r) * DK + j, d1[r]);
                four_rows<CJ>(kw, su + tw * LDV + i, LDV, d1);
            }
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int c = 0; c < CJ; ++c) {
                    kw[t][c] *= ew[tw + t];
                    fw[t] = fmaf(sk[(tw + t) * LDK + j + c], kw[t][c], fw[t]);
                }
            for (int t = tw; t < CHUNK; ++t) {
                float qc[CJ], kc[CJ], p[2][4], g[2][4];
                vec_of<CJ>(sq + t * LDK + j, qc);
                vec_of<CJ>(sk + t * LDK + j, kc);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    vec_of<4>(dP + t * LDC + tw + 4 * e, p[e]);
                    vec_of<4>(dG + t * LDC + tw + 4 * e, g[e]);
                }
#pragma unroll
                for (int s = 0; s < 8; ++s)
#pragma unroll
                    for (int c = 0; c < CJ; ++c) kw[s][c] = fmaf(p[s / 4][s % 4], qc[c], fmaf(g[s / 4][s % 4], kc[c], kw[s][c]));
            }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            in8[t] = fw[t];
            if (on) {
#pragma unroll
                for (int c = 0; c < CJ; ++c) {
                    if (tw + t < m) {
                        static_cast<TI*>(a.grad_q)[(tok + tw + t) * DK + j + c] = from_f32<TI>(dq[t][c]);
                        static_cast<TI*>(a.grad_k)[(tok + tw + t) * DK + j + c] = from_f32<TI>(kr[t][c] + kw[t][c]);
                    }
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                c8[t] += __shfl_xor_sync(0xffffffffu, c8[t], o);
                in8[t] += __shfl_xor_sync(0xffffffffu, in8[t], o);
            }
            if (lane == 0) {
                sc[tw + t] = c8[t];
                si[tw + t] = in8[t];
            }
        }
    }
    float x = 0.f;
    for (long long i = tid; i < size; i += GRAD_THREADS) x = fmaf(__ldg(S0 + i), __ldg(D1 + i), x);
    x = block_sum(x, share);                 // (and the tokens' shares are in shared memory)
    if (warp == 0) {
        // gradients of the log decays: reads of S0 from the chunk's end, writes to D1 from its beginning
        float c[2], f[2], across[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            c[e] = sc[t];
            f[e] = si[t];
            across[e] = 0.f;
#pragma unroll
            for (int w = 0; w < GRAD_THREADS / 32; ++w) across[e] += sw[w * CHUNK + t];
        }
        float s = c[0] + c[1], pre = f[0] + f[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float z = __shfl_down_sync(0xffffffffu, s, o), y = __shfl_up_sync(0xffffffffu, pre, o);
            if (lane + o < 32) s += z;
            if (lane >= o) pre += y;
        }
        const float before = __shfl_up_sync(0xffffffffu, pre, 1);
        const float rest = eg[CHUNK - 1] * x + (lane > 0 ? before : 0.f);   // (tokens behind the chunk's last have no decay)
        const float above = __shfl_down_sync(0xffffffffu, s, 1);
        const float ga[2] = {(s + rest) + across[0], (((lane < 31 ? above : 0.f) + c[1]) + (rest + f[0])) + across[1]};
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            if (t < m) {
                static_cast<TI*>(a.grad_d)[tok + t] = from_f32<TI>(-A * ga[e]);
                sum = fmaf(-sd[t], ga[e], sum);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (in.sum_A && lane == 0) in.sum_A[slot * a.H + h] = sum;
    }
}

// ---- one token -------------------------------------------------------------

constexpr int STEP_THREADS = 256, STEP_UNR = 4;

// DK / 4 lanes to a state row, four columns a lane; the row's three dots (S k,
// S q, k q) are one round of shuffles, and o = a S q + u (k.q) needs no second
// one.  A state element is read and written once: bound by HBM.  UNR rows a
// lane keep more loads in flight where there are many (us of 2048 heads of 128 x
// 128 with UNR 1, 2, 4: 55.1, 54.9, 53.3, 74 % of what a copy reaches; of 256:
// 8.05, 8.27, 8.33).
template <typename TI, typename TO, int DK, int UNR>
__global__ void __launch_bounds__(STEP_THREADS) delta_step_kernel(const DeltaArgs a, const float* state, float* next) {
    constexpr int LPR = DK / 4, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31, sub = lane / LPR, col = lane % LPR * 4;
    const long long rows = static_cast<long long>(a.B) * a.H * a.dv;
    const long long first = (static_cast<long long>(blockIdx.x) * (STEP_THREADS / 32) + (threadIdx.x >> 5)) * RPW * UNR + sub;
    float4 S[UNR];
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
        const long long row = first + u * RPW;
        S[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < rows) S[u] = __ldcs(reinterpret_cast<const float4*>(state + row * DK + col));
    }
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
        const long long row = first + u * RPW;
        const bool on = row < rows;
        const long long bh = on ? row / a.dv : 0;
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f), q = k;
        float v = 0.f, al = 0.f, be = 0.f;
        if (on) {
            k = load4(static_cast<const TI*>(a.k) + bh * DK + col);
            q = load4(static_cast<const TI*>(a.q) + bh * DK + col);
            v = to_f32(static_cast<const TI*>(a.v)[row]);
            al = expf(-a.A[bh % a.H] * to_f32(static_cast<const TI*>(a.d)[bh]));
            be = to_f32(static_cast<const TI*>(a.beta)[bh]);
        }
        float p[3];
        p[0] = S[u].x * k.x + S[u].y * k.y + (S[u].z * k.z + S[u].w * k.w);
        p[1] = S[u].x * q.x + S[u].y * q.y + (S[u].z * q.z + S[u].w * q.w);
        p[2] = k.x * q.x + k.y * q.y + (k.z * q.z + k.w * q.w);
        row_sums<LPR>(p);
        const float w = be * (v - al * p[0]);
        if (on) {
            __stcs(reinterpret_cast<float4*>(next + row * DK + col),
                   make_float4(fmaf(w, k.x, al * S[u].x), fmaf(w, k.y, al * S[u].y), fmaf(w, k.z, al * S[u].z),
                               fmaf(w, k.w, al * S[u].w)));
            if (lane % LPR == 0) static_cast<TO*>(a.out)[row] = from_f32<TO>(fmaf(w, p[2], al * p[1]));
        }
    }
}

// ---- host --------------------------------------------------------------------

template <typename F>
kdn_status by_type(kdn_dtype in, kdn_dtype out, F f) {
    if (in == KDN_BF16) return out == KDN_BF16 ? f(__nv_bfloat16(), __nv_bfloat16()) : f(__nv_bfloat16(), float());
    return out == KDN_BF16 ? f(float(), __nv_bfloat16()) : f(float(), float());
}
template <typename F>
kdn_status by_size(int dk, F f) {
    switch (dk) {
        case 16: return f(std::integral_constant<int, 16>());
        case 32: return f(std::integral_constant<int, 32>());
        case 64: return f(std::integral_constant<int, 64>());
        default: return f(std::integral_constant<int, 128>());
    }
}

template <typename K>
kdn_status set_smem(K kernel, size_t bytes) {
    return from_cuda(allow_smem(reinterpret_cast<const void*>(kernel), bytes));
}

long long state_rows(const DeltaArgs& a) { return static_cast<long long>(a.offsets ? a.nseq : a.B) * a.H; }

template <int DK>
long long walk_blocks(const DeltaArgs& a) {
    return state_rows(a) * ((a.dv + Shape<DK>::ROWS - 1) / Shape<DK>::ROWS);
}
constexpr long long kMostBlocks = 0x7fffffffLL;

// A call's stream-ordered scratch, freed on the stream when it leaves scope.
struct Scratch {
    cudaStream_t stream;
    void* p = nullptr;
    explicit Scratch(cudaStream_t s) : stream(s) {}
    kdn_status take(long long bytes) { return from_cuda(cudaMallocAsync(&p, static_cast<size_t>(bytes), stream)); }
    ~Scratch() {
        if (p) cudaFreeAsync(p, stream);
    }
};

long long rounded(long long bytes) { return (bytes + 255) / 256 * 256; }

// The backward's scratch: states, adjoints, r, y, shares of dA.
struct BackLayout {
    long long states, rows, shares;
    BackLayout(int B, int H, int T, int dk, int dv, int nseq) {
        const long long slots = slots_of(B, T, nseq);
        states = rounded(slots * H * dv * dk * 4);
        rows = rounded(static_cast<long long>(B) * H * T * dv * 4);
        shares = rounded(slots * H * 4);
    }
    long long bytes() const { return 2 * states + 2 * rows + shares; }
};

}  // namespace
}  // namespace delta

using namespace delta;

bool delta_fits(int B, int H, int T, int dk, int dv, int nseq, kdn_dtype in_dtype, bool back) {
    if (T == 0 || !(back || tc_takes_fwd(B, H, T, dk, dv, nseq, in_dtype))) return true;
    return slots_of(B, T, nseq) * H <= kMostBlocks;
}

long long delta_fwd_workspace_bytes(int B, int H, int T, int dk, int dv, int nseq, kdn_dtype in_dtype) {
    return tc_takes_fwd(B, H, T, dk, dv, nseq, in_dtype) ? tc_fwd_bytes(B, H, T, nseq) : 0;
}

long long delta_bwd_workspace_bytes(int B, int H, int T, int dk, int dv, int nseq, kdn_dtype in_dtype) {
    if (T == 0) return 0;
    const long long bytes = BackLayout(B, H, T, dk, dv, nseq).bytes();
    // (the type of grad_out, which this does not know, decides the form)
    const long long tc = tc_takes(B, H, dk, dv, nseq, in_dtype) ? tc_bwd_bytes(B, H, T, nseq) : 0;
    return tc > bytes ? tc : bytes;
}

kdn_status delta_fwd_launch(const DeltaArgs& a, cudaStream_t stream, long long wait_ns) {
    if (tc_takes_fwd(a.B, a.H, a.T, a.dk, a.dv, a.nseq, a.in_dtype)) {
        Scratch scratch(stream);
        char* ws = static_cast<char*>(a.workspace);
        if (!ws) {
            const kdn_status s = scratch.take(tc_fwd_bytes(a.B, a.H, a.T, a.nseq));
            if (s != KDN_OK) return s;
            ws = static_cast<char*>(scratch.p);
        }
        return tc_fwd(a, ws, stream, wait_ns);
    }
    return by_type(a.in_dtype, a.out_dtype, [&](auto ti, auto to) {
        return by_size(a.dk, [&](auto dk) {
            using TI = decltype(ti);
            using TO = decltype(to);
            constexpr int DK = decltype(dk)::value;
            const long long blocks = walk_blocks<DK>(a);
            if (blocks > kMostBlocks) return KDN_ERR_INVALID_ARG;
            constexpr int smem = WalkShared<TI, TI, DK>::BYTES;
            auto kernel = delta_walk_kernel<TI, TO, DK, false>;
            const kdn_status s = set_smem(kernel, smem);
            if (s != KDN_OK) return s;
            kernel<<<static_cast<unsigned>(blocks), WALK_ALL, smem, stream>>>(a, Keep{});
            return from_cuda(cudaGetLastError());
        });
    });
}

kdn_status delta_bwd_launch(const DeltaArgs& a, cudaStream_t stream, long long wait_ns) {
    if (a.T == 0) {   // the state passes through, and no token has a share of dA
        cudaError_t e = cudaSuccess;
        const size_t bytes = static_cast<size_t>(state_rows(a)) * a.dv * a.dk * 4;
        if (a.grad_S0)
            e = a.grad_final_state ? cudaMemcpyAsync(a.grad_S0, a.grad_final_state, bytes, cudaMemcpyDeviceToDevice, stream)
                                   : cudaMemsetAsync(a.grad_S0, 0, bytes, stream);
        if (e == cudaSuccess && a.grad_A) e = cudaMemsetAsync(a.grad_A, 0, sizeof(float) * a.H, stream);
        return from_cuda(e);
    }
    const BackLayout lay(a.B, a.H, a.T, a.dk, a.dv, a.nseq);
    const long long slots = slots_of(a.B, a.T, a.nseq);
    Scratch scratch(stream);
    char* ws = static_cast<char*>(a.workspace);
    if (!ws) {
        const kdn_status s = scratch.take(delta_bwd_workspace_bytes(a.B, a.H, a.T, a.dk, a.dv, a.nseq, a.in_dtype));
        if (s != KDN_OK) return s;
        ws = static_cast<char*>(scratch.p);
    }
    if (tc_takes(a.B, a.H, a.dk, a.dv, a.nseq, a.in_dtype) && a.out_dtype == KDN_BF16) return tc_bwd(a, ws, stream, wait_ns);
    float* states = reinterpret_cast<float*>(ws);
    float* adjoints = reinterpret_cast<float*>(ws + lay.states);
    float* r = reinterpret_cast<float*>(ws + 2 * lay.states);
    float* y = reinterpret_cast<float*>(ws + 2 * lay.states + lay.rows);
    float* shares = reinterpret_cast<float*>(ws + 2 * lay.states + 2 * lay.rows);
    return by_type(a.in_dtype, a.out_dtype, [&](auto ti, auto to) {
        return by_size(a.dk, [&](auto dk) {
            using TI = decltype(ti);
            using TO = decltype(to);
            constexpr int DK = decltype(dk)::value;
            const long long blocks = walk_blocks<DK>(a);
            if (blocks > kMostBlocks) return KDN_ERR_INVALID_ARG;
            auto walk = delta_walk_kernel<TI, float, DK, true>;
            auto back = delta_back_kernel<TI, TO, DK>;
            auto grad = delta_grad_kernel<TI, TO, DK>;
            constexpr int walk_smem = WalkShared<TI, TI, DK>::BYTES, back_smem = WalkShared<TI, TO, DK>::BYTES;
            kdn_status s = set_smem(walk, walk_smem);
            if (s == KDN_OK) s = set_smem(back, back_smem);
            if (s == KDN_OK) s = set_smem(grad, grad_smem<DK>(128));
            if (s != KDN_OK) return s;
            walk<<<static_cast<unsigned>(blocks), WALK_ALL, walk_smem, stream>>>(a, Keep{states, r});
            back<<<static_cast<unsigned>(blocks), WALK_ALL, back_smem, stream>>>(a, Keep{adjoints, y});
            grad<<<static_cast<unsigned>(slots * a.H), GRAD_THREADS, grad_smem<DK>(a.dv), stream>>>(
                a, GradIn{states, adjoints, r, y, a.grad_A ? shares : nullptr});
            s = from_cuda(cudaGetLastError());
            if (s == KDN_OK && a.grad_A)
                s = from_cuda(sum_rows(shares, slots, a.H, a.grad_A, nullptr, a.H, stream));
            return s;
        });
    });
}

kdn_status delta_step_launch(const DeltaArgs& a, const float* state, float* next, cudaStream_t stream) {
    return by_type(a.in_dtype, a.out_dtype, [&](auto ti, auto to) {
        return by_size(a.dk, [&](auto dk) {
            using TI = decltype(ti);
            using TO = decltype(to);
            constexpr int DK = decltype(dk)::value, RPW = 32 / (DK / 4), NW = STEP_THREADS / 32;
            const long long rows = static_cast<long long>(a.B) * a.H * a.dv;
            auto go = [&](auto unr) {
                constexpr int UNR = decltype(unr)::value;
                const long long blocks = (rows + NW * RPW * UNR - 1) / (NW * RPW * UNR);
                if (blocks > kMostBlocks) return KDN_ERR_INVALID_ARG;
                delta_step_kernel<TI, TO, DK, UNR><<<static_cast<unsigned>(blocks), STEP_THREADS, 0, stream>>>(a, state, next);
                return from_cuda(cudaGetLastError());
            };
            // few rows want every SM, many want loads in flight
            if (rows < static_cast<long long>(NW) * RPW * STEP_UNR * sm_count() * 8) return go(std::integral_constant<int, 1>());
            return go(std::integral_constant<int, STEP_UNR>());
        });
    });
}

}  // namespace kdn
