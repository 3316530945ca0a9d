// delta_tc.cu -- the gated delta rule in chunks of 64 tokens on the tensor
// cores, for bf16 inputs and heads of 128 (narrower ones have zeros behind;
// delta_device.cuh has the rule, delta_scan.cu the token-by-token form for the
// rest).
//
// With g_t the log decay since the chunk began and E_ts = e^{g_t - g_s}, and S
// the state before the chunk,
//     G = (K K^T) . E (s < t),   P = (Q K^T) . E (s <= t),
//     T = -G (1 + beta G)^{-1}   (strictly lower),
//     Z = V - e^g K S^T,   R = Z + T (beta Z),   U = beta R,
//     O = e^g Q S^T + P U,
//     S' = e^{g_C} S + U^T (e^{g_C - g} K).
// T and P need no state: delta_prep_kernel makes them for all chunks side by
// side, and delta_chunk_kernel walks a head's chunks with five products each.
//
// Precision.  The inputs are bf16 and the results as exact as fp32 arithmetic
// makes them: every other operand is a pair of fp16 numbers hi + lo (22 bits;
// two products with an input, three of two such pairs, fp32 sums in tensor
// memory).  Pairs of bf16 would keep 16 bits at the same cost; the state was
// then 3e-6 off, and the gradient of A, a sum over all tokens whose chunks'
// errors add up, up to 8e-5.  fp16 has 5 bits of exponent, so operands are
// scaled by exact powers of two, undone where the fp32 sums are read: inputs
// and the chunk's T and P by one for their tile, Z, U and S by one for each
// state row, from the row's largest magnitude (rows do not touch one another,
// whatever their sizes).  An element is exact to 2^-38 of the largest.
#include <type_traits>
#include <utility>

#include <cuda_fp16.h>

#include "delta_device.cuh"
#include "delta_tc.h"
#include "kdn.h"
#include "kdn_device.cuh"
#include "kdn_internal.h"
#include "kernel_setup.h"
#include "sum_rows.cuh"

namespace kdn {
namespace delta {
namespace {

__device__ int g_delta_error = 0;

constexpr int D = 128;                       // d_k = d_v
constexpr int C = CHUNK;
// Shared tiles are made of core matrices of 8 rows x 16 bytes, 128 contiguous
// bytes each, one after another along the columns: element (r, c) of a tile
// with W columns of 2 bytes is at (r / 8) * (W / 8) * 128 + (c / 8) * 128 +
// (r % 8) * 16 + (c % 8) * 2.
constexpr int ROWS_D = (D / 8) * 128;        // 8 rows of a tile of 128 columns
constexpr int ROWS_C = (C / 8) * 128;        // 8 rows of a tile of 64 columns
constexpr int TILE_X = C * D * 2;            // a chunk's q, k or v
constexpr int TILE_T = C * C * 2;            // hi or lo of T or P
__host__ __device__ constexpr int at_d(int r, int c8) { return (r / 8) * ROWS_D + c8 * 128 + (r % 8) * 16; }
__host__ __device__ constexpr int at_c(int r, int c8) { return (r / 8) * ROWS_C + c8 * 128 + (r % 8) * 16; }

// What the preparation leaves of a chunk, as the walk reads it.
constexpr int PREP_KQ = 0;                   // k and q, one tile of 2 x 64 rows
constexpr int PREP_T = 2 * TILE_X;           // T hi, lo
constexpr int PREP_P = PREP_T + 2 * TILE_T;  // P hi, lo
constexpr int PREP_GATES = PREP_P + 2 * TILE_T;   // fp32: five rows of 64, then single values
constexpr int G_E = 0, G_W = C, G_BETA = 2 * C, G_HI = 3 * C, G_LO = 4 * C;   // e^g, e^{g_C - g}, beta, log2 e . g
// e^{g_C}, and the powers of two that undo the scales of k, q, do, T and P
constexpr int G_END = 5 * C, G_KDN = G_END + 1, G_QDN = G_END + 2, G_XDN = G_END + 3, G_TDN = G_END + 4, G_PDN = G_END + 5,
              G_ALL = G_END + 6;
constexpr int PREP_BYTES = PREP_GATES + 1408;
static_assert(G_ALL * 4 <= 1408, "the gates' room");
constexpr int PREP_STEP = PREP_BYTES + TILE_X;   // (backward: do behind it)
// What the backward's walks leave of a chunk beside it, fp32: a state (S before
// the chunk, or its adjoint D behind it) as [i][j] and the rows R and Y as
// [i][t]; four columns of all 128 rows i, then the next four.
constexpr int STATE_BYTES = D * D * 4, ROWS_BYTES = D * C * 4;
__host__ __device__ constexpr int at_f(int i, int c4) { return c4 * D * 16 + i * 16; }

// x as fp16 pairs hi + lo: hi rounded to nearest, lo what is left, rounded:
// within 2^-22 of x (2^-25 where lo is subnormal).
__device__ __forceinline__ void halves(float2 x, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __float22half2_rn(x);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const float2 d = __ffma2_rn(__half22float2(h), make_float2(-1.f, -1.f), x);
    const __half2 l = __float22half2_rn(d);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}

// The power of two that brings the largest magnitude m to [2^13, 2^14), and its
// inverse.  (What is below 2^-113 counts as that; infinities stay infinite.)
__device__ __forceinline__ void scale_of(float m, float& up, float& down) {
    const uint32_t e = max(__float_as_uint(m) >> 23, 14u);
    up = __uint_as_float((267u - e) << 23);
    down = __uint_as_float((e - 13u) << 23);
}
// ... of an input's tile: at most 2^60, so that products of two stay floats.
__device__ __forceinline__ void input_scale(float m, float& up, float& down) {
    scale_of(fmaxf(m, 0x1p-47f), up, down);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// The largest magnitude; NaN where there is one.
__device__ __forceinline__ float largest(float m, const float2 (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(x[e].x), "f"(x[e].y));
    return m;
}
// The instruction descriptor's types: fp16 operands where the bf16 form has bf16's bits.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool a_mn = false, bool b_mn = false) {
    return umma_idesc_bf16_f32(m, n, a_mn, b_mn) & ~((7u << 7) | (7u << 10));
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 16 bytes into shared memory, or zeros.
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// n tokens of k, then of q, as one tile of 2 x 64 rows (zeros behind the last
// token and the last of dk columns), by `threads` threads.  A warp instruction moves 8 tokens x 4 of
// their 16-byte pieces, so that its writes hit each bank group four times.
__device__ __forceinline__ void load_kq(uint32_t tile, const __nv_bfloat16* k, const __nv_bfloat16* q, int n, int dk,
                                        int tid, int threads) {
    const int lane = tid & 31, a = lane & 7, b = lane >> 3;
    for (int w = tid >> 5; w < 2 * C / 8 * 4; w += threads >> 5) {
        const int r = (w >> 2) * 8 + a, c8 = (w & 3) * 4 + b, t = r & (C - 1);
        const bool there = t < n && c8 * 8 < dk;
        copy16_or_zero(tile + at_d(r, c8), (r < C ? k : q) + (there ? static_cast<long long>(t) * dk + c8 * 8 : 0), there);
    }
}

// 8 bf16 numbers as fp16, times a power of two.
__device__ __forceinline__ uint4 to_half(uint4 w, float up) {
    uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = make_float2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u));
        const __half2 h = __float22half2_rn(__fmul2_rn(f, both(up)));
        u[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// 8 bf16 numbers without those that are not finite (0 in their place; `all`
// turns false where there are such).
__device__ __forceinline__ uint4 finite_bf16(uint4 w, bool* all = nullptr) {
    uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t bad = __vcmpeq2(u[e] & 0x7f807f80u, 0x7f807f80u);
        if (all) *all = *all && bad == 0u;
        u[e] &= ~bad;
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}
// The largest magnitude of 8 bf16 numbers, as bits of two.
__device__ __forceinline__ uint32_t largest_bf16(uint32_t m, uint4 w) {
    m = __vmaxu2(m, w.x & 0x7fff7fffu);
    m = __vmaxu2(m, w.y & 0x7fff7fffu);
    m = __vmaxu2(m, w.z & 0x7fff7fffu);
    return __vmaxu2(m, w.w & 0x7fff7fffu);
}

// Piece i (of 8 columns) of rows of D, of which there are dv in memory and zeros behind.
template <bool FULL>
__device__ __forceinline__ uint4 piece(const __nv_bfloat16* p, int i, int dv) {
    if (FULL) return reinterpret_cast<const uint4*>(p)[i];
    const int c = i % (D / 8) * 8;
    return c < dv ? *reinterpret_cast<const uint4*>(p + static_cast<long long>(i / (D / 8)) * dv + c) : make_uint4(0u, 0u, 0u, 0u);
}

// ---- preparation -------------------------------------------------------------

constexpr int PREP_THREADS = 128;
constexpr int LG = C + 4, LX = 36;           // a row of G, T and of X in shared memory
// G (then T, block by block in its place), N = G beta and X lie where k and q
// lay before the product: five CTAs to an SM hide one another's waits.
constexpr int P_OFF_KQ = 0, P_OFF_G = 0, P_OFF_N = P_OFF_G + C * LG * 4, P_OFF_X = P_OFF_N + C * LG * 4,
              P_OFF_GATE = P_OFF_X + 32 * LX * 4, P_SMEM = P_OFF_GATE + 3 * C * 4 + 128;
static_assert(P_OFF_GATE >= 2 * TILE_X, "the gates lie behind k and q");

// acc[r] += sum_s A[r * RS][s] B[s] for R rows and 4 columns: A's rows in shared
// memory LA apart, B's LB apart.
template <int R, int RS, int N>
__device__ __forceinline__ void small_product(const float* A, int LA, const float* B, int LB, float2 (&acc)[R][2]) {
#pragma unroll
    for (int s = 0; s < N; s += 4) {
        float4 b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = *reinterpret_cast<const float4*>(B + (s + e) * LB);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float4 f = *reinterpret_cast<const float4*>(A + r * RS * LA + s);
            const float x[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[r][0] = __ffma2_rn(make_float2(x[e], x[e]), make_float2(b[e].x, b[e].y), acc[r][0]);
                acc[r][1] = __ffma2_rn(make_float2(x[e], x[e]), make_float2(b[e].z, b[e].w), acc[r][1]);
            }
        }
    }
}

// T21 = -(X + T2 (beta2 X)), X = G21 + N21 T1 with N = G beta, of pairs of
// blocks of SIZE: a thread has 4 columns of R rows, 16 apart.
template <int SIZE>
__device__ __forceinline__ void join_blocks(float* sT, const float* sN, float* sXb, const float* sb) {
    constexpr int PER = PREP_THREADS * 2 * SIZE / C, R = SIZE / 16;
    const int p = threadIdx.x / PER, i = threadIdx.x % PER, o = 2 * SIZE * p;
    const int c4 = (i % (SIZE / 4)) * 4, r0 = i / (SIZE / 4);
    float* Xb = sXb + p * SIZE * LX;
    float2 x[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float4 f = *reinterpret_cast<const float4*>(sT + (o + SIZE + r0 + 16 * r) * LG + o + c4);   // G21
        x[r][0] = make_float2(f.x, f.y);
        x[r][1] = make_float2(f.z, f.w);
    }
    small_product<R, 16, SIZE>(sN + (o + SIZE + r0) * LG + o, LG, sT + o * LG + o + c4, LG, x);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float b = sb[o + SIZE + r0 + 16 * r];
        *reinterpret_cast<float4*>(Xb + (r0 + 16 * r) * LX + c4) =
            make_float4(b * x[r][0].x, b * x[r][0].y, b * x[r][1].x, b * x[r][1].y);
    }
    __syncthreads();
    small_product<R, 16, SIZE>(sT + (o + SIZE + r0) * LG + o + SIZE, LG, Xb + c4, LX, x);
#pragma unroll
    for (int r = 0; r < R; ++r)
        *reinterpret_cast<float4*>(sT + (o + SIZE + r0 + 16 * r) * LG + o + c4) =
            make_float4(-x[r][0].x, -x[r][0].y, -x[r][1].x, -x[r][1].y);
    __syncthreads();
}

// A CTA makes one chunk's T and P: one product [K; Q] K^T (M = 128, N = 64),
// then T from G by blocks.  With T1, T2 the blocks' own,
//     T21 = -(1 + T2 beta2) G21 (1 + beta1 T1),
// from 16 x 16 blocks that a warp solves row after row.  No power of G is
// formed: keys that are alike make those large.  Bound by the waits of the solve's
// steps and by HBM: 8192 chunks of 128 193 us, 811 MB, 62 % of what a copy moves.
template <bool FULL>
__global__ void __launch_bounds__(PREP_THREADS) delta_prep_kernel(const DeltaArgs a, char* prep, long long wait_ns) {
    extern __shared__ __align__(128) unsigned char smem[];
    float* sG = reinterpret_cast<float*>(smem + P_OFF_G);        // [t][s]
    float* sN = reinterpret_cast<float*>(smem + P_OFF_N);        // G beta
    float* gh = reinterpret_cast<float*>(smem + P_OFF_GATE);     // log2 decay since the chunk began, as two floats
    float* gl = gh + C;
    float* sb = gl + C;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + P_OFF_GATE + 3 * C * 4);
    uint32_t* holder = reinterpret_cast<uint32_t*>(bar + 1);
    uint32_t* tops = holder + 1;                                 // [4 warps][k, q, do], then [4] of T
    int* gone = reinterpret_cast<int*>(tops + 16);               // the first token whose k, beta or decay is not finite
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = static_cast<int>(blockIdx.x % a.H);
    const long long slot = blockIdx.x / a.H;
    long long n, row;
    int t0, m;
    if (!chunk_of(a, slot, &n, &t0, &m, &row)) return;
    const long long tok = (row * a.H + h) * a.T + t0;
    const int bytes = a.grad_out ? PREP_STEP : PREP_BYTES;
    char* out = prep + (slot * a.H + h) * static_cast<long long>(bytes);

    const int dk = FULL ? D : a.dk, dv = FULL ? D : a.dv;
    const __nv_bfloat16* go = static_cast<const __nv_bfloat16*>(a.grad_out) + (a.grad_out ? tok * dv : 0);
    load_kq(smem_addr(smem), static_cast<const __nv_bfloat16*>(a.k) + tok * dk,
            static_cast<const __nv_bfloat16*>(a.q) + tok * dk, m, dk, tid, PREP_THREADS);
    if (warp == 0) {
        tmem_alloc(holder, 64);
    } else if (warp == 1) {
        if (lane == 0) {
            mbar_init(bar, 1);
            mbar_init_fence();
        }
        // sums in 64 bits: the differences of a long chunk's decays keep their bits.  A token's own
        // decay of 2^-1024 is 0 in fp32 alike.
        const double A = -1.4426950408889634 * a.A[h];
        double g[2];
        float b[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            g[e] = t < m ? A * to_f32(static_cast<const __nv_bfloat16*>(a.d)[tok + t]) : 0.0;
            if (g[e] < -1024.0) g[e] = -1024.0;
            b[e] = t < m ? to_f32(static_cast<const __nv_bfloat16*>(a.beta)[tok + t]) : 0.f;
        }
        double s = g[0] + g[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += x;
        }
        const double end = __shfl_sync(0xffffffffu, s, 31), before = __shfl_up_sync(0xffffffffu, s, 1);
        if (lane > 0) g[0] += before;            // (not s - g[1]: the second token's may be no number)
        g[1] = s;
        float* gates = reinterpret_cast<float*>(out + PREP_GATES);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            gh[t] = static_cast<float>(g[e]);
            gl[t] = static_cast<float>(g[e] - gh[t]);
            sb[t] = b[e];
            gates[G_E + t] = exp2f(static_cast<float>(g[e]));
            gates[G_W + t] = exp2f(static_cast<float>(end - g[e]));
            gates[G_BETA + t] = b[e];
            gates[G_HI + t] = gh[t];
            gates[G_LO + t] = gl[t];
        }
        const bool fine0 = isfinite(g[0]) && isfinite(b[0]), fine1 = isfinite(g[1]) && isfinite(b[1]);
        const int first = __reduce_min_sync(0xffffffffu, !fine0 ? 2 * lane : !fine1 ? 2 * lane + 1 : C);
        if (lane == 0) {
            gates[G_END] = exp2f(static_cast<float>(end));
            *gone = first;
        }
    }
    uint32_t top[3] = {0u, 0u, 0u};
    if (a.grad_out)
        for (int i = tid; i < m * (D / 8); i += PREP_THREADS) top[2] = largest_bf16(top[2], piece<FULL>(go, i, dv));
    copies_done();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *holder, base = smem_addr(smem);
    for (int i = tid; i < C * (D / 8); i += PREP_THREADS) {
        top[0] = largest_bf16(top[0], *reinterpret_cast<const uint4*>(smem + P_OFF_KQ + i * 16));
        top[1] = largest_bf16(top[1], *reinterpret_cast<const uint4*>(smem + P_OFF_KQ + TILE_X + i * 16));
    }
#pragma unroll
    for (int e = 0; e < 3; ++e) {
        const uint32_t x = __reduce_max_sync(0xffffffffu, max(top[e] >> 16, top[e] & 0xffffu));
        if (lane == 0) tops[3 * warp + e] = x;
    }
    if (tid == 0) {
        constexpr uint32_t IDESC = umma_idesc_bf16_f32(128, C);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t d = umma_desc_kmajor(base + P_OFF_KQ + ks * 256, 128, ROWS_D);
            umma_bf16(tmem, d, d, IDESC, ks > 0 ? 1u : 0u);
        }
        if (t0 / C != a.stall) umma_commit(bar);
    }
    __syncthreads();   // the magnitudes are here
    uint32_t most3[3];
#pragma unroll
    for (int e = 0; e < 3; ++e) most3[e] = max(max(tops[e], tops[3 + e]), max(tops[6 + e], tops[9 + e]));
    // What is not finite is to spoil its own token's outputs and all behind, nothing before: scales
    // come from the rest, and the solve leaves out the tokens from the first such k on (0 times NaN
    // is NaN).  Their own Z is not finite, which the walk looks at.
    if (max(most3[0], max(most3[1], most3[2])) >= 0x7f80u) {
        __syncthreads();
        uint32_t t3[3] = {0u, 0u, 0u};
        for (int i = tid; i < C * (D / 8); i += PREP_THREADS) {
            bool k_fine = true;
            t3[0] = largest_bf16(t3[0], finite_bf16(*reinterpret_cast<const uint4*>(smem + P_OFF_KQ + i * 16), &k_fine));
            t3[1] = largest_bf16(t3[1], finite_bf16(*reinterpret_cast<const uint4*>(smem + P_OFF_KQ + TILE_X + i * 16)));
            if (!k_fine) atomicMin(gone, i / (D / 8 * 8) * 8 + i % 8);   // (piece i of the tile: its row)
            if (a.grad_out && i < m * (D / 8)) t3[2] = largest_bf16(t3[2], finite_bf16(piece<FULL>(go, i, dv)));
        }
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            const uint32_t x = __reduce_max_sync(0xffffffffu, max(t3[e] >> 16, t3[e] & 0xffffu));
            if (lane == 0) tops[3 * warp + e] = x;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 3; ++e) most3[e] = max(max(tops[e], tops[3 + e]), max(tops[6 + e], tops[9 + e]));
    }
    const int bad = *gone;
    float ups[3], downs[3];
#pragma unroll
    for (int e = 0; e < 3; ++e) input_scale(__uint_as_float(most3[e] << 16), ups[e], downs[e]);
    if (tid >= bad && tid < C) sb[tid] = 0.f;    // (for the solve; read behind the next barrier)
    for (int i = tid; i < 2 * C * (D / 8); i += PREP_THREADS)
        *reinterpret_cast<uint4*>(out + PREP_KQ + i * 16) =
            to_half(*reinterpret_cast<const uint4*>(smem + P_OFF_KQ + i * 16), i < C * (D / 8) ? ups[0] : ups[1]);
    if (a.grad_out) {
        for (int i = tid; i < C * (D / 8); i += PREP_THREADS) {
            const int t = i / (D / 8), c8 = i % (D / 8);
            *reinterpret_cast<uint4*>(out + PREP_BYTES + at_d(t, c8)) = t < m ? to_half(piece<FULL>(go, i, dv), ups[2]) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    const bool late = !mbar_wait(bar, 0, wait_ns);
    if (__syncthreads_or(late)) {      // given up: what the product may still read and write is left as it is
        if (warp == 0) {
            mbar_wait(bar, 0, wait_ns);
            tc_fence_after_sync();
            tmem_dealloc(tmem, 64);
            if (lane == 0) record_error(&g_delta_error, KDN_ERR_TIMEOUT);
        }
        return;
    }
    // the product is done and k and q are read: they may be overwritten
    tc_fence_after_sync();
    // |P| <= 128 max|k| max|q|: scaled by both and by 2^-21 it is below 2^14
    const float p_up = ups[0] * ups[1] * 0x1p-21f;
    if (tid == 0) {
        float* gates = reinterpret_cast<float*>(out + PREP_GATES);
#pragma unroll
        for (int e = 0; e < 3; ++e) gates[G_KDN + e] = downs[e];
        gates[G_PDN] = downs[0] * downs[1] * 0x1p21f;
    }
    {   // row tid: K K^T of token tid, or Q K^T of token tid - 64
        const int t = tid & (C - 1);
        const bool reads = tid < C;          // k_t reads the state before its token, q_t the one after
        const float2 th = make_float2(gh[t], gh[t]), tl = make_float2(gl[t], gl[t]), minus = make_float2(-1.f, -1.f);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float x[32];
            tmem_ld32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + 32 * half, x);
            if (__any_sync(0xffffffffu, 32 * half <= t)) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const int s = 32 * half + e;
                    const float4 h = *reinterpret_cast<const float4*>(gh + s), l = *reinterpret_cast<const float4*>(gl + s);
                    const float2 w0 = __fadd2_rn(__ffma2_rn(make_float2(h.x, h.y), minus, th),
                                                 __ffma2_rn(make_float2(l.x, l.y), minus, tl));
                    const float2 w1 = __fadd2_rn(__ffma2_rn(make_float2(h.z, h.w), minus, th),
                                                 __ffma2_rn(make_float2(l.z, l.w), minus, tl));
                    const int last = !reads ? t : t < bad ? t - 1 : -1;
                    x[e] = s <= last ? x[e] * ex2(w0.x) : 0.f;
                    x[e + 1] = s + 1 <= last ? x[e + 1] * ex2(w0.y) : 0.f;
                    x[e + 2] = s + 2 <= last ? x[e + 2] * ex2(w1.x) : 0.f;
                    x[e + 3] = s + 3 <= last ? x[e + 3] * ex2(w1.y) : 0.f;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = 0.f;
            }
            if (reads) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const int s = 32 * half + e;
                    const float4 b = *reinterpret_cast<const float4*>(sb + s);
                    *reinterpret_cast<float4*>(sG + t * LG + s) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                    *reinterpret_cast<float4*>(sN + t * LG + s) =
                        make_float4(x[e] * b.x, x[e + 1] * b.y, x[e + 2] * b.z, x[e + 3] * b.w);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) halves(make_float2(p_up * x[e + 2 * p], p_up * x[e + 2 * p + 1]), hi[p], lo[p]);
                    const int off = PREP_P + at_c(t, 4 * half + e / 8);
                    *reinterpret_cast<uint4*>(out + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(out + off + TILE_T) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();   // G is in shared memory; tensor memory is read
    if (warp == 0) tmem_dealloc(tmem, 64);
    {   // 16 x 16 blocks on the diagonal: lane c has column c, T_t = -(G_t + sum_{s < t} N_ts T_s) row after row
        const int o = 16 * warp, c = lane & 15;
        float col[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float x = sG[(o + t) * LG + o + c], y = 0.f;
#pragma unroll
            for (int s4 = 0; s4 < t; s4 += 4) {
                const float4 f = *reinterpret_cast<const float4*>(sN + (o + t) * LG + o + s4);
                x = fmaf(f.x, col[s4], x);
                if (s4 + 1 < t) y = fmaf(f.y, col[s4 + 1], y);
                if (s4 + 2 < t) x = fmaf(f.z, col[s4 + 2], x);
                if (s4 + 3 < t) y = fmaf(f.w, col[s4 + 3], y);
            }
            col[t] = -(x + y);               // (0 above and on the diagonal: G is, and the rows before are)
        }
        __syncwarp();
        if (lane < 16)
#pragma unroll
            for (int t = 0; t < 16; ++t) sG[(o + t) * LG + o + c] = col[t];
    }
    __syncthreads();
    join_blocks<16>(sG, sN, reinterpret_cast<float*>(smem + P_OFF_X), sb);
    join_blocks<32>(sG, sN, reinterpret_cast<float*>(smem + P_OFF_X), sb);
    float2 x[4][4];
    float most = 0.f;
#pragma unroll
    for (int n4 = 0; n4 < 4; ++n4) {
        const int i = tid + n4 * PREP_THREADS, t = i & (C - 1), c8 = i / C;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            x[n4][p] = *reinterpret_cast<const float2*>(sG + t * LG + 8 * c8 + 2 * p);
            most = fmaxf(most, fmaxf(fabsf(x[n4][p].x), fabsf(x[n4][p].y)));
        }
    }
    static_assert(C * (C / 8) == 4 * PREP_THREADS, "four pieces a thread");
    const uint32_t warp_most = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    if (lane == 0) tops[12 + warp] = warp_most;
    __syncthreads();
    float up, down;
    scale_of(__uint_as_float(max(max(tops[12], tops[13]), max(tops[14], tops[15]))), up, down);
    if (tid == 0) reinterpret_cast<float*>(out + PREP_GATES)[G_TDN] = down;
#pragma unroll
    for (int n4 = 0; n4 < 4; ++n4) {
        const int i = tid + n4 * PREP_THREADS, t = i & (C - 1), c8 = i / C;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) halves(__fmul2_rn(x[n4][p], both(up)), hi[p], lo[p]);
        const int off = PREP_T + at_c(t, c8);
        *reinterpret_cast<uint4*>(out + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(out + off + TILE_T) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// ---- the walk ------------------------------------------------------------------

// Warps 0-15 work on the state's rows (thread = row i = lane of tensor memory,
// warp / 4 = quarter of the columns and of the tokens); a thread's 32 columns of
// S stay in its registers.  Warp 16 issues the products, warp 17 brings the
// tiles, one chunk ahead.  Sixteen row warps: with eight, two to a scheduler,
// their dependent steps took 1.6 times as long.  Bound by that chain (exchange of
// a row's largest, halves, product, sums, four times a chunk): 128 heads of 4096
// tokens 244 us, 7600 cycles a chunk, the tensor pipe busy in 30 % of them.
constexpr int ROW_WARPS = 16, MMA_WARP = ROW_WARPS, CH_THREADS = (ROW_WARPS + 2) * 32;
// shared memory: two stages of a prepared chunk and v (backward: do);
// two arrays of the rows' largest magnitudes, one value of each quarter
constexpr int ST_V = PREP_BYTES, STAGE_BYTES = ST_V + TILE_X;
static_assert(ST_V % 128 == 0, "tiles on 128 bytes");
constexpr int CH_OFF_TOP = 2 * STAGE_BYTES, CH_OFF_BAR = CH_OFF_TOP + 2 * 4 * D * 4, CH_SMEM = CH_OFF_BAR + 192;
// ... and the adjoint's e^g do, hi and lo
constexpr int AD_OFF_X = (CH_SMEM + 127) / 128 * 128, AD_SMEM = AD_OFF_X + 2 * D * C * 2;
static_assert(AD_SMEM <= 227 * 1024, "shared memory");
// tensor memory: the chunk's share of S (fp32) and the halves of S as packed
// pairs (an A operand's layout), the accumulators of Z (then of R, then U's
// halves), of Q S^T and of P U, and the halves of beta Z (then of e^{g_C - g} U)
constexpr uint32_t COL_S = 0, COL_SH = 128, COL_SL = 192, COL_Z = 256, COL_QS = 320, COL_O = 384, COL_W = 448;

// Waits that end: the first that runs out marks the CTA, and the others return
// at once.  The rows then run through their chunks without waiting (their
// barriers still match), copies and products are no longer issued, and those in
// flight are waited for before the CTA ends.
struct Waits {
    volatile int* dead;
    long long limit;
    __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) const {
        if (mbar_try_wait(bar, parity)) return;
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(bar, parity)) {
            if (*dead) return;
            if (static_cast<long long>(globaltimer_ns() - t0) > limit) {
                *dead = 1;
                return;
            }
        }
    }
};

// Issue by a whole warp, whose values are all uniform: one thread of it is
// elected for the instruction.  (Out of a branch of one lane each operand went
// through vector registers, and a product took 56 cycles to issue.)
// D (TMEM) = A (TMEM, two fp16 numbers to a column, lane = row) * B^T (smem)
__device__ __forceinline__ void umma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// ... the same with A in shared memory.
__device__ __forceinline__ void umma_sa(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_done(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tmem_st8w(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_get16(uint32_t taddr, float2 (&x)[8]) {
    float v[16];
    tmem_ld16_async(taddr, v);
    tmem_wait_ld16(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = make_float2(v[2 * e], v[2 * e + 1]);
}
// 16 consecutive floats of shared memory (16-byte aligned).
__device__ __forceinline__ void get16(const float* p, float2 (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float4 f = reinterpret_cast<const float4*>(p)[e];
        x[2 * e] = make_float2(f.x, f.y);
        x[2 * e + 1] = make_float2(f.z, f.w);
    }
}
// Column i of 16 rows of [t][D] bf16.
__device__ __forceinline__ void get_column(const __nv_bfloat16* p, float2 (&x)[8]) {
    const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = make_float2(__uint_as_float(static_cast<uint32_t>(u[2 * e * D]) << 16),
                           __uint_as_float(static_cast<uint32_t>(u[(2 * e + 1) * D]) << 16));
}


// The largest of a row's four quarters: each puts its own, and all four warps of
// a lane quarter meet.  (Two arrays in turn: an array's readers are past it when
// the next but one exchange writes it.)  A negative number says that the quarter
// has values that are not finite; `first`: the first such quarter, or 4.
__device__ __forceinline__ float row_top(float* tops, float mine, int q4, int part, int i, int* first = nullptr) {
    tops[part * D + i] = mine;
    asm volatile("bar.sync %0, 128;" ::"r"(1 + q4) : "memory");
    const float t[4] = {tops[i], tops[D + i], tops[2 * D + i], tops[3 * D + i]};
    if (first) {
        const uint32_t sign = __float_as_uint(t[0]) | __float_as_uint(t[1]) | __float_as_uint(t[2]) | __float_as_uint(t[3]);
        *first = 4;
        if (sign >> 31) *first = signbit(t[0]) ? 0 : signbit(t[1]) ? 1 : signbit(t[2]) ? 2 : 3;
    }
    return fmaxf(fmaxf(fabsf(t[0]), fabsf(t[1])), fmaxf(fabsf(t[2]), fabsf(t[3])));
}

__device__ __forceinline__ bool finite(float top) { return top < __int_as_float(0x7f800000); }
// Takes the values from the first that is not finite (or from `from` on) out of
// an operand: the place of that one.  In a product its 0 weights would make NaN of
// the tokens before it.
__device__ __forceinline__ int cut_off(float2 (&x)[8], int from) {
    int n = 16;
#pragma unroll
    for (int t = 15; t >= 0; --t)
        if (t >= from || !isfinite(t & 1 ? x[t / 2].y : x[t / 2].x)) n = t;
#pragma unroll
    for (int t = 0; t < 16; ++t)
        if (t >= n) (t & 1 ? x[t / 2].y : x[t / 2].x) = 0.f;
    return n;
}

// The halves of 16 values times a power of two, one K step.
__device__ __forceinline__ void put_scaled(uint32_t taddr, const float2 (&x)[8], float up) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) halves(__fmul2_rn(x[e], both(up)), hi[e], lo[e]);
    tmem_st8w(taddr, hi);
    tmem_st8w(taddr + 8, lo);
}

// Four consecutive values and more of a kept tile, from column c4 * 4 on.
template <int N>
__device__ __forceinline__ void keep_row(char* tile, int i, int c4, const float2* x) {
#pragma unroll
    for (int e = 0; e < N / 2; ++e)
        *reinterpret_cast<float4*>(tile + at_f(i, c4 + e)) =
            make_float4(x[2 * e].x, x[2 * e].y, x[2 * e + 1].x, x[2 * e + 1].y);
}

// Chunks' tiles by one thread: what the preparation left, and v where it is given
// (with do behind the rest and the last chunk first where not); `zeros`: no values.
__device__ __forceinline__ void load_chunks(unsigned char* smem, uint64_t* full, uint64_t* empty, const Waits& wait,
                                            const __nv_bfloat16* v, int dv, bool zeros, const char* prep, long long step,
                                            int len, int chunks, int stall) {
    int sent = -1;                                   // the last one whose copies were issued
    for (int n = 0; n < chunks; ++n) {
        const int c = v ? n : chunks - 1 - n, st = n & 1, m = zeros ? 0 : min(C, len - c * C);
        if (n >= 2) wait(empty + st, ((n >> 1) - 1) & 1);
        if (*wait.dead) break;
        if (n == stall) continue;                    // (fault injection)
        sent = n;
        unsigned char* stage = smem + st * STAGE_BYTES;
        if (v) {
            // rows as they are; no token: zeros, not what lay there before
            for (int e = m * D * 2; e < TILE_X; e += 16) *reinterpret_cast<uint4*>(stage + ST_V + e) = make_uint4(0u, 0u, 0u, 0u);
            mbar_arrive_expect_tx(full + st, PREP_BYTES + m * dv * 2);
            bulk_g2s(stage, prep + c * step, PREP_BYTES, full + st);
            const __nv_bfloat16* src = v + static_cast<long long>(c) * C * dv;
            if (dv == D) {
                if (m > 0) bulk_g2s(stage + ST_V, src, m * D * 2, full + st);
            } else {   // (the columns behind are zeros from the start)
                for (int t = 0; t < m; ++t) bulk_g2s(stage + ST_V + t * D * 2, src + t * dv, dv * 2, full + st);
            }
        } else {
            mbar_arrive_expect_tx(full + st, PREP_STEP);
            bulk_g2s(stage, prep + c * step, PREP_STEP, full + st);
        }
    }
    // no copy outlives the CTA
    for (int n = max(sent - 1, 0); n <= sent; ++n)
        if (n != stall && !mbar_wait(full + (n & 1), (n >> 1) & 1, wait.limit)) *wait.dead = 1;
}

// A walk's kept tiles; null in a forward call.
struct KeepTiles {
    char* states;      // STATE_BYTES a chunk
    char* rows;        // ROWS_BYTES a chunk
};

// How a walk is cut along the tokens: `parts` parts of `len` chunks.
struct Parts {
    int parts, len;
    const float* starts;   // [rows,parts,D,D]: a part's first state (null: one part, from S0)
    float* ends;           // ENDS: [rows,parts - 1,2,D,D]
};
// OUTPUTS; TILES: no outputs, but the state before each chunk and R; ENDS: of a
// part its end alone, from a zero state (N) or, without values, from the
// identity (M): S behind the part is S M + N whatever S.
enum Walk { OUTPUTS, TILES, ENDS };

template <typename TO, Walk WALK, bool FULL>
__global__ void __launch_bounds__(CH_THREADS, 1) delta_chunk_kernel(const DeltaArgs a, const char* prep, int prep_bytes,
                                                                    const KeepTiles keep, const Parts cut, long long wait_ns) {
    constexpr bool KEEP = WALK != OUTPUTS;             // no outputs
    extern __shared__ __align__(128) unsigned char smem[];
    float* tops = reinterpret_cast<float*>(smem + CH_OFF_TOP);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + CH_OFF_BAR);   // [2] a stage is here
    uint64_t* empty = full + 2;                                        // [2] a stage is read
    uint64_t* done_z = empty + 2;                                      // products: Z, R, S, O
    uint64_t* done_r = done_z + 1;
    uint64_t* done_s = done_r + 1;                                     // [2] (columns 0-63 and 64-127)
    uint64_t* done_o = done_s + 2;
    uint64_t* have_s = done_o + 1;                                     // operands: S [2], beta Z, wU, U
    uint64_t* have_z = have_s + 2;
    uint64_t* have_w = have_z + 1;
    uint64_t* have_u = have_w + 1;
    uint64_t* read_o = have_u + 1;                                     // Q S^T and P U are read
    uint64_t* done_all = read_o + 1;                                   // no product is left
    uint32_t* holder = reinterpret_cast<uint32_t*>(done_all + 1);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int jobs = WALK == ENDS ? 2 * (cut.parts - 1) : cut.parts;   // of a state row
    const long long sr = blockIdx.x / jobs, n = sr / a.H;
    const int job = static_cast<int>(blockIdx.x % jobs), piece = WALK == ENDS ? job >> 1 : job;
    const bool identity = WALK == ENDS && (job & 1);
    const int h = static_cast<int>(sr % a.H);
    Span sp = span_of(a, n);
    if (cut.parts > 1) {   // this part's tokens and chunks
        sp.lo += piece * cut.len * C;
        sp.slot += piece * cut.len;
        if (sp.hi - sp.lo > cut.len * C) sp.hi = sp.lo + cut.len * C;
    }
    const int len = max(sp.hi - sp.lo, 0), chunks = (len + C - 1) / C;
    const int dk = FULL ? D : a.dk, dv = FULL ? D : a.dv;
    const long long tok = (sp.row * a.H + h) * a.T + sp.lo, size = static_cast<long long>(dv) * dk;
    // (the parts' states are whole, as the fold reads and writes them)
    const float* S0 = WALK == ENDS ? nullptr : cut.starts ? cut.starts + blockIdx.x * static_cast<long long>(D * D)
                                            : a.S0 ? a.S0 + sr * size : nullptr;
    const int s_ld = FULL || cut.starts ? D : dk, s_rows = FULL || cut.starts ? D : dv;
    const int f_ld = FULL || WALK == ENDS ? D : dk, f_rows = FULL || WALK == ENDS ? D : dv;
    float* final_state = WALK == ENDS ? cut.ends + blockIdx.x * static_cast<long long>(D * D)
                         : WALK == OUTPUTS && a.final_state && piece == cut.parts - 1 ? a.final_state + sr * size : nullptr;
    if (chunks == 0) {
        if (final_state)
            for (int i = tid; i < size / 4; i += CH_THREADS)
                reinterpret_cast<float4*>(final_state)[i] =
                    S0 ? reinterpret_cast<const float4*>(S0)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1 + ROW_WARPS);
            mbar_init(done_s + s, 1);
            mbar_init(have_s + s, ROW_WARPS / 2);
        }
        for (uint64_t* b : {done_z, done_r, done_o, done_all}) mbar_init(b, 1);
        for (uint64_t* b : {have_z, have_w, have_u, read_o}) mbar_init(b, ROW_WARPS);
        mbar_init_fence();
        *dead = 0;
    }
    if (!FULL && dv < D) {   // zeros behind v's columns in both stages
        for (int e = tid; e < 2 * TILE_X / 16; e += CH_THREADS)
            *reinterpret_cast<uint4*>(smem + e / (TILE_X / 16) * STAGE_BYTES + ST_V + e % (TILE_X / 16) * 16) = make_uint4(0u, 0u, 0u, 0u);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == MMA_WARP) tmem_alloc(holder, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *holder, base = smem_addr(smem);
    const Waits wait{dead, wait_ns};
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
        wait(bar, parity);
        __syncwarp();
        tc_fence_after_sync();
    };

    if (warp >= MMA_WARP) {
        if (warp > MMA_WARP) {
            // ---- tiles ------------------------------------------------------------------
            if (lane == 0)
                load_chunks(smem, full, empty, wait, static_cast<const __nv_bfloat16*>(a.v) + tok * dv, dv, identity,
                            prep + (sp.slot * a.H + h) * static_cast<long long>(prep_bytes),
                            static_cast<long long>(a.H) * prep_bytes, len, chunks, a.stall);
        } else {
            // ---- products ---------------------------------------------------------------
            constexpr uint32_t ID_T = idesc_f16(128, C), ID_S = idesc_f16(128, D / 2, false, true);
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                const uint32_t par = c & 1, pr = base + st * STAGE_BYTES, kq = pr + PREP_KQ;
                wait_warp(full + st, (c >> 1) & 1);
                if (__any_sync(0xffffffffu, *dead)) break;
                if (!KEEP && c > 0) wait_warp(done_o, par ^ 1);   // (U's halves were read out of COL_Z)
                // S K^T, from the columns of S as they come
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    wait_warp(have_s + half, par);
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) {
                        const int ks = half * (D / 32) + e;
                        const uint64_t b = umma_desc_kmajor(kq + ks * 256, 128, ROWS_D);
                        umma_ta(tmem + COL_Z, tmem + COL_SH + 8 * ks, b, ID_T, ks > 0 ? 1u : 0u);
                        umma_ta(tmem + COL_Z, tmem + COL_SL + 8 * ks, b, ID_T, 1u);
                    }
                }
                umma_done(done_z);
                // S Q^T, while the rows work on Z
                if (!KEEP && c > 0) wait_warp(read_o, par ^ 1);
#pragma unroll
                for (int ks = 0; ks < (KEEP ? 0 : D / 16); ++ks) {
                    const uint64_t b = umma_desc_kmajor(kq + TILE_X + ks * 256, 128, ROWS_D);
                    umma_ta(tmem + COL_QS, tmem + COL_SH + 8 * ks, b, ID_T, ks > 0 ? 1u : 0u);
                    umma_ta(tmem + COL_QS, tmem + COL_SL + 8 * ks, b, ID_T, 1u);
                }
                wait_warp(have_z, par);
                // (beta Z)^T T^T: hi hi, hi lo, lo hi
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks) {
                    const uint64_t hi = umma_desc_kmajor(pr + PREP_T + ks * 256, 128, ROWS_C);
                    const uint64_t lo = umma_desc_kmajor(pr + PREP_T + TILE_T + ks * 256, 128, ROWS_C);
                    const uint32_t z = tmem + COL_W + 16 * ks;
                    umma_ta(tmem + COL_Z, z, hi, ID_T, ks > 0 ? 1u : 0u);
                    umma_ta(tmem + COL_Z, z, lo, ID_T, 1u);
                    umma_ta(tmem + COL_Z, z + 8, hi, ID_T, 1u);
                }
                umma_done(done_r);
                wait_warp(have_w, par);
                // (e^{g_C - g} U)^T K, in two halves of its columns
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks) {
                        const uint64_t b = umma_desc_mnmajor(kq + ks * 2 * ROWS_D + half * (D / 16) * 128, ROWS_D, 128);
                        umma_ta(tmem + COL_S + half * (D / 2), tmem + COL_W + 16 * ks, b, ID_S, ks > 0 ? 1u : 0u);
                        umma_ta(tmem + COL_S + half * (D / 2), tmem + COL_W + 16 * ks + 8, b, ID_S, 1u);
                    }
                    umma_done(done_s + half);
                }
                if (!KEEP) {
                    wait_warp(have_u, par);
                    // U^T P^T
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks) {
                        const uint64_t hi = umma_desc_kmajor(pr + PREP_P + ks * 256, 128, ROWS_C);
                        const uint64_t lo = umma_desc_kmajor(pr + PREP_P + TILE_T + ks * 256, 128, ROWS_C);
                        const uint32_t u = tmem + COL_Z + 16 * ks;
                        umma_ta(tmem + COL_O, u, hi, ID_T, ks > 0 ? 1u : 0u);
                        umma_ta(tmem + COL_O, u, lo, ID_T, 1u);
                        umma_ta(tmem + COL_O, u + 8, hi, ID_T, 1u);
                    }
                    umma_done(done_o);
                }
                umma_done(empty + st);
            }
            umma_done(done_all);
            if (!mbar_wait(done_all, 0, wait_ns)) *dead = 1;   // no product outlives the CTA
        }
    } else {
        // ---- rows -------------------------------------------------------------------
        const int q4 = warp & 3, part = warp >> 2, i = 32 * q4 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q4) << 16);
        const int cb = 32 * part, tb = 16 * part;        // its columns of S, its tokens
        float* tops2 = tops + 4 * D;
        auto arrive = [&](uint64_t* bar) {
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        float2 S[2][8];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                const int j = cb + 16 * p + 2 * e;
                if (S0 && (FULL || (i < s_rows && j < s_ld))) f = *reinterpret_cast<const float4*>(S0 + static_cast<long long>(i) * s_ld + j);
                if (identity) f = make_float4(j == i, j + 1 == i, j + 2 == i, j + 3 == i);
                S[p][e] = make_float2(f.x, f.y);
                S[p][e + 1] = make_float2(f.z, f.w);
            }
        TO* out = static_cast<TO*>(a.out) + tok * dv + i;
        float s_down = 1.f, w_down = 1.f, u_down = 1.f, end = 1.f;   // of the chunk before: what undoes the scales, e^{g_C}
        int lost = 16;                                   // ... its tokens here whose outputs are not numbers, from this one on
        bool row_lost = false;                           // ... and whether the row has such: its state is none either
        auto take = [&](int c) {                         // S behind chunk c
            wait_warp(done_s + (part >> 1), c & 1);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float2 x[8];
                tmem_get16(tl + COL_S + cb + 16 * p, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) S[p][e] = __ffma2_rn(x[e], both(w_down), __fmul2_rn(S[p][e], both(end)));
                if (row_lost) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) S[p][e] = both(__int_as_float(0x7fffffff));
                }
            }
        };
        auto finish = [&](int c, float before) {         // outputs of chunk c, whose S had the scale `before`
            const float* gates = reinterpret_cast<const float*>(smem + (c & 1) * STAGE_BYTES + PREP_GATES);
            const float fq = before * gates[G_QDN], fo = u_down * gates[G_PDN];
            wait_warp(done_o, c & 1);
            float2 o[8], q[8];
            tmem_get16(tl + COL_O + tb, o);
            tmem_get16(tl + COL_QS + tb, q);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float4 g = *reinterpret_cast<const float4*>(gates + G_E + tb + 2 * e);
                o[e] = __ffma2_rn(o[e], both(fo), __fmul2_rn(__fmul2_rn(q[e], both(fq)), make_float2(g.x, g.y)));
                o[e + 1] = __ffma2_rn(o[e + 1], both(fo), __fmul2_rn(__fmul2_rn(q[e + 1], both(fq)), make_float2(g.z, g.w)));
            }
            if (lost < 16) {
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (t >= lost) (t & 1 ? o[t / 2].y : o[t / 2].x) = __int_as_float(0x7fffffff);
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(read_o);
                mbar_arrive(empty + (c & 1));
            }
            const int m = FULL || i < dv ? len - c * C - tb : 0;
            TO* dst = out + (static_cast<long long>(c) * C + tb) * dv;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (2 * e < m) dst[2 * e * dv] = from_f32<TO>(o[e].x);
                if (2 * e + 1 < m) dst[(2 * e + 1) * dv] = from_f32<TO>(o[e].y);
            }
        };
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            const uint32_t par = c & 1;
            unsigned char* stage = smem + st * STAGE_BYTES;
            const float* gates = reinterpret_cast<const float*>(stage + PREP_GATES);
            if (c > 0) take(c - 1);
            float up;
            const float before = s_down;
            {   // the state's halves
                scale_of(row_top(tops, largest(largest(0.f, S[0]), S[1]), q4, part, i), up, s_down);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) halves(__fmul2_rn(S[p][e], both(up)), hi[e], lo[e]);
                    tmem_st8w(tl + COL_SH + (cb + 16 * p) / 2, hi);
                    tmem_st8w(tl + COL_SL + (cb + 16 * p) / 2, lo);
                }
            }
            arrive(have_s + (part >> 1));
            if (WALK == TILES) {
                char* to = keep.states + ((sp.slot + c) * a.H + h) * STATE_BYTES;
                keep_row<8>(to, i, cb / 4, S[0]);
                keep_row<8>(to, i, cb / 4 + 4, S[1]);
            } else if (WALK == OUTPUTS && c > 0) {
                finish(c - 1, before);
            }
            wait_warp(full + st, (c >> 1) & 1);
            end = gates[G_END];
            float2 z[8], x[8];
            get_column(reinterpret_cast<const __nv_bfloat16*>(stage + ST_V) + tb * D + i, z);
            float z_down;
            {   // z = v - e^g S k
                const float f = -s_down * gates[G_KDN];
                wait_warp(done_z, par);
                tmem_get16(tl + COL_Z + tb, x);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 g = *reinterpret_cast<const float4*>(gates + G_E + tb + 2 * e);
                    const float4 b = *reinterpret_cast<const float4*>(gates + G_BETA + tb + 2 * e);
                    z[e] = __ffma2_rn(__fmul2_rn(x[e], both(f)), make_float2(g.x, g.y), z[e]);
                    z[e + 1] = __ffma2_rn(__fmul2_rn(x[e + 1], both(f)), make_float2(g.z, g.w), z[e + 1]);
                    x[e] = __fmul2_rn(make_float2(b.x, b.y), z[e]);
                    x[e + 1] = __fmul2_rn(make_float2(b.z, b.w), z[e + 1]);
                }
                int mine = 16, first;
                float top = largest(0.f, x);
                if (!finite(top)) {
                    mine = cut_off(x, 16);
                    top = largest(0.f, x);
                }
                scale_of(row_top(tops2, mine < 16 ? -top : top, q4, part, i, &first), up, z_down);
                lost = first < part ? 0 : mine;
                put_scaled(tl + COL_W + tb, x, up);
                arrive(have_z);
            }
            {   // r = z + T beta z, u = beta r
                const float f = z_down * gates[G_TDN];
                wait_warp(done_r, par);
                tmem_get16(tl + COL_Z + tb, x);
                if (KEEP) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[e] = __ffma2_rn(x[e], both(f), z[e]);
                    if (lost < 16) {
#pragma unroll
                        for (int t = 0; t < 16; ++t)
                            if (t >= lost) (t & 1 ? z[t / 2].y : z[t / 2].x) = __int_as_float(0x7fffffff);
                    }
                    if (WALK == TILES) keep_row<8>(keep.rows + ((sp.slot + c) * a.H + h) * ROWS_BYTES, i, tb / 4, z);
                }
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 b = *reinterpret_cast<const float4*>(gates + G_BETA + tb + 2 * e);
                    const float4 w = *reinterpret_cast<const float4*>(gates + G_W + tb + 2 * e);
                    if (!KEEP) {
                        z[e] = __ffma2_rn(x[e], both(f), z[e]);
                        z[e + 1] = __ffma2_rn(x[e + 1], both(f), z[e + 1]);
                    }
                    z[e] = __fmul2_rn(make_float2(b.x, b.y), z[e]);
                    z[e + 1] = __fmul2_rn(make_float2(b.z, b.w), z[e + 1]);
                    x[e] = __fmul2_rn(make_float2(w.x, w.y), z[e]);
                    x[e + 1] = __fmul2_rn(make_float2(w.z, w.w), z[e + 1]);
                }
                float top = largest(0.f, x);
                if (lost < 16 || !finite(top)) {
                    // w u and u are 0 from the first place on where r is none; where w alone is none, the outputs are
                    lost = cut_off(z, lost);
                    top = cut_off(x, lost) < lost ? __int_as_float(0x7f800000) : largest(0.f, x);
                }
                int first;
                top = row_top(tops, lost < 16 ? -top : top, q4, part, i, &first);
                scale_of(top, up, w_down);
                row_lost = first < 4 || isinf(top);
                if (first < part) lost = 0;
                w_down *= gates[G_KDN];
                put_scaled(tl + COL_W + tb, x, up);
                arrive(have_w);
                if (KEEP) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(empty + st);
                } else {
                    scale_of(row_top(tops2, largest(0.f, z), q4, part, i), up, u_down);
                    put_scaled(tl + COL_Z + tb, z, up);
                    arrive(have_u);
                }
            }
        }
        if (WALK != TILES) take(chunks - 1);
        if (WALK == OUTPUTS) finish(chunks - 1, s_down);
        if (final_state) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float* dst = final_state + static_cast<long long>(i) * f_ld + cb + 16 * p;
                if (!FULL && (i >= f_rows || cb + 16 * p >= f_ld)) continue;
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    *reinterpret_cast<float4*>(dst + 2 * e) = make_float4(S[p][e].x, S[p][e].y, S[p][e + 1].x, S[p][e + 1].y);
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && *dead) record_error(&g_delta_error, KDN_ERR_TIMEOUT);
}

// The parts' first states from their ends: S_{p+1} = S_p M_p + N_p.  A CTA has
// 16 rows of a head's state, a thread two of them by four columns.
constexpr int FOLD_ROWS = 16, FOLD_THREADS = 256;
__global__ void __launch_bounds__(FOLD_THREADS) delta_fold_kernel(const float* S0, const float* ends, float* starts, int parts, int dk,
                                                                  int dv) {
    __shared__ float S[FOLD_ROWS][D];
    constexpr int PER = D / FOLD_ROWS;
    const long long row = blockIdx.x / PER, size = static_cast<long long>(D) * D;
    const int i0 = static_cast<int>(blockIdx.x % PER) * FOLD_ROWS;
    const int r = 2 * (threadIdx.x / 32), c = 4 * (threadIdx.x % 32);
    float4 x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const long long at = (row * dv + i0 + r + e) * dk + c;
        x[e] = S0 && i0 + r + e < dv && c < dk ? *reinterpret_cast<const float4*>(S0 + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int p = 0; p < parts; ++p) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            *reinterpret_cast<float4*>(&S[r + e][c]) = x[e];
            *reinterpret_cast<float4*>(starts + (row * parts + p) * size + static_cast<long long>(i0 + r + e) * D + c) = x[e];
        }
        if (p == parts - 1) break;
        __syncwarp();                                  // (a warp's two rows are its own)
        const float* N = ends + (row * (parts - 1) + p) * 2 * size;
        const float* M = N + size;
#pragma unroll
        for (int e = 0; e < 2; ++e) x[e] = *reinterpret_cast<const float4*>(N + static_cast<long long>(i0 + r + e) * D + c);
#pragma unroll 8
        for (int j = 0; j < D; ++j) {
            const float4 m = __ldg(reinterpret_cast<const float4*>(M + static_cast<long long>(j) * D + c));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float s = S[r + e][j];
                x[e].x = fmaf(s, m.x, x[e].x);
                x[e].y = fmaf(s, m.y, x[e].y);
                x[e].z = fmaf(s, m.z, x[e].z);
                x[e].w = fmaf(s, m.w, x[e].w);
            }
        }
        __syncwarp();
    }
}

// ---- the adjoint's walk --------------------------------------------------------

// D, the adjoint of the state behind a chunk, walks to the chunk before it:
//     dU = P^T dO + e^{g_C - g} (K D^T),   Y = dU + T^T (beta dU),   L = beta Y,
//     D' = e^{g_C} D + dO^T (e^g Q) - L^T (e^g K),
// with the forward's shape (D for S, dU for Z, Y for R).  P^T dO and dO^T (e^g
// Q) do not wait for D.  dV = L; D (behind the chunk) and Y are kept.  P^T dO
// lies in COL_W until beta dU's halves do; e^g dO is an operand in shared memory.
// (128 heads of 4096 tokens 334 us, bound as the forward's walk is.)
constexpr uint32_t COL_X = 320;              // dO^T (e^g Q), 128 columns

// END: of a part but the first its end alone, from zero (the last one's from the
// final state's gradient): nothing is kept or written but that.
template <bool FULL, bool END>
__global__ void __launch_bounds__(CH_THREADS, 1) delta_adjoint_kernel(const DeltaArgs a, const char* prep, const KeepTiles keep,
                                                                      const Parts cut, long long wait_ns) {
    extern __shared__ __align__(128) unsigned char smem[];
    float* tops = reinterpret_cast<float*>(smem + CH_OFF_TOP);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + CH_OFF_BAR);
    uint64_t* empty = full + 2;
    uint64_t* done_p = empty + 2;                                      // products: P^T dO, K D^T, T^T beta dU, D
    uint64_t* done_z = done_p + 1;
    uint64_t* done_r = done_z + 1;
    uint64_t* done_s = done_r + 1;                                     // [2]
    uint64_t* have_s = done_s + 2;                                     // operands: D [2], e^g dO, beta dU, L
    uint64_t* have_x = have_s + 2;
    uint64_t* have_z = have_x + 1;
    uint64_t* have_w = have_z + 1;
    uint64_t* done_all = have_w + 1;                                   // no product is left
    uint32_t* holder = reinterpret_cast<uint32_t*>(done_all + 1);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int jobs = END ? cut.parts - 1 : cut.parts;                  // of a state row
    const long long sr = blockIdx.x / jobs, n = sr / a.H;
    const int piece = static_cast<int>(blockIdx.x % jobs) + (END ? 1 : 0);
    const int h = static_cast<int>(sr % a.H);
    Span sp = span_of(a, n);
    if (cut.parts > 1) {   // this part's tokens and chunks
        sp.lo += piece * cut.len * C;
        sp.slot += piece * cut.len;
        if (sp.hi - sp.lo > cut.len * C) sp.hi = sp.lo + cut.len * C;
    }
    const int len = max(sp.hi - sp.lo, 0), chunks = (len + C - 1) / C;
    const int dk = FULL ? D : a.dk, dv = FULL ? D : a.dv;
    const long long tok = (sp.row * a.H + h) * a.T + sp.lo, size = static_cast<long long>(dv) * dk;
    constexpr long long WHOLE = D * D;                                 // (the parts' states, as the folds have them)
    const bool begun = !END && cut.starts;
    const float* D1 = begun ? cut.starts + blockIdx.x * WHOLE
                      : a.grad_final_state && piece == cut.parts - 1 ? a.grad_final_state + sr * size : nullptr;
    float* D0 = END ? cut.ends + (sr * (cut.parts - 1) + piece - 1) * 2 * WHOLE
                : a.grad_S0 && piece == 0 ? a.grad_S0 + sr * size : nullptr;
    const int s_ld = FULL || begun ? D : dk, s_rows = FULL || begun ? D : dv;
    const int f_ld = FULL || END ? D : dk, f_rows = FULL || END ? D : dv;
    if (chunks == 0) {
        if (D0)
            for (int i = tid; i < size / 4; i += CH_THREADS)
                reinterpret_cast<float4*>(D0)[i] =
                    D1 ? reinterpret_cast<const float4*>(D1)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1 + ROW_WARPS);
            mbar_init(done_s + s, 1);
            mbar_init(have_s + s, ROW_WARPS / 2);
        }
        for (uint64_t* b : {done_p, done_z, done_r, done_all}) mbar_init(b, 1);
        for (uint64_t* b : {have_x, have_z, have_w}) mbar_init(b, ROW_WARPS);
        mbar_init_fence();
        *dead = 0;
    }
    if (warp == MMA_WARP) tmem_alloc(holder, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *holder, base = smem_addr(smem);
    const Waits wait{dead, wait_ns};
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
        wait(bar, parity);
        __syncwarp();
        tc_fence_after_sync();
    };

    if (warp >= MMA_WARP) {
        if (warp > MMA_WARP) {
            if (lane == 0)
                load_chunks(smem, full, empty, wait, nullptr, D, false, prep + (sp.slot * a.H + h) * static_cast<long long>(PREP_STEP),
                            static_cast<long long>(a.H) * PREP_STEP, len, chunks, a.stall);
        } else {
            constexpr uint32_t ID_T = idesc_f16(128, C), ID_TN = idesc_f16(128, C, false, true),
                               ID_P = idesc_f16(128, C, true, true), ID_S = idesc_f16(128, D / 2, false, true),
                               ID_Q = idesc_f16(128, D, false, true);
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                const uint32_t par = c & 1, pr = base + st * STAGE_BYTES, kq = pr + PREP_KQ;
                wait_warp(full + st, (c >> 1) & 1);
                if (__any_sync(0xffffffffu, *dead)) break;
                if (c > 0) wait_warp(done_s + 1, par ^ 1);   // (L's halves were read out of COL_W)
                // dO^T P
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks) {
                    const uint64_t g = umma_desc_mnmajor(kq + ST_V + ks * 2 * ROWS_D, ROWS_D, 128);
                    const uint64_t hi = umma_desc_mnmajor(pr + PREP_P + ks * 2 * ROWS_C, ROWS_C, 128);
                    const uint64_t lo = umma_desc_mnmajor(pr + PREP_P + TILE_T + ks * 2 * ROWS_C, ROWS_C, 128);
                    umma_sa(tmem + COL_W, g, hi, ID_P, ks > 0 ? 1u : 0u);
                    umma_sa(tmem + COL_W, g, lo, ID_P, 1u);
                }
                umma_done(done_p);
                // D K^T
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    wait_warp(have_s + half, par);
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) {
                        const int ks = half * (D / 32) + e;
                        const uint64_t b = umma_desc_kmajor(kq + ks * 256, 128, ROWS_D);
                        umma_ta(tmem + COL_Z, tmem + COL_SH + 8 * ks, b, ID_T, ks > 0 ? 1u : 0u);
                        umma_ta(tmem + COL_Z, tmem + COL_SL + 8 * ks, b, ID_T, 1u);
                    }
                }
                umma_done(done_z);
                wait_warp(have_x, par);
                // (e^g dO)^T Q, while the rows work on dU
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks) {
                    const uint64_t b = umma_desc_mnmajor(kq + TILE_X + ks * 2 * ROWS_D, ROWS_D, 128);
                    const uint32_t x = base + AD_OFF_X + ks * 256;
                    umma_sa(tmem + COL_X, umma_desc_kmajor(x, 128, ROWS_C), b, ID_Q, ks > 0 ? 1u : 0u);
                    umma_sa(tmem + COL_X, umma_desc_kmajor(x + D * C * 2, 128, ROWS_C), b, ID_Q, 1u);
                }
                wait_warp(have_z, par);
                // (beta dU)^T T: hi hi, hi lo, lo hi
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks) {
                    const uint64_t hi = umma_desc_mnmajor(pr + PREP_T + ks * 2 * ROWS_C, ROWS_C, 128);
                    const uint64_t lo = umma_desc_mnmajor(pr + PREP_T + TILE_T + ks * 2 * ROWS_C, ROWS_C, 128);
                    const uint32_t z = tmem + COL_W + 16 * ks;
                    umma_ta(tmem + COL_Z, z, hi, ID_TN, ks > 0 ? 1u : 0u);
                    umma_ta(tmem + COL_Z, z, lo, ID_TN, 1u);
                    umma_ta(tmem + COL_Z, z + 8, hi, ID_TN, 1u);
                }
                umma_done(done_r);
                wait_warp(have_w, par);
                // -(e^g L)^T K, in two halves of its columns
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks) {
                        const uint64_t b = umma_desc_mnmajor(kq + ks * 2 * ROWS_D + half * (D / 16) * 128, ROWS_D, 128);
                        umma_ta(tmem + COL_S + half * (D / 2), tmem + COL_W + 16 * ks, b, ID_S, ks > 0 ? 1u : 0u);
                        umma_ta(tmem + COL_S + half * (D / 2), tmem + COL_W + 16 * ks + 8, b, ID_S, 1u);
                    }
                    umma_done(done_s + half);
                }
                umma_done(empty + st);
            }
            umma_done(done_all);
            if (!mbar_wait(done_all, 0, wait_ns)) *dead = 1;   // no product outlives the CTA
        }
    } else {
        const int q4 = warp & 3, part = warp >> 2, i = 32 * q4 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q4) << 16);
        const int cb = 32 * part, tb = 16 * part;
        float* tops2 = tops + 4 * D;
        auto arrive = [&](uint64_t* bar) {
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        float2 S[2][8];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (D1 && (FULL || (i < s_rows && cb + 16 * p < s_ld)))
                    f = *reinterpret_cast<const float4*>(D1 + static_cast<long long>(i) * s_ld + cb + 16 * p + 2 * e);
                S[p][e] = make_float2(f.x, f.y);
                S[p][e + 1] = make_float2(f.z, f.w);
            }
        __nv_bfloat16* gv = static_cast<__nv_bfloat16*>(a.grad_v) + tok * dv + i;
        float s_down = 1.f, x_down = 1.f, w_down = 1.f, end = 1.f;
        auto take = [&](int c) {                         // D before what was chunk c of the walk
            wait_warp(done_s + (part >> 1), c & 1);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float2 x[8];
                tmem_get16(tl + COL_S + cb + 16 * p, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) S[p][e] = __ffma2_rn(x[e], both(w_down), __fmul2_rn(S[p][e], both(end)));
                tmem_get16(tl + COL_X + cb + 16 * p, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) S[p][e] = __ffma2_rn(x[e], both(x_down), S[p][e]);
            }
        };
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1, chunk = chunks - 1 - c;
            const uint32_t par = c & 1;
            const unsigned char* stage = smem + st * STAGE_BYTES;
            const float* gates = reinterpret_cast<const float*>(stage + PREP_GATES);
            const long long slot = (sp.slot + chunk) * a.H + h;
            if (c > 0) take(c - 1);
            float up;
            {
                scale_of(row_top(tops, largest(largest(0.f, S[0]), S[1]), q4, part, i), up, s_down);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) halves(__fmul2_rn(S[p][e], both(up)), hi[e], lo[e]);
                    tmem_st8w(tl + COL_SH + (cb + 16 * p) / 2, hi);
                    tmem_st8w(tl + COL_SL + (cb + 16 * p) / 2, lo);
                }
            }
            arrive(have_s + (part >> 1));
            if (!END) {
                keep_row<8>(keep.states + slot * STATE_BYTES, i, cb / 4, S[0]);
                keep_row<8>(keep.states + slot * STATE_BYTES, i, cb / 4 + 4, S[1]);
            }
            wait_warp(full + st, (c >> 1) & 1);
            end = gates[G_END];
            float2 z[8], x[8];
            {   // e^g dO
                const unsigned char* go = stage + ST_V + at_d(tb, i / 8) + (i % 8) * 2;
                const float f = gates[G_XDN];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 g = *reinterpret_cast<const float4*>(gates + G_E + tb + 2 * e);
                    float v[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int t = 2 * e + w;
                        v[w] = __half2float(*reinterpret_cast<const __half*>(go + (t / 8) * ROWS_D + (t % 8) * 16));
                    }
                    x[e] = __fmul2_rn(make_float2(v[0] * f, v[1] * f), make_float2(g.x, g.y));
                    x[e + 1] = __fmul2_rn(make_float2(v[2] * f, v[3] * f), make_float2(g.z, g.w));
                }
                scale_of(row_top(tops2, largest(0.f, x), q4, part, i), up, x_down);
                x_down *= gates[G_QDN];
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) halves(__fmul2_rn(x[e + w], both(up)), hi[w], lo[w]);
                    unsigned char* to = smem + AD_OFF_X + at_c(i, tb / 8 + e / 4);
                    *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(to + D * C * 2) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(have_x);
            }
            float z_down;
            {   // du = P^T dO + e^{g_C - g} K D^T
                const float f = s_down * gates[G_KDN], fp = gates[G_XDN] * gates[G_PDN];
                wait_warp(done_p, par);
                tmem_get16(tl + COL_W + tb, z);
                wait_warp(done_z, par);
                tmem_get16(tl + COL_Z + tb, x);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 w = *reinterpret_cast<const float4*>(gates + G_W + tb + 2 * e);
                    const float4 b = *reinterpret_cast<const float4*>(gates + G_BETA + tb + 2 * e);
                    z[e] = __ffma2_rn(__fmul2_rn(x[e], both(f)), make_float2(w.x, w.y), __fmul2_rn(z[e], both(fp)));
                    z[e + 1] = __ffma2_rn(__fmul2_rn(x[e + 1], both(f)), make_float2(w.z, w.w), __fmul2_rn(z[e + 1], both(fp)));
                    x[e] = __fmul2_rn(make_float2(b.x, b.y), z[e]);
                    x[e + 1] = __fmul2_rn(make_float2(b.z, b.w), z[e + 1]);
                }
                scale_of(row_top(tops, largest(0.f, x), q4, part, i), up, z_down);
                put_scaled(tl + COL_W + tb, x, up);
                arrive(have_z);
            }
            {   // y = du + T^T (beta du), l = beta y
                const float f = z_down * gates[G_TDN];
                wait_warp(done_r, par);
                tmem_get16(tl + COL_Z + tb, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = __ffma2_rn(x[e], both(f), z[e]);
                if (!END) keep_row<8>(keep.rows + slot * ROWS_BYTES, i, tb / 4, z);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 b = *reinterpret_cast<const float4*>(gates + G_BETA + tb + 2 * e);
                    const float4 g = *reinterpret_cast<const float4*>(gates + G_E + tb + 2 * e);
                    z[e] = __fmul2_rn(make_float2(b.x, b.y), z[e]);
                    z[e + 1] = __fmul2_rn(make_float2(b.z, b.w), z[e + 1]);
                    x[e] = __fmul2_rn(make_float2(-g.x, -g.y), z[e]);
                    x[e + 1] = __fmul2_rn(make_float2(-g.z, -g.w), z[e + 1]);
                }
                scale_of(row_top(tops2, largest(0.f, x), q4, part, i), up, w_down);
                w_down *= gates[G_KDN];
                put_scaled(tl + COL_W + tb, x, up);
                arrive(have_w);
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + st);
                const int m = !END && (FULL || i < dv) ? len - chunk * C - tb : 0;
                __nv_bfloat16* dst = gv + (static_cast<long long>(chunk) * C + tb) * dv;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (2 * e < m) dst[2 * e * dv] = __float2bfloat16_rn(z[e].x);
                    if (2 * e + 1 < m) dst[(2 * e + 1) * dv] = __float2bfloat16_rn(z[e].y);
                }
            }
        }
        if (D0) {
            take(chunks - 1);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float* dst = D0 + static_cast<long long>(i) * f_ld + cb + 16 * p;
                if (!FULL && (i >= f_rows || cb + 16 * p >= f_ld)) continue;
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    *reinterpret_cast<float4*>(dst + 2 * e) = make_float4(S[p][e].x, S[p][e].y, S[p][e + 1].x, S[p][e + 1].y);
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && *dead) record_error(&g_delta_error, KDN_ERR_TIMEOUT);
}

// The adjoints behind the parts from their ends: D_{p-1} = D_p M_p^T + N_p, the
// last part's end having begun with the final state's gradient.  As the states'
// fold otherwise; an end lies where N of the part before it was.
__global__ void __launch_bounds__(FOLD_THREADS) delta_fold_back_kernel(const float* D1, const float* ends, float* starts, int parts,
                                                                       int dk, int dv) {
    __shared__ float S[FOLD_ROWS][D];
    constexpr int PER = D / FOLD_ROWS;
    const long long row = blockIdx.x / PER, size = static_cast<long long>(D) * D;
    const int i0 = static_cast<int>(blockIdx.x % PER) * FOLD_ROWS;
    const int r = 2 * (threadIdx.x / 32), lane = threadIdx.x % 32;   // two rows, columns lane + 32 e
    float x[2][4];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int i = i0 + r + e, c = lane + 32 * w;
            x[e][w] = D1 && i < dv && c < dk ? D1[(row * dv + i) * dk + c] : 0.f;
        }
    for (int p = parts - 1; p >= 0; --p) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                S[r + e][lane + 32 * w] = x[e][w];
                starts[(row * parts + p) * size + static_cast<long long>(i0 + r + e) * D + lane + 32 * w] = x[e][w];
            }
        if (p == 0) break;
        __syncwarp();                                  // (a warp's two rows are its own)
        const float* N = ends + (row * (parts - 1) + p - 1) * 2 * size;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int w = 0; w < 4; ++w) x[e][w] = N[static_cast<long long>(i0 + r + e) * D + lane + 32 * w];
        if (p < parts - 1) {
            const float* M = ends + ((row * (parts - 1) + p) * 2 + 1) * size;
#pragma unroll 4
            for (int j = 0; j < D; j += 4) {
                const float4 s0 = *reinterpret_cast<const float4*>(&S[r][j]), s1 = *reinterpret_cast<const float4*>(&S[r + 1][j]);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float4 m = __ldg(reinterpret_cast<const float4*>(M + static_cast<long long>(lane + 32 * w) * D + j));
                    x[0][w] = fmaf(s0.x, m.x, fmaf(s0.y, m.y, fmaf(s0.z, m.z, fmaf(s0.w, m.w, x[0][w]))));
                    x[1][w] = fmaf(s1.x, m.x, fmaf(s1.y, m.y, fmaf(s1.z, m.z, fmaf(s1.w, m.w, x[1][w]))));
                }
            }
        }
        __syncwarp();
    }
}

// ---- the gradients of a chunk ----------------------------------------------------

// A CTA makes one chunk's gradients of one head from its tiles and the walks'
// kept ones (see delta_scan.cu for the formulas), transposed: a thread of a row
// warp is a column j of d_k, its registers are tokens.  With u = beta R and l =
// beta Y the products use R and Y as they are kept, and beta, E and the signs
// come in with the sums:
//     [s x t]  R dO^T, R Y^T -> dP^T, dG^T (E, masks) and dbeta_t = R_t . Y_t,
//              K Q^T, K K^T -> W = dP . (Q K^T) + dG . (K K^T), summed pair by pair,
//     [j x t]  S0^T dO^T, S0^T Y^T, K^T dP^T, K^T dG^T -> dq, dk as a reader,
//     [j x s]  Q^T dP, K^T dG, D1^T R^T -> dk as a writer.
// The kept fp32 tiles become pairs of fp16 in their place, each tile (dP and dG
// too) with one power of two (its values meet in sums); D1 follows S0 there.  <S0, D1> is
// taken in fp32: the gradient of A is a sum over all tokens to which it adds the
// same in every token of its chunk.  Bound by the latency of these steps with one
// CTA to an SM: 8192 chunks 708 us (655 without W), 13 us a chunk, its 260 KB 5.8 at
// a copy's rate.
constexpr int GR_WARPS = 16, GR_THREADS = GR_WARPS * 32 + 32;
constexpr int GR_KQ = 0, GR_DO = 2 * TILE_X, GR_R = GR_DO + TILE_X, GR_Y = GR_R + ROWS_BYTES, GR_S = GR_Y + ROWS_BYTES,
              GR_P = GR_S + STATE_BYTES, GR_MISC = GR_P + 2 * C * 2 * C * 2;
// fp32: the gates, of each lane quarter what a token reads of S0 and writes to D1, sums of W (GR_X: across a
// token, from the 16 tokens that it is in, of each 32 writers and of dP and dG; GR_W: of a writer, all of 16 readers;
// GR_NEAR: K Q^T and K K^T on the diagonal), row warps' sums and magnitudes
constexpr int GR_GATES = GR_MISC, GR_C = GR_GATES + (G_ALL + 3) / 4 * 16, GR_F = GR_C + 4 * C * 4, GR_X = GR_F + 4 * C * 4,
              GR_W = GR_X + 4 * C * 4, GR_NEAR = GR_W + 8 * C * 4, GR_SUM = GR_NEAR + 2 * C * 16,
              GR_TOP = GR_SUM + GR_WARPS * 4, GR_BAR = GR_TOP + 5 * GR_WARPS * 4, GR_SMEM = GR_BAR + 128;
static_assert(GR_SMEM <= 227 * 1024, "shared memory");
// (CG_A: R dO^T and R Y^T, then K^T dG in its first half; CG_W, CG_W2: K K^T and K Q^T first; CG_Q2: K^T dP^T, K^T dG^T)
constexpr uint32_t CG_A = 0, CG_Q = 128, CG_R = 192, CG_W = 256, CG_W2 = 320, CG_Q2 = 384;

// Sums over the lanes of 16 values each: lane l holds value l % 16's (both
// halves of a warp the same).
__device__ __forceinline__ float lane_sums(float (&v)[16], int lane) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int e = 0; e < o; ++e) {
            const float mine = up ? v[e + o] : v[e], other = up ? v[e] : v[e + o];
            v[e] = mine + __shfl_xor_sync(0xffffffffu, other, o);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

__device__ __forceinline__ void prefetch_l2(const void* p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

struct GradTiles {
    const char* prep;
    const char* states;
    const char* adjoints;
    const char* r;
    const char* y;
    float* sum_A;           // [slots,H] or null
    int ahead;              // tiles between this CTA's and the one that follows it on its SM
};

// The largest magnitude that the row warps (or those that sync on `bar`) have:
// one slot of `tops` each.
__device__ __forceinline__ float block_top(float* tops, float mine, int bar, int threads, int warps, int warp) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(mine));
    if ((threadIdx.x & 31) == 0) tops[warp] = __uint_as_float(m);
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
    const int l = threadIdx.x & 31;
    return __uint_as_float(__reduce_max_sync(0xffffffffu, l < warps ? __float_as_uint(tops[l]) : 0u));
}

// The largest of what half of the warps put there (behind that).
__device__ __forceinline__ float warps_top(const float* tops) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(tops[threadIdx.x & (GR_WARPS / 2 - 1)])));
}

// 8 values of a row as a 16-byte piece of halves each.
__device__ __forceinline__ void half_pieces(unsigned char* hi_at, unsigned char* lo_at, const float2* x, float up) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) halves(__fmul2_rn(x[e], both(up)), hi[e], lo[e]);
    *reinterpret_cast<uint4*>(hi_at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(lo_at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

template <bool FULL>
__global__ void __launch_bounds__(GR_THREADS, 1) delta_tc_grad_kernel(const DeltaArgs a, const GradTiles in, long long wait_ns) {
    extern __shared__ __align__(128) unsigned char smem[];
    float* gates = reinterpret_cast<float*>(smem + GR_GATES);
    float* sc = reinterpret_cast<float*>(smem + GR_C);
    float* sf = reinterpret_cast<float*>(smem + GR_F);
    float* sx = reinterpret_cast<float*>(smem + GR_X);                // [2 which + half of the writers][t]
    float* sw = reinterpret_cast<float*>(smem + GR_W);                // [4 which + 16 readers][s]
    float* ssum = reinterpret_cast<float*>(smem + GR_SUM);
    float* tops = reinterpret_cast<float*>(smem + GR_TOP);            // [5][GR_WARPS]: R, Y, S0, dP and dG, D1
    uint64_t* in_ry = reinterpret_cast<uint64_t*>(smem + GR_BAR);   // kept rows and S0 are here
    uint64_t* in_s = in_ry + 1;
    uint64_t* done_a = in_s + 1;                                       // products
    uint64_t* done_b = done_a + 1;
    uint64_t* done_c = done_b + 1;
    uint64_t* done_d = done_c + 1;
    uint64_t* have_ry = done_d + 1;                                    // operands: R and Y, S0, dP and dG, D1
    uint64_t* have_s = have_ry + 1;
    uint64_t* have_p = have_s + 1;
    uint64_t* have_d = have_p + 1;
    uint32_t* holder = reinterpret_cast<uint32_t*>(have_d + 1);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = static_cast<int>(blockIdx.x % a.H);
    const long long slot = blockIdx.x / a.H, tile = blockIdx.x;
    long long n, row;
    int t0, m;
    if (!chunk_of(a, slot, &n, &t0, &m, &row)) {
        if (in.sum_A && tid == 0) in.sum_A[tile] = 0.f;
        return;
    }
    const long long tok = (row * a.H + h) * a.T + t0;
    const char* adjoint = in.adjoints + tile * STATE_BYTES;
    if (tid == 0) {
        for (uint64_t* b : {in_ry, in_s, done_a, done_b, done_c, done_d}) mbar_init(b, 1);
        for (uint64_t* b : {have_ry, have_s, have_p, have_d}) mbar_init(b, GR_WARPS);
        mbar_init_fence();
        *dead = 0;
        const char* prep = in.prep + tile * PREP_STEP;
        if (t0 / C != a.stall) {
            mbar_arrive_expect_tx(in_ry, 2 * ROWS_BYTES + 3 * TILE_X);
            bulk_g2s(smem + GR_KQ, prep + PREP_KQ, 2 * TILE_X, in_ry);
            bulk_g2s(smem + GR_DO, prep + PREP_BYTES, TILE_X, in_ry);
            bulk_g2s(smem + GR_R, in.r + tile * ROWS_BYTES, ROWS_BYTES, in_ry);
            bulk_g2s(smem + GR_Y, in.y + tile * ROWS_BYTES, ROWS_BYTES, in_ry);
        }
        mbar_arrive_expect_tx(in_s, STATE_BYTES);
        bulk_g2s(smem + GR_S, in.states + tile * STATE_BYTES, STATE_BYTES, in_s);
        // one CTA to an SM: what the next one reads comes to L2 while this one works
        const long long next = tile + in.ahead;
        if (next < gridDim.x) {
            prefetch_l2(in.prep + next * PREP_STEP, PREP_STEP);
            prefetch_l2(in.r + next * ROWS_BYTES, ROWS_BYTES);
            prefetch_l2(in.y + next * ROWS_BYTES, ROWS_BYTES);
            prefetch_l2(in.states + next * STATE_BYTES, STATE_BYTES);
            prefetch_l2(in.adjoints + next * STATE_BYTES, STATE_BYTES);
        }
    }
    if (warp == GR_WARPS) {
        tmem_alloc(holder, 512);
    } else {
        const float* g = reinterpret_cast<const float*>(in.prep + tile * PREP_STEP + PREP_GATES);
        if (tid < G_ALL) gates[tid] = g[tid];
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *holder, base = smem_addr(smem);
    const Waits wait{dead, wait_ns};
    auto wait_warp = [&](uint64_t* bar) {
        wait(bar, 0);
        __syncwarp();
        tc_fence_after_sync();
    };
    if (warp == GR_WARPS) {
        constexpr uint32_t ID_AK = idesc_f16(128, C, true, false), ID_AN = idesc_f16(128, C, true, true),
                           ID_A2 = idesc_f16(128, 2 * C, true, true), ID_KQ = idesc_f16(128, 2 * C);
        auto rows_of = [&](int off, int ks, int lo) {                  // a K step of a tile of 128 columns, MN-major
            return umma_desc_mnmajor(base + off + ks * 2 * ROWS_D + lo * (C / 8) * 128, ROWS_D, 128);
        };
        wait_warp(in_ry);                                              // (k, q and do, as they came)
        wait_warp(have_ry);
        // [s x t]: R dO^T, R Y^T (rows 64-127 are of no use)
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t rh = rows_of(GR_R, ks, 0), rl = rows_of(GR_R, ks, 1);
            const uint64_t g = umma_desc_kmajor(base + GR_DO + ks * 256, 128, ROWS_D);
            const uint64_t yh = rows_of(GR_Y, ks, 0), yl = rows_of(GR_Y, ks, 1);
            umma_sa(tmem + CG_A, rh, g, ID_AK, ks > 0 ? 1u : 0u);
            umma_sa(tmem + CG_A, rl, g, ID_AK, 1u);
            umma_sa(tmem + CG_A + C, rh, yh, ID_AN, ks > 0 ? 1u : 0u);
            umma_sa(tmem + CG_A + C, rh, yl, ID_AN, 1u);
            umma_sa(tmem + CG_A + C, rl, yh, ID_AN, 1u);
        }
        // [s x t]: K K^T, K Q^T (nor here)
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t kq = umma_desc_kmajor(base + GR_KQ + ks * 256, 128, ROWS_D);
            umma_sa(tmem + CG_W, kq, kq, ID_KQ, ks > 0 ? 1u : 0u);
        }
        umma_done(done_a);
        wait_warp(have_s);
        // [j x t]: S0^T dO^T, S0^T Y^T
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t sh = rows_of(GR_S, ks, 0), sl = rows_of(GR_S + D * D * 2, ks, 0);
            const uint64_t g = umma_desc_kmajor(base + GR_DO + ks * 256, 128, ROWS_D);
            const uint64_t yh = rows_of(GR_Y, ks, 0), yl = rows_of(GR_Y, ks, 1);
            umma_sa(tmem + CG_Q, sh, g, ID_AK, ks > 0 ? 1u : 0u);
            umma_sa(tmem + CG_Q, sl, g, ID_AK, 1u);
            umma_sa(tmem + CG_R, sh, yh, ID_AN, ks > 0 ? 1u : 0u);
            umma_sa(tmem + CG_R, sh, yl, ID_AN, 1u);
            umma_sa(tmem + CG_R, sl, yh, ID_AN, 1u);
        }
        umma_done(done_b);
        wait_warp(have_p);
        // [j x t]: K^T [dP^T | dG^T];  [j x s]: Q^T dP, K^T dG
#pragma unroll
        for (int ks = 0; ks < C / 16; ++ks) {
            const uint64_t k = rows_of(GR_KQ, ks, 0);
            umma_sa(tmem + CG_Q2, k, rows_of(GR_P, ks, 0), ID_A2, ks > 0 ? 1u : 0u);
            umma_sa(tmem + CG_Q2, k, rows_of(GR_P + C * 2 * C * 2, ks, 0), ID_A2, 1u);
        }
#pragma unroll
        for (int ks = 0; ks < C / 16; ++ks) {
            const uint64_t k = rows_of(GR_KQ, ks, 0), q = rows_of(GR_KQ + TILE_X, ks, 0);
#pragma unroll
            for (int lo = 0; lo < 2; ++lo) {
                const uint32_t p = base + GR_P + lo * C * 2 * C * 2 + ks * 256;
                umma_sa(tmem + CG_W2, q, umma_desc_kmajor(p, 128, ROWS_D), ID_AK, ks > 0 || lo > 0 ? 1u : 0u);
                umma_sa(tmem + CG_A, k, umma_desc_kmajor(p + (C / 8) * 128, 128, ROWS_D), ID_AK, ks > 0 || lo > 0 ? 1u : 0u);
            }
        }
        umma_done(done_c);
        wait_warp(have_d);
        // [j x s]: D1^T R^T
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t dh = rows_of(GR_S, ks, 0), dl = rows_of(GR_S + D * D * 2, ks, 0);
            const uint64_t rh = rows_of(GR_R, ks, 0), rl = rows_of(GR_R, ks, 1);
            umma_sa(tmem + CG_W, dh, rh, ID_AN, ks > 0 ? 1u : 0u);
            umma_sa(tmem + CG_W, dh, rl, ID_AN, 1u);
            umma_sa(tmem + CG_W, dl, rh, ID_AN, 1u);
        }
        umma_done(done_d);
        // neither a copy nor a product outlives the CTA
        bool ok = mbar_wait(done_d, 0, wait_ns);
        ok = mbar_wait(in_ry, 0, wait_ns) && mbar_wait(in_s, 0, wait_ns) && ok;
        if (!ok) *dead = 1;
    } else {
        const int q4 = warp & 3, part = warp >> 2, tb = 16 * part;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q4) << 16);
        const int i = tid & (D - 1), quarter = tid / D;      // a row of the kept tiles, a quarter of its columns
        auto arrive = [&](uint64_t* bar) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        float r_down, y_down, s_down, p_down, g_down, d_down, up;
        {   // R and Y in halves
            float2 x[8], y[8];
            wait_warp(in_ry);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 f = *reinterpret_cast<const float4*>(smem + GR_R + at_f(i, 4 * quarter + e));
                const float4 g = *reinterpret_cast<const float4*>(smem + GR_Y + at_f(i, 4 * quarter + e));
                x[2 * e] = make_float2(f.x, f.y);
                x[2 * e + 1] = make_float2(f.z, f.w);
                y[2 * e] = make_float2(g.x, g.y);
                y[2 * e + 1] = make_float2(g.z, g.w);
            }
            // (the second exchange's barrier is past every thread's loads too)
            scale_of(block_top(tops, largest(0.f, x), 1, GR_WARPS * 32, GR_WARPS, warp), up, r_down);
            float y_up;
            scale_of(block_top(tops + GR_WARPS, largest(0.f, y), 1, GR_WARPS * 32, GR_WARPS, warp), y_up, y_down);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                unsigned char* to = smem + GR_R + at_d(i, 2 * quarter + e);
                half_pieces(to, to + (C / 8) * 128, x + 4 * e, up);
                to = smem + GR_Y + at_d(i, 2 * quarter + e);
                half_pieces(to, to + (C / 8) * 128, y + 4 * e, y_up);
            }
            arrive(have_ry);
        }
        float d_up;
        {   // <S0, D1>, and S0 in halves
            float4 g[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = __ldg(reinterpret_cast<const float4*>(adjoint + at_f(i, 8 * quarter + e)));
            float dot = 0.f, top = 0.f, d_top = 0.f;
            wait_warp(in_s);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float4 f = *reinterpret_cast<const float4*>(smem + GR_S + at_f(i, 8 * quarter + e));
                dot = fmaf(f.x, g[e].x, fmaf(f.y, g[e].y, fmaf(f.z, g[e].z, fmaf(f.w, g[e].w, dot))));
                top = fmaxf(fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y))), fmaxf(fabsf(f.z), fabsf(f.w)));
                d_top = fmaxf(fmaxf(d_top, fmaxf(fabsf(g[e].x), fabsf(g[e].y))), fmaxf(fabsf(g[e].z), fabsf(g[e].w)));
                g[e] = f;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            if (lane == 0) ssum[warp] = dot;
            scale_of(block_top(tops + 2 * GR_WARPS, top, 1, GR_WARPS * 32, GR_WARPS, warp), up, s_down);
            scale_of(block_top(tops + 4 * GR_WARPS, d_top, 1, GR_WARPS * 32, GR_WARPS, warp), d_up, d_down);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x[4] = {make_float2(g[2 * e].x, g[2 * e].y), make_float2(g[2 * e].z, g[2 * e].w),
                                     make_float2(g[2 * e + 1].x, g[2 * e + 1].y), make_float2(g[2 * e + 1].z, g[2 * e + 1].w)};
                unsigned char* to = smem + GR_S + at_d(i, 4 * quarter + e);
                half_pieces(to, to + D * D * 2, x, up);
            }
            arrive(have_s);
        }
        float w[16];
        {   // dP^T, dG^T and W.  Their sums lie in 64 lanes of tensor memory, half of the warps': those copy what is
            // needed of them to where dP and dG will be, and all warps take 16 tokens of a row s of one of the two.
            // Of each [s][t] the groups of four columns with t >= s are copied; K Q^T and K K^T go, turned by half a
            // turn, where the groups before them would be, those of the groups on the diagonal to a place of their own
            unsigned char* raw = smem + GR_P;
            if (q4 < 2) {
                const int s = 32 * q4 + lane, which = part >> 1;
                unsigned char* near = smem + GR_NEAR + (C * which + s) * 16;
                wait_warp(done_a);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    float x[16];
                    tmem_ld16_async(tl + CG_A + 32 * part + 16 * p, x);
                    tmem_ld16_async(tl + CG_W + (32 * part + 16 * p + C) % (2 * C), w);
                    tmem_wait_ld16(x);
                    tmem_wait_ld16(w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = 32 * (part & 1) + 16 * p + 4 * e;      // four tokens from this one on
                        unsigned char* to = raw + ((16 * which + t / 4) * C + s) * 16;
                        unsigned char* turned = raw + ((16 * which + (C - 4 - t) / 4) * C + C - 1 - s) * 16;
                        if (t + 3 >= s) {
                            *reinterpret_cast<float4*>(to) = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                            *reinterpret_cast<float4*>(t > s ? turned : near) =
                                make_float4(w[4 * e + 3], w[4 * e + 2], w[4 * e + 1], w[4 * e]);
                        }
                    }
                }
                tc_fence_before_sync();
            }
            asm volatile("bar.sync 1, %0;" ::"n"(GR_WARPS * 32) : "memory");
            const int s = tid & (C - 1), g16 = tid / C, which = g16 >> 2, t1 = 16 * (g16 & 3);
            const float sh = gates[G_HI + s], sl = gates[G_LO + s];
            const float bs = gates[G_BETA + s] * r_down * (which == 1 ? -y_down : gates[G_XDN]);
            float2 x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 f = *reinterpret_cast<const float4*>(raw + ((4 * g16 + e) * C + s) * 16);
                x[2 * e] = make_float2(f.x, f.y);
                x[2 * e + 1] = make_float2(f.z, f.w);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 f = *reinterpret_cast<const float4*>(
                    t1 + 4 * e > s ? raw + ((16 * which + (C - 4 - t1) / 4 - e) * C + C - 1 - s) * 16
                                   : smem + GR_NEAR + (C * which + s) * 16);
                w[4 * e] = f.w;
                w[4 * e + 1] = f.z;
                w[4 * e + 2] = f.y;
                w[4 * e + 3] = f.x;
            }
            const int first = which == 1 ? s + 1 : s;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int t = t1 + 2 * e;
                const float2 gh = *reinterpret_cast<const float2*>(gates + G_HI + t);
                const float2 gl = *reinterpret_cast<const float2*>(gates + G_LO + t);
                if (which == 1) {   // R_s . Y_s
                    const float2 gb = *reinterpret_cast<const float2*>(gates + G_BETA + t);
                    if ((t == s || t + 1 == s) && s < m)
                        static_cast<__nv_bfloat16*>(a.grad_beta)[tok + s] =
                            __float2bfloat16_rn((t == s ? x[e].x : x[e].y) * r_down * y_down);
                    x[e] = __fmul2_rn(x[e], gb);
                }
                // (first the scales, then the decay: theirs may be 2^-116, and its product with that no float)
                x[e] = __fmul2_rn(x[e], both(bs));
                x[e].x = t >= first ? x[e].x * ex2((gh.x - sh) + (gl.x - sl)) : 0.f;
                x[e].y = t + 1 >= first ? x[e].y * ex2((gh.y - sh) + (gl.y - sl)) : 0.f;
            }
            {   // sums of W from each of the 16 tokens on, of one writer before it; of all 16
                const float f = gates[G_KDN] * (which == 1 ? gates[G_KDN] : gates[G_QDN]);
                float sum = 0.f;
#pragma unroll
                for (int t = 15; t >= 0; --t) {
                    if (t1 + t > s) sum = fmaf(f * w[t], t & 1 ? x[t / 2].y : x[t / 2].x, sum);
                    w[t] = t1 + t > s ? sum : 0.f;
                }
                sw[g16 * C + s] = sum;
            }
            // dP and dG have a power of two each (queries of 2^-40 make dG so much smaller beside dP): warps 0-7 have
            // dP, 8-15 dG.  (The exchange's barrier is past every thread's loads.)
            float g_up;
            block_top(tops + 3 * GR_WARPS, largest(0.f, x), 1, GR_WARPS * 32, GR_WARPS, warp);
            scale_of(warps_top(tops + 3 * GR_WARPS), up, p_down);
            scale_of(warps_top(tops + 3 * GR_WARPS + GR_WARPS / 2), g_up, g_down);
            if (which == 1) up = g_up;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                unsigned char* to = smem + GR_P + at_d(s, 2 * g16 + e);
                half_pieces(to, to + C * 2 * C * 2, x + 4 * e, up);
            }
            arrive(have_p);
        }
        {   // D1 in halves, where S0 was
            float4 g[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = __ldg(reinterpret_cast<const float4*>(adjoint + at_f(i, 8 * quarter + e)));
            wait_warp(done_b);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x[4] = {make_float2(g[2 * e].x, g[2 * e].y), make_float2(g[2 * e].z, g[2 * e].w),
                                     make_float2(g[2 * e + 1].x, g[2 * e + 1].y), make_float2(g[2 * e + 1].z, g[2 * e + 1].w)};
                unsigned char* to = smem + GR_S + at_d(i, 4 * quarter + e);
                half_pieces(to, to + D * D * 2, x, d_up);
            }
            arrive(have_d);
        }
        {   // ... over all writers, of dP or dG
            const int s0 = warp & 1, g16 = warp >> 1;
            const float across = lane_sums(w, lane);
            if (lane < 16) sx[(2 * (g16 >> 2) + s0) * C + 16 * (g16 & 3) + lane] = across;
        }
        const int j = 32 * q4 + lane, dk = FULL ? D : a.dk;
        const int mine = FULL || j < dk ? m - tb : 0;          // tokens of a column that there is
        const float kdn = gates[G_KDN], qdn = gates[G_QDN];
        float cc[16];
        float2 kr[8], kj[8];
        auto column = [&](const unsigned char* p, float down, float2 (&v)[8]) {
#pragma unroll
            for (int t = 0; t < 16; ++t) {
                const float f = down * __half2float(*reinterpret_cast<const __half*>(p + (t / 8) * ROWS_D + (t % 8) * 16));
                if (t & 1) v[t / 2].y = f;
                else v[t / 2].x = f;
            }
        };
        const unsigned char* at = smem + GR_KQ + at_d(tb, j / 8) + (j % 8) * 2;
        {
            float2 x[8], y[8], g[8];
            get16(gates + G_E + tb, g);
            tmem_get16(tl + CG_Q + tb, x);
            wait_warp(done_c);
            tmem_get16(tl + CG_Q2 + tb, y);
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.grad_q) + (tok + tb) * dk + j;
            column(at + TILE_X, qdn, kj);
            const float f = s_down * gates[G_XDN], fp = p_down * kdn;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = __fmul2_rn(__fmul2_rn(g[e], both(f)), x[e]);
                y[e] = __ffma2_rn(y[e], both(fp), x[e]);
                if (2 * e < mine) dst[2 * e * dk] = __float2bfloat16_rn(y[e].x);
                if (2 * e + 1 < mine) dst[(2 * e + 1) * dk] = __float2bfloat16_rn(y[e].y);
                cc[2 * e] = kj[e].x * x[e].x;
                cc[2 * e + 1] = kj[e].y * x[e].y;
            }
            tmem_get16(tl + CG_R + tb, x);
            tmem_get16(tl + CG_Q2 + C + tb, y);
            float2 b[8];
            get16(gates + G_BETA + tb, b);
            column(at, kdn, kj);
            const float fr = -s_down * y_down, fg = g_down * kdn;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = __fmul2_rn(__fmul2_rn(__fmul2_rn(g[e], both(fr)), b[e]), x[e]);
                kr[e] = __ffma2_rn(y[e], both(fg), x[e]);
                cc[2 * e] = fmaf(kj[e].x, x[e].x, cc[2 * e]);
                cc[2 * e + 1] = fmaf(kj[e].y, x[e].y, cc[2 * e + 1]);
            }
        }
        {
            float2 x[8], y[8];
            tmem_get16(tl + CG_W2 + tb, y);
            tmem_get16(tl + CG_A + tb, x);
            const float fq = p_down * qdn, fk = g_down * kdn;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[e] = __ffma2_rn(y[e], both(fq), __fmul2_rn(x[e], both(fk)));
                kr[e] = __fadd2_rn(kr[e], y[e]);
            }
        }
        const float c1 = lane_sums(cc, lane);
        {
            float2 x[8], g[8], b[8];
            float f[16];
            get16(gates + G_W + tb, g);
            get16(gates + G_BETA + tb, b);
            const float fd = d_down * r_down;
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = __fmul2_rn(__fmul2_rn(g[e], both(fd)), b[e]);
            wait_warp(done_d);
            tmem_get16(tl + CG_W + tb, x);
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.grad_k) + (tok + tb) * dk + j;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = __fmul2_rn(g[e], x[e]);
                f[2 * e] = kj[e].x * x[e].x;
                f[2 * e + 1] = kj[e].y * x[e].y;
                x[e] = __fadd2_rn(x[e], kr[e]);
                if (2 * e < mine) dst[2 * e * dk] = __float2bfloat16_rn(x[e].x);
                if (2 * e + 1 < mine) dst[(2 * e + 1) * dk] = __float2bfloat16_rn(x[e].y);
            }
            const float f1 = lane_sums(f, lane);
            if (lane < 16) {
                sc[q4 * C + tb + lane] = c1;
                sf[q4 * C + tb + lane] = f1;
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == GR_WARPS) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
    if (warp == 0) {
        // gradients of the log decays: all that is read from a token on of what was written before it.  Reads of S0
        // from the chunk's end, writes to D1 from its beginning, W of the pairs that stand across, <D1, S0>: each term
        // has the token's decay in it.  (As sums of q.dq + k.dk the other pairs cancel but for their roundings, which
        // are larger than the gradient of a strong decay: of decays of e^-5 to e^-20 some had no digit right.)
        float c[2], f[2], w[2], x = lane < GR_WARPS ? ssum[lane] : 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            c[e] = (sc[t] + sc[C + t]) + (sc[2 * C + t] + sc[3 * C + t]);
            f[e] = (sf[t] + sf[C + t]) + (sf[2 * C + t] + sf[3 * C + t]);
            w[e] = (sx[t] + sx[C + t]) + (sx[2 * C + t] + sx[3 * C + t]);
        }
#pragma unroll
        for (int g = 1; g < 4; ++g) {        // readers of a later 16
            const float2 u = *reinterpret_cast<const float2*>(sw + g * C + 2 * lane);
            const float2 v = *reinterpret_cast<const float2*>(sw + (4 + g) * C + 2 * lane);
            const float first = u.x + v.x;
            float s = first + (u.y + v.y);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float z = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += z;
            }
            float before = __shfl_up_sync(0xffffffffu, s, 1);
            if (lane == 0) before = 0.f;
            if (lane < 8 * g) {
                w[0] += before;
                w[1] += before + first;
            }
        }
        float s = c[0] + c[1], pre = f[0] + f[1];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float z = __shfl_down_sync(0xffffffffu, s, o), y = __shfl_up_sync(0xffffffffu, pre, o);
            if (lane + o < 32) s += z;
            if (lane >= o) pre += y;
        }
        const float above = __shfl_down_sync(0xffffffffu, s, 1), below = __shfl_up_sync(0xffffffffu, pre, 1);
        const float rest = fmaf(gates[G_END], x, lane > 0 ? below : 0.f);
        const float ga[2] = {(s + rest) + w[0], (((lane < 31 ? above : 0.f) + c[1]) + (rest + f[0])) + w[1]};
        const float A = a.A[h];
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            if (t < m) {
                static_cast<__nv_bfloat16*>(a.grad_d)[tok + t] = __float2bfloat16_rn(-A * ga[e]);
                sum = fmaf(-to_f32(static_cast<const __nv_bfloat16*>(a.d)[tok + t]), ga[e], sum);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
            if (in.sum_A) in.sum_A[tile] = sum;
            if (*dead) record_error(&g_delta_error, KDN_ERR_TIMEOUT);
        }
    }
}

}  // namespace

// Heads narrower than 128 are taken with zeros behind, at the cost of whole ones:
// us here / token by token, forward then backward, of 16 x 32 x 4096 x 64 x 64 1739
// / 2567, 5717 / 13385; of 128 heads x 2048 of 64 x 32 235 / 382, 775 / 1213, but of
// 2048 x 256 471 / 308, 1503 / 1476: smaller ones where each has an SM of its own
// (of 32 x 32 and less the gain, 234 / 360, is not worth ten times the scratch).
bool tc_takes(int B, int H, int dk, int dv, int nseq, kdn_dtype in_dtype) {
    const long long rows = static_cast<long long>(nseq > 0 ? nseq : B) * H;
    return in_dtype == KDN_BF16 && (dk * dv >= 64 * 64 || (dk * dv >= 64 * 32 && rows <= sm_count()));
}

// Against the walk token by token (us for heads x tokens, here / there): few heads
// wait for two launches here, 16 x 48 19.1 / 13.7, 16 x 64 18.3 / 16.9, 16 x 96
// 21 / 24, 64 x 48 19.3 / 18.3, 64 x 64 18.7 / 22.9; many cost a chunk's work
// however few its tokens, 128 x 24 20.6 / 20.0, 256 x 16 34 / 25, 256 x 32 33 / 41,
// 2048 x 16 211 / 157, 2048 x 32 204 / 264.  Narrower heads, 128 x 64: 16 x 64 26 /
// 21, 16 x 128 28 / 34, 2048 x 32 204 / 139, 2048 x 64 190 / 251; 64 x 64: 16 x 64
// 25 / 20, 16 x 128 27 / 30, 2048 x 64 180 / 153, 2048 x 128 280 / 294.  (Backward
// calls gain at any length: 16 x 8 44 / 65, 2048 x 8 546 / 1140, 2048 x 256 1620 /
// 7740; of 64 x 64 16 x 32 53 / 55, 2048 x 32 520 / 666.)
bool tc_takes_fwd(int B, int H, int T, int dk, int dv, int nseq, kdn_dtype in_dtype) {
    const bool few = static_cast<long long>(nseq > 0 ? nseq : B) * H <= 64;
    const int least = dk * dv == D * D ? (few ? 64 : 28) : dk * dv >= D * D / 2 ? (few ? 96 : 48) : 112;
    return tc_takes(B, H, dk, dv, nseq, in_dtype) && T / (nseq > 0 ? nseq : 1) >= least;
}

namespace {

// Few heads and long sequences: parts walk side by side once their first states
// are known, for which each part but the last is walked twice more (N and M) and
// the ends are folded one after another.  In units of a chunk's walk: an end's
// costs 0.8, a fold about one, the launches four.  No split unless it takes three
// quarters of the time.  (Packed sequences' lengths are the device's.)
Parts cut_of(int B, int H, int T, int nseq) {
    Parts best{1, 0, nullptr, nullptr};
    if (nseq > 0) return best;
    const long long rows = static_cast<long long>(B) * H, sms = sm_count();
    const int chunks = (T + C - 1) / C;
    const auto rounds = [&](long long jobs) { return static_cast<double>((jobs + sms - 1) / sms); };
    double least = 0.75 * rounds(rows) * chunks;
    if (rows >= sms) return best;
    for (int p = 2; p <= 64 && p <= chunks / 2; ++p) {
        const int len = (chunks + p - 1) / p, parts = (chunks + len - 1) / len;
        if (parts < 2) break;
        const double cost = (rounds(rows * parts) + 0.8 * rounds(2 * rows * (parts - 1))) * len + parts + 4.0;
        if (cost < least) {
            least = cost;
            best.parts = parts;
            best.len = len;
        }
    }
    return best;
}
long long rounded(long long bytes) { return (bytes + 255) / 256 * 256; }

// The first states of all parts.
cudaError_t states_of_parts(const DeltaArgs& a, const char* prep, int step, const Parts& cut, float* starts, long long rows,
                            cudaStream_t stream, long long wait_ns) {
    auto kernel = a.dk == D && a.dv == D ? delta_chunk_kernel<float, ENDS, true> : delta_chunk_kernel<float, ENDS, false>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), CH_SMEM);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(rows * 2 * (cut.parts - 1)), CH_THREADS, CH_SMEM, stream>>>(a, prep, step, KeepTiles{}, cut, wait_ns);
    delta_fold_kernel<<<static_cast<unsigned>(rows * (D / FOLD_ROWS)), FOLD_THREADS, 0, stream>>>(a.S0, cut.ends, starts, cut.parts,
                                                                                                 a.dk, a.dv);
    return cudaGetLastError();
}

}  // namespace

long long tc_fwd_bytes(int B, int H, int T, int nseq) {
    const Parts cut = cut_of(B, H, T, nseq);
    const long long rows = static_cast<long long>(B) * H, states = cut.parts > 1 ? rows * (3LL * cut.parts - 2) : 0;
    return slots_of(B, T, nseq) * H * PREP_BYTES + states * D * D * 4;
}

kdn_status tc_fwd(const DeltaArgs& a, char* ws, cudaStream_t stream, long long wait_ns) {
    const long long blocks = slots_of(a.B, a.T, a.nseq) * a.H;
    const long long rows = static_cast<long long>(a.offsets ? a.nseq : a.B) * a.H;
    if (blocks > 0x7fffffffLL || rows > 0x7fffffffLL) return KDN_ERR_INVALID_ARG;
    const bool full = a.dk == D && a.dv == D, bf16 = a.out_dtype == KDN_BF16;
    cudaError_t e;
    auto prepare = full ? delta_prep_kernel<true> : delta_prep_kernel<false>;
    if ((e = allow_smem(reinterpret_cast<const void*>(prepare), P_SMEM)) != cudaSuccess) return from_cuda(e);
    prepare<<<static_cast<unsigned>(blocks), PREP_THREADS, P_SMEM, stream>>>(a, ws, wait_ns);
    if ((e = cudaGetLastError()) != cudaSuccess) return from_cuda(e);
    Parts cut = cut_of(a.B, a.H, a.T, a.nseq);
    if (cut.parts > 1) {
        cut.ends = reinterpret_cast<float*>(ws + blocks * PREP_BYTES);
        float* starts = cut.ends + rows * 2 * (cut.parts - 1) * D * D;
        if ((e = states_of_parts(a, ws, PREP_BYTES, cut, starts, rows, stream, wait_ns)) != cudaSuccess) return from_cuda(e);
        cut.starts = starts;
    }
    auto kernel = full ? (bf16 ? delta_chunk_kernel<__nv_bfloat16, OUTPUTS, true> : delta_chunk_kernel<float, OUTPUTS, true>)
                       : (bf16 ? delta_chunk_kernel<__nv_bfloat16, OUTPUTS, false> : delta_chunk_kernel<float, OUTPUTS, false>);
    if ((e = allow_smem(reinterpret_cast<const void*>(kernel), CH_SMEM)) != cudaSuccess) return from_cuda(e);
    kernel<<<static_cast<unsigned>(rows * cut.parts), CH_THREADS, CH_SMEM, stream>>>(a, ws, PREP_BYTES, KeepTiles{}, cut, wait_ns);
    return from_cuda(cudaGetLastError());
}

long long tc_bwd_bytes(int B, int H, int T, int nseq) {
    const long long tiles = slots_of(B, T, nseq) * H;
    const Parts cut = cut_of(B, H, T, nseq);
    const long long states = cut.parts > 1 ? static_cast<long long>(B) * H * (3LL * cut.parts - 2) : 0;
    return tiles * (PREP_STEP + 2 * STATE_BYTES + 2 * ROWS_BYTES) + rounded(tiles * 4) + states * STATE_BYTES;
}

kdn_status tc_bwd(const DeltaArgs& a, char* ws, cudaStream_t stream, long long wait_ns) {
    const long long slots = slots_of(a.B, a.T, a.nseq), tiles = slots * a.H;
    const long long rows = static_cast<long long>(a.offsets ? a.nseq : a.B) * a.H;
    if (tiles > 0x7fffffffLL || rows > 0x7fffffffLL) return KDN_ERR_INVALID_ARG;
    char* prep = ws;
    const KeepTiles fwd{prep + tiles * PREP_STEP, prep + tiles * (PREP_STEP + 2 * STATE_BYTES)};
    const KeepTiles bwd{fwd.states + tiles * STATE_BYTES, fwd.rows + tiles * ROWS_BYTES};
    float* shares = reinterpret_cast<float*>(bwd.rows + tiles * ROWS_BYTES);
    const bool full = a.dk == D && a.dv == D;
    auto prepare = full ? delta_prep_kernel<true> : delta_prep_kernel<false>;
    auto walk = full ? delta_chunk_kernel<float, TILES, true> : delta_chunk_kernel<float, TILES, false>;
    auto adjoint = full ? delta_adjoint_kernel<true, false> : delta_adjoint_kernel<false, false>;
    auto gradients = full ? delta_tc_grad_kernel<true> : delta_tc_grad_kernel<false>;
    const std::pair<const void*, int> kernels[] = {{reinterpret_cast<const void*>(prepare), P_SMEM},
                                                   {reinterpret_cast<const void*>(walk), CH_SMEM},
                                                   {reinterpret_cast<const void*>(adjoint), AD_SMEM},
                                                   {reinterpret_cast<const void*>(gradients), GR_SMEM}};
    cudaError_t e = cudaSuccess;
    for (const auto& k : kernels)
        if ((e = allow_smem(k.first, k.second)) != cudaSuccess) return from_cuda(e);
    prepare<<<static_cast<unsigned>(tiles), PREP_THREADS, P_SMEM, stream>>>(a, prep, wait_ns);
    Parts cut = cut_of(a.B, a.H, a.T, a.nseq), back = cut;
    float* starts = nullptr;
    if (cut.parts > 1) {
        cut.ends = back.ends = reinterpret_cast<float*>(reinterpret_cast<char*>(shares) + rounded(tiles * 4));
        starts = cut.ends + rows * 2 * (cut.parts - 1) * D * D;
        if ((e = states_of_parts(a, prep, PREP_STEP, cut, starts, rows, stream, wait_ns)) != cudaSuccess) return from_cuda(e);
        cut.starts = back.starts = starts;
    }
    const unsigned walks = static_cast<unsigned>(rows * cut.parts);
    walk<<<walks, CH_THREADS, CH_SMEM, stream>>>(a, prep, PREP_STEP, fwd, cut, wait_ns);
    if (cut.parts > 1) {   // (what the forward's ends and first states lie in is free, but M)
        auto ends = full ? delta_adjoint_kernel<true, true> : delta_adjoint_kernel<false, true>;
        if ((e = allow_smem(reinterpret_cast<const void*>(ends), AD_SMEM)) != cudaSuccess) return from_cuda(e);
        ends<<<static_cast<unsigned>(rows * (cut.parts - 1)), CH_THREADS, AD_SMEM, stream>>>(a, prep, bwd, back, wait_ns);
        delta_fold_back_kernel<<<static_cast<unsigned>(rows * (D / FOLD_ROWS)), FOLD_THREADS, 0, stream>>>(
            a.grad_final_state, back.ends, starts, cut.parts, a.dk, a.dv);
    }
    adjoint<<<walks, CH_THREADS, AD_SMEM, stream>>>(a, prep, bwd, back, wait_ns);
    gradients<<<static_cast<unsigned>(tiles), GR_THREADS, GR_SMEM, stream>>>(
        a, GradTiles{prep, fwd.states, bwd.states, fwd.rows, bwd.rows, a.grad_A ? shares : nullptr, sm_count()}, wait_ns);
    if ((e = cudaGetLastError()) != cudaSuccess || !a.grad_A) return from_cuda(e);
    return from_cuda(sum_rows(shares, slots, a.H, a.grad_A, nullptr, a.H, stream));
}

}  // namespace delta

cudaError_t delta_take_device_error(int* status) {
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, delta::g_delta_error, sizeof(int));
    if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(delta::g_delta_error, &zero, sizeof(int));
    *status = v;
    return e;
}

}  // namespace kdn
