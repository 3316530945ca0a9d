// delta_tc.cu -- the gated delta rule in chunks of 64 tokens on the tensor
// cores, for bf16 inputs and d_k = d_v = 128 (delta_device.cuh has the rule,
// delta_scan.cu the token-by-token form for the rest).
//
// With g_t the log decay since the chunk began and E_ts = e^{g_t - g_s}, and S
// the state before the chunk,
//     G = (K K^T) . E (s < t),   P = (Q K^T) . E (s <= t),
//     T = -G (1 + beta G)^{-1}   (strictly lower),
//     Z = V - e^g K S^T,   R = Z + T (beta Z),   U = beta R,
//     O = e^g Q S^T + P U,
//     S' = e^{g_C} S + U^T (e^{g_C - g} K).
// T and P need no state: delta_prep_kernel makes them for all chunks side by
// side, and delta_chunk_kernel walks a head's chunks with four products each.
#include <type_traits>

#include "delta_device.cuh"
#include "delta_tc.h"
#include "kdn.h"
#include "kdn_device.cuh"
#include "kdn_internal.h"
#include "kernel_setup.h"

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
constexpr int TILE_T = C * C * 2;            // one bf16 half of T or P
__host__ __device__ constexpr int at_d(int r, int c8) { return (r / 8) * ROWS_D + c8 * 128 + (r % 8) * 16; }
__host__ __device__ constexpr int at_c(int r, int c8) { return (r / 8) * ROWS_C + c8 * 128 + (r % 8) * 16; }

// What the preparation leaves of a chunk, as the walk reads it.
constexpr int PREP_T = 0;                    // T hi, lo
constexpr int PREP_P = 2 * TILE_T;           // P hi, lo
constexpr int PREP_GATES = 4 * TILE_T;       // e^g, e^{g_C - g}, beta: [3][64] fp32, then e^{g_C}
constexpr int PREP_BYTES = PREP_GATES + 1024;

// x as bf16 pairs hi + lo: hi rounded to nearest, lo what is left, rounded:
// within 2^-17 of x, and 2^-20 in the mean.
__device__ __forceinline__ void halves(float2 x, uint32_t& hi, uint32_t& lo) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const float2 up = make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
    const float2 d = __ffma2_rn(up, make_float2(-1.f, -1.f), x);
    const __nv_bfloat162 l = __floats2bfloat162_rn(d.x, d.y);
    lo = *reinterpret_cast<const uint32_t*>(&l);
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
// token), by `threads` threads.  A warp instruction moves 8 tokens x 4 of
// their 16-byte pieces, so that its writes hit each bank group four times.
__device__ __forceinline__ void load_kq(uint32_t tile, const __nv_bfloat16* k, const __nv_bfloat16* q, int n, int tid,
                                        int threads) {
    const int lane = tid & 31, a = lane & 7, b = lane >> 3;
    for (int w = tid >> 5; w < 2 * C / 8 * 4; w += threads >> 5) {
        const int r = (w >> 2) * 8 + a, c8 = (w & 3) * 4 + b, t = r & (C - 1);
        const __nv_bfloat16* src = (r < C ? k : q) + (t < n ? static_cast<long long>(t) * D : 0) + c8 * 8;
        copy16_or_zero(tile + at_d(r, c8), src, t < n);
    }
}

// ---- preparation -------------------------------------------------------------

constexpr int PREP_THREADS = 128;
constexpr int LG = C + 4, LX = 36;           // a row of G, T and of X in shared memory
// G (then T, block by block in its place), N = G beta and X lie where k and q
// lay before the product: five CTAs to an SM hide one another's waits.
constexpr int P_OFF_KQ = 0, P_OFF_G = 0, P_OFF_N = P_OFF_G + C * LG * 4, P_OFF_X = P_OFF_N + C * LG * 4,
              P_OFF_GATE = P_OFF_X + 32 * LX * 4, P_SMEM = P_OFF_GATE + 3 * C * 4 + 64;
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
// formed: keys that are alike make those large.
__global__ void __launch_bounds__(PREP_THREADS) delta_prep_kernel(const DeltaArgs a, char* prep, long long wait_ns) {
    extern __shared__ __align__(128) unsigned char smem[];
    float* sG = reinterpret_cast<float*>(smem + P_OFF_G);        // [t][s]
    float* sN = reinterpret_cast<float*>(smem + P_OFF_N);        // G beta
    float* gh = reinterpret_cast<float*>(smem + P_OFF_GATE);     // log2 decay since the chunk began, as two floats
    float* gl = gh + C;
    float* sb = gl + C;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + P_OFF_GATE + 3 * C * 4);
    uint32_t* holder = reinterpret_cast<uint32_t*>(bar + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = static_cast<int>(blockIdx.x % a.H);
    const long long slot = blockIdx.x / a.H;
    long long n, row;
    int t0, m;
    if (!chunk_of(a, slot, &n, &t0, &m, &row)) return;
    const long long tok = (row * a.H + h) * a.T + t0;
    char* out = prep + (slot * a.H + h) * static_cast<long long>(PREP_BYTES);

    load_kq(smem_addr(smem), static_cast<const __nv_bfloat16*>(a.k) + tok * D,
            static_cast<const __nv_bfloat16*>(a.q) + tok * D, m, tid, PREP_THREADS);
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
        const double end = __shfl_sync(0xffffffffu, s, 31);
        g[0] = s - g[1];
        g[1] = s;
        float* gates = reinterpret_cast<float*>(out + PREP_GATES);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            gh[t] = static_cast<float>(g[e]);
            gl[t] = static_cast<float>(g[e] - gh[t]);
            sb[t] = b[e];
            gates[t] = exp2f(static_cast<float>(g[e]));
            gates[C + t] = exp2f(static_cast<float>(end - g[e]));
            gates[2 * C + t] = b[e];
        }
        if (lane == 0) gates[3 * C] = exp2f(static_cast<float>(end));
    }
    copies_done();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *holder, base = smem_addr(smem);
    if (tid == 0) {
        constexpr uint32_t IDESC = umma_idesc_bf16_f32(128, C);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t d = umma_desc_kmajor(base + P_OFF_KQ + ks * 256, 128, ROWS_D);
            umma_bf16(tmem, d, d, IDESC, ks > 0 ? 1u : 0u);
        }
        umma_commit(bar);
    }
    const bool ok = mbar_wait(bar, 0, wait_ns);
    tc_fence_after_sync();
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
                    const int last = reads ? t - 1 : t;
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
                    for (int p = 0; p < 4; ++p) halves(make_float2(x[e + 2 * p], x[e + 2 * p + 1]), hi[p], lo[p]);
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
    for (int i = tid; i < C * (C / 8); i += PREP_THREADS) {
        const int t = i & (C - 1), c8 = i / C;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int s = 8 * c8 + 2 * p;
            halves(*reinterpret_cast<const float2*>(sG + t * LG + s), hi[p], lo[p]);
        }
        const int off = PREP_T + at_c(t, c8);
        *reinterpret_cast<uint4*>(out + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(out + off + TILE_T) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    if (!ok) record_error(&g_delta_error, KDN_ERR_TIMEOUT);
}

// ---- the walk ------------------------------------------------------------------

// Warps 0-15 work on the state's rows (thread = row i = lane of tensor memory,
// warp / 4 = quarter of the columns and of the tokens), warp 16 issues the
// products, warps 17 and 18 bring the tiles, one chunk ahead.  Sixteen row
// warps: with eight, two to a scheduler, their dependent steps took 1.6 times
// as long (a chunk 7900 cycles).
constexpr int ROW_WARPS = 16, MMA_WARP = ROW_WARPS, LOAD_WARPS = 2, CH_THREADS = (ROW_WARPS + 1 + LOAD_WARPS) * 32;
// shared memory: two stages of [k; q], v and the prepared chunk
constexpr int ST_V = 2 * TILE_X, ST_PREP = ST_V + TILE_X, STAGE_BYTES = ST_PREP + PREP_BYTES;
constexpr int CH_OFF_BAR = 2 * STAGE_BYTES, CH_SMEM = CH_OFF_BAR + 128;
static_assert(CH_SMEM <= 227 * 1024, "shared memory");
// tensor memory: S (fp32) and its bf16 halves as packed pairs (an A operand's
// layout), the accumulators of Z (then of R, then U's halves) and of Q S^T, of
// P U, and the halves of beta Z (then of e^{g_C - g} U)
constexpr uint32_t COL_S = 0, COL_SH = 128, COL_SL = 192, COL_Z = 256, COL_QS = 320, COL_O = 384, COL_W = 448;

// Waits that end: the first that runs out marks the CTA, and the others return
// at once.
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
// D (TMEM) = A (TMEM, bf16 pairs packed per column, lane = row) * B^T (smem)
__device__ __forceinline__ void umma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
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
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const float2 (&x)[8]) {
    float v[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[2 * e] = x[e].x;
        v[2 * e + 1] = x[e].y;
    }
    tmem_st16(taddr, v);
}
// The halves of 16 tokens' values, one K step: hi in 8 columns, lo in the 8 behind them.
__device__ __forceinline__ void put_halves(uint32_t taddr, const float2 (&x)[8]) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) halves(x[e], hi[e], lo[e]);
    tmem_st8w(taddr, hi);
    tmem_st8w(taddr + 8, lo);
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

template <typename TO>
__global__ void __launch_bounds__(CH_THREADS, 1) delta_chunk_kernel(const DeltaArgs a, const char* prep, long long wait_ns) {
    extern __shared__ __align__(128) unsigned char smem[];
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
    uint32_t* holder = reinterpret_cast<uint32_t*>(have_u + 1);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long sr = blockIdx.x, n = sr / a.H;
    const int h = static_cast<int>(sr % a.H);
    const Span sp = span_of(a, n);
    const int len = max(sp.hi - sp.lo, 0), chunks = (len + C - 1) / C;
    const long long tok = (sp.row * a.H + h) * a.T + sp.lo, size = static_cast<long long>(D) * D;
    const float* S0 = a.S0 ? a.S0 + sr * size : nullptr;
    float* final_state = a.final_state ? a.final_state + sr * size : nullptr;
    if (chunks == 0) {
        if (final_state)
            for (int i = tid; i < size / 4; i += CH_THREADS)
                reinterpret_cast<float4*>(final_state)[i] =
                    S0 ? reinterpret_cast<const float4*>(S0)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(full + s, LOAD_WARPS * 32 + 1);
            mbar_init(empty + s, 1 + ROW_WARPS);
        }
        for (uint64_t* b : {done_z, done_r, done_s, done_s + 1, done_o}) mbar_init(b, 1);
        for (uint64_t* b : {have_z, have_w, have_u}) mbar_init(b, ROW_WARPS);
        for (uint64_t* b : {have_s, have_s + 1}) mbar_init(b, ROW_WARPS / 2);
        mbar_init_fence();
        *dead = 0;
    }
    if (warp == MMA_WARP) tmem_alloc(holder, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *holder, base = smem_addr(smem);
    const Waits wait{dead, wait_ns};

    if (warp > MMA_WARP) {
        // ---- tiles ------------------------------------------------------------------
        const int l = tid - (MMA_WARP + 1) * 32;
        const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + tok * D;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + tok * D;
        const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + tok * D;
        const char* mine = prep + (sp.slot * a.H + h) * static_cast<long long>(PREP_BYTES);
        int sent = -1;                                   // the last chunk whose copies were issued
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1, m = min(C, len - c * C);
            if (c >= 2) wait(empty + st, ((c >> 1) - 1) & 1);
            if (*dead) break;
            sent = c;
            unsigned char* stage = smem + st * STAGE_BYTES;
            const long long row = static_cast<long long>(c) * C * D;
            if (l == 0) {
                mbar_arrive_expect_tx(full + st, m * D * 2 + PREP_BYTES);
                bulk_g2s(stage + ST_V, v + row, m * D * 2, full + st);
                bulk_g2s(stage + ST_PREP, mine + c * static_cast<long long>(a.H) * PREP_BYTES, PREP_BYTES, full + st);
            }
            load_kq(smem_addr(stage), k + row, q + row, m, l, LOAD_WARPS * 32);
            // no token: zeros, not what lay there before
            for (int e = l; e < (C - m) * (D / 8); e += LOAD_WARPS * 32)
                *reinterpret_cast<uint4*>(stage + ST_V + m * D * 2 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
            copies_done();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(full + st);
        }
        // no copy outlives the CTA
        if (l == 0 && sent >= 0 && !mbar_wait(full + (sent & 1), (sent >> 1) & 1, wait_ns)) *dead = 1;
    } else if (warp == MMA_WARP) {
        // ---- products ---------------------------------------------------------------
        {
            auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
                wait(bar, parity);
                __syncwarp();
                tc_fence_after_sync();
            };
            constexpr uint32_t ID_T = umma_idesc_bf16_f32(128, C), ID_S = umma_idesc_bf16_f32(128, D / 2, false, true);
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                const uint32_t par = c & 1, kq = base + st * STAGE_BYTES, pr = kq + ST_PREP;
                wait_warp(full + st, (c >> 1) & 1);
                if (c > 0) wait_warp(done_o, par ^ 1);   // (U's halves were read out of COL_Z)
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
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
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
                // S += (e^{g_C - g} U)^T K, in two halves of its columns
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks) {
                        const uint64_t b = umma_desc_mnmajor(kq + ks * 2 * ROWS_D + half * (D / 16) * 128, ROWS_D, 128);
                        umma_ta(tmem + COL_S + half * (D / 2), tmem + COL_W + 16 * ks, b, ID_S, 1u);
                        umma_ta(tmem + COL_S + half * (D / 2), tmem + COL_W + 16 * ks + 8, b, ID_S, 1u);
                    }
                    umma_done(done_s + half);
                }
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
                umma_done(empty + st);
            }
            if (!mbar_wait(done_o, (chunks - 1) & 1, wait_ns)) *dead = 1;   // nor does a product
        }
    } else {
        // ---- rows -------------------------------------------------------------------
        const int q4 = warp & 3, part = warp >> 2, i = 32 * q4 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q4) << 16);
        const int cb = 32 * part, tb = 16 * part;        // its columns of S, its tokens
        auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
            wait(bar, parity);
            __syncwarp();
            tc_fence_after_sync();
        };
        auto arrive = [&](uint64_t* bar) {
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float2 x[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (S0) f = *reinterpret_cast<const float4*>(S0 + static_cast<long long>(i) * D + cb + 16 * p + 2 * e);
                x[e] = make_float2(f.x, f.y);
                x[e + 1] = make_float2(f.z, f.w);
            }
            tmem_put16(tl + COL_S + cb + 16 * p, x);
        }
        tmem_wait_st();
        TO* out = static_cast<TO*>(a.out) + tok * D + i;
        float2 qs[8];                                    // e^g Q S^T of the chunk before
        auto finish = [&](int c) {                       // outputs of chunk c
            wait_warp(done_o, c & 1);
            float2 o[8];
            tmem_get16(tl + COL_O + tb, o);
            const int m = len - c * C - tb;
            TO* dst = out + (static_cast<long long>(c) * C + tb) * D;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 y = __fadd2_rn(o[e], qs[e]);
                if (2 * e < m) dst[2 * e * D] = from_f32<TO>(y.x);
                if (2 * e + 1 < m) dst[(2 * e + 1) * D] = from_f32<TO>(y.y);
            }
        };
        auto read_qs = [&](int c) {                      // (the last use of its stage)
            wait_warp(done_s + (part >> 1), c & 1);
            float2 eg[8];
            tmem_get16(tl + COL_QS + tb, qs);
            get16(reinterpret_cast<const float*>(smem + (c & 1) * STAGE_BYTES + ST_PREP + PREP_GATES) + tb, eg);
#pragma unroll
            for (int e = 0; e < 8; ++e) qs[e] = __fmul2_rn(qs[e], eg[e]);
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + (c & 1));
        };
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            const uint32_t par = c & 1;
            unsigned char* stage = smem + st * STAGE_BYTES;
            const float* eg = reinterpret_cast<const float*>(stage + ST_PREP + PREP_GATES) + tb;
            const float *ew = eg + C, *be = ew + C;
            if (c > 0) read_qs(c - 1);
            wait_warp(full + st, (c >> 1) & 1);
            {   // the state's halves, and its decay over the chunk in place
                const float end = *(reinterpret_cast<const float*>(stage + ST_PREP + PREP_GATES) + 3 * C);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    float2 x[8];
                    tmem_get16(tl + COL_S + cb + 16 * p, x);
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) halves(x[e], hi[e], lo[e]);
                    tmem_st8w(tl + COL_SH + (cb + 16 * p) / 2, hi);
                    tmem_st8w(tl + COL_SL + (cb + 16 * p) / 2, lo);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = __fmul2_rn(x[e], make_float2(end, end));
                    tmem_put16(tl + COL_S + cb + 16 * p, x);
                }
            }
            arrive(have_s + (part >> 1));
            if (c > 0) finish(c - 1);
            float2 z[8], b[8];
            get_column(reinterpret_cast<const __nv_bfloat16*>(stage + ST_V) + tb * D + i, z);
            get16(be, b);
            {   // z = v - e^g S k
                float2 x[8], g[8];
                get16(eg, g);
                wait_warp(done_z, par);
                tmem_get16(tl + COL_Z + tb, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = __fmul2_rn(x[e], g[e]);
                    z[e] = __ffma2_rn(x[e], make_float2(-1.f, -1.f), z[e]);
                    x[e] = __fmul2_rn(b[e], z[e]);
                }
                put_halves(tl + COL_W + tb, x);
                arrive(have_z);
            }
            {   // r = z + T beta z, u = beta r
                float2 x[8], w[8];
                get16(ew, w);
                wait_warp(done_r, par);
                tmem_get16(tl + COL_Z + tb, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    z[e] = __fmul2_rn(b[e], __fadd2_rn(z[e], x[e]));
                    x[e] = __fmul2_rn(w[e], z[e]);
                }
                put_halves(tl + COL_W + tb, x);
                arrive(have_w);
                put_halves(tl + COL_Z + tb, z);
                arrive(have_u);
            }
        }
        read_qs(chunks - 1);
        finish(chunks - 1);
        if (final_state) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float2 x[8];
                tmem_get16(tl + COL_S + cb + 16 * p, x);
                float* dst = final_state + static_cast<long long>(i) * D + cb + 16 * p;
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    *reinterpret_cast<float4*>(dst + 2 * e) = make_float4(x[e].x, x[e].y, x[e + 1].x, x[e + 1].y);
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

}  // namespace

bool tc_takes(int T, int dk, int dv, int nseq, kdn_dtype in_dtype) {
    return in_dtype == KDN_BF16 && dk == D && dv == D && T / (nseq > 0 ? nseq : 1) >= 32;
}

long long tc_fwd_bytes(int B, int H, int T, int nseq) { return slots_of(B, T, nseq) * H * PREP_BYTES; }

kdn_status tc_fwd(const DeltaArgs& a, char* ws, cudaStream_t stream, long long wait_ns) {
    const long long blocks = slots_of(a.B, a.T, a.nseq) * a.H;
    const long long rows = static_cast<long long>(a.offsets ? a.nseq : a.B) * a.H;
    if (blocks > 0x7fffffffLL || rows > 0x7fffffffLL) return KDN_ERR_INVALID_ARG;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(delta_prep_kernel), P_SMEM);
    if (e != cudaSuccess) return from_cuda(e);
    delta_prep_kernel<<<static_cast<unsigned>(blocks), PREP_THREADS, P_SMEM, stream>>>(a, ws, wait_ns);
    if ((e = cudaGetLastError()) != cudaSuccess) return from_cuda(e);
    auto kernel = a.out_dtype == KDN_BF16 ? delta_chunk_kernel<__nv_bfloat16> : delta_chunk_kernel<float>;
    if ((e = allow_smem(reinterpret_cast<const void*>(kernel), CH_SMEM)) != cudaSuccess) return from_cuda(e);
    kernel<<<static_cast<unsigned>(rows), CH_THREADS, CH_SMEM, stream>>>(a, ws, wait_ns);
    return from_cuda(cudaGetLastError());
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
