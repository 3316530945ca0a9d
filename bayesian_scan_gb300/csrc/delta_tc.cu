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

// x0, x1 as bf16 pairs hi + lo: hi rounded to nearest, lo what is left,
// rounded: within 2^-17 of x, and 2^-20 in the mean.
__device__ __forceinline__ void halves(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const __nv_bfloat162 l =
        __floats2bfloat162_rn(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xffff0000u));
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
constexpr int LG = C + 4;                    // a row of G and T in shared memory
constexpr int P_OFF_KQ = 0, P_OFF_G = 2 * TILE_X, P_OFF_T = P_OFF_G + C * LG * 4, P_OFF_X = P_OFF_T + C * LG * 4,
              P_OFF_GATE = P_OFF_X + 32 * 36 * 4, P_SMEM = P_OFF_GATE + 5 * C * 4 + 64;

// A CTA makes one chunk's T and P: one product [K; Q] K^T (M = 128, N = 64),
// then T from G by blocks.  With T1, T2 the blocks' own,
//     T21 = -(1 + T2 beta2) G21 (1 + beta1 T1),
// from 16 x 16 blocks that a warp solves row after row.  No power of G is
// formed: keys that are alike make those large.
__global__ void __launch_bounds__(PREP_THREADS) delta_prep_kernel(const DeltaArgs a, char* prep, long long wait_ns) {
    extern __shared__ __align__(128) unsigned char smem[];
    float* sG = reinterpret_cast<float*>(smem + P_OFF_G);        // [t][s]
    float* sT = reinterpret_cast<float*>(smem + P_OFF_T);
    float* sX = reinterpret_cast<float*>(smem + P_OFF_X);        // [32][36]
    float* gh = reinterpret_cast<float*>(smem + P_OFF_GATE);     // log2 decay since the chunk began, as two floats
    float* gl = gh + C;
    float* sb = gl + C;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + P_OFF_GATE + 5 * C * 4);
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
    for (int i = tid; i < C * LG; i += PREP_THREADS) sT[i] = 0.f;
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
        const float th = gh[t], tl = gl[t];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float x[32];
            tmem_ld32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + 32 * half, x);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const int s = 32 * half + e;
                const float w = ex2((th - gh[s]) + (tl - gl[s]));
                x[e] = (tid < C ? s < t : s <= t) ? x[e] * w : 0.f;
            }
            if (tid < C) {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4*>(sG + t * LG + 32 * half + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            } else {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) halves(x[e + 2 * p], x[e + 2 * p + 1], hi[p], lo[p]);
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
    {   // 16 x 16 blocks on the diagonal: lane c has column c, rows one after another
        const int o = 16 * warp, c = lane & 15;
        float col[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float x = sG[(o + t) * LG + o + c];
#pragma unroll
            for (int s = 0; s < t; ++s) x = fmaf(sG[(o + t) * LG + o + s] * sb[o + s], col[s], x);
            col[t] = -x;                     // (0 above and on the diagonal: G is, and the rows before are)
        }
        if (lane < 16)
#pragma unroll
            for (int t = 0; t < 16; ++t) sT[(o + t) * LG + o + c] = col[t];
    }
    __syncthreads();
    // pairs of blocks of `size`: X = G21 + G21 beta1 T1, T21 = -(X + T2 beta2 X)
#pragma unroll
    for (int size = 16; size < C; size *= 2) {
        const int pairs = C / (2 * size), per = PREP_THREADS / pairs;      // threads to a pair: 64, 128
        const int p = tid / per, i = tid % per, o = 2 * size * p;
        const int c4 = (i % (size / 4)) * 4, r0 = i / (size / 4);
        const int step = per / (size / 4);                                  // 16, 16
        float* X = sX + p * 16 * 36;
        for (int r = r0; r < size; r += step) {
            float4 x = *reinterpret_cast<const float4*>(sG + (o + size + r) * LG + o + c4);
            for (int s = 0; s < size; ++s) {
                const float g = sG[(o + size + r) * LG + o + s] * sb[o + s];
                const float4 y = *reinterpret_cast<const float4*>(sT + (o + s) * LG + o + c4);
                x.x = fmaf(g, y.x, x.x);
                x.y = fmaf(g, y.y, x.y);
                x.z = fmaf(g, y.z, x.z);
                x.w = fmaf(g, y.w, x.w);
            }
            *reinterpret_cast<float4*>(X + r * 36 + c4) = x;
        }
        __syncthreads();
        for (int r = r0; r < size; r += step) {
            float4 x = *reinterpret_cast<const float4*>(X + r * 36 + c4);
            for (int s = 0; s < r; ++s) {    // (T2 is strictly lower)
                const float g = sT[(o + size + r) * LG + o + size + s] * sb[o + size + s];
                const float4 y = *reinterpret_cast<const float4*>(X + s * 36 + c4);
                x.x = fmaf(g, y.x, x.x);
                x.y = fmaf(g, y.y, x.y);
                x.z = fmaf(g, y.z, x.z);
                x.w = fmaf(g, y.w, x.w);
            }
            *reinterpret_cast<float4*>(sT + (o + size + r) * LG + o + c4) = make_float4(-x.x, -x.y, -x.z, -x.w);
        }
        __syncthreads();
    }
    for (int i = tid; i < C * (C / 8); i += PREP_THREADS) {
        const int t = i & (C - 1), c8 = i / C;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int s = 8 * c8 + 2 * p;
            halves(sT[t * LG + s], sT[t * LG + s + 1], hi[p], lo[p]);
        }
        const int off = PREP_T + at_c(t, c8);
        *reinterpret_cast<uint4*>(out + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(out + off + TILE_T) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    if (!ok) record_error(&g_delta_error, KDN_ERR_TIMEOUT);
}

// ---- the walk ------------------------------------------------------------------

// Warps 0-7 work on the state's rows (thread = row i = lane of tensor memory,
// warp / 4 = half of the columns), warp 8 issues the products, warps 9 and 10
// bring the tiles, one chunk ahead.
constexpr int ROW_WARPS = 8, MMA_WARP = 8, LOAD_WARPS = 2, CH_THREADS = (ROW_WARPS + 1 + LOAD_WARPS) * 32;
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

// D (TMEM) = A (TMEM, bf16 pairs packed per column, lane = row) * B^T (smem)
__device__ __forceinline__ void umma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st16w(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// The halves of 32 tokens' values: hi in 16 columns, lo in the 16 behind them.
__device__ __forceinline__ void put_halves(uint32_t taddr, const float (&x)[32]) {
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) halves(x[2 * e], x[2 * e + 1], hi[e], lo[e]);
    tmem_st16w(taddr, hi);
    tmem_st16w(taddr + 16, lo);
}
// ... and where K step ks (16 tokens) of such halves lies.
__device__ __forceinline__ uint32_t half_at(int ks) { return 32 * (ks >> 1) + 8 * (ks & 1); }

template <typename TO>
__global__ void __launch_bounds__(CH_THREADS, 1) delta_chunk_kernel(const DeltaArgs a, const char* prep, long long wait_ns) {
    extern __shared__ __align__(128) unsigned char smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + CH_OFF_BAR);   // [2] a stage is here
    uint64_t* empty = full + 2;                                        // [2] a stage is read
    uint64_t* done_z = empty + 2;                                      // products: Z and Q S^T, R, S, O
    uint64_t* done_r = done_z + 1;
    uint64_t* done_s = done_r + 1;
    uint64_t* done_o = done_s + 1;
    uint64_t* have_s = done_o + 1;                                     // operands: S, beta Z, wU, U
    uint64_t* have_z = have_s + 1;
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
        for (uint64_t* b : {done_z, done_r, done_s, done_o}) mbar_init(b, 1);
        for (uint64_t* b : {have_s, have_z, have_w, have_u}) mbar_init(b, ROW_WARPS);
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
            copies_done();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(full + st);
        }
        // no copy outlives the CTA
        if (l == 0 && sent >= 0 && !mbar_wait(full + (sent & 1), (sent >> 1) & 1, wait_ns)) *dead = 1;
    } else if (warp == MMA_WARP) {
        // ---- products ---------------------------------------------------------------
        if (lane == 0) {
            constexpr uint32_t ID_N128 = umma_idesc_bf16_f32(128, 128), ID_N64 = umma_idesc_bf16_f32(128, C),
                               ID_S = umma_idesc_bf16_f32(128, D, false, true);
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                const uint32_t par = c & 1, kq = base + st * STAGE_BYTES, pr = kq + ST_PREP;
                wait(full + st, (c >> 1) & 1);
                wait(have_s, par);
                if (c > 0) wait(done_o, par ^ 1);        // (U's halves were read out of COL_Z)
                tc_fence_after_sync();
                // [S K^T | S Q^T]
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint64_t b = umma_desc_kmajor(kq + ks * 256, 128, ROWS_D);
                    umma_ta(tmem + COL_Z, tmem + COL_SH + 8 * ks, b, ID_N128, ks > 0 ? 1u : 0u);
                    umma_ta(tmem + COL_Z, tmem + COL_SL + 8 * ks, b, ID_N128, 1u);
                }
                umma_commit(done_z);
                wait(have_z, par);
                tc_fence_after_sync();
                // (beta Z)^T T^T: hi hi, hi lo, lo hi
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks) {
                    const uint64_t hi = umma_desc_kmajor(pr + PREP_T + ks * 256, 128, ROWS_C);
                    const uint64_t lo = umma_desc_kmajor(pr + PREP_T + TILE_T + ks * 256, 128, ROWS_C);
                    const uint32_t z = tmem + COL_W + half_at(ks);
                    umma_ta(tmem + COL_Z, z, hi, ID_N64, ks > 0 ? 1u : 0u);
                    umma_ta(tmem + COL_Z, z, lo, ID_N64, 1u);
                    umma_ta(tmem + COL_Z, z + 16, hi, ID_N64, 1u);
                }
                umma_commit(done_r);
                wait(have_w, par);
                tc_fence_after_sync();
                // S += (e^{g_C - g} U)^T K
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks) {
                    const uint64_t b = umma_desc_mnmajor(kq + ks * 2 * ROWS_D, ROWS_D, 128);
                    umma_ta(tmem + COL_S, tmem + COL_W + half_at(ks), b, ID_S, 1u);
                    umma_ta(tmem + COL_S, tmem + COL_W + half_at(ks) + 16, b, ID_S, 1u);
                }
                umma_commit(done_s);
                wait(have_u, par);
                tc_fence_after_sync();
                // U^T P^T
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks) {
                    const uint64_t hi = umma_desc_kmajor(pr + PREP_P + ks * 256, 128, ROWS_C);
                    const uint64_t lo = umma_desc_kmajor(pr + PREP_P + TILE_T + ks * 256, 128, ROWS_C);
                    const uint32_t u = tmem + COL_Z + half_at(ks);
                    umma_ta(tmem + COL_O, u, hi, ID_N64, ks > 0 ? 1u : 0u);
                    umma_ta(tmem + COL_O, u, lo, ID_N64, 1u);
                    umma_ta(tmem + COL_O, u + 16, hi, ID_N64, 1u);
                }
                umma_commit(done_o);
                umma_commit(empty + st);
            }
            if (!mbar_wait(done_o, (chunks - 1) & 1, wait_ns)) *dead = 1;   // nor does a product
        }
        __syncwarp();
    } else {
        // ---- rows -------------------------------------------------------------------
        const int q4 = warp & 3, half = warp >> 2, i = 32 * q4 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q4) << 16);
        const int cb = 64 * half, tb = 32 * half;        // its columns of S, its tokens
        auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
            wait(bar, parity);
            __syncwarp();
            tc_fence_after_sync();
        };
        auto arrive = [&](uint64_t* bar) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float x[32];
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (S0) f = *reinterpret_cast<const float4*>(S0 + static_cast<long long>(i) * D + cb + 32 * p + j);
                x[j] = f.x;
                x[j + 1] = f.y;
                x[j + 2] = f.z;
                x[j + 3] = f.w;
            }
            tmem_st32(tl + COL_S + cb + 32 * p, x);
        }
        tmem_wait_st();
        TO* out = static_cast<TO*>(a.out) + tok * D + i;
        float qs[32];                                    // e^g Q S^T of the chunk before
        auto finish = [&](int c) {                       // outputs of chunk c
            wait_warp(done_o, c & 1);
            float o[32];
            tmem_ld32(tl + COL_O + tb, o);
            const int m = len - c * C - tb;
            TO* dst = out + (static_cast<long long>(c) * C + tb) * D;
#pragma unroll
            for (int t = 0; t < 32; ++t)
                if (t < m) dst[static_cast<long long>(t) * D] = from_f32<TO>(o[t] + qs[t]);
        };
        auto read_qs = [&](int c) {                      // (the last use of its stage)
            wait_warp(done_s, c & 1);
            tmem_ld32(tl + COL_QS + tb, qs);
            const float* eg = reinterpret_cast<const float*>(smem + (c & 1) * STAGE_BYTES + ST_PREP + PREP_GATES) + tb;
#pragma unroll
            for (int t = 0; t < 32; ++t) qs[t] *= eg[t];
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + (c & 1));
        };
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1, m = min(C, len - c * C);
            const uint32_t par = c & 1;
            unsigned char* stage = smem + st * STAGE_BYTES;
            const float* eg = reinterpret_cast<const float*>(stage + ST_PREP + PREP_GATES);
            const float *ew = eg + C, *be = ew + C;
            if (c > 0) read_qs(c - 1);
            wait_warp(full + st, (c >> 1) & 1);
            {   // the state's halves, and its decay over the chunk in place
                const float end = eg[3 * C];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    float x[32];
                    tmem_ld32(tl + COL_S + cb + 32 * p, x);
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) halves(x[2 * e], x[2 * e + 1], hi[e], lo[e]);
                    tmem_st16w(tl + COL_SH + (cb + 32 * p) / 2, hi);
                    tmem_st16w(tl + COL_SL + (cb + 32 * p) / 2, lo);
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] *= end;
                    tmem_st32(tl + COL_S + cb + 32 * p, x);
                }
                tmem_wait_st();
            }
            arrive(have_s);
            if (c > 0) finish(c - 1);
            // z = v - e^g S k
            float z[32];
            {
                wait_warp(done_z, par);
                float x[32];
                tmem_ld32(tl + COL_Z + tb, x);
                const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(stage + ST_V) + tb * D + i;
#pragma unroll
                for (int t = 0; t < 32; ++t) {
                    z[t] = fmaf(-eg[tb + t], x[t], to_f32(v[t * D]));
                    if (tb + t >= m) z[t] = 0.f;         // (no token: what lies there is old)
                    x[t] = be[tb + t] * z[t];
                }
                put_halves(tl + COL_W + tb, x);
                tmem_wait_st();
                arrive(have_z);
            }
            {   // r = z + T beta z, u = beta r
                wait_warp(done_r, par);
                float x[32];
                tmem_ld32(tl + COL_Z + tb, x);
#pragma unroll
                for (int t = 0; t < 32; ++t) {
                    z[t] = be[tb + t] * (z[t] + x[t]);
                    x[t] = ew[tb + t] * z[t];
                }
                put_halves(tl + COL_W + tb, x);
                tmem_wait_st();
                arrive(have_w);
                put_halves(tl + COL_Z + tb, z);
                tmem_wait_st();
                arrive(have_u);
            }
        }
        read_qs(chunks - 1);
        finish(chunks - 1);
        if (final_state) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float x[32];
                tmem_ld32(tl + COL_S + cb + 32 * p, x);
                float* dst = final_state + static_cast<long long>(i) * D + cb + 32 * p;
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<float4*>(dst + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
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
