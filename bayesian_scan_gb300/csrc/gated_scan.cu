// gated_scan.cu -- the gated recurrence with one gate per channel,
//     h_t = alpha_t h_{t-1} + w_t x_t,  alpha_t = exp(-A d_t),  w_t = 1 or
//     1 - alpha_t ("Kalman Linear Attention (KLA)", Metodologia 2: the affine
//     recursion of the information mean),
// its backward pass and its one-token step.
//
// Backward, with u_t = alpha_t (g_t + u_{t+1}) the gradient that reaches
// h_{t-1} (g the incoming gradient, u_T+1 the final state's):
//     grad x_t = w_t (g_t + u_{t+1}),   grad d_t = -A u_t (h_{t-1} - leak x_t),
//     grad A = -sum d_t u_t (h_{t-1} - leak x_t),   grad h_0 = u_0:
// the same recurrence in the other direction.
//
// Layout.  Tokens lie C elements apart, so lanes run along the channels (V
// each, 128 bytes a warp) and every warp owns K consecutive tokens of a tile
// of NW * K.  A warp composes its tokens from a zero state (the affine map
// h -> alpha h + s of its span), the warps' maps are folded through shared
// memory, and a second pass over the tokens writes the states.  So every
// element is read once and written once, and HBM bounds the kernel: 6 bytes
// per element forward (bf16), 10 backward.
//
// One CTA walks one sequence of one slab of channels, tile after tile, the
// rows of the next tiles on their way.  Where that makes too few CTAs a
// cluster of S of them takes S consecutive tiles per round: each CTA sends
// its tile's map to all others' shared memory, and every CTA then knows the
// state before its tile and before the next round.  Where even clusters leave
// SMs free (a long sequence of few channels) the tokens are cut into parts;
// a first kernel takes maps of 512 tokens, a second read of two tensors.
// The order of composition is fixed, so results do not depend on the
// schedule.
#include <cfloat>
#include <map>
#include <mutex>
#include <type_traits>
#include <utility>

#include "gated_device.cuh"
#include "kdn_device.cuh"
#include "kdn_internal.h"
#include "kernel_setup.h"
#include "sum_rows.cuh"

namespace kdn {
namespace {

using namespace gated;

// The largest portable cluster.  (Nine CTAs, four such clusters to a GPC's 38
// slots, took as long as eight on 65536 x 2048.)
constexpr int MAX_CLUSTER = 8;
constexpr int NW = 8;             // warps per CTA
constexpr int FWD_K = 16, BWD_K = 8;
constexpr int STAGES = 2;
constexpr int MAP_TOKENS = 512, MAP_WARPS = 16;   // of one map where a sequence is cut into parts

__device__ int g_gated_error = 0;

// How one call is cut: slabs of 32 V channels, clusters of S CTAs, parts of
// `len` tokens (one part: the sequence).
struct Cut {
    int slabs, S, parts, len;
    const float4* maps;    // [state row, T / MAP_TOKENS, C]: {a, e, s, z}
    long long wait_ns;     // limit of one wait inside a cluster
    int stall;             // fault injection: the rank that sends nothing (-1: none)
};

// A warp's place: its channels, its part's tokens [lo, hi) of the T-token row
// `row`, the sequence's first token, and the rounds of its CTA.
template <int V, int K>
struct Place {
    int warp, lane, S, rank, part, c0, c, lo, hi, begin, rounds;
    long long sr, row;     // state row n*H + h, row of the tensors

    __device__ __forceinline__ Place(const GatedArgs& p, const Cut& cut) {
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        S = cut.S;
        rank = static_cast<int>(blockIdx.x % S);
        const long long unit = blockIdx.x / S, u = unit / cut.slabs;
        c0 = static_cast<int>(unit - u * cut.slabs) * 32 * V;
        c = c0 + lane * V;
        sr = u / cut.parts;
        part = static_cast<int>(u - sr * cut.parts);
        row = sr;
        lo = 0;
        hi = p.T;
        if (p.offsets) {
            const long long n = sr / p.H;
            row = sr - n * p.H;
            lo = min(max(p.offsets[n], 0), p.T);
            hi = min(max(p.offsets[n + 1], lo), p.T);
        }
        begin = lo;
        if (cut.parts > 1) {
            lo = static_cast<int>(min(static_cast<long long>(hi), static_cast<long long>(part) * cut.len));
            hi = static_cast<int>(min(static_cast<long long>(hi), static_cast<long long>(lo) + cut.len));
        }
        rounds = (hi - lo + S * NW * K - 1) / (S * NW * K);
    }
};

// An affine map h -> (a + e) h + s of a lane's V channels over a span of
// tokens, z its exponent (a + e = 2^z), as shared-memory words that one
// 16-byte access per channel moves: {a, e, s, z}, or {a0, a1, e0, e1} and
// {s0, s1, z0, z1}.
template <int V>
struct Map {
    float a[V], e[V], s[V], z[V];
};
template <int V>
using MapWords = float4[V][32];

template <int V>
__device__ __forceinline__ Map<V> map_of(const float (&z)[V], const float (&s)[V]) {
    Map<V> m;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Gate g = gate(z[v]);
        m.a[v] = g.a;
        m.e[v] = g.e;
        m.s[v] = s[v];
        m.z[v] = z[v];
    }
    return m;
}

template <int V>
__device__ __forceinline__ void put_map(MapWords<V>& w, int lane, const Map<V>& m) {
    if constexpr (V == 1) {
        w[0][lane] = make_float4(m.a[0], m.e[0], m.s[0], m.z[0]);
    } else {
        w[0][lane] = make_float4(m.a[0], m.a[1], m.e[0], m.e[1]);
        w[1][lane] = make_float4(m.s[0], m.s[1], m.z[0], m.z[1]);
    }
}

template <int V>
__device__ __forceinline__ Map<V> get_map(const MapWords<V>& w, int lane) {
    Map<V> m;
    const float4 q = w[0][lane];
    if constexpr (V == 1) {
        m.a[0] = q.x;
        m.e[0] = q.y;
        m.s[0] = q.z;
        m.z[0] = q.w;
    } else {
        const float4 r = w[1][lane];
        m.a[0] = q.x;
        m.a[1] = q.y;
        m.e[0] = q.z;
        m.e[1] = q.w;
        m.s[0] = r.x;
        m.s[1] = r.y;
        m.z[0] = r.z;
        m.z[1] = r.w;
    }
    return m;
}

template <int V>
__device__ __forceinline__ void apply(const Map<V>& m, float (&h)[V]) {
    if constexpr (V == 1) {
        h[0] = decay_add(m.a[0], m.e[0], h[0], m.s[0]);
    } else {
        const F2 hh{h[0], h[1]};
        const F2 n = fma2(F2{m.a[0], m.a[1]}, hh, fma2(F2{m.e[0], m.e[1]}, hh, F2{m.s[0], m.s[1]}));
        h[0] = n.x;
        h[1] = n.y;
    }
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Folding the maps of a round.  Every warp hands in its map; on return
// `start` is the state before the warp's tokens and `carry` the one after the
// round's last tile, both from the carry before the round.  One warp, another
// each round, does what the CTA has in common (by all warps alike it was a
// fifth of the kernel's instructions: 65536 x 2048 247 us, so 210 us).
//
// In a cluster the tile's map goes to every CTA's shared memory by stores
// that complete on the receiver's mbarrier: no fence waits for the round's
// global stores, as the cluster barrier's release would (an eighth of the
// time).  A CTA sends round r after a barrier that the reader of its round r -
// 2 has passed, and receives all of round r - 1 before it sends round r, so no
// store finds its buffer in use.
template <int V>
struct Fold {
    MapWords<V> warp[2][NW];           // a round's maps; alone [0], and in [1] the warps' starts
    uint64_t full[2];
    // a CTA alone has no memory from here on
    MapWords<V> cta[2][MAX_CLUSTER];
    float start[V][32], carry[V][32];
    int late;                          // a wait ran out: no more sends and waits

    __device__ __forceinline__ float* starts(int w) { return reinterpret_cast<float*>(warp[1]) + w * V * 32; }

    // Every CTA of the cluster runs, its barriers set up, before one sends.
    __device__ __forceinline__ void begin(int S) {
        if (S > 1) {
            if (threadIdx.x == 0) {
                mbar_init(&full[0], 1);
                mbar_init(&full[1], 1);
                mbar_init_fence();
                late = 0;
            }
            cluster_sync();
        }
    }
    // No CTA leaves while another may still send to it.
    __device__ __forceinline__ void end(int S) {
        if (S > 1) {
            cluster_sync();
            if (late) {   // what was sent and not waited for arrives in the meantime
                const unsigned long long t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 100000) __nanosleep(1000);
            }
        }
    }
};

__device__ __forceinline__ bool full_try(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded: after limit_ns it records an error and returns false.  (The timer
// is read once per 64 tries: a read costs more than a try.)
__device__ __forceinline__ bool full_wait(uint64_t* bar, uint32_t parity, long long limit_ns) {
    unsigned long long t0 = 0;
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (full_try(bar, parity)) return true;
        const unsigned long long t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (static_cast<long long>(t - t0) > limit_ns) {
            record_error(&g_gated_error, KDN_ERR_TIMEOUT);
            return false;
        }
    }
}

__device__ __forceinline__ void send(uint32_t dst, float4 v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ uint32_t at_rank(const void* p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ float from_rank(const float* p, int rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at_rank(p, rank)) : "memory");
    return v;
}

template <int V>
__device__ __forceinline__ void fold_round(Fold<V>& f, const Cut& cut, int r, int rank, int warp, int lane,
                                           const float (&z)[V], const float (&s)[V], float (&carry)[V],
                                           float (&start)[V]) {
    const int S = cut.S;
    if (S == 1) {
        // the folding warp works out every warp's start; the next round's first barrier comes after
        // all have read theirs
        put_map<V>(f.warp[0][warp], lane, map_of<V>(z, s));
        __syncthreads();
        if (warp == r % NW) {
            float h[V];
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = carry[v];
#pragma unroll
            for (int w = 0; w < NW; ++w) {
#pragma unroll
                for (int v = 0; v < V; ++v) f.starts(w)[v * 32 + lane] = h[v];
                apply<V>(get_map<V>(f.warp[0][w], lane), h);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) f.starts(NW)[v * 32 + lane] = h[v];
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            start[v] = f.starts(warp)[v * 32 + lane];
            carry[v] = f.starts(NW)[v * 32 + lane];
        }
        return;
    }
    const int buf = r & 1;
    put_map<V>(f.warp[buf][warp], lane, map_of<V>(z, s));
    __syncthreads();
    if (warp == r % NW) {
        // it composes the tile's map, sends it to every CTA and takes the round's maps in
        const bool late = f.late;
        if (lane == 0 && !late) mbar_arrive_expect_tx(&f.full[buf], S * sizeof(MapWords<V>));
        float h[V], zz[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = zz[v] = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const Map<V> m = get_map<V>(f.warp[buf][w], lane);
            apply<V>(m, h);
#pragma unroll
            for (int v = 0; v < V; ++v) zz[v] += m.z[v];
        }
        const Map<V> m = map_of<V>(zz, h);
        for (int j = 0; j < S && !late && rank != cut.stall; ++j) {
            const uint32_t to = at_rank(&f.cta[buf][rank][0][lane], j), bar = at_rank(&f.full[buf], j);
            if constexpr (V == 1) {
                send(to, make_float4(m.a[0], m.e[0], m.s[0], m.z[0]), bar);
            } else {
                send(to, make_float4(m.a[0], m.a[1], m.e[0], m.e[1]), bar);
                send(to + 512, make_float4(m.s[0], m.s[1], m.z[0], m.z[1]), bar);
            }
        }
        if (!late && !full_wait(&f.full[buf], (r >> 1) & 1, cut.wait_ns)) f.late = 1;
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = carry[v];
        for (int j = 0; j < S; ++j) {
            if (j == rank)
#pragma unroll
                for (int v = 0; v < V; ++v) f.start[v][lane] = h[v];
            apply<V>(get_map<V>(f.cta[buf][j], lane), h);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) f.carry[v][lane] = h[v];
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        start[v] = f.start[v][lane];
        carry[v] = f.carry[v][lane];
    }
    for (int w = 0; w < warp; ++w) apply<V>(get_map<V>(f.warp[buf][w], lane), start);
}

// The state that a part starts from: the sequence's carry through the maps of
// the tokens before the part (those after it, backward).  Each warp composes
// a share of the maps; all fold the shares.
template <int V, bool BWD>
__device__ __forceinline__ void through_parts(const GatedArgs& p, const Cut& cut, Fold<V>& f, long long sr, int part,
                                              int warp, int lane, int c, float (&carry)[V]) {
    if (cut.parts == 1) return;
    const int all = (p.T + MAP_TOKENS - 1) / MAP_TOKENS, edge = (part + (BWD ? 1 : 0)) * (cut.len / MAP_TOKENS);
    const int n = BWD ? max(all - edge, 0) : edge, share = (n + NW - 1) / NW;
    float z[V], s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        z[v] = s[v] = 0.f;
        if (c + v >= p.C) continue;
        const float4* m = cut.maps + sr * all * p.C + c + v;
#pragma unroll 8
        for (int i = warp * share; i < min(n, (warp + 1) * share); ++i) {
            const float4 q = m[static_cast<long long>(BWD ? all - 1 - i : i) * p.C];
            s[v] = decay_add(q.x, q.y, s[v], q.z);
            z[v] += q.w;
        }
    }
    put_map<V>(f.warp[0][warp], lane, map_of<V>(z, s));
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) apply<V>(get_map<V>(f.warp[0][w], lane), carry);
    __syncthreads();
}

// A warp's rows come through shared memory, STAGES rounds ahead: by
// asynchronous copies of SIZE = 16 or 4 bytes, whichever the tensors' rows
// allow, or, for rows of an odd number of bf16, by element (SIZE = 2, not
// asynchronous); what lies outside the sequence or the channels becomes
// zeros (d = x = 0: alpha = 1, nothing added).  With SIZE = 16 results leave
// through shared memory too, in 16-byte pieces, else straight from the
// registers.  A warp reads only rows that it copied itself, so no barrier
// beyond the fold's is needed.
//
// 16-byte pieces matter: single loads and stores of a lane's channels, with
// their addresses and predicates, were half of all instructions (8 x 4096 x
// 2048 bf16: 212 us, against 117 us in pieces).
template <typename TI, typename TO, int V, int K>
struct FwdShared {
    static constexpr int ROW = 32 * V * static_cast<int>(sizeof(TI)), OROW = 32 * V * static_cast<int>(sizeof(TO));
    struct __align__(16) Stage {
        char x[K * ROW], d[K * ROW];                 // out overwrites both
    };
    Stage st[STAGES][NW];
    Fold<V> fold;
};

// Measured (GB300; 16-bit in and out, 134 M elements, 805 MB, where 118 us is
// the copy's rate): as 16 x 4096 x 2048 142 us, 4 x 16384 x 2048 (clusters of
// 2) 167 us, 1 x 65536 x 2048 (clusters of 8) 190 us, 213 us of the convex
// form; 2 CTAs per SM (128 registers), 18.7 instructions per element, 24.5
// with clusters of 8.
template <typename TI, typename TO, int V, int K, bool LEAK, int SIZE>
__global__ void __launch_bounds__(NW * 32, 2)
gated_fwd_kernel(const __grid_constant__ GatedArgs p, const __grid_constant__ Cut cut) {
    using Sh = FwdShared<TI, TO, V, K>;
    static_assert(Sh::OROW * K <= static_cast<int>(sizeof(typename Sh::Stage)), "out takes the stage's place");
    extern __shared__ __align__(16) char smem[];
    Sh& sh = *reinterpret_cast<Sh*>(smem);
    const Place<V, K> at(p, cut);
    const int lane = at.lane, c = at.c;
    const long long arow = (at.sr % p.H) * p.C;

    float rate[V], carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        rate[v] = c + v < p.C ? -LOG2E * p.A[arow + c + v] : 0.f;
        carry[v] = c + v < p.C && p.h0 ? p.h0[at.sr * p.C + c + v] : 0.f;
    }
    const int t0 = at.lo + (at.rank * NW + at.warp) * K, step = at.S * NW * K;
    const long long xld = p.x_ld * sizeof(TI), dld = p.d_ld * sizeof(TI);
    const char* xp = static_cast<const char*>(p.x) + (at.row * p.T + t0) * xld + at.c0 * sizeof(TI);
    const char* dp = static_cast<const char*>(p.d) + (at.row * p.T + t0) * dld + at.c0 * sizeof(TI);
    TO* op = static_cast<TO*>(p.out) + (at.row * p.T + t0) * p.C + at.c0;
    const int width = (p.C - at.c0) * static_cast<int>(sizeof(TI)), owidth = (p.C - at.c0) * static_cast<int>(sizeof(TO));

    auto fetch = [&](int r) {
        const int n = at.hi - t0 - r * step;               // tokens left
        if (n > 0) {
            typename Sh::Stage& st = sh.st[r % STAGES][at.warp];
            rows_in<SIZE, Sh::ROW, K>(st.x, p.x, xp + static_cast<long long>(r) * step * xld, xld, 0, n, width, lane);
            rows_in<SIZE, Sh::ROW, K>(st.d, p.d, dp + static_cast<long long>(r) * step * dld, dld, 0, n, width, lane);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
        if (i < at.rounds) fetch(i);
        else copy_commit();
    through_parts<V, false>(p, cut, sh.fold, at.sr, at.part, at.warp, lane, c, carry);
    sh.fold.begin(at.S);
    for (int r = 0; r < at.rounds; ++r) {
        const int n = at.hi - t0 - r * step;
        char* xs = sh.st[r % STAGES][at.warp].x;
        const char* ds = sh.st[r % STAGES][at.warp].d;
        copy_wait<STAGES - 1>();
        __syncwarp();
        float a[K][V], b[K][V], z[V], s[V], h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = s[v] = 0.f;
        if (n > 0) {                                        // (the warp as one)
#pragma unroll
            for (int i = 0; i < K * V / 2; ++i) {
                // two channels of a token, or (V = 1) two tokens of a channel
                const int k0 = 2 * i / V, v0 = 2 * i % V, k1 = (2 * i + 1) / V, v1 = (2 * i + 1) % V;
                const Vec<TI, V> d0 = peek<TI, V>(ds + k0 * Sh::ROW + lane * V * sizeof(TI)),
                                 x0 = peek<TI, V>(xs + k0 * Sh::ROW + lane * V * sizeof(TI));
                Vec<TI, V> d1 = d0, x1 = x0;
                if (V == 1) {
                    d1 = peek<TI, V>(ds + k1 * Sh::ROW + lane * V * sizeof(TI));
                    x1 = peek<TI, V>(xs + k1 * Sh::ROW + lane * V * sizeof(TI));
                }
                const F2 zz = mul2(F2{rate[v0], rate[v1]}, F2{d0.get(v0), d1.get(v1)});
                const Gate2 gg = gate2<LEAK, sizeof(TO) == 4>(zz);
                F2 x{x0.get(v0), x1.get(v1)};
                if (LEAK) x = mul2(x, gg.w);
                a[k0][v0] = gg.a.x;
                a[k1][v1] = gg.a.y;
                b[k0][v0] = x.x;
                b[k1][v1] = x.y;
                if constexpr (V == 1) {
                    z[0] += zz.x + zz.y;
                    s[0] = fmaf(gg.a.y, fmaf(gg.a.x, s[0], x.x), x.y);
                } else {
                    const F2 m = fma2(gg.a, F2{s[0], s[1]}, x), zs = add2(F2{z[0], z[1]}, zz);
                    s[0] = m.x;
                    s[1] = m.y;
                    z[0] = zs.x;
                    z[1] = zs.y;
                }
            }
        }
        fold_round<V>(sh.fold, cut, r, at.rank, at.warp, lane, z, s, carry, h);
        if (n > 0) {
            TO* o = op + static_cast<long long>(r) * step * p.C;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if constexpr (V == 1) {
                    h[0] = fmaf(a[k][0], h[0], b[k][0]);
                } else {
                    const F2 m = fma2(F2{a[k][0], a[k][1]}, F2{h[0], h[1]}, F2{b[k][0], b[k][1]});
                    h[0] = m.x;
                    h[1] = m.y;
                }
                if (SIZE == 16) {
                    Vec<TO, V> q;
                    q.set(h);
                    poke<TO, V>(xs + k * Sh::OROW + lane * V * sizeof(TO), q);
                } else if (k < n) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (c + v < p.C) __stcs(o + static_cast<long long>(k) * p.C + lane * V + v, from_f32<TO>(h[v]));
                }
            }
            __syncwarp();
            if (SIZE == 16) {
                rows_out<Sh::OROW, K>(reinterpret_cast<char*>(o), p.C * static_cast<long long>(sizeof(TO)), xs, 0, n,
                                      owidth, lane);
                __syncwarp();
            }
        }
        if (r + STAGES < at.rounds) fetch(r + STAGES);
        else copy_commit();
    }
    sh.fold.end(at.S);
    if (p.final_state && at.rank == 0 && at.warp == 0 && at.part == cut.parts - 1)
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c + v < p.C) p.final_state[at.sr * p.C + c + v] = carry[v];
}

// grad d overwrites d; grad x overwrites x, or, where K is twice BWD_K and
// there is no room for x, g.
template <typename TI, typename TO, int V, int K, bool LEAK>
struct BwdShared {
    static constexpr int ROW = 32 * V * static_cast<int>(sizeof(TI)), OROW = 32 * V * static_cast<int>(sizeof(TO));
    static constexpr bool X = K == BWD_K;
    static_assert(X || (!LEAK && sizeof(TI) == sizeof(TO)), "g takes grad x");
    struct __align__(16) Stage {
        char d[K * ROW], x[X ? K * ROW : 16], g[K * OROW], h[K * OROW];
        __device__ __forceinline__ char* grad_x() { return X ? x : g; }
    };
    Stage st[STAGES][NW];
    float dA[V][32];
    Fold<V> fold;
};

// The same walk from the last token to the first.  `sums` [sequence, part, H,
// C] takes the shares of grad A (the sums themselves where there is one).
template <typename TI, typename TO, int V, int K, bool LEAK, int SIZE>
__global__ void __launch_bounds__(NW * 32, 2)
gated_bwd_kernel(const __grid_constant__ GatedArgs p, const __grid_constant__ Cut cut, float* sums) {
    using Sh = BwdShared<TI, TO, V, K, LEAK>;
    extern __shared__ __align__(16) char smem[];
    Sh& sh = *reinterpret_cast<Sh*>(smem);
    const Place<V, K> at(p, cut);
    const int lane = at.lane, c = at.c;
    const long long arow = (at.sr % p.H) * p.C;

    float nA[V], rate[V], carry[V], dA[V], first[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const bool on = c + v < p.C;
        nA[v] = on ? -p.A[arow + c + v] : 0.f;
        rate[v] = LOG2E * nA[v];
        carry[v] = on && p.grad_final_state ? p.grad_final_state[at.sr * p.C + c + v] : 0.f;
        first[v] = on && p.h0 ? p.h0[at.sr * p.C + c + v] : 0.f;
        dA[v] = 0.f;
    }
    // a warp's rows of round r are tokens base - r step .. + K - 1, walked from the last
    const int base = at.hi - (at.rank * NW + at.warp + 1) * K, step = at.S * NW * K;
    const long long dld = p.d_ld * sizeof(TI), xld = p.x_ld * sizeof(TI), tld = p.C * static_cast<long long>(sizeof(TO));
    const long long row = at.row * p.T;
    const int width = (p.C - at.c0) * static_cast<int>(sizeof(TI)), owidth = (p.C - at.c0) * static_cast<int>(sizeof(TO));

    auto fetch = [&](int r) {
        const int t = base - r * step;
        if (t + K > at.lo) {
            typename Sh::Stage& st = sh.st[r % STAGES][at.warp];
            const int f = max(at.lo - t, 0);               // rows before the part
            rows_in<SIZE, Sh::ROW, K>(st.d, p.d, static_cast<const char*>(p.d) + (row + t) * dld + at.c0 * sizeof(TI), dld,
                                      f, K, width, lane);
            if (LEAK)
                rows_in<SIZE, Sh::ROW, K>(st.x, p.x, static_cast<const char*>(p.x) + (row + t) * xld + at.c0 * sizeof(TI),
                                          xld, f, K, width, lane);
            rows_in<SIZE, Sh::OROW, K>(st.g, p.grad_out,
                                       static_cast<const char*>(p.grad_out) + (row + t) * tld + at.c0 * sizeof(TO), tld, f,
                                       K, owidth, lane);
            // the states before: one token earlier (h0 for the sequence's first one, below)
            rows_in<SIZE, Sh::OROW, K>(st.h, p.out,
                                       static_cast<const char*>(p.out) + (row + t - 1) * tld + at.c0 * sizeof(TO), tld,
                                       f + (t + f == at.begin), K, owidth, lane);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
        if (i < at.rounds) fetch(i);
        else copy_commit();
    through_parts<V, true>(p, cut, sh.fold, at.sr, at.part, at.warp, lane, c, carry);
    sh.fold.begin(at.S);
    for (int r = 0; r < at.rounds; ++r) {
        const int t = base - r * step;
        const bool any = t + K > at.lo;                     // (the warp as one)
        typename Sh::Stage& st = sh.st[r % STAGES][at.warp];
        copy_wait<STAGES - 1>();
        __syncwarp();
        float a[K][V], w[LEAK ? K : 1][V], z[V], s[V], u[V];
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = s[v] = 0.f;
        if (any) {
            // u = alpha (g + u): the map of a token is (alpha, alpha g); index k counts back from the last
#pragma unroll
            for (int i = 0; i < K * V / 2; ++i) {
                const int k0 = 2 * i / V, v0 = 2 * i % V, k1 = (2 * i + 1) / V, v1 = (2 * i + 1) % V;
                const int j0 = K - 1 - k0, j1 = K - 1 - k1;
                const Vec<TI, V> d0 = peek<TI, V>(st.d + j0 * Sh::ROW + lane * V * sizeof(TI));
                const Vec<TO, V> g0 = peek<TO, V>(st.g + j0 * Sh::OROW + lane * V * sizeof(TO));
                Vec<TI, V> d1 = d0;
                Vec<TO, V> g1 = g0;
                if (V == 1) {
                    d1 = peek<TI, V>(st.d + j1 * Sh::ROW + lane * V * sizeof(TI));
                    g1 = peek<TO, V>(st.g + j1 * Sh::OROW + lane * V * sizeof(TO));
                }
                const F2 zz = mul2(F2{rate[v0], rate[v1]}, F2{d0.get(v0), d1.get(v1)});
                const Gate2 gg = gate2<LEAK, sizeof(TI) == 4>(zz);
                a[k0][v0] = gg.a.x;
                a[k1][v1] = gg.a.y;
                if (LEAK) {
                    w[LEAK ? k0 : 0][v0] = gg.w.x;
                    w[LEAK ? k1 : 0][v1] = gg.w.y;
                }
                if constexpr (V == 1) {
                    z[0] += zz.x + zz.y;
                    s[0] = gg.a.y * (gg.a.x * (s[0] + g0.get(0)) + g1.get(0));
                } else {
                    const F2 m = mul2(gg.a, add2(F2{s[0], s[1]}, F2{g0.get(0), g0.get(1)}));
                    const F2 zs = add2(F2{z[0], z[1]}, zz);
                    s[0] = m.x;
                    s[1] = m.y;
                    z[0] = zs.x;
                    z[1] = zs.y;
                }
            }
        }
        fold_round<V>(sh.fold, cut, r, at.rank, at.warp, lane, z, s, carry, u);
        if (any) {
            TI* gx_out = static_cast<TI*>(p.grad_x) + (row + t) * p.C + at.c0;
            TI* gd_out = static_cast<TI*>(p.grad_d) + (row + t) * p.C + at.c0;
            // (a tile with tokens before the part: d = 0 there, but their m may be NaN.  Code of its own:
            // a predicate in every tile costs the convex layer 153 -> 156 us)
            auto walk = [&](auto edge) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int j = K - 1 - k;
                    const Vec<TI, V> dv = peek<TI, V>(st.d + j * Sh::ROW + lane * V * sizeof(TI));
                    const Vec<TO, V> gv = peek<TO, V>(st.g + j * Sh::OROW + lane * V * sizeof(TO));
                    const Vec<TO, V> hv = peek<TO, V>(st.h + j * Sh::OROW + lane * V * sizeof(TO));
                    Vec<TI, V> xv = dv;
                    if (LEAK) xv = peek<TI, V>(st.x + j * Sh::ROW + lane * V * sizeof(TI));
                    float gx[V], gd[V], prev[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) prev[v] = t + j == at.begin ? first[v] : hv.get(v);
                    if constexpr (V == 1) {
                        const float dh = u[0] + gv.get(0);
                        u[0] = a[k][0] * dh;
                        gx[0] = dh;
                        if (LEAK) {
                            prev[0] -= xv.get(0);
                            gx[0] = w[LEAK ? k : 0][0] * dh;
                        }
                        const float m = u[0] * prev[0];
                        gd[0] = nA[0] * m;
                        if (!decltype(edge)::value || t + j >= at.lo) dA[0] = fmaf(dv.get(0), m, dA[0]);
                    } else {
                        const F2 dh = add2(F2{u[0], u[1]}, F2{gv.get(0), gv.get(1)});
                        const F2 n = mul2(F2{a[k][0], a[k][1]}, dh);
                        F2 x = dh, before{prev[0], prev[1]};
                        if (LEAK) {
                            before = add2(before, F2{-xv.get(0), -xv.get(1)});
                            x = mul2(F2{w[LEAK ? k : 0][0], w[LEAK ? k : 0][1]}, dh);
                        }
                        const F2 m = mul2(n, before), d = mul2(F2{nA[0], nA[1]}, m);
                        const F2 sum = fma2(F2{dv.get(0), dv.get(1)}, m, F2{dA[0], dA[1]});
                        u[0] = n.x;
                        u[1] = n.y;
                        gx[0] = x.x;
                        gx[1] = x.y;
                        gd[0] = d.x;
                        gd[1] = d.y;
                        if (!decltype(edge)::value || t + j >= at.lo) {
                            dA[0] = sum.x;
                            dA[1] = sum.y;
                        }
                    }
                    if (SIZE == 16) {
                        Vec<TI, V> q;
                        q.set(gx);
                        poke<TI, V>(st.grad_x() + j * Sh::ROW + lane * V * sizeof(TI), q);
                        q.set(gd);
                        poke<TI, V>(st.d + j * Sh::ROW + lane * V * sizeof(TI), q);
                    } else if (t + j >= at.lo) {
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            if (c + v < p.C) {
                                __stcs(gx_out + static_cast<long long>(j) * p.C + lane * V + v, from_f32<TI>(gx[v]));
                                __stcs(gd_out + static_cast<long long>(j) * p.C + lane * V + v, from_f32<TI>(gd[v]));
                            }
                    }
                }
            };
            if (t >= at.lo) walk(std::false_type());
            else walk(std::true_type());
            __syncwarp();
            if (SIZE == 16) {
                const int f = max(at.lo - t, 0);
                const long long ld = p.C * static_cast<long long>(sizeof(TI));
                rows_out<Sh::ROW, K>(reinterpret_cast<char*>(gx_out), ld, st.grad_x(), f, K, width, lane);
                rows_out<Sh::ROW, K>(reinterpret_cast<char*>(gd_out), ld, st.d, f, K, width, lane);
                __syncwarp();
            }
        }
        if (r + STAGES < at.rounds) fetch(r + STAGES);
        else copy_commit();
    }
    if (sums) {
        // the warps' shares, in order, then the cluster's
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) sh.fold.warp[0][at.warp][v][lane].x = dA[v];
        __syncthreads();
        if (at.warp == 0)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float sum = 0.f;
                for (int i = 0; i < NW; ++i) sum += sh.fold.warp[0][i][v][lane].x;
                sh.dA[v][lane] = sum;
            }
        if (at.S == 1) __syncwarp();
    }
    sh.fold.end(at.S);
    if (at.rank == 0 && at.warp == 0)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (p.grad_h0 && at.part == 0 && c + v < p.C) p.grad_h0[at.sr * p.C + c + v] = carry[v];
            if (sums) {
                float sum = 0.f;
                for (int j = 0; j < at.S; ++j)
                    sum += at.S == 1 ? sh.dA[v][lane] : from_rank(&sh.dA[v][lane], j);
                const long long n = at.sr / p.H, hd = at.sr % p.H;
                if (c + v < p.C) sums[((n * cut.parts + at.part) * p.H + hd) * p.C + c + v] = -sum;
            }
        }
    if (sums && at.S > 1) cluster_sync();   // rank 0 has read the others' sums
}

// The maps of every MAP_TOKENS tokens of long sequences of few channels: {a,
// e, s, z}, [state row, T / MAP_TOKENS, C].  A warp composes a
// sixteenth of them, a channel per lane, UN tokens' loads in flight.
template <typename TI, typename TO, bool LEAK, bool BWD>
__global__ void __launch_bounds__(MAP_WARPS * 32) gated_maps_kernel(const __grid_constant__ GatedArgs p, float4* maps) {
    constexpr int UN = 16, sub = MAP_TOKENS / MAP_WARPS;
    __shared__ float4 share[MAP_WARPS][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slabs = (p.C + 31) / 32, c = static_cast<int>(blockIdx.x % slabs) * 32 + lane;
    const int all = (p.T + MAP_TOKENS - 1) / MAP_TOKENS;
    const long long u = blockIdx.x / slabs, sr = u / all;
    const int chunk = static_cast<int>(u - sr * all);
    const bool on = c < p.C;
    const long long from = min(static_cast<long long>(p.T), static_cast<long long>(chunk) * MAP_TOKENS + warp * sub);
    const long long to = min(static_cast<long long>(p.T), from + sub);
    const float rate = on ? -LOG2E * p.A[(sr % p.H) * p.C + c] : 0.f;
    const TI* d = static_cast<const TI*>(p.d) + sr * p.T * p.d_ld + c;
    const TI* x = static_cast<const TI*>(p.x) + sr * p.T * p.x_ld + c;
    const TO* g = static_cast<const TO*>(p.grad_out) + sr * p.T * p.C + c;
    float z = 0.f, s = 0.f, sz = 0.f;
    for (long long t = from; t < to; t += UN) {
        float dv[UN], xv[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const long long k = BWD ? to - 1 - (t - from) - i : t + i;
            const bool ok = on && k >= from && k < to;
            dv[i] = ok ? to_f32(d[k * p.d_ld]) : 0.f;
            xv[i] = !ok ? 0.f : BWD ? to_f32(g[k * p.C]) : to_f32(x[k * p.x_ld]);
        }
        // spans of UN tokens are composed by their exponents' sum, as a warp's are in the walk
        float zz = 0.f, ss = 0.f;
#pragma unroll
        for (int i = 0; i < UN; i += 2) {
            const F2 e = mul2(both(rate), F2{dv[i], dv[i + 1]});
            const Gate2 q = gate2<LEAK && !BWD, sizeof(TO) == 4>(e);
            zz += e.x + e.y;
            if (BWD) ss = q.a.y * (q.a.x * (ss + xv[i]) + xv[i + 1]);
            else if (LEAK) ss = fmaf(q.a.y, fmaf(q.a.x, ss, q.w.x * xv[i]), q.w.y * xv[i + 1]);
            else ss = fmaf(q.a.y, fmaf(q.a.x, ss, xv[i]), xv[i + 1]);
        }
        const Gate q = gate(zz);
        s = decay_add(q, s, ss);
        z += zz;
        sz = z;
    }
    share[warp][lane] = make_float4(0.f, 0.f, s, sz);
    __syncthreads();
    if (warp > 0 || !on) return;
    z = s = 0.f;
    for (int i = 0; i < MAP_WARPS; ++i) {
        const float4 m = share[BWD ? MAP_WARPS - 1 - i : i][lane];
        const Gate q = gate(m.w);
        s = decay_add(q, s, m.z);
        z += m.w;
    }
    const Gate q = gate(z);
    maps[(sr * all + chunk) * p.C + c] = make_float4(q.a, q.e, s, z);
}

// A step moves 4 (state) + 4 + 2 + 2 + 2 bytes per element (bf16) once, so a
// large batch is bound by HBM and a small one by its launch; N elements per
// thread where rows and addresses allow.
template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(NW * 32)
gated_step_kernel(const TI* __restrict__ x, const TI* __restrict__ d, const float* __restrict__ A, bool leak,
                  const float* state, float* new_state, TO* __restrict__ out, long long n, long long HC) {
    const long long i = (static_cast<long long>(blockIdx.x) * (NW * 32) + threadIdx.x) * N;
    if (i >= n) return;
    const long long j = i % HC;
    float xv[N], dv[N], s[N], Av[N], h[N];
    load_n<N>(x + i, xv);
    load_n<N>(d + i, dv);
    load_n<N>(A + j, Av);
    load_n<N>(state + i, s);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const Gate g = gate(-LOG2E * (Av[k] * dv[k]));
        h[k] = decay_add(g, s[k], leak ? g.w * xv[k] : xv[k]);
    }
    store_n<N>(new_state + i, h);
    store_n<N>(out + i, h);
}

template <typename F>
kdn_status by_type(kdn_dtype in, kdn_dtype out, F f) {
    if (in == KDN_BF16)
        return out == KDN_BF16 ? f(__nv_bfloat16(), __nv_bfloat16()) : f(__nv_bfloat16(), float());
    return out == KDN_BF16 ? f(float(), __nv_bfloat16()) : f(float(), float());
}

long long state_rows(const GatedArgs& a) { return static_cast<long long>(a.nseq > 0 ? a.nseq : a.B) * a.H; }

// Whether every row of every tensor starts on a multiple of `bytes` and is a
// multiple of it long.
bool rows_ok(const GatedArgs& a, long long bytes) {
    const long long is = a.in_dtype == KDN_BF16 ? 2 : 4, os = a.out_dtype == KDN_BF16 ? 2 : 4;
    const void* ptrs[] = {a.x, a.d, a.grad_x, a.grad_d, a.out, a.grad_out};
    for (const void* q : ptrs)
        if (reinterpret_cast<uintptr_t>(q) % bytes) return false;
    return a.C * is % bytes == 0 && a.C * os % bytes == 0 && a.d_ld * is % bytes == 0 &&
           (!a.x || a.x_ld * is % bytes == 0);
}

// What the current device holds of a kernel at once: clusters of 1 .. MAX_CLUSTER
// CTAs (0: none).  Asked once per device and kernel, when the kernel's shared
// memory is set up too.
struct Resident {
    int clusters[MAX_CLUSTER];
};

cudaError_t resident(const void* kernel, size_t alone, size_t smem, Resident* out) try {
    static std::mutex lock;
    static std::map<std::pair<int, const void*>, Resident> known;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const std::lock_guard<std::mutex> hold(lock);
    auto it = known.find({dev, kernel});
    if (it == known.end()) {
        Resident r{};
        e = allow_smem(kernel, smem);
        if (e != cudaSuccess) return e;
        int n = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, NW * 32, alone);
        if (e != cudaSuccess) return e;
        r.clusters[0] = n * sm_count();
        for (int S = 2; S <= MAX_CLUSTER; ++S) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(S);
            cfg.blockDim = dim3(NW * 32);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute at{};
            at.id = cudaLaunchAttributeClusterDimension;
            at.val.clusterDim.x = S;
            at.val.clusterDim.y = at.val.clusterDim.z = 1;
            cfg.attrs = &at;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&r.clusters[S - 1], kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                r.clusters[S - 1] = 0;
            }
        }
        it = known.emplace(std::make_pair(dev, kernel), r).first;
    }
    *out = it->second;
    return cudaSuccess;
} catch (...) {   // no exception leaves a C entry point
    return cudaErrorMemoryAllocation;
}

int maps_of(int T) { return (T + MAP_TOKENS - 1) / MAP_TOKENS; }

// A bound of the parts that plan() takes, whatever the types and kernels: one
// map each at least, and no more than fill the device.
long long most_parts(long long rows, int C, int T) {
    const long long n = 2LL * sm_count() / (rows * ((C + 63) / 64));
    return n < 1 ? 1 : n < maps_of(T) ? n : maps_of(T) > 0 ? maps_of(T) : 1;
}

// Cluster size and parts, by a model in rounds of a full device (two CTAs per
// SM, 2.5 us): waves x (rounds x cost + START).
//
// A wave is what the device holds at once: its CTA slots, or fewer for
// clusters, which a GPC holds whole.  A cluster's round costs more than a
// CTA's alone (the exchange), by what was measured on 134 M elements: 8 %
// with two CTAs, 14 % with four, 25 % with eight; an SM with one CTA does a
// round in about two thirds of the time that it takes for two; starting a CTA
// costs about 1.5 rounds.  So 8 x 4096 x 2048 runs without clusters (with an
// earlier fold 80 us, 91 with two CTAs each), 65536 x 2048 with eight.
//
// Parts add a pass over two tensors (the walk's own time again: its loads are
// single elements) and a launch (`fixed` rounds; three and a half, nine with scratch of its own), and make
// units enough that no or small clusters do: 65536 x 64 144 -> 41 us, backward
// 265 -> 54 us.
//
// Packed sequences have one length on average and may have others; a long
// average gets a cluster whatever the grid, for the longest walks that are
// left alone at the end: of two CTAs where the grid fills the device three
// times, of four where it fills it, of eight else.  65536 bf16 tokens, us:
//   32 sequences of 4096 channels, random lengths / one of half the tokens:
//     two 324 / 323 (backward 546 / 544), four 397 / 404 (664 / 669);
//   16 of 2048: two 215 / 256, four 176 / 180 (300 / 304), eight 228 / 234
//     (382 / 388);
//   8 of 1024: four 140 / 138 (250 / 247), eight 123 / 104 (213 / 184).
kdn_status plan(const GatedArgs& a, const void* kernel, size_t alone, size_t smem, int V, int K, double fixed, Cut* cut) {
    Resident held;
    const cudaError_t e = resident(kernel, alone, smem, &held);
    if (e != cudaSuccess) return from_cuda(e);
    cut->slabs = (a.C + 32 * V - 1) / (32 * V);
    cut->S = cut->parts = 1;
    cut->len = a.T;
    const int tile = NW * K;
    const long long rows = state_rows(a), units = rows * cut->slabs;
    const long long len = a.nseq > 0 ? (a.T + a.nseq - 1) / a.nseq : a.T;
    static const double cost[MAX_CLUSTER] = {1, 1.08, 1.11, 1.14, 1.17, 1.20, 1.23, 1.25};
    constexpr double START = 1.5, SECOND_READ = 1.0;
    double best = DBL_MAX;
    auto consider = [&](long long parts, long long tokens, double more) {
        const long long tiles = (tokens + tile - 1) / tile, n = units * parts;
        for (int S = 1; S <= MAX_CLUSTER && (S == 1 || S <= tiles); ++S) {
            const int h = held.clusters[S - 1];
            if (h < 1) continue;
            double t = static_cast<double>((n + h - 1) / h) *
                       (static_cast<double>((tiles + S - 1) / S) * cost[S - 1] + START);
            if (n * S <= sm_count()) t *= 0.65;
            if (t + more < best * 0.98) {
                best = t + more;
                cut->S = S;
                cut->parts = static_cast<int>(parts);
                cut->len = static_cast<int>(tokens);
            }
        }
    };
    consider(1, len, 0.0);
    if (a.nseq > 0) {
        const long long most = units > 3LL * held.clusters[0] ? 2 : units > held.clusters[0] ? 4 : MAX_CLUSTER;
        const long long s = len / tile / 4 < most ? len / tile / 4 : most;
        if (cut->S < s && held.clusters[s - 1] > 0) cut->S = static_cast<int>(s);
        return KDN_OK;
    }
    const long long bound = most_parts(rows, a.C, a.T), maps = maps_of(a.T);
    long long n = held.clusters[0] / units;
    if (n > bound) n = bound;
    if (n > 1) {
        const long long each = (maps + n - 1) / n;                    // maps of a part
        const long long tokens = each * MAP_TOKENS;
        const double again = SECOND_READ * static_cast<double>(units * ((a.T + tile - 1) / tile)) / held.clusters[0];
        consider((maps + each - 1) / each, tokens, again + fixed);
    }
    if (cut->parts == 1) cut->len = a.T;
    return KDN_OK;
}

// A kernel's shared memory, and without what only clusters use.
template <typename Sh>
struct Sizes {
    static constexpr size_t alone = sizeof(Sh) - sizeof(Sh::fold.cta) - sizeof(Sh::fold.start) - sizeof(Sh::fold.carry) - sizeof(Sh::fold.late);
    static constexpr size_t smem() { return sizeof(Sh); }
    static size_t of(const Cut& cut) { return cut.S > 1 ? smem() : alone; }
};

template <typename... KArgs, typename... Args>
kdn_status launch_walk(void (*kernel)(KArgs...), long long rows, const Cut& cut, size_t smem, cudaStream_t stream, Args... args) {
    const long long blocks = rows * cut.parts * cut.slabs * cut.S;
    if (blocks > 0x7fffffffLL) return KDN_ERR_INVALID_ARG;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cut.S;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = cut.S > 1 ? 1 : 0;
    return from_cuda(cudaLaunchKernelEx(&cfg, kernel, args...));
}

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

template <typename TI, typename TO, bool LEAK, bool BWD>
kdn_status launch_maps(const GatedArgs& a, float4* maps, cudaStream_t stream) {
    // (parts are for few channels: this is under 2^31)
    const long long blocks = state_rows(a) * maps_of(a.T) * ((a.C + 31) / 32);
    gated_maps_kernel<TI, TO, LEAK, BWD><<<static_cast<unsigned>(blocks), MAP_WARPS * 32, 0, stream>>>(a, maps);
    return from_cuda(cudaGetLastError());
}

long long maps_bytes(long long rows, long long parts, int C, int T) {
    return parts > 1 ? rows * maps_of(T) * C * 16 : 0;
}

}  // namespace

long long gated_bwd_workspace_bytes(int B, int H, int T, int C, int nseq) {
    const long long rows = static_cast<long long>(nseq > 0 ? nseq : B) * H;
    const long long parts = nseq > 0 ? 1 : most_parts(rows, C, T);
    return maps_bytes(rows, parts, C, T) + (rows / H * parts > 1 ? rows * parts * C * 4 : 0);
}

kdn_status gated_fwd_launch(const GatedArgs& a, cudaStream_t stream, long long wait_ns, int stall) {
    return by_type(a.in_dtype, a.out_dtype, [&](auto ti, auto to) {
        using TI = decltype(ti);
        using TO = decltype(to);
        constexpr int V = std::is_same<TI, __nv_bfloat16>::value ? 2 : 1;
        auto go = [&](auto leak, auto size) {
            constexpr bool L = decltype(leak)::value;
            auto kernel = gated_fwd_kernel<TI, TO, V, FWD_K, L, decltype(size)::value>;
            using Sh = FwdShared<TI, TO, V, FWD_K>;
            Cut cut{};
            cut.wait_ns = wait_ns;
            cut.stall = stall;
            kdn_status s = plan(a, reinterpret_cast<const void*>(kernel), Sizes<Sh>::alone, Sizes<Sh>::smem(), V, FWD_K, 9.0, &cut);
            if (s != KDN_OK) return s;
            Scratch scratch(stream);
            if (cut.parts > 1) {
                s = scratch.take(maps_bytes(state_rows(a), cut.parts, a.C, a.T));
                if (s != KDN_OK) return s;
                cut.maps = static_cast<float4*>(scratch.p);
                s = launch_maps<TI, TO, L, false>(a, static_cast<float4*>(scratch.p), stream);
                if (s != KDN_OK) return s;
            }
            return launch_walk(kernel, state_rows(a), cut, Sizes<Sh>::of(cut), stream, a, cut);
        };
        auto sized = [&](auto leak) {
            if (rows_ok(a, 16)) return go(leak, std::integral_constant<int, 16>());
            if (sizeof(TI) == 4 && sizeof(TO) == 4) return go(leak, std::integral_constant<int, 4>());
            if (rows_ok(a, 4)) return go(leak, std::integral_constant<int, 4>());
            return go(leak, std::integral_constant<int, 2>());
        };
        return a.leak ? sized(std::true_type()) : sized(std::false_type());
    });
}

kdn_status gated_bwd_launch(const GatedArgs& a, cudaStream_t stream, long long wait_ns, int stall) {
    return by_type(a.in_dtype, a.out_dtype, [&](auto ti, auto to) {
        using TI = decltype(ti);
        using TO = decltype(to);
        constexpr int V = std::is_same<TI, __nv_bfloat16>::value ? 2 : 1;
        auto go = [&](auto leak, auto size) {
            constexpr bool L = decltype(leak)::value;
            constexpr int SIZE = decltype(size)::value;
            auto kernel = gated_bwd_kernel<TI, TO, V, BWD_K, L, SIZE>;
            using Sh = BwdShared<TI, TO, V, BWD_K, L>;
            Cut cut{};
            cut.wait_ns = wait_ns;
            cut.stall = stall;
            kdn_status s = plan(a, reinterpret_cast<const void*>(kernel), Sizes<Sh>::alone, Sizes<Sh>::smem(), V, BWD_K,
                                a.workspace ? 3.5 : 9.0, &cut);
            if (s != KDN_OK) return s;
            size_t smem = Sizes<Sh>::of(cut);
            // twice the tokens a round where that still leaves two CTAs to an SM: 16-bit rows, no x,
            // no cluster
            if constexpr (!L && SIZE == 16 && sizeof(TI) == 2 && sizeof(TO) == 2) {
                using Wide = BwdShared<TI, TO, V, 2 * BWD_K, L>;
                auto wide = gated_bwd_kernel<TI, TO, V, 2 * BWD_K, L, SIZE>;
                if (cut.S == 1 && cut.parts == 1) {
                    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(wide), Sizes<Wide>::alone);
                    if (e != cudaSuccess) return from_cuda(e);
                    kernel = wide;
                    smem = Sizes<Wide>::alone;
                }
            }
            const long long rows = state_rows(a), shares = rows / a.H * cut.parts;
            const long long maps = maps_bytes(rows, cut.parts, a.C, a.T), HC = static_cast<long long>(a.H) * a.C;
            const long long bytes = maps + (shares > 1 && a.grad_A ? shares * HC * 4 : 0);
            Scratch scratch(stream);
            char* ws = static_cast<char*>(a.workspace);
            if (bytes > 0 && !ws) {
                s = scratch.take(bytes);
                if (s != KDN_OK) return s;
                ws = static_cast<char*>(scratch.p);
            }
            if (cut.parts > 1) {
                cut.maps = reinterpret_cast<float4*>(ws);
                s = launch_maps<TI, TO, L, true>(a, reinterpret_cast<float4*>(ws), stream);
                if (s != KDN_OK) return s;
            }
            float* sums = !a.grad_A ? nullptr : shares > 1 ? reinterpret_cast<float*>(ws + maps) : a.grad_A;
            s = launch_walk(kernel, rows, cut, smem, stream, a, cut, sums);
            if (s == KDN_OK && a.grad_A && shares > 1)
                s = from_cuda(sum_rows(sums, shares, HC, a.grad_A, nullptr, HC, stream));
            return s;
        };
        auto sized = [&](auto leak) {
            if (rows_ok(a, 16)) return go(leak, std::integral_constant<int, 16>());
            if (sizeof(TI) == 4 && sizeof(TO) == 4) return go(leak, std::integral_constant<int, 4>());
            if (rows_ok(a, 4)) return go(leak, std::integral_constant<int, 4>());
            return go(leak, std::integral_constant<int, 2>());
        };
        return a.leak ? sized(std::true_type()) : sized(std::false_type());
    });
}

cudaError_t gated_take_device_error(int* status) {
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_gated_error, sizeof(int));
    if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(g_gated_error, &zero, sizeof(int));
    *status = v;
    return e;
}

kdn_status gated_step_launch(const void* x, const void* d, const float* A, bool leak, const float* state,
                             float* new_state, void* out, int B, int H, int C, kdn_dtype in_dtype,
                             kdn_dtype out_dtype, cudaStream_t stream) {
    const long long HC = static_cast<long long>(H) * C, n = HC * B;
    const void* ptrs[] = {x, d, A, state, new_state, out};
    bool wide = HC % 4 == 0 && n >= 4LL * NW * 32 * sm_count();   // (a small call wants threads, not width)
    for (const void* q : ptrs) wide = wide && reinterpret_cast<uintptr_t>(q) % 16 == 0;
    const long long per = wide ? 4 : 1, blocks = (n / per + NW * 32 - 1) / (NW * 32);
    if (blocks > 0x7fffffffLL) return KDN_ERR_INVALID_ARG;
    return by_type(in_dtype, out_dtype, [&](auto ti, auto to) {
        using TI = decltype(ti);
        using TO = decltype(to);
        auto kernel = wide ? gated_step_kernel<TI, TO, 4> : gated_step_kernel<TI, TO, 1>;
        kernel<<<static_cast<unsigned>(blocks), NW * 32, 0, stream>>>(
            static_cast<const TI*>(x), static_cast<const TI*>(d), A, leak, state, new_state, static_cast<TO*>(out), n, HC);
        return from_cuda(cudaGetLastError());
    });
}

}  // namespace kdn
