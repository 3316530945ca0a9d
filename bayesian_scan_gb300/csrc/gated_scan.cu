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
// memory, and a second pass over the tokens, still in registers, writes the
// states.  So every element is read once and written once, and HBM bounds the
// kernel: 6 bytes per element forward (bf16), 10 backward.
//
// One CTA walks one sequence of one slab of channels, tile after tile, the
// next tile's loads in flight.  Where that makes too few CTAs a cluster of S
// of them takes S consecutive tiles per round: each CTA sends its tile's map
// to all others' shared memory and one cluster barrier later every CTA knows
// the state before its tile and before the next round.  The composition's
// order is fixed, so results do not depend on the schedule.
#include <type_traits>

#include "gated_device.cuh"
#include "kdn_device.cuh"
#include "kdn_internal.h"
#include "sum_rows.cuh"

namespace kdn {
namespace {

using namespace gated;

constexpr int MAX_CLUSTER = 8;
constexpr int THREADS = 256;      // of the kernels without tiles
constexpr int FWD_WARPS = 8, BWD_WARPS = 8;

__device__ int g_gated_error = 0;

// The tokens of state row n*H + h (a batch, or a packed sequence): [lo, hi)
// of the T-token row `row`.
struct Span {
    long long row;
    int lo, hi;
};

__device__ __forceinline__ Span span_of(const GatedArgs& p, long long sr) {
    Span s{sr, 0, p.T};
    if (p.offsets) {
        const long long n = sr / p.H;
        s.row = sr - n * p.H;
        s.lo = min(max(p.offsets[n], 0), p.T);
        s.hi = min(max(p.offsets[n + 1], s.lo), p.T);
    }
    return s;
}

// How one call is cut: slabs of 32 V channels, clusters of S CTAs.
struct Cut {
    int slabs, S;
    long long wait_ns;     // limit of one wait inside a cluster
};

// An affine map h -> (a + e) h + s of a lane's V channels over a span of
// tokens, z its exponent (a + e = exp(z)), as shared-memory words that one
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
// round's last tile, both from the carry before the round.  Rounds alternate
// between two buffers, so one barrier a round is enough.
//
// In a cluster the tile's map goes to every CTA's shared memory by stores
// that complete on the receiver's mbarrier: no fence waits for the round's
// global stores, as the cluster barrier's release would (an eighth of the
// time).  A CTA sends round r only after all its warps have read round r - 2,
// and receives all of round r - 1 before it sends round r, so no store finds
// its buffer in use.
template <int V, int NW>
struct Fold {
    MapWords<V> warp[2][NW];
    MapWords<V> cta[2][MAX_CLUSTER];
    uint64_t full[2];

    // Every CTA of the cluster runs, its barriers set up, before one sends.
    __device__ __forceinline__ void begin(int S) {
        if (S > 1) {
            if (threadIdx.x == 0) {
                mbar_init(&full[0], 1);
                mbar_init(&full[1], 1);
                mbar_init_fence();
            }
            cluster_sync();
        }
    }
    // No CTA leaves while another may still send to it.
    __device__ __forceinline__ void end(int S, bool late) {
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

// Bounded: after limit_ns it records an error and no later round waits.
__device__ __forceinline__ void full_wait(uint64_t* bar, uint32_t parity, long long limit_ns, bool& late) {
    if (late || full_try(bar, parity)) return;
    const unsigned long long t0 = globaltimer_ns();
    while (!full_try(bar, parity))
        if (static_cast<long long>(globaltimer_ns() - t0) > limit_ns) {
            record_error(&g_gated_error, KDN_ERR_TIMEOUT);
            late = true;
            return;
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

template <int V, int NW>
__device__ __forceinline__ void fold_round(Fold<V, NW>& f, int r, int S, int rank, int warp, int lane,
                                           long long limit_ns, bool& late, const float (&z)[V], const float (&s)[V],
                                           float (&carry)[V], float (&start)[V]) {
    const int buf = r & 1;
    put_map<V>(f.warp[buf][warp], lane, map_of<V>(z, s));
    __syncthreads();
    if (S > 1) {
        if (threadIdx.x == 0) mbar_arrive_expect_tx(&f.full[buf], S * sizeof(MapWords<V>));
        if (warp < S) {
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
            for (int j = warp; j < S; j += NW) {
                const uint32_t to = at_rank(&f.cta[buf][rank][0][lane], j), bar = at_rank(&f.full[buf], j);
                if constexpr (V == 1) {
                    send(to, make_float4(m.a[0], m.e[0], m.s[0], m.z[0]), bar);
                } else {
                    send(to, make_float4(m.a[0], m.a[1], m.e[0], m.e[1]), bar);
                    send(to + 512, make_float4(m.s[0], m.s[1], m.z[0], m.z[1]), bar);
                }
            }
        }
        full_wait(&f.full[buf], (r >> 1) & 1, limit_ns, late);
#pragma unroll
        for (int v = 0; v < V; ++v) start[v] = carry[v];
        for (int j = 0; j < S; ++j) {
            if (j == rank)
#pragma unroll
                for (int v = 0; v < V; ++v) start[v] = carry[v];
            apply<V>(get_map<V>(f.cta[buf][j], lane), carry);
        }
        for (int w = 0; w < warp; ++w) apply<V>(get_map<V>(f.warp[buf][w], lane), start);
    } else {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w == warp)
#pragma unroll
                for (int v = 0; v < V; ++v) start[v] = carry[v];
            apply<V>(get_map<V>(f.warp[buf][w], lane), carry);
        }
    }
}

template <typename TI, typename TO, int V, int K, int NW, bool LEAK>
__global__ void __launch_bounds__(NW * 32, 16 / NW) gated_fwd_kernel(const GatedArgs p, const Cut cut) {
    __shared__ Fold<V, NW> fold;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = cut.S, rank = blockIdx.x % S;
    const long long unit = blockIdx.x / S;
    const long long sr = unit / cut.slabs;
    const int c = (static_cast<int>(unit - sr * cut.slabs) * 32 + lane) * V;
    const bool on = c < p.C;
    const Span sp = span_of(p, sr);
    const int rounds = (sp.hi - sp.lo + S * NW * K - 1) / (S * NW * K);
    const long long arow = (sr % p.H) * p.C;

    float nA[V], carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        nA[v] = on ? -p.A[arow + c + v] : 0.f;
        carry[v] = on && p.h0 ? p.h0[sr * p.C + c + v] : 0.f;
    }
    const TI* xp = static_cast<const TI*>(p.x) + sp.row * p.T * p.x_ld + c;
    const TI* dp = static_cast<const TI*>(p.d) + sp.row * p.T * p.d_ld + c;
    TO* op = static_cast<TO*>(p.out) + sp.row * p.T * p.C + c;

    Vec<TI, V> xr[K], dr[K];
    auto fetch = [&](int r) {
        const int t = sp.lo + ((r * S + rank) * NW + warp) * K;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xr[k] = Vec<TI, V>{};
            dr[k] = Vec<TI, V>{};
            if (on && t + k < sp.hi) {
                xr[k] = load<TI, V>(xp + static_cast<long long>(t + k) * p.x_ld);
                dr[k] = load<TI, V>(dp + static_cast<long long>(t + k) * p.d_ld);
            }
        }
    };
    if (rounds > 0) fetch(0);
    fold.begin(S);
    bool late = false;
    for (int r = 0; r < rounds; ++r) {
        const int t = sp.lo + ((r * S + rank) * NW + warp) * K;
        // tokens behind the end have d = x = 0: alpha = 1, nothing added
        float a[K][V], b[K][V], z[V], s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = s[v] = 0.f;
#pragma unroll
        for (int i = 0; i < K * V / 2; ++i) {
            const int k0 = 2 * i / V, v0 = 2 * i % V, k1 = (2 * i + 1) / V, v1 = (2 * i + 1) % V;
            const F2 zz = mul2(F2{nA[v0], nA[v1]}, F2{dr[k0].get(v0), dr[k1].get(v1)});
            const Gate2 gg = gate2<LEAK>(zz);
            a[k0][v0] = gg.a.x;
            a[k1][v1] = gg.a.y;
            F2 x{xr[k0].get(v0), xr[k1].get(v1)};
            if (LEAK) x = mul2(x, gg.w);
            b[k0][v0] = x.x;
            b[k1][v1] = x.y;
            if (V == 1) {
                z[0] += zz.x + zz.y;
                s[0] = fmaf(gg.a.x, s[0], x.x);
                s[0] = fmaf(gg.a.y, s[0], x.y);
            } else {
                const F2 ss{s[v0], s[v1]};
                const F2 n = fma2(gg.a, ss, x), zs = add2(F2{z[v0], z[v1]}, zz);
                s[v0] = n.x;
                s[v1] = n.y;
                z[v0] = zs.x;
                z[v1] = zs.y;
            }
        }
        if (r + 1 < rounds) fetch(r + 1);
        float h[V];
        fold_round<V, NW>(fold, r, S, rank, warp, lane, cut.wait_ns, late, z, s, carry, h);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (V == 1) {
                h[0] = fmaf(a[k][0], h[0], b[k][0]);
            } else {
#pragma unroll
                for (int v = 0; v < V; v += 2) {
                    const F2 hh{h[v], h[v + 1]};
                    const F2 n = fma2(F2{a[k][v], a[k][v + 1]}, hh, F2{b[k][v], b[k][v + 1]});
                    h[v] = n.x;
                    h[v + 1] = n.y;
                }
            }
            if (on && t + k < sp.hi) {
                Vec<TO, V> o;
                o.set(h);
                store<TO, V>(op + static_cast<long long>(t + k) * p.C, o);
            }
        }
    }
    fold.end(S, late);
    if (p.final_state && rank == 0 && warp == 0 && on)
#pragma unroll
        for (int v = 0; v < V; ++v) p.final_state[sr * p.C + c + v] = carry[v];
}

// The same walk from the last token to the first.  `part` [sequence, rank,
// H, C] takes each CTA's share of grad A.
template <typename TI, typename TO, int V, int K, int NW, bool LEAK>
__global__ void __launch_bounds__(NW * 32, 16 / NW)
gated_bwd_kernel(const GatedArgs p, const Cut cut, float* part) {
    __shared__ Fold<V, NW> fold;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = cut.S, rank = blockIdx.x % S;
    const long long unit = blockIdx.x / S;
    const long long sr = unit / cut.slabs;
    const int c = (static_cast<int>(unit - sr * cut.slabs) * 32 + lane) * V;
    const bool on = c < p.C;
    const Span sp = span_of(p, sr);
    const int rounds = (sp.hi - sp.lo + S * NW * K - 1) / (S * NW * K);
    const long long arow = (sr % p.H) * p.C;

    float nA[V], carry[V], dA[V], first[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        nA[v] = on ? -p.A[arow + c + v] : 0.f;
        carry[v] = on && p.grad_final_state ? p.grad_final_state[sr * p.C + c + v] : 0.f;
        first[v] = on && p.h0 ? p.h0[sr * p.C + c + v] : 0.f;
        dA[v] = 0.f;
    }
    const TI* dp = static_cast<const TI*>(p.d) + sp.row * p.T * p.d_ld + c;
    const TI* xp = LEAK ? static_cast<const TI*>(p.x) + sp.row * p.T * p.x_ld + c : nullptr;
    const long long row = sp.row * p.T * p.C + c;
    const TO* hp = static_cast<const TO*>(p.out) + row;
    const TO* gp = static_cast<const TO*>(p.grad_out) + row;
    TI* gxp = static_cast<TI*>(p.grad_x) + row;
    TI* gdp = static_cast<TI*>(p.grad_d) + row;

    Vec<TI, V> dn[K];
    Vec<TO, V> gn[K];
    auto fetch = [&](int r) {
        const int t = sp.hi - 1 - ((r * S + rank) * NW + warp) * K;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            dn[k] = Vec<TI, V>{};
            gn[k] = Vec<TO, V>{};
            if (on && t - k >= sp.lo) {
                dn[k] = load<TI, V>(dp + static_cast<long long>(t - k) * p.d_ld);
                gn[k] = load<TO, V>(gp + static_cast<long long>(t - k) * p.C);
            }
        }
    };
    if (rounds > 0) fetch(0);
    fold.begin(S);
    bool late = false;
    for (int r = 0; r < rounds; ++r) {
        const int t = sp.hi - 1 - ((r * S + rank) * NW + warp) * K;
        Vec<TO, V> hr[K];
        Vec<TI, V> xr[K], dr[K];
        Vec<TO, V> gr[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            hr[k] = Vec<TO, V>{};
            xr[k] = Vec<TI, V>{};
            if (on && t - k > sp.lo) hr[k] = load<TO, V>(hp + static_cast<long long>(t - k - 1) * p.C);
            if (LEAK && on && t - k >= sp.lo) xr[k] = load<TI, V>(xp + static_cast<long long>(t - k) * p.x_ld);
            dr[k] = dn[k];
            gr[k] = gn[k];
        }
        float a[K][V], z[V], s[V], w[LEAK ? K : 1][V];
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = s[v] = 0.f;
        // u = alpha (g + u): the map of a token is (alpha, alpha g)
#pragma unroll
        for (int i = 0; i < K * V / 2; ++i) {
            const int k0 = 2 * i / V, v0 = 2 * i % V, k1 = (2 * i + 1) / V, v1 = (2 * i + 1) % V;
            const F2 zz = mul2(F2{nA[v0], nA[v1]}, F2{dr[k0].get(v0), dr[k1].get(v1)});
            const Gate2 gg = gate2<LEAK>(zz);
            a[k0][v0] = gg.a.x;
            a[k1][v1] = gg.a.y;
            if (LEAK) {
                w[LEAK ? k0 : 0][v0] = gg.w.x;
                w[LEAK ? k1 : 0][v1] = gg.w.y;
            }
            if (V == 1) {
                z[0] += zz.x + zz.y;
                const float d0 = s[0] + gr[k0].get(0);
                s[0] = gg.a.x * d0;
                const float d1 = s[0] + gr[k1].get(0);
                s[0] = gg.a.y * d1;
            } else {
                const F2 dh = add2(F2{s[v0], s[v1]}, F2{gr[k0].get(v0), gr[k0].get(v1)});
                const F2 n = mul2(gg.a, dh), zs = add2(F2{z[v0], z[v1]}, zz);
                s[v0] = n.x;
                s[v1] = n.y;
                z[v0] = zs.x;
                z[v1] = zs.y;
            }
        }
        if (r + 1 < rounds) fetch(r + 1);
        float u[V];
        fold_round<V, NW>(fold, r, S, rank, warp, lane, cut.wait_ns, late, z, s, carry, u);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float gx[V], gd[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float dh = u[v] + gr[k].get(v);
                u[v] = a[k][v] * dh;
                float prev = t - k > sp.lo ? hr[k].get(v) : first[v];
                gx[v] = dh;
                if (LEAK) {
                    prev -= xr[k].get(v);
                    gx[v] = w[LEAK ? k : 0][v] * dh;
                }
                const float m = u[v] * prev;
                gd[v] = nA[v] * m;
                if (t - k >= sp.lo) dA[v] = fmaf(-dr[k].get(v), m, dA[v]);
            }
            if (on && t - k >= sp.lo) {
                Vec<TI, V> o;
                o.set(gx);
                store<TI, V>(gxp + static_cast<long long>(t - k) * p.C, o);
                o.set(gd);
                store<TI, V>(gdp + static_cast<long long>(t - k) * p.C, o);
            }
        }
    }
    fold.end(S, late);
    if (p.grad_h0 && rank == 0 && warp == 0 && on)
#pragma unroll
        for (int v = 0; v < V; ++v) p.grad_h0[sr * p.C + c + v] = carry[v];
    if (part) {
        // the warps' shares, in order
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) fold.warp[0][warp][v][lane].x = dA[v];
        __syncthreads();
        if (warp == 0 && on)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float sum = 0.f;
                for (int w = 0; w < NW; ++w) sum += fold.warp[0][w][v][lane].x;
                part[((sr / p.H * S + rank) * p.H + sr % p.H) * p.C + c + v] = sum;
            }
    }
}

// The staged form: a warp's rows come through shared memory, STAGES rounds
// ahead by asynchronous copies of SIZE bytes that fill what lies outside the
// sequence or the channels with zeros, and with SIZE = 16 leave through it
// too, in 16-byte pieces (a 4-byte SIZE takes rows that are only aligned to
// that, and stores straight from the registers).  A warp reads only rows that
// it copied itself, so no barrier beyond the fold's is needed.
constexpr int STAGES = 2;

template <typename TI, typename TO, int V, int K, int NW>
struct FwdShared {
    static constexpr int ROW = 32 * V * static_cast<int>(sizeof(TI)), OROW = 32 * V * static_cast<int>(sizeof(TO));
    struct __align__(16) Stage {
        char x[K * ROW], d[K * ROW];                 // out overwrites both
    };
    Stage st[STAGES][NW];
    Fold<V, NW> fold;
};

template <typename TI, typename TO, int V, int K, int NW, bool LEAK, int SIZE>
__global__ void __launch_bounds__(NW * 32, 16 / NW) gated_fwd_staged(const GatedArgs p, const Cut cut) {
    using Sh = FwdShared<TI, TO, V, K, NW>;
    static_assert(Sh::OROW * K <= static_cast<int>(sizeof(typename Sh::Stage)), "out takes the stage's place");
    extern __shared__ __align__(16) char smem[];
    Sh& sh = *reinterpret_cast<Sh*>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = cut.S, rank = blockIdx.x % S;
    const long long unit = blockIdx.x / S;
    const long long sr = unit / cut.slabs;
    const int c0 = static_cast<int>(unit - sr * cut.slabs) * 32 * V, c = c0 + lane * V;
    const Span sp = span_of(p, sr);
    const int rounds = (sp.hi - sp.lo + S * NW * K - 1) / (S * NW * K);
    const long long arow = (sr % p.H) * p.C;

    float nA[V], carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        nA[v] = c + v < p.C ? -p.A[arow + c + v] : 0.f;
        carry[v] = c + v < p.C && p.h0 ? p.h0[sr * p.C + c + v] : 0.f;
    }
    const int t0 = sp.lo + (rank * NW + warp) * K, step = S * NW * K;
    const long long xld = p.x_ld * sizeof(TI), dld = p.d_ld * sizeof(TI);
    const char* xp = static_cast<const char*>(p.x) + (sp.row * p.T + t0) * xld + c0 * sizeof(TI);
    const char* dp = static_cast<const char*>(p.d) + (sp.row * p.T + t0) * dld + c0 * sizeof(TI);
    TO* op = static_cast<TO*>(p.out) + (sp.row * p.T + t0) * p.C + c0;
    const int width = (p.C - c0) * static_cast<int>(sizeof(TI)), owidth = (p.C - c0) * static_cast<int>(sizeof(TO));

    auto fetch = [&](int r) {
        const int n = sp.hi - t0 - r * step;               // tokens left
        if (n > 0) {
            typename Sh::Stage& st = sh.st[r % STAGES][warp];
            const uint32_t sm = static_cast<uint32_t>(__cvta_generic_to_shared(st.x));
            rows_in<SIZE, Sh::ROW, K>(sm, p.x, xp + static_cast<long long>(r) * step * xld, xld, 0, n, width, lane);
            rows_in<SIZE, Sh::ROW, K>(sm + K * Sh::ROW, p.d, dp + static_cast<long long>(r) * step * dld, dld, 0, n, width, lane);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
        if (i < rounds) fetch(i);
        else copy_commit();
    sh.fold.begin(S);
    bool late = false;
    for (int r = 0; r < rounds; ++r) {
        const int n = sp.hi - t0 - r * step;
        char* xs = sh.st[r % STAGES][warp].x;
        const char* ds = sh.st[r % STAGES][warp].d;
        copy_wait<STAGES - 1>();
        __syncwarp();
        float a[K][V], b[K][V], z[V], s[V], h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = s[v] = 0.f;
        if (n > 0) {                                        // (the warp as one)
#pragma unroll
            for (int i = 0; i < K * V / 2; ++i) {
                const int k0 = 2 * i / V, v0 = 2 * i % V, k1 = (2 * i + 1) / V, v1 = (2 * i + 1) % V;
                const Vec<TI, V> d0 = peek<TI, V>(ds + k0 * Sh::ROW + lane * V * sizeof(TI)),
                                 x0 = peek<TI, V>(xs + k0 * Sh::ROW + lane * V * sizeof(TI));
                Vec<TI, V> d1 = d0, x1 = x0;
                if (V == 1) {
                    d1 = peek<TI, V>(ds + k1 * Sh::ROW + lane * V * sizeof(TI));
                    x1 = peek<TI, V>(xs + k1 * Sh::ROW + lane * V * sizeof(TI));
                }
                const F2 zz = mul2(F2{nA[v0], nA[v1]}, F2{d0.get(v0), d1.get(v1)});
                const Gate2 gg = gate2<LEAK>(zz);
                a[k0][v0] = gg.a.x;
                a[k1][v1] = gg.a.y;
                F2 x{x0.get(v0), x1.get(v1)};
                if (LEAK) x = mul2(x, gg.w);
                b[k0][v0] = x.x;
                b[k1][v1] = x.y;
                if constexpr (V == 1) {
                    z[0] += zz.x + zz.y;
                    s[0] = fmaf(gg.a.x, s[0], x.x);
                    s[0] = fmaf(gg.a.y, s[0], x.y);
                } else {
                    const F2 ss{s[0], s[1]};
                    const F2 m = fma2(gg.a, ss, x), zs = add2(F2{z[0], z[1]}, zz);
                    s[0] = m.x;
                    s[1] = m.y;
                    z[0] = zs.x;
                    z[1] = zs.y;
                }
            }
        }
        fold_round<V, NW>(sh.fold, r, S, rank, warp, lane, cut.wait_ns, late, z, s, carry, h);
        if (n > 0) {
            TO* o = op + static_cast<long long>(r) * step * p.C;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if constexpr (V == 1) {
                    h[0] = fmaf(a[k][0], h[0], b[k][0]);
                } else {
                    const F2 hh{h[0], h[1]};
                    const F2 m = fma2(F2{a[k][0], a[k][1]}, hh, F2{b[k][0], b[k][1]});
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
        if (r + STAGES < rounds) fetch(r + STAGES);
        else copy_commit();
    }
    sh.fold.end(S, late);
    if (p.final_state && rank == 0 && warp == 0)
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c + v < p.C) p.final_state[sr * p.C + c + v] = carry[v];
}

template <typename TI, typename TO, int V, int K, int NW>
struct BwdShared {
    static constexpr int ROW = 32 * V * static_cast<int>(sizeof(TI)), OROW = 32 * V * static_cast<int>(sizeof(TO));
    struct __align__(16) Stage {
        char d[K * ROW], x[K * ROW], g[K * OROW], h[K * OROW];   // grad d overwrites d, grad x x
    };
    Stage st[STAGES][NW];
    Fold<V, NW> fold;
};

template <typename TI, typename TO, int V, int K, int NW, bool LEAK, int SIZE>
__global__ void __launch_bounds__(NW * 32, 16 / NW)
gated_bwd_staged(const GatedArgs p, const Cut cut, float* part) {
    using Sh = BwdShared<TI, TO, V, K, NW>;
    extern __shared__ __align__(16) char smem[];
    Sh& sh = *reinterpret_cast<Sh*>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = cut.S, rank = blockIdx.x % S;
    const long long unit = blockIdx.x / S;
    const long long sr = unit / cut.slabs;
    const int c0 = static_cast<int>(unit - sr * cut.slabs) * 32 * V, c = c0 + lane * V;
    const Span sp = span_of(p, sr);
    const int rounds = (sp.hi - sp.lo + S * NW * K - 1) / (S * NW * K);
    const long long arow = (sr % p.H) * p.C;

    float nA[V], carry[V], dA[V], first[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const bool on = c + v < p.C;
        nA[v] = on ? -p.A[arow + c + v] : 0.f;
        carry[v] = on && p.grad_final_state ? p.grad_final_state[sr * p.C + c + v] : 0.f;
        first[v] = on && p.h0 ? p.h0[sr * p.C + c + v] : 0.f;
        dA[v] = 0.f;
    }
    // a warp's rows of round r are tokens base - r step .. + K - 1, walked from the last
    const int base = sp.hi - (rank * NW + warp + 1) * K, step = S * NW * K;
    const long long dld = p.d_ld * sizeof(TI), xld = p.x_ld * sizeof(TI), old_ = p.C * static_cast<long long>(sizeof(TO));
    const long long row = sp.row * p.T;
    const int width = (p.C - c0) * static_cast<int>(sizeof(TI)), owidth = (p.C - c0) * static_cast<int>(sizeof(TO));

    auto fetch = [&](int r) {
        const int t = base - r * step;
        if (t + K > sp.lo) {
            typename Sh::Stage& st = sh.st[r % STAGES][warp];
            const int f = max(sp.lo - t, 0);               // rows before the sequence
            const uint32_t sm = static_cast<uint32_t>(__cvta_generic_to_shared(st.d));
            constexpr int N = K * Sh::ROW, M = K * Sh::OROW;
            rows_in<SIZE, Sh::ROW, K>(sm, p.d, static_cast<const char*>(p.d) + (row + t) * dld + c0 * sizeof(TI), dld, f, K,
                                      width, lane);
            if (LEAK)
                rows_in<SIZE, Sh::ROW, K>(sm + N, p.x, static_cast<const char*>(p.x) + (row + t) * xld + c0 * sizeof(TI), xld,
                                          f, K, width, lane);
            rows_in<SIZE, Sh::OROW, K>(sm + 2 * N, p.grad_out, static_cast<const char*>(p.grad_out) + (row + t) * old_ + c0 * sizeof(TO),
                                       old_, f, K, owidth, lane);
            // the states before: one token earlier (h0 for the first one, below)
            rows_in<SIZE, Sh::OROW, K>(sm + 2 * N + M, p.out, static_cast<const char*>(p.out) + (row + t - 1) * old_ + c0 * sizeof(TO),
                                       old_, f + (t + f == sp.lo), K, owidth, lane);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
        if (i < rounds) fetch(i);
        else copy_commit();
    sh.fold.begin(S);
    bool late = false;
    for (int r = 0; r < rounds; ++r) {
        const int t = base - r * step;
        const bool any = t + K > sp.lo;
        typename Sh::Stage& st = sh.st[r % STAGES][warp];
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
                const F2 zz = mul2(F2{nA[v0], nA[v1]}, F2{d0.get(v0), d1.get(v1)});
                const Gate2 gg = gate2<LEAK>(zz);
                a[k0][v0] = gg.a.x;
                a[k1][v1] = gg.a.y;
                if (LEAK) {
                    w[LEAK ? k0 : 0][v0] = gg.w.x;
                    w[LEAK ? k1 : 0][v1] = gg.w.y;
                }
                if constexpr (V == 1) {
                    z[0] += zz.x + zz.y;
                    const float h0 = s[0] + g0.get(0);
                    s[0] = gg.a.x * h0;
                    const float h1 = s[0] + g1.get(0);
                    s[0] = gg.a.y * h1;
                } else {
                    const F2 dh = add2(F2{s[0], s[1]}, F2{g0.get(0), g0.get(1)});
                    const F2 m = mul2(gg.a, dh), zs = add2(F2{z[0], z[1]}, zz);
                    s[0] = m.x;
                    s[1] = m.y;
                    z[0] = zs.x;
                    z[1] = zs.y;
                }
            }
        }
        fold_round<V, NW>(sh.fold, r, S, rank, warp, lane, cut.wait_ns, late, z, s, carry, u);
        if (any) {
            TI* gx_out = static_cast<TI*>(p.grad_x) + (row + t) * p.C + c0;
            TI* gd_out = static_cast<TI*>(p.grad_d) + (row + t) * p.C + c0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int j = K - 1 - k;
                const Vec<TI, V> dv = peek<TI, V>(st.d + j * Sh::ROW + lane * V * sizeof(TI));
                const Vec<TO, V> gv = peek<TO, V>(st.g + j * Sh::OROW + lane * V * sizeof(TO));
                const Vec<TO, V> hv = peek<TO, V>(st.h + j * Sh::OROW + lane * V * sizeof(TO));
                Vec<TI, V> xv = dv;
                if (LEAK) xv = peek<TI, V>(st.x + j * Sh::ROW + lane * V * sizeof(TI));
                float gx[V], gd[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float dh = u[v] + gv.get(v);
                    u[v] = a[k][v] * dh;
                    float prev = t + j == sp.lo ? first[v] : hv.get(v);
                    gx[v] = dh;
                    if (LEAK) {
                        prev -= xv.get(v);
                        gx[v] = w[LEAK ? k : 0][v] * dh;
                    }
                    const float m = u[v] * prev;
                    gd[v] = nA[v] * m;
                    dA[v] = fmaf(-dv.get(v), m, dA[v]);     // (d = 0 outside the sequence)
                }
                if (SIZE == 16) {
                    Vec<TI, V> q;
                    q.set(gx);
                    poke<TI, V>(st.x + j * Sh::ROW + lane * V * sizeof(TI), q);
                    q.set(gd);
                    poke<TI, V>(st.d + j * Sh::ROW + lane * V * sizeof(TI), q);
                } else if (t + j >= sp.lo) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (c + v < p.C) {
                            __stcs(gx_out + static_cast<long long>(j) * p.C + lane * V + v, from_f32<TI>(gx[v]));
                            __stcs(gd_out + static_cast<long long>(j) * p.C + lane * V + v, from_f32<TI>(gd[v]));
                        }
                }
            }
            __syncwarp();
            if (SIZE == 16) {
                const int f = max(sp.lo - t, 0);
                const long long ld = p.C * static_cast<long long>(sizeof(TI));
                rows_out<Sh::ROW, K>(reinterpret_cast<char*>(gx_out), ld, st.x, f, K, width, lane);
                rows_out<Sh::ROW, K>(reinterpret_cast<char*>(gd_out), ld, st.d, f, K, width, lane);
                __syncwarp();
            }
        }
        if (r + STAGES < rounds) fetch(r + STAGES);
        else copy_commit();
    }
    sh.fold.end(S, late);
    if (p.grad_h0 && rank == 0 && warp == 0)
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c + v < p.C) p.grad_h0[sr * p.C + c + v] = carry[v];
    if (part) {
        // the warps' shares, in order
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) sh.fold.warp[0][warp][v][lane].x = dA[v];
        __syncthreads();
        if (warp == 0)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float sum = 0.f;
                for (int i = 0; i < NW; ++i) sum += sh.fold.warp[0][i][v][lane].x;
                if (c + v < p.C) part[((sr / p.H * S + rank) * p.H + sr % p.H) * p.C + c + v] = sum;
            }
    }
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(THREADS)
gated_step_kernel(const TI* __restrict__ x, const TI* __restrict__ d, const float* __restrict__ A, bool leak,
                  const float* state, float* new_state, TO* __restrict__ out, long long n, long long HC) {
    const long long i = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
    if (i >= n) return;
    const Gate g = gate(-A[i % HC] * to_f32(d[i]));
    const float xi = to_f32(x[i]);
    const float h = decay_add(g, state[i], leak ? g.w * xi : xi);
    new_state[i] = h;
    out[i] = from_f32<TO>(h);
}

template <typename F>
kdn_status by_type(const GatedArgs& a, F f) {
    if (a.in_dtype == KDN_BF16)
        return a.out_dtype == KDN_BF16 ? f(__nv_bfloat16(), __nv_bfloat16()) : f(__nv_bfloat16(), float());
    return a.out_dtype == KDN_BF16 ? f(float(), __nv_bfloat16()) : f(float(), float());
}

long long state_rows(const GatedArgs& a) { return static_cast<long long>(a.nseq > 0 ? a.nseq : a.B) * a.H; }

// CTAs per cluster: as many as keep the grid within the GPU's two CTAs per
// SM, no more than a sequence has tiles.  The exchange of a round costs a
// cluster more than half of the round itself (2.5 us alone on two CTAs per
// SM, 3.3 us with four, 4.0 us with eight), so a grid that fills the SMs
// without clusters stays without (8 x 4096 x 2048: 80 us, 91 with two), and
// one that does not gains from every CTA (65536 x 2048: 257 us with eight).
// Packed sequences have one length on average and may have others, so a long
// average gets a cluster whatever the grid.
int cluster_size(const GatedArgs& a, int V) {
    constexpr int TILE = FWD_WARPS * 16;
    const long long units = state_rows(a) * ((a.C + 32 * V - 1) / (32 * V));
    const long long len = a.nseq > 0 ? (a.T + a.nseq - 1) / a.nseq : a.T, tiles = (len + TILE - 1) / TILE;
    long long S = 2LL * sm_count() / units;
    if (a.nseq > 0 && S < tiles / 4) S = tiles / 4;
    if (S > tiles) S = tiles;
    return static_cast<int>(S < 1 ? 1 : S > MAX_CLUSTER ? MAX_CLUSTER : S);
}

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

// One launch of a walk kernel over all (state row, slab) units.
template <typename... KArgs, typename... Args>
kdn_status launch_walk(void (*kernel)(KArgs...), int threads, long long rows, const Cut& cut, size_t smem, cudaStream_t stream,
                       Args... args) {
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess) return from_cuda(e);
    }
    const long long blocks = rows * cut.slabs * cut.S;
    if (blocks > 0x7fffffffLL) return KDN_ERR_INVALID_ARG;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(threads);
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

}  // namespace

long long gated_bwd_workspace_bytes(int B, int H, int T, int C, int nseq) {
    GatedArgs a{};
    a.B = B;
    a.H = H;
    a.T = T;
    a.C = C;
    a.nseq = nseq;
    return state_rows(a) * cluster_size(a, 2) * C * 4;   // (V = 1 makes clusters no larger)
}

kdn_status gated_fwd_launch(const GatedArgs& a, cudaStream_t stream, long long wait_ns) {
    const long long rows = state_rows(a);
    Cut cut{0, 1, wait_ns};
    return by_type(a, [&](auto ti, auto to) {
        using TI = decltype(ti);
        using TO = decltype(to);
        constexpr int V = std::is_same<TI, __nv_bfloat16>::value ? 2 : 1, K = 16, NW = FWD_WARPS;
        auto go = [&](auto kernel, int v, size_t smem) {
            cut.slabs = (a.C + 32 * v - 1) / (32 * v);
            cut.S = cluster_size(a, v);
            return launch_walk(kernel, NW * 32, rows, cut, smem, stream, a, cut);
        };
        auto leak = [&](auto l) {
            constexpr bool L = decltype(l)::value;
            if (rows_ok(a, 16))
                return go(gated_fwd_staged<TI, TO, V, K, NW, L, 16>, V, sizeof(FwdShared<TI, TO, V, K, NW>));
            if (rows_ok(a, 4))
                return go(gated_fwd_staged<TI, TO, V, K, NW, L, 4>, V, sizeof(FwdShared<TI, TO, V, K, NW>));
            return go(gated_fwd_kernel<TI, TO, 1, K, NW, L>, 1, 0);
        };
        return a.leak ? leak(std::true_type()) : leak(std::false_type());
    });
}

kdn_status gated_bwd_launch(const GatedArgs& a, cudaStream_t stream, long long wait_ns) {
    const long long rows = state_rows(a);
    Cut cut{0, 1, wait_ns};
    float* part = a.grad_A ? static_cast<float*>(a.workspace) : nullptr;
    const bool own = a.grad_A && !part;
    if (own) {
        const kdn_status s = from_cuda(cudaMallocAsync(&part, rows * cluster_size(a, 2) * a.C * 4, stream));
        if (s != KDN_OK) return s;
    }
    kdn_status s = by_type(a, [&](auto ti, auto to) {
        using TI = decltype(ti);
        using TO = decltype(to);
        constexpr int V = std::is_same<TI, __nv_bfloat16>::value ? 2 : 1, K = 8, NW = BWD_WARPS;
        auto go = [&](auto kernel, int v, size_t smem) {
            cut.slabs = (a.C + 32 * v - 1) / (32 * v);
            cut.S = cluster_size(a, v);
            return launch_walk(kernel, NW * 32, rows, cut, smem, stream, a, cut, part);
        };
        auto leak = [&](auto l) {
            constexpr bool L = decltype(l)::value;
            if (rows_ok(a, 16)) return go(gated_bwd_staged<TI, TO, V, K, NW, L, 16>, V, sizeof(BwdShared<TI, TO, V, K, NW>));
            if (rows_ok(a, 4)) return go(gated_bwd_staged<TI, TO, V, K, NW, L, 4>, V, sizeof(BwdShared<TI, TO, V, K, NW>));
            return go(gated_bwd_kernel<TI, TO, 1, K, NW, L>, 1, 0);
        };
        return a.leak ? leak(std::true_type()) : leak(std::false_type());
    });
    if (s == KDN_OK && a.grad_A) {
        const long long HC = static_cast<long long>(a.H) * a.C;
        s = from_cuda(sum_rows(part, rows / a.H * cut.S, HC, a.grad_A, nullptr, HC, stream));
    }
    if (own) {
        const kdn_status f = from_cuda(cudaFreeAsync(part, stream));
        if (s == KDN_OK) s = f;
    }
    return s;
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
    const long long blocks = (n + THREADS - 1) / THREADS;
    if (blocks > 0x7fffffffLL) return KDN_ERR_INVALID_ARG;
    GatedArgs t{};
    t.in_dtype = in_dtype;
    t.out_dtype = out_dtype;
    return by_type(t, [&](auto ti, auto to) {
        using TI = decltype(ti);
        using TO = decltype(to);
        gated_step_kernel<TI, TO><<<static_cast<unsigned>(blocks), THREADS, 0, stream>>>(
            static_cast<const TI*>(x), static_cast<const TI*>(d), A, leak, state, new_state,
            static_cast<TO*>(out), n, HC);
        return from_cuda(cudaGetLastError());
    });
}

}  // namespace kdn
