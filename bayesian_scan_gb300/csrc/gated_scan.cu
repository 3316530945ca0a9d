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
// of WARPS * K.  A warp composes its tokens from a zero state (the affine map
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
#include <cooperative_groups.h>

#include <type_traits>

#include "gated_device.cuh"
#include "kdn_internal.h"

namespace kdn {
namespace {

namespace cg = cooperative_groups;
using namespace gated;

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int MAX_CLUSTER = 8;

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
};

// An affine map h -> (a + e) h + s of one channel over a span of tokens.
struct __align__(16) Map {
    float a, e, s, z;      // z: the exponent's sum, alpha = exp(z)
};

__device__ __forceinline__ Map map_of(float z, float s) {
    const Gate g = gate(z);
    return Map{g.a, g.e, s, z};
}
__device__ __forceinline__ float apply(const Map& m, float h) { return decay_add(m.a, m.e, h, m.s); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Folding the maps of a round.  Every warp hands in its map; on return
// `start` is the state before the warp's tokens and `carry` the one after the
// round's last tile, both from the carry before the round.
template <int V>
struct Fold {
    Map warp[2][WARPS][V][32];
    Map cta[2][MAX_CLUSTER][V][32];
};

template <int V>
__device__ __forceinline__ void fold_round(Fold<V>& f, int buf, int S, int rank, int warp, int lane,
                                           const float (&z)[V], const float (&s)[V], float (&carry)[V],
                                           float (&start)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) f.warp[buf][warp][v][lane] = map_of(z[v], s[v]);
    __syncthreads();
    if (S > 1) {
        // warp j sends the tile's map to CTA j
        if (warp < S) {
            cg::cluster_group cl = cg::this_cluster();
            Map* to = cl.map_shared_rank(&f.cta[buf][rank][0][lane], warp);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float h = 0.f, zz = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const Map m = f.warp[buf][w][v][lane];
                    h = apply(m, h);
                    zz += m.z;
                }
                to[v * 32] = map_of(zz, h);
            }
        }
        cluster_arrive();
        cluster_wait();
        float c[V];
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = start[v] = carry[v];
        for (int j = 0; j < S; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (j == rank) start[v] = c[v];
                c[v] = apply(f.cta[buf][j][v][lane], c[v]);
            }
#pragma unroll
        for (int v = 0; v < V; ++v) carry[v] = c[v];
        for (int w = 0; w < warp; ++w)
#pragma unroll
            for (int v = 0; v < V; ++v) start[v] = apply(f.warp[buf][w][v][lane], start[v]);
    } else {
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (w == warp) start[v] = carry[v];
                carry[v] = apply(f.warp[buf][w][v][lane], carry[v]);
            }
    }
}

// Pairs of gates: two channels of a token, or (V = 1) two tokens of a channel.
template <int V, int K>
struct Gates {
    float a[K][V];
    uint32_t e[K * V / 2];   // bf16 pairs: e is under 2^-25, three digits of it are plenty
    __device__ __forceinline__ F2 err(int i) const {
        return F2{__uint_as_float(e[i] << 16), __uint_as_float(e[i] & 0xffff0000u)};
    }
    __device__ __forceinline__ float err1(int k, int v) const {
        const F2 f = err((k * V + v) / 2);
        return (k * V + v) & 1 ? f.y : f.x;
    }
    __device__ __forceinline__ void put(int i, F2 x) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
        e[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
};

template <typename TI, typename TO, int V, int K, bool LEAK>
__global__ void __launch_bounds__(THREADS, 2) gated_fwd_kernel(const GatedArgs p, const Cut cut) {
    __shared__ Fold<V> fold;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = cut.S, rank = blockIdx.x % S;
    const long long unit = blockIdx.x / S;
    const long long sr = unit / cut.slabs;
    const int c = (static_cast<int>(unit - sr * cut.slabs) * 32 + lane) * V;
    const bool on = c < p.C;
    const Span sp = span_of(p, sr);
    const int rounds = (sp.hi - sp.lo + S * WARPS * K - 1) / (S * WARPS * K);
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
        const int t = sp.lo + ((r * S + rank) * WARPS + warp) * K;
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
    if (S > 1) {   // every CTA of the cluster runs before its shared memory is written
        cluster_arrive();
        cluster_wait();
    }
    for (int r = 0; r < rounds; ++r) {
        const int t = sp.lo + ((r * S + rank) * WARPS + warp) * K;
        // tokens behind the end have d = x = 0: alpha = 1, nothing added
        Gates<V, K> g;
        float b[K][V], z[V], s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = s[v] = 0.f;
#pragma unroll
        for (int i = 0; i < K * V / 2; ++i) {
            const int k0 = 2 * i / V, v0 = 2 * i % V, k1 = (2 * i + 1) / V, v1 = (2 * i + 1) % V;
            const F2 zz = mul2(F2{nA[v0], nA[v1]}, F2{dr[k0].get(v0), dr[k1].get(v1)});
            const Gate2 gg = gate2(zz);
            g.a[k0][v0] = gg.a.x;
            g.a[k1][v1] = gg.a.y;
            g.put(i, gg.e);
            F2 x{xr[k0].get(v0), xr[k1].get(v1)};
            if (LEAK) x = mul2(x, gg.w);
            b[k0][v0] = x.x;
            b[k1][v1] = x.y;
            if (V == 1) {
                z[0] += zz.x + zz.y;
                s[0] = decay_add(gg.a.x, gg.e.x, s[0], x.x);
                s[0] = decay_add(gg.a.y, gg.e.y, s[0], x.y);
            } else {
                const F2 ss{s[v0], s[v1]};
                const F2 n = fma2(gg.a, ss, fma2(gg.e, ss, x)), zs = add2(F2{z[v0], z[v1]}, zz);
                s[v0] = n.x;
                s[v1] = n.y;
                z[v0] = zs.x;
                z[v1] = zs.y;
            }
        }
        if (r + 1 < rounds) fetch(r + 1);
        float h[V];
        fold_round<V>(fold, r & 1, S, rank, warp, lane, z, s, carry, h);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (V == 1) {
                h[0] = decay_add(g.a[k][0], g.err1(k, 0), h[0], b[k][0]);
            } else {
#pragma unroll
                for (int v = 0; v < V; v += 2) {
                    const F2 hh{h[v], h[v + 1]};
                    const F2 n = fma2(F2{g.a[k][v], g.a[k][v + 1]}, hh,
                                      fma2(g.err((k * V + v) / 2), hh, F2{b[k][v], b[k][v + 1]}));
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
    if (p.final_state && rank == 0 && warp == 0 && on)
#pragma unroll
        for (int v = 0; v < V; ++v) p.final_state[sr * p.C + c + v] = carry[v];
}

// The same walk from the last token to the first.  `part` [state row, rank, C]
// takes each CTA's share of grad A.
template <typename TI, typename TO, int V, int K, bool LEAK>
__global__ void __launch_bounds__(THREADS, 2)
gated_bwd_kernel(const GatedArgs p, const Cut cut, float* part) {
    __shared__ Fold<V> fold;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = cut.S, rank = blockIdx.x % S;
    const long long unit = blockIdx.x / S;
    const long long sr = unit / cut.slabs;
    const int c = (static_cast<int>(unit - sr * cut.slabs) * 32 + lane) * V;
    const bool on = c < p.C;
    const Span sp = span_of(p, sr);
    const int rounds = (sp.hi - sp.lo + S * WARPS * K - 1) / (S * WARPS * K);
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
        const int t = sp.hi - 1 - ((r * S + rank) * WARPS + warp) * K;
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
    if (S > 1) {
        cluster_arrive();
        cluster_wait();
    }
    for (int r = 0; r < rounds; ++r) {
        const int t = sp.hi - 1 - ((r * S + rank) * WARPS + warp) * K;
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
        Gates<V, K> g;
        float z[V], s[V], w[LEAK ? K : 1][V];
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = s[v] = 0.f;
        // u = alpha (g + u): the map of a token is (alpha, alpha g)
#pragma unroll
        for (int i = 0; i < K * V / 2; ++i) {
            const int k0 = 2 * i / V, v0 = 2 * i % V, k1 = (2 * i + 1) / V, v1 = (2 * i + 1) % V;
            const F2 zz = mul2(F2{nA[v0], nA[v1]}, F2{dr[k0].get(v0), dr[k1].get(v1)});
            const Gate2 gg = gate2(zz);
            g.a[k0][v0] = gg.a.x;
            g.a[k1][v1] = gg.a.y;
            if (LEAK) {   // e follows from w
                w[LEAK ? k0 : 0][v0] = gg.w.x;
                w[LEAK ? k1 : 0][v1] = gg.w.y;
            } else {
                g.put(i, gg.e);
            }
            if (V == 1) {
                z[0] += zz.x + zz.y;
                const float d0 = s[0] + gr[k0].get(0);
                s[0] = decay_add(gg.a.x, gg.e.x, d0, 0.f);
                const float d1 = s[0] + gr[k1].get(0);
                s[0] = decay_add(gg.a.y, gg.e.y, d1, 0.f);
            } else {
                const F2 dh = add2(F2{s[v0], s[v1]}, F2{gr[k0].get(v0), gr[k0].get(v1)});
                const F2 n = fma2(gg.a, dh, mul2(gg.e, dh)), zs = add2(F2{z[v0], z[v1]}, zz);
                s[v0] = n.x;
                s[v1] = n.y;
                z[v0] = zs.x;
                z[v1] = zs.y;
            }
        }
        if (r + 1 < rounds) fetch(r + 1);
        float u[V];
        fold_round<V>(fold, r & 1, S, rank, warp, lane, z, s, carry, u);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float gx[V], gd[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float a = g.a[k][v], e = LEAK ? -w[LEAK ? k : 0][v] - (a - 1.f) : g.err1(k, v);
                const float dh = u[v] + gr[k].get(v);
                u[v] = fmaf(a, dh, e * dh);
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
    if (p.grad_h0 && rank == 0 && warp == 0 && on)
#pragma unroll
        for (int v = 0; v < V; ++v) p.grad_h0[sr * p.C + c + v] = carry[v];
    if (part) {
        // the warps' shares, in order
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) fold.warp[0][warp][v][lane].s = dA[v];
        __syncthreads();
        if (warp == 0 && on)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float sum = 0.f;
                for (int w = 0; w < WARPS; ++w) sum += fold.warp[0][w][v][lane].s;
                part[(sr * S + rank) * p.C + c + v] = sum;
            }
    }
}

// grad A: the shares of one head's state rows, in order.
__global__ void __launch_bounds__(THREADS)
gated_dA_kernel(const float* __restrict__ part, float* __restrict__ grad_A, long long rows, int H, int C, int S) {
    const int cb = (C + THREADS - 1) / THREADS;
    const int c = static_cast<int>(blockIdx.x % cb) * THREADS + threadIdx.x;
    if (c >= C) return;
    const int hd = blockIdx.x / cb;
    float s = 0.f;
    for (long long r = hd; r < rows; r += H)
        for (int j = 0; j < S; ++j) s += part[(r * S + j) * C + c];
    grad_A[static_cast<long long>(hd) * C + c] = s;
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

// CTAs per cluster: enough to fill the GPU's two CTAs per SM, no more than
// the sequence has tiles.
int cluster_size(long long rows, int C, int T) {
    const long long slabs = (C + 63) / 64, want = 2LL * sm_count();
    int S = 1;
    while (S < MAX_CLUSTER && rows * slabs * S < want && S * 128 < T) S *= 2;
    return S;
}

// Whether every row of every tensor takes V-element accesses.
bool vector_ok(const GatedArgs& a, int V) {
    if (a.C % V) return false;
    const uintptr_t is = (a.in_dtype == KDN_BF16 ? 2 : 4) * V, os = (a.out_dtype == KDN_BF16 ? 2 : 4) * V;
    const void* ins[] = {a.x, a.d, a.grad_x, a.grad_d};
    const void* outs[] = {a.out, a.grad_out};
    for (const void* q : ins)
        if (reinterpret_cast<uintptr_t>(q) % is) return false;
    for (const void* q : outs)
        if (reinterpret_cast<uintptr_t>(q) % os) return false;
    return (!a.x || a.x_ld % V == 0) && a.d_ld % V == 0;
}

// One launch of a walk kernel over all (state row, slab) units.
template <typename... KArgs, typename... Args>
kdn_status launch_walk(void (*kernel)(KArgs...), long long rows, const Cut& cut, cudaStream_t stream, Args... args) {
    const long long blocks = rows * cut.slabs * cut.S;
    if (blocks > 0x7fffffffLL) return KDN_ERR_INVALID_ARG;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(THREADS);
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
    const long long rows = static_cast<long long>(nseq > 0 ? nseq : B) * H;
    return rows * cluster_size(rows, C, T) * C * 4;
}

kdn_status gated_fwd_launch(const GatedArgs& a, cudaStream_t stream) {
    const long long rows = state_rows(a);
    Cut cut{0, cluster_size(rows, a.C, a.T)};
    return by_type(a, [&](auto ti, auto to) {
        using TI = decltype(ti);
        using TO = decltype(to);
        constexpr int VV = std::is_same<TI, __nv_bfloat16>::value ? 2 : 1;
        auto go = [&](auto kernel, int V) {
            cut.slabs = (a.C + 32 * V - 1) / (32 * V);
            return launch_walk(kernel, rows, cut, stream, a, cut);
        };
        if (VV > 1 && vector_ok(a, VV))
            return a.leak ? go(gated_fwd_kernel<TI, TO, VV, 16, true>, VV)
                          : go(gated_fwd_kernel<TI, TO, VV, 16, false>, VV);
        return a.leak ? go(gated_fwd_kernel<TI, TO, 1, 16, true>, 1)
                      : go(gated_fwd_kernel<TI, TO, 1, 16, false>, 1);
    });
}

kdn_status gated_bwd_launch(const GatedArgs& a, cudaStream_t stream) {
    const long long rows = state_rows(a);
    Cut cut{0, cluster_size(rows, a.C, a.T)};
    float* part = a.grad_A ? static_cast<float*>(a.workspace) : nullptr;
    const bool own = a.grad_A && !part;
    if (own) {
        const kdn_status s = from_cuda(cudaMallocAsync(&part, rows * cut.S * a.C * 4, stream));
        if (s != KDN_OK) return s;
    }
    kdn_status s = by_type(a, [&](auto ti, auto to) {
        using TI = decltype(ti);
        using TO = decltype(to);
        constexpr int VV = std::is_same<TI, __nv_bfloat16>::value ? 2 : 1;
        auto go = [&](auto kernel, int V) {
            cut.slabs = (a.C + 32 * V - 1) / (32 * V);
            return launch_walk(kernel, rows, cut, stream, a, cut, part);
        };
        if (VV > 1 && vector_ok(a, VV))
            return a.leak ? go(gated_bwd_kernel<TI, TO, VV, 8, true>, VV)
                          : go(gated_bwd_kernel<TI, TO, VV, 8, false>, VV);
        return a.leak ? go(gated_bwd_kernel<TI, TO, 1, 8, true>, 1)
                      : go(gated_bwd_kernel<TI, TO, 1, 8, false>, 1);
    });
    if (s == KDN_OK && a.grad_A) {
        const long long blocks = static_cast<long long>((a.C + THREADS - 1) / THREADS) * a.H;
        gated_dA_kernel<<<static_cast<unsigned>(blocks), THREADS, 0, stream>>>(part, a.grad_A, rows, a.H, a.C, cut.S);
        s = from_cuda(cudaGetLastError());
    }
    if (own) {
        const kdn_status f = from_cuda(cudaFreeAsync(part, stream));
        if (s == KDN_OK) s = f;
    }
    return s;
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
