// gated_scan.cu -- the gated recurrence with one gate per channel,
//     h_t = alpha_t h_{t-1} + w_t x_t,  alpha_t = exp(-A d_t),  w_t = 1 or
//     1 - alpha_t ("Kalman Linear Attention (KLA)", Metodologia 2: the affine
//     recursion of the information mean),
// its backward pass and its one-token step.
//
// Backward, with u_t = alpha_t (g_t + u_{t+1}) the gradient that reaches
// h_{t-1} (g the incoming gradient, u_T+1 the final state's):
//     grad x_t = w_t (g_t + u_{t+1}),   grad d_t = -A u_t (h_{t-1} - leak x_t),
//     grad A = -sum d_t u_t (h_{t-1} - leak x_t),   grad h_0 = u_0.
//
// A thread walks one channel of one sequence.
#include <cstdint>

#include "gated_device.cuh"
#include "kdn_internal.h"

namespace kdn {
namespace {

using namespace gated;

constexpr int THREADS = 128;

// The tokens of state row n (a batch, or a packed sequence): [lo, hi) of the
// T-token row `row`.
struct Span {
    long long row;
    int lo, hi;
};

__device__ __forceinline__ Span span_of(const int* offsets, int H, int T, long long n, int h) {
    Span s{n * H + h, 0, T};
    if (offsets) {
        s.row = h;
        s.lo = min(max(offsets[n], 0), T);
        s.hi = min(max(offsets[n + 1], s.lo), T);
    }
    return s;
}

template <typename TI, typename TO, bool LEAK>
__global__ void __launch_bounds__(THREADS) gated_fwd_kernel(GatedArgs p) {
    const int cb = (p.C + THREADS - 1) / THREADS;
    const int c = static_cast<int>(blockIdx.x % cb) * THREADS + threadIdx.x;
    if (c >= p.C) return;
    const long long sr = blockIdx.x / cb;                  // state row n*H + h
    const long long n = sr / p.H;
    const int hd = static_cast<int>(sr - n * p.H);
    const Span s = span_of(p.offsets, p.H, p.T, n, hd);
    const float nA = -p.A[static_cast<long long>(hd) * p.C + c];
    float h = p.h0 ? p.h0[sr * p.C + c] : 0.f;
    for (int t = s.lo; t < s.hi; ++t) {
        const long long r = s.row * p.T + t;
        const float x = to_f32(static_cast<const TI*>(p.x)[r * p.x_ld + c]);
        const Gate g = gate(nA * to_f32(static_cast<const TI*>(p.d)[r * p.d_ld + c]));
        h = decay_add(g, h, LEAK ? g.w * x : x);
        static_cast<TO*>(p.out)[r * p.C + c] = from_f32<TO>(h);
    }
    if (p.final_state) p.final_state[sr * p.C + c] = h;
}

template <typename TI, typename TO, bool LEAK>
__global__ void __launch_bounds__(THREADS) gated_bwd_kernel(GatedArgs p, float* part) {
    const int cb = (p.C + THREADS - 1) / THREADS;
    const int c = static_cast<int>(blockIdx.x % cb) * THREADS + threadIdx.x;
    if (c >= p.C) return;
    const long long sr = blockIdx.x / cb;
    const long long n = sr / p.H;
    const int hd = static_cast<int>(sr - n * p.H);
    const Span s = span_of(p.offsets, p.H, p.T, n, hd);
    const float nA = -p.A[static_cast<long long>(hd) * p.C + c];
    float u = p.grad_final_state ? p.grad_final_state[sr * p.C + c] : 0.f;
    float dA = 0.f;
    for (int t = s.hi - 1; t >= s.lo; --t) {
        const long long r = s.row * p.T + t;
        const float d = to_f32(static_cast<const TI*>(p.d)[r * p.d_ld + c]);
        const Gate g = gate(nA * d);
        float prev = t > s.lo ? to_f32(static_cast<const TO*>(p.out)[(r - 1) * p.C + c])
                              : (p.h0 ? p.h0[sr * p.C + c] : 0.f);
        if (LEAK) prev -= to_f32(static_cast<const TI*>(p.x)[r * p.x_ld + c]);
        const float dh = to_f32(static_cast<const TO*>(p.grad_out)[r * p.C + c]) + u;
        u = fmaf(g.a, dh, g.e * dh);
        const float m = u * prev;
        dA = fmaf(-d, m, dA);
        static_cast<TI*>(p.grad_x)[r * p.C + c] = from_f32<TI>(LEAK ? g.w * dh : dh);
        static_cast<TI*>(p.grad_d)[r * p.C + c] = from_f32<TI>(nA * m);
    }
    if (p.grad_h0) p.grad_h0[sr * p.C + c] = u;
    if (part) part[sr * p.C + c] = dA;
}

// grad A: the state rows' sums of one head, in order
__global__ void __launch_bounds__(THREADS)
gated_dA_kernel(const float* __restrict__ part, float* __restrict__ grad_A, long long rows, int H, int C) {
    const int c = blockIdx.x * THREADS + threadIdx.x;
    if (c >= C) return;
    const int hd = blockIdx.y;
    float s = 0.f;
    for (long long r = hd; r < rows; r += H) s += part[r * C + c];
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

}  // namespace

long long gated_bwd_workspace_bytes(int B, int H, int, int C, int nseq) {
    return static_cast<long long>(nseq > 0 ? nseq : B) * H * C * 4;
}

kdn_status gated_fwd_launch(const GatedArgs& a, cudaStream_t stream) {
    const long long rows = static_cast<long long>(a.nseq > 0 ? a.nseq : a.B) * a.H;
    const long long blocks = rows * ((a.C + THREADS - 1) / THREADS);
    if (blocks > 0x7fffffffLL) return KDN_ERR_INVALID_ARG;
    const unsigned grid = static_cast<unsigned>(blocks);
    return by_type(a, [&](auto ti, auto to) {
        using TI = decltype(ti);
        using TO = decltype(to);
        if (a.leak) gated_fwd_kernel<TI, TO, true><<<grid, THREADS, 0, stream>>>(a);
        else gated_fwd_kernel<TI, TO, false><<<grid, THREADS, 0, stream>>>(a);
        return from_cuda(cudaGetLastError());
    });
}

kdn_status gated_bwd_launch(const GatedArgs& a, cudaStream_t stream) {
    const long long rows = static_cast<long long>(a.nseq > 0 ? a.nseq : a.B) * a.H;
    const int cb = (a.C + THREADS - 1) / THREADS;
    if (rows * cb > 0x7fffffffLL) return KDN_ERR_INVALID_ARG;
    const unsigned grid = static_cast<unsigned>(rows * cb);
    float* part = static_cast<float*>(a.workspace);
    if (a.grad_A && !part) {
        const kdn_status s = from_cuda(cudaMallocAsync(&part, rows * a.C * 4, stream));
        if (s != KDN_OK) return s;
    }
    kdn_status s = by_type(a, [&](auto ti, auto to) {
        using TI = decltype(ti);
        using TO = decltype(to);
        if (a.leak) gated_bwd_kernel<TI, TO, true><<<grid, THREADS, 0, stream>>>(a, a.grad_A ? part : nullptr);
        else gated_bwd_kernel<TI, TO, false><<<grid, THREADS, 0, stream>>>(a, a.grad_A ? part : nullptr);
        return from_cuda(cudaGetLastError());
    });
    if (s == KDN_OK && a.grad_A) {
        const dim3 g2(cb, a.H);
        gated_dA_kernel<<<g2, THREADS, 0, stream>>>(part, a.grad_A, rows, a.H, a.C);
        s = from_cuda(cudaGetLastError());
    }
    if (part && part != a.workspace) {
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
