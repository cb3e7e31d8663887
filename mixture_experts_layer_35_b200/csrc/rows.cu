// rows.cu -- tokens sorted by expert and back, with their gradients.
//
//   dispatch           xs[inv[k, m]] = x[m]
//   combine            y[m] = sum_k w[m, k] ys[inv[k, m]]      (w = 1: the gradient of dispatch)
//   combine backward   dys[inv[k, m]] = w[m, k] dy[m],  dw[m, k] = <dy[m], ys[inv[k, m]]>
//
// All three go token by token, so that the [M, H] side moves once and only the [P, H] side
// carries the top-k factor; a gather by sorted rows would read each token K times.  Rows
// move in 16-byte chunks, each warp taking 32 * U neighbouring chunks of one token.  They
// are bound by memory.  A slot whose row lies outside [0, P) was dropped: it is not written, adds
// nothing, and its weight's gradient is zero.  Sums are FP32, over k in ascending order,
// rounded once; nothing is accumulated with atomics, so results do not change from run to run.
// Measured: dispatch of 8192 x 2560, top 10, 8 % of the slots dropped, 69 us (96 % of the copy rate); combine of
// 4096 x 2048, top 8, 28 us (83 %) and without weights 27 us; its gradient in FP32, 2047 x 2688, top 6, 49 us (90 %).
#include "experts.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Rows of token m's slots: lane k holds inv[k, m], or -1 for a dropped one.
__device__ __forceinline__ int slot_row(const RowsArgs& a, int m, int lane) {
    const int p = lane < a.K ? a.inv[(size_t)lane * a.M + m] : -1;
    return (unsigned)p < (unsigned)a.P ? p : -1;
}

template <typename T, int U>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const RowsArgs a) {
    chain();
    const int lane = threadIdx.x & 31;
    const int nch = a.H / Chunk<T>::V, spans = cdiv(nch, 32 * U);
    const long long n = (long long)a.M * spans, step = (long long)gridDim.x * (kThreads / 32);
    const uint4* x = static_cast<const uint4*>(a.src);
    uint4* xs = static_cast<uint4*>(a.dst);
    for (long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < n; i += step) {
        const int m = (int)(i / spans), c0 = (int)(i - (long long)m * spans) * 32 * U + lane;
        const int row = slot_row(a, m, lane);
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + 32 * u < nch) v[u] = ld_stream16(x + (size_t)m * nch + c0 + 32 * u);
        for (int k = 0; k < a.K; ++k) {
            const int p = __shfl_sync(0xffffffffu, row, k);
            if (p < 0) continue;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + 32 * u < nch) xs[(size_t)p * nch + c0 + 32 * u] = v[u];
        }
    }
}

// Eight loads in flight per lane; the next token's rows and weights are loaded meanwhile.
template <typename T, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads, 4) combine_kernel(const RowsArgs a) {
    chain();
    constexpr int V = Chunk<T>::V, KU = 8;
    const int lane = threadIdx.x & 31;
    const int nch = a.H / V, spans = cdiv(nch, 32);
    const long long n = (long long)a.M * spans, step = (long long)gridDim.x * (kThreads / 32);
    const uint4* ys = static_cast<const uint4*>(a.src);
    uint4* y = static_cast<uint4*>(a.dst);
    long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    int row = -1;
    float wt = 1.0f;
    auto load_slots = [&](long long unit) {
        const int m = (int)(unit / spans);
        row = slot_row(a, m, lane);
        if (WEIGHTED && lane < a.K) wt = a.w[(size_t)m * a.K + lane];
    };
    if (i < n) load_slots(i);
    for (; i < n; i += step) {
        const int m = (int)(i / spans), c = (int)(i - (long long)m * spans) * 32 + lane;
        const bool in = c < nch;
        const int row_m = row;
        const float wt_m = wt;
        float acc[V];
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = 0.0f;
        for (int k0 = 0; k0 < a.K; k0 += KU) {
            uint4 v[KU];
            uint32_t use = 0;
#pragma unroll
            for (int kk = 0; kk < KU; ++kk) {
                const int p = __shfl_sync(0xffffffffu, row_m, (k0 + kk) & 31);
                if (k0 + kk < a.K && p >= 0) {
                    use |= 1u << kk;
                    if (in) v[kk] = ld_stream16(ys + (size_t)p * nch + c);
                }
            }
            if (k0 == 0 && i + step < n) load_slots(i + step);
#pragma unroll
            for (int kk = 0; kk < KU; ++kk) {
                const float w = WEIGHTED ? __shfl_sync(0xffffffffu, wt_m, (k0 + kk) & 31) : 1.0f;
                if (!(use >> kk & 1u)) continue;
                float f[V];
                Chunk<T>::unpack(v[kk], f);
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] = WEIGHTED ? fmaf(w, f[j], acc[j]) : acc[j] + f[j];
            }
        }
        if (in) y[(size_t)m * nch + c] = Chunk<T>::pack(acc);
    }
}

// One warp per slot, slots of a token next to each other, so that a token's dy row is read
// from memory once and from L1 by the other slots' warps of the block.
template <typename T>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const RowsArgs a) {
    chain();
    constexpr int V = Chunk<T>::V, U = 4;
    const int lane = threadIdx.x & 31;
    const int nch = a.H / V;
    const long long n = (long long)a.M * a.K, step = (long long)gridDim.x * (kThreads / 32);
    const uint4* dy = static_cast<const uint4*>(a.dy);
    const uint4* ys = static_cast<const uint4*>(a.src);
    uint4* dys = static_cast<uint4*>(a.dst);
    for (long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < n; i += step) {
        const int m = (int)(i / a.K), k = (int)(i - (long long)m * a.K);
        const int p = a.inv[(size_t)k * a.M + m];
        float dot = 0.0f;
        if ((unsigned)p < (unsigned)a.P) {
            const float w = a.w[i];
            for (int c0 = lane; c0 < nch; c0 += 32 * U) {
                uint4 g[U], v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool in = c0 + 32 * u < nch;
                    g[u] = in ? ld_nc16(dy + (size_t)m * nch + c0 + 32 * u) : make_uint4(0, 0, 0, 0);
                    v[u] = in ? ld_stream16(ys + (size_t)p * nch + c0 + 32 * u) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (c0 + 32 * u >= nch) continue;
                    float gf[V], vf[V];
                    Chunk<T>::unpack(g[u], gf);
                    Chunk<T>::unpack(v[u], vf);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        dot = fmaf(gf[j], vf[j], dot);
                        gf[j] = __fmul_rn(w, gf[j]);
                    }
                    dys[(size_t)p * nch + c0 + 32 * u] = Chunk<T>::pack(gf);
                }
            }
            dot = warp_sum(dot);
        }
        if (lane == 0) a.dw[i] = dot;
    }
}

int grid_for(long long warps, int sms, int blocks_per_sm) {
    const long long blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    return (int)std::max<long long>(1, std::min<long long>(blocks, (long long)sms * blocks_per_sm));
}

template <typename T>
cudaError_t dispatch_t(const RowsArgs& a, int sms, cudaStream_t s) {
    const int nch = a.H / Chunk<T>::V;
    if ((long long)a.M * cdiv(nch, 128) >= 8LL * sms)
        return launch_k(dispatch_kernel<T, 4>, dim3(grid_for((long long)a.M * cdiv(nch, 128), sms, 32)), dim3(kThreads),
                        0, s, true, a);
    return launch_k(dispatch_kernel<T, 1>, dim3(grid_for((long long)a.M * cdiv(nch, 32), sms, 8)), dim3(kThreads), 0, s, true, a);
}
template <typename T, bool WEIGHTED>
cudaError_t combine_t(const RowsArgs& a, int sms, cudaStream_t s) {
    const long long n = (long long)a.M * cdiv(a.H / Chunk<T>::V, 32);
    return launch_k(combine_kernel<T, WEIGHTED>, dim3(grid_for(n, sms, 4)), dim3(kThreads), 0, s, true, a);
}

}  // namespace

cudaError_t launch_dispatch(const RowsArgs& a, bool f32, int sms, cudaStream_t s) {
    return f32 ? dispatch_t<float>(a, sms, s) : dispatch_t<bf16>(a, sms, s);
}
cudaError_t launch_combine(const RowsArgs& a, bool f32, int sms, cudaStream_t s) {
    if (a.w) return f32 ? combine_t<float, true>(a, sms, s) : combine_t<bf16, true>(a, sms, s);
    return f32 ? combine_t<float, false>(a, sms, s) : combine_t<bf16, false>(a, sms, s);
}
cudaError_t launch_combine_backward(const RowsArgs& a, bool f32, int sms, cudaStream_t s) {
    const int grid = grid_for((long long)a.M * a.K, sms, 8);
    if (f32) return launch_k(combine_backward_kernel<float>, dim3(grid), dim3(kThreads), 0, s, true, a);
    return launch_k(combine_backward_kernel<bf16>, dim3(grid), dim3(kThreads), 0, s, true, a);
}

}  // namespace moe
