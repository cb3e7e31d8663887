// quantize.cu -- 8-bit blocks with one FP32 scale each, and the activation between an
// expert's two products.
//
// A block's largest magnitude a gives its scale s = a / fmax and its values
// q = round(v * (fmax / a)) (to nearest even, e4m3: fmax 448, e5m2: fmax 57344); v ~ s q.
//   rows      1 x 128: the A operand of a product over the columns
//   columns   128 x 1 inside each expert: the operands of the weight gradient (contraction over rows)
//   blocks    128 x 128: weights
// Every value is read once, kept in registers between the maximum and the rounding, and
// written once; all of them are bound by memory.  Measured: rows 32768 x 2048 44 us (71 % of the copy
// rate), quantised dispatch of 8192 x 2560, top 10, 52 us (77 %), columns 24570 x 1856 of 128 experts 36.6 us
// (58 %), blocks 128 x 1856 x 2688 322 us (92 %); SwiGLU of 32768 x 512 18 us (85 %), to 8 bits 19 us (70 %), its
// gradient 30 us (88 %); ReLU^2 of 24576 x 1856 31 us (92 %).
#include "experts.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t amax8(const float (&f)[8], uint32_t m) {
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(f[j]));
    return m;
}

// Sixteen lanes take the 128 columns of one block, eight each; a warp takes two neighbouring
// blocks of a row, U times.
template <typename T, int SRC, bool QUANT, bool E5M2, int U>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantArgs a) {
    chain();
    const int lane = threadIdx.x & 31, sub = lane >> 4;
    const int nb = cdiv(a.C, kQBlock), spans = cdiv(nb, 2 * U);
    const int ld = SRC == QS_SWIGLU ? 2 * a.C : a.C;
    const long long n = (long long)a.M * spans, step = (long long)gridDim.x * (kThreads / 32);
    const T* src = static_cast<const T*>(a.src);
    const float fmax = fp8_max(E5M2);
    for (long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < n; i += step) {
        const int m = (int)(i / spans), b0 = (int)(i - (long long)m * spans) * 2 * U + sub;
        int row = -1;
        if (QUANT && a.inv) {
            row = lane < a.K ? a.inv[(size_t)lane * a.M + m] : -1;
            if ((unsigned)row >= (unsigned)a.P) row = -1;
        }
        Raw8<T> v[U], w[SRC == QS_SWIGLU ? U : 1];  // as they lie: all loads in flight at once
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (b0 + 2 * u) * kQBlock + (lane & 15) * 8;
            v[u].zero();
            if (SRC == QS_SWIGLU) w[SRC == QS_SWIGLU ? u : 0].zero();
            if (c < a.C) {
                v[u].load(src + (size_t)m * ld + c);
                if (SRC == QS_SWIGLU) w[SRC == QS_SWIGLU ? u : 0].load(src + (size_t)m * ld + a.C + c);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + 2 * u, c = b * kQBlock + (lane & 15) * 8;
            float f[8];
            v[u].get(f);
            if (SRC == QS_SWIGLU) {
                float g[8];
                w[SRC == QS_SWIGLU ? u : 0].get(g);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = quick_swiglu(f[j], g[j]);
            } else if (SRC == QS_RELU2) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = relu2_nan(f[j]);
            }
            if (!QUANT) {
                if (c < a.C) store8(static_cast<T*>(a.h) + (size_t)m * a.C + c, f);
                continue;
            }
            uint32_t mx = amax8(f, 0u);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            float scale, factor;
            block_scale(mx, fmax, scale, factor);
            const uint2 out = pack8_fp8<E5M2>(f, factor);
            for (int k = 0; k < a.K; ++k) {
                const int p = a.inv ? __shfl_sync(0xffffffffu, row, k) : m;
                if (p < 0) continue;
                if (c < a.C) *reinterpret_cast<uint2*>(a.q + (size_t)p * a.C + c) = out;
                if ((lane & 15) == 0 && b < nb) a.scales[(size_t)p * nb + b] = scale;
            }
        }
    }
}

// 128 x 128 weight blocks, one per CTA: thread t takes columns 8 (t % 16) .. + 7 of rows
// t / 16 + 16 i.
template <typename T, bool E5M2>
__global__ void __launch_bounds__(kThreads) quantize_blocks_kernel(const T* __restrict__ w, int N, int C,
                                                                   uint8_t* __restrict__ q,
                                                                   float* __restrict__ scales) {
    __shared__ uint32_t s_max[kThreads / 32];
    chain();
    const int nk = cdiv(C, kQBlock), nn = cdiv(N, kQBlock);
    const int kb = blockIdx.x % nk, rest = blockIdx.x / nk, nb = rest % nn, e = rest / nn;
    const int c = kb * kQBlock + (threadIdx.x & 15) * 8, r0 = nb * kQBlock + (threadIdx.x >> 4);
    const size_t base = (size_t)e * N * C;
    Raw8<T> v[8];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i].zero();
        if (c < C && r0 + 16 * i < N) v[i].load(w + base + (size_t)(r0 + 16 * i) * C + c);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        v[i].get(f);
        mx = amax8(f, mx);
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) mx = max(mx, s_max[i]);
    float scale, factor;
    block_scale(mx, fp8_max(E5M2), scale, factor);
    if (threadIdx.x == 0) scales[blockIdx.x] = scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        v[i].get(f);
        if (c < C && r0 + 16 * i < N)
            *reinterpret_cast<uint2*>(q + base + (size_t)(r0 + 16 * i) * C + c) = pack8_fp8<E5M2>(f, factor);
    }
}

// 128-row blocks inside each expert, 128 columns at a time: as quantize_blocks, but the
// maximum is one per column, and rows past the expert's end are written as zeros.  Offsets may reach
// past the P rows (a row limit).  The weight gradient, which reads these blocks, knows the room for
// them alone and not P, so the blocks are laid out by offsets clamped to the room here too, and one whose
// rows are all missing is written as zeros, its scales as well.
template <typename T, bool E5M2>
__global__ void __launch_bounds__(kThreads) quantize_columns_kernel(const T* __restrict__ x, int P, int C,
                                                                    const int32_t* __restrict__ offsets, int E,
                                                                    uint8_t* __restrict__ q,
                                                                    float* __restrict__ scales, int blocks) {
    __shared__ int s_off[MOE_MAX_EXPERTS + 1], s_first[MOE_MAX_EXPERTS + 1], s_warp[33];
    __shared__ __align__(16) uint32_t s_max[kThreads / 32][kQBlock];
    __shared__ __align__(16) float s_factor[kQBlock];
    chain();
    expert_blocks<kQBlock>(offsets, E, offsets ? blocks * kQBlock : P, s_off, s_first, s_warp);
    const int nc = cdiv(C, kQBlock), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // Without offsets every block is the one expert's: one that P leaves empty is written as zero rows.
    const int used = offsets ? min(s_first[E], blocks) : blocks;
    const int col = (threadIdx.x & 15) * 8, r0 = threadIdx.x >> 4;
    for (long long t = blockIdx.x; t < (long long)used * nc; t += gridDim.x) {
        const int b = (int)(t / nc), cb = (int)(t - (long long)b * nc) * kQBlock, c = cb + col;
        const int e = expert_of(s_first, E, b, 1);
        const int row0 = s_off[e] + (b - s_first[e]) * kQBlock, have = min(kQBlock, min(s_off[e + 1], P) - row0);
        Raw8<T> v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i].zero();
            if (c < C && r0 + 16 * i < have) v[i].load(x + (size_t)(row0 + r0 + 16 * i) * C + c);
        }
        uint32_t mx[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f[8];
            v[i].get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) mx[j] = max(mx[j], abs_bits(f[j]));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) mx[j] = max(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 16));
        if (lane < 16) {
            *reinterpret_cast<uint4*>(&s_max[warp][col]) = make_uint4(mx[0], mx[1], mx[2], mx[3]);
            *reinterpret_cast<uint4*>(&s_max[warp][col + 4]) = make_uint4(mx[4], mx[5], mx[6], mx[7]);
        }
        __syncthreads();
        if (threadIdx.x < kQBlock) {  // one thread per column: its maximum and the two quotients
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kThreads / 32; ++i) m = max(m, s_max[i][threadIdx.x]);
            float scale, factor;
            block_scale(m, fp8_max(E5M2), scale, factor);
            s_factor[threadIdx.x] = factor;
            if (cb + (int)threadIdx.x < C) scales[(size_t)b * C + cb + threadIdx.x] = have > 0 ? scale : 0.0f;
        }
        __syncthreads();
        float factor[8];
        const float4 fa = *reinterpret_cast<const float4*>(s_factor + col);
        const float4 fb = *reinterpret_cast<const float4*>(s_factor + col + 4);
        factor[0] = fa.x, factor[1] = fa.y, factor[2] = fa.z, factor[3] = fa.w;
        factor[4] = fb.x, factor[5] = fb.y, factor[6] = fb.z, factor[7] = fb.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f[8];
            v[i].get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], factor[j]);
            if (c < C)
                *reinterpret_cast<uint2*>(q + ((size_t)b * kQBlock + r0 + 16 * i) * C + c) = pack8_fp8<E5M2>(f, 1.0f);
        }
    }
}

// h = silu(g) u:  dg = dh u (sg + g sg (1 - sg)),  du = dh g sg,  sg = 1 / (1 + e^-g).
// h = relu(g)^2:  dg = 2 relu(g) dh.
template <typename T, bool SWIGLU>
__global__ void __launch_bounds__(kThreads) activation_backward_kernel(const T* __restrict__ y,
                                                                       const T* __restrict__ dh, int P, int I,
                                                                       T* __restrict__ dy) {
    chain();
    const int nch = I / 8, ld = SWIGLU ? 2 * I : I;
    // This thread's chunks of eight, as (row, chunk) pairs advanced without a division.
    const long long first = (long long)blockIdx.x * kThreads + threadIdx.x, step = (long long)gridDim.x * kThreads;
    const int step_p = (int)(step / nch), step_c = (int)(step - (long long)step_p * nch) * 8;
    size_t p = (size_t)(first / nch);
    int c = (int)(first - (long long)p * nch) * 8;
    for (; p < (size_t)P; p += step_p) {
        float g[8], u[8], d[8], dg[8], du[8];
        load8(y + p * ld + c, g);
        if (SWIGLU) load8(y + p * ld + I + c, u);
        load8(dh + p * I + c, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (SWIGLU) {
                const float sg = quick_sigmoid(g[j]);
                const float si = g[j] * sg;
                dg[j] = d[j] * u[j] * fmaf(si, 1.0f - sg, sg);
                du[j] = d[j] * si;
            } else {
                dg[j] = g[j] <= 0.0f ? 0.0f * d[j] : 2.0f * g[j] * d[j];
            }
        }
        store8(dy + p * ld + c, dg);
        if (SWIGLU) store8(dy + p * ld + I + c, du);
        c += step_c;
        if (c >= I) {
            c -= I;
            ++p;
        }
    }
}

int grid_for(long long blocks, int sms, int per_sm) {
    return (int)std::max<long long>(1, std::min<long long>(blocks, (long long)sms * per_sm));
}

template <typename T, int SRC, bool QUANT, bool E5M2>
cudaError_t rows_t(const QuantArgs& a, int sms, cudaStream_t s) {
    const int nb = cdiv(a.C, kQBlock);
    // Blocks per warp: with four (two halves of a warp) enough bytes are in flight; eight for plain
    // rows written once (32768 x 2048: 50 -> 44 us; rows written to K places go slower, 51 -> 53, and
    // SwiGLU's two operands are eight loads already, 18 -> 31); two while there are few warps.
    const long long pairs = (long long)a.M * cdiv(nb, 2);
    const bool once = SRC != QS_SWIGLU && !a.inv;
    if constexpr (SRC != QS_SWIGLU) {
        if (once && pairs >= 32LL * sms)
            return launch_k(quantize_rows_kernel<T, SRC, QUANT, E5M2, 4>,
                            dim3(grid_for(((long long)a.M * cdiv(nb, 8) + 7) / 8, sms, 16)), dim3(kThreads), 0, s, true, a);
    }
    if (pairs >= 16LL * sms)
        return launch_k(quantize_rows_kernel<T, SRC, QUANT, E5M2, 2>,
                        dim3(grid_for(((long long)a.M * cdiv(nb, 4) + 7) / 8, sms, 16)), dim3(kThreads), 0, s, true, a);
    return launch_k(quantize_rows_kernel<T, SRC, QUANT, E5M2, 1>, dim3(grid_for((pairs + 7) / 8, sms, 16)), dim3(kThreads),
                    0, s, true, a);
}
template <typename T, int SRC>
cudaError_t rows_src(const QuantArgs& a, int sms, cudaStream_t s) {
    if (a.q) return a.e5m2 ? rows_t<T, SRC, true, true>(a, sms, s) : rows_t<T, SRC, true, false>(a, sms, s);
    if constexpr (SRC != QS_ROWS) return rows_t<T, SRC, false, false>(a, sms, s);
    return cudaErrorInvalidValue;
}
template <typename T>
cudaError_t rows_type(const QuantArgs& a, int src, int sms, cudaStream_t s) {
    if (src == QS_SWIGLU) return rows_src<T, QS_SWIGLU>(a, sms, s);
    if (src == QS_RELU2) return rows_src<T, QS_RELU2>(a, sms, s);
    return rows_src<T, QS_ROWS>(a, sms, s);
}
template <typename T>
cudaError_t blocks_t(const void* w, int E, int N, int C, int e5m2, uint8_t* q, float* scales, cudaStream_t s) {
    const dim3 grid((unsigned)(E * cdiv(N, kQBlock) * cdiv(C, kQBlock)));
    auto kern = e5m2 ? quantize_blocks_kernel<T, true> : quantize_blocks_kernel<T, false>;
    return launch_k(kern, grid, dim3(kThreads), 0, s, true, static_cast<const T*>(w), N, C, q, scales);
}
template <typename T>
cudaError_t columns_t(const void* x, int P, int C, const int32_t* offsets, int E, int e5m2, uint8_t* q, float* scales,
                      int blocks, int sms, cudaStream_t s) {
    const long long tiles = (long long)std::min(blocks, P / kQBlock + std::min(E, P)) * cdiv(C, kQBlock);
    auto kern = e5m2 ? quantize_columns_kernel<T, true> : quantize_columns_kernel<T, false>;
    return launch_k(kern, dim3(grid_for(tiles, sms, 4)), dim3(kThreads), 0, s, true, static_cast<const T*>(x), P, C,
                    offsets, E, q, scales, blocks);
}
template <typename T>
cudaError_t act_backward_t(const void* y, const void* dh, bool swiglu, int P, int I, void* dy, int sms,
                           cudaStream_t s) {
    const long long n = (long long)P * (I / 8);
    auto kern = swiglu ? activation_backward_kernel<T, true> : activation_backward_kernel<T, false>;
    return launch_k(kern, dim3(grid_for((n + kThreads - 1) / kThreads, sms, 16)), dim3(kThreads), 0, s, true,
                    static_cast<const T*>(y), static_cast<const T*>(dh), P, I, static_cast<T*>(dy));
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantArgs& a, int src, bool f32, int sms, cudaStream_t s) {
    return f32 ? rows_type<float>(a, src, sms, s) : rows_type<bf16>(a, src, sms, s);
}
cudaError_t launch_quantize_blocks(const void* w, bool f32, int E, int N, int C, int e5m2, uint8_t* q, float* scales,
                                   cudaStream_t s) {
    return f32 ? blocks_t<float>(w, E, N, C, e5m2, q, scales, s) : blocks_t<bf16>(w, E, N, C, e5m2, q, scales, s);
}
cudaError_t launch_quantize_columns(const void* x, bool f32, int P, int C, const int32_t* offsets, int E, int e5m2,
                                    uint8_t* q, float* scales, int blocks, int sms, cudaStream_t s) {
    return f32 ? columns_t<float>(x, P, C, offsets, E, e5m2, q, scales, blocks, sms, s)
               : columns_t<bf16>(x, P, C, offsets, E, e5m2, q, scales, blocks, sms, s);
}
cudaError_t launch_activation_backward(const void* y, const void* dh, bool f32, bool swiglu, int P, int I, void* dy,
                                       int sms, cudaStream_t s) {
    return f32 ? act_backward_t<float>(y, dh, swiglu, P, I, dy, sms, s)
               : act_backward_t<bf16>(y, dh, swiglu, P, I, dy, sms, s);
}

}  // namespace moe
