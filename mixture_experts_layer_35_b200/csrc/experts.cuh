// experts.cuh -- launch interfaces and device helpers of the expert operators: rows sorted
// by expert and back (rows.cu), block quantisers and the activation (quantize.cu), and the
// grouped 8-bit product (product.cu).  Their host side is experts_api.cu.
#pragma once
#include <cuda_fp8.h>

#include "kernels.cuh"

namespace moe {

constexpr int kQBlock = 128;         // columns or rows that share one scale
constexpr float kAmaxFloor = 0x1p-96f;  // smallest block maximum a scale is made from

// The operators' kernels are launched so that each may start while the kernel before it in the
// stream drains.  Called before the first access to global memory: waits until that kernel is
// complete, and lets the next one start its own prologue.
__device__ __forceinline__ void chain() {
    pdl_wait();
    pdl_trigger();
}

// ---------------------------------------------------------------- 16-byte chunks of a row
template <typename T>
struct Chunk;  // V values of T in 16 bytes, as FP32
template <>
struct Chunk<bf16> {
    static constexpr int V = 8;
    static __device__ __forceinline__ void unpack(const uint4& c, float (&f)[V]) {
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16lo(w[i]);
            f[2 * i + 1] = bf16hi(w[i]);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[V]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (uint32_t)f2bf_bits(f[2 * i]) | ((uint32_t)f2bf_bits(f[2 * i + 1]) << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Chunk<float> {
    static constexpr int V = 4;
    static __device__ __forceinline__ void unpack(const uint4& c, float (&f)[V]) {
        f[0] = __uint_as_float(c.x);
        f[1] = __uint_as_float(c.y);
        f[2] = __uint_as_float(c.z);
        f[3] = __uint_as_float(c.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[V]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

// Eight consecutive values of a row as FP32 (one 16-byte load of BF16, two of FP32).
__device__ __forceinline__ void load8(const bf16* p, float (&f)[8]) { Chunk<bf16>::unpack(ld_stream16(p), f); }
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    float a[4], b[4];
    Chunk<float>::unpack(ld_stream16(p), a);
    Chunk<float>::unpack(ld_stream16(p + 4), b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = a[i];
        f[4 + i] = b[i];
    }
}
// The same eight values as they lie in memory, for code that keeps many of them at once.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16> {
    uint4 a;
    __device__ __forceinline__ void load(const bf16* p) { a = ld_stream16(p); }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const { Chunk<bf16>::unpack(a, f); }
};
template <>
struct Raw8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = ld_stream16(p);
        b = ld_stream16(p + 4);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        float x[4], y[4];
        Chunk<float>::unpack(a, x);
        Chunk<float>::unpack(b, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = x[i];
            f[4 + i] = y[i];
        }
    }
};
__device__ __forceinline__ void store8(bf16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = Chunk<bf16>::pack(f);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    const float a[4] = {f[0], f[1], f[2], f[3]}, b[4] = {f[4], f[5], f[6], f[7]};
    *reinterpret_cast<uint4*>(p) = Chunk<float>::pack(a);
    *reinterpret_cast<uint4*>(p + 4) = Chunk<float>::pack(b);
}

// ---------------------------------------------------------------- 8-bit blocks
// The largest magnitude of a block is kept as the bits of |v|: their order as integers is
// the order of the values, with infinity above every number and NaN above infinity, so a
// NaN reaches the scale instead of being skipped.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// A block whose largest magnitude is a (at least 2^-96, so that the factor stays finite):
// scale a / fmax, and the factor fmax / a its values are multiplied by before the rounding.
__device__ __forceinline__ void block_scale(uint32_t amax_bits, float fmax, float& scale, float& factor) {
    const float a = __uint_as_float(max(amax_bits, __float_as_uint(kAmaxFloor)));
    scale = __fdiv_rn(a, fmax);
    factor = __fdiv_rn(fmax, a);
}
__host__ __device__ inline float fp8_max(int e5m2) { return e5m2 ? 57344.0f : 448.0f; }
// Eight values times the factor, rounded to nearest even, in 8 bytes.
template <bool E5M2>
__device__ __forceinline__ uint2 pack8_fp8(const float (&f)[8], float factor) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(f[2 * i], factor), __fmul_rn(f[2 * i + 1], factor)),
                                        __NV_SATFINITE, E5M2 ? __NV_E5M2 : __NV_E4M3);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// ---------------------------------------------------------------- activation
// As the fused layer's, except that the quotient is the two-instruction one (off by at most 2
// units in the last place for divisors up to 2^126; 0 above, where the sigmoid is below 2^-126),
// and that a NaN stays one through ReLU^2.  The correctly rounded quotient's slow path took
// 10 us of a 128 x 256 tile of the fused product (250 against 160 us for 10240 rows of 256 experts).
__device__ __forceinline__ float quick_sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }
__device__ __forceinline__ float quick_swiglu(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }
__device__ __forceinline__ float relu2_nan(float g) { return g > 0.0f ? g * g : (g == g ? 0.0f : g); }

// ---------------------------------------------------------------- rows of each expert
// off[0..E]: the row offsets, clamped to [0, P] and to the largest one before (no offsets: one
// expert with all rows), so that whatever they hold, experts' rows lie in [0, P), do not overlap and
// are at most P.  first[0..E]: exclusive prefix over the experts of ceil(rows / UNIT).  By the whole
// CTA (a multiple of 32 threads); s_warp: 33 ints.
template <int UNIT>
__device__ __forceinline__ void expert_blocks(const int32_t* offsets, int E, int P, int* off, int* first, int* s_warp) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    const int per = cdiv(E, (int)blockDim.x), e0 = min(tid * per, E), e1 = min(e0 + per, E);  // this thread's experts
    int top = offsets ? min(max(offsets[0], 0), P) : 0;
    if (tid == 0) off[0] = top;
    for (int e = e0; e < e1; ++e) {
        top = max(top, offsets ? min(offsets[e + 1], P) : P);
        off[e + 1] = top;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, top, o);
        if (lane >= o) top = max(top, n);
    }
    if (lane == 31) s_warp[warp] = top;
    top = __shfl_up_sync(0xffffffffu, top, 1);  // the largest of the lanes before
    if (lane == 0) top = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) top = max(top, s_warp[w]);
    for (int e = e0; e < e1; ++e) off[e + 1] = max(off[e + 1], top);
    __syncthreads();
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += cdiv(off[e + 1] - off[e], UNIT);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += s_warp[w];
    for (int e = e0; e < e1; ++e) {
        first[e] = run;
        run += cdiv(off[e + 1] - off[e], UNIT);
    }
    if (tid == 0) {
        int total = 0;
        for (int w = 0; w < nw; ++w) total += s_warp[w];
        first[E] = total;
    }
    __syncthreads();
}
// The last expert e with first[e] * scale <= i (i below the total): the one that holds i.
__device__ __forceinline__ int expert_of(const int* first, int E, int i, int scale) {
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] * scale <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ---------------------------------------------------------------- launches
struct RowsArgs {
    const void* src;       // dispatch: x [M, H]; combine: ys [P, H]
    const void* dy;        // combine backward: dy [M, H]
    const int32_t* inv;    // [K, M]
    const float* w;        // [M, K] or null (ones)
    void* dst;             // dispatch: xs [P, H]; combine: y [M, H]; backward: dys [P, H]
    float* dw;             // combine backward: [M, K]
    int M, K, H, P;
};
cudaError_t launch_dispatch(const RowsArgs& a, bool f32, int sms, cudaStream_t s);
cudaError_t launch_combine(const RowsArgs& a, bool f32, int sms, cudaStream_t s);
cudaError_t launch_combine_backward(const RowsArgs& a, bool f32, int sms, cudaStream_t s);

enum QuantSrc { QS_ROWS = 0, QS_SWIGLU = 1, QS_RELU2 = 2 };
struct QuantArgs {
    const void* src;       // [M, C], or [M, 2C] for SwiGLU
    const int32_t* inv;    // [K, M] rows to write, or null: row m
    uint8_t* q;            // 8-bit rows, or null
    float* scales;         // [rows, ceil(C / 128)]
    void* h;               // rows of the source's type when q is null
    int M, K, C, P;
    int e5m2;
};
// One scale per row and 128 columns (of the rows, or of their activation), written to row m
// or to the rows inv names; or the activation alone.
cudaError_t launch_quantize_rows(const QuantArgs& a, int src, bool f32, int sms, cudaStream_t s);
cudaError_t launch_quantize_blocks(const void* w, bool f32, int E, int N, int C, int e5m2, uint8_t* q, float* scales,
                                   cudaStream_t s);
cudaError_t launch_quantize_columns(const void* x, bool f32, int P, int C, const int32_t* offsets, int E, int e5m2,
                                    uint8_t* q, float* scales, int blocks, int sms, cudaStream_t s);
cudaError_t launch_activation_backward(const void* y, const void* dh, bool f32, bool swiglu, int P, int I, void* dy,
                                       int sms, cudaStream_t s);

enum ProductKind { PK_FORWARD = 0, PK_INPUT_GRAD = 1 };
struct ProductArgs {
    int rows;              // weight gradient: output rows per expert (N)
    int cols;              // output columns: N, C, C; I for a fused activation
    int P, E;
    int nbl;               // blocks of 128 along the contraction (forward, input gradient)
    int wn, wk;            // weight scale blocks along N and C
    const int32_t* offsets;
    const float* sa;       // row scales [P, nbl]; weight gradient: dy's [blocks, N]
    const float* sb;       // weight scales [E, wn, wk]; weight gradient: x's [blocks, C]
    int blocks;            // weight gradient: 128-row blocks in the padded operands (P = 128 * blocks)
    int a_e5m2, b_e5m2;    // types of the rows (dy); weight gradient: of x
    int out_f32, accumulate;
    int up;                // SwiGLU: row of the first up feature
    int h_e5m2;
    void* out;
    float* out_scales;     // fused activation: [P, ceil(I / 128)]
};
// Forward, input gradient: a = rows, b = weights.  Weight gradient: a = dy, b = x, out = dw.
struct ProductMaps {
    CUtensorMap a, b, out;
};
// Rows per tile of a forward product or input gradient when its experts have few rows
// (launch_product_few), or 0 (launch_product).
int product_few_rows(int act, const ProductArgs& a);
constexpr int kRowBox = 32;  // rows per TMA box of the row operand
cudaError_t launch_product(int kind, int act, const ProductArgs& a, const ProductMaps& m, int sms, cudaStream_t s);
cudaError_t launch_product_few(int kind, int act, int tile_rows, const ProductArgs& a, const ProductMaps& m, int sms,
                               cudaStream_t s);
cudaError_t launch_weight_grad(const ProductArgs& a, const ProductMaps& m, int sms, cudaStream_t s);
// Addresses of the error words on the current device; and all of them read and cleared, after the
// work on `s` so far (synchronises it).
cudaError_t product_error_word(int** p);
cudaError_t product_few_error_word(int** p);
cudaError_t weight_grad_error_word(int** p);
cudaError_t product_error(int* code, cudaStream_t s);

}  // namespace moe
