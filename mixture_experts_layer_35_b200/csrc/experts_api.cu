// experts_api.cu -- the C ABI of the expert operators: host-side validation, tensor maps and
// launches.  Nothing here allocates or synchronises (except moe_product_get_error).
#include <cstring>
#include <initializer_list>

#include "experts.cuh"

using namespace moe;

namespace {

bool bad_ptr(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15u); }
bool bad_opt(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u); }
bool bad_dtype(int t) { return t != MOE_DT_BF16 && t != MOE_DT_FP32; }
bool bad_fp8(int t) { return t != MOE_DT_E4M3 && t != MOE_DT_E5M2; }
size_t dt_bytes(int t) { return t == MOE_DT_FP32 ? 4 : 2; }
// A buffer's bytes; null: not given.
struct Span {
    const void* p;
    size_t n;
};
bool overlaps(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}
// An output that shares memory with an input or with another output.
bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span* p = outs.begin(); p != o; ++p)
            if (overlaps(*o, *p)) return true;
        for (const Span& i : ins)
            if (overlaps(*o, i)) return true;
    }
    return false;
}
size_t scale_bytes(size_t rows, int cols) { return rows * cdiv(cols, kQBlock) * sizeof(float); }
size_t slot_bytes(int M, int K) { return (size_t)M * K * 4; }  // inv, weights
size_t offset_bytes(int E) { return ((size_t)E + 1) * sizeof(int32_t); }
int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
    return n;
}
moe_status_t launched(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// M tokens of K slots with H features, and P rows.
moe_status_t check_slots(int dtype, int M, int K, int H, int P, int multiple) {
    if (bad_dtype(dtype) || M < 0 || K < 1 || P < 0 || H < 1 || H % multiple) return MOE_ERR_INVALID_ARG;
    if (K > MOE_MAX_TOPK || (long long)M * K > MOE_MAX_ROWS || P > MOE_MAX_ROWS || H > MOE_MAX_FEATURES)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
// P rows of E experts.
moe_status_t check_experts(int P, const int32_t* offsets, int E) {
    if (P < 0 || E < 1 || bad_opt(offsets) || (!offsets && E != 1)) return MOE_ERR_INVALID_ARG;
    if (P > MOE_MAX_ROWS || E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
moe_status_t check_features(int n, int multiple) {
    if (n < 1 || n % multiple) return MOE_ERR_INVALID_ARG;
    return n > MOE_MAX_FEATURES ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Tensor maps over bytes: boxes of 128 bytes by `rows`, in the 128-byte swizzle.
bool bytes_map(CUtensorMap* m, const void* base, int dim, uint64_t inner, uint64_t rows, uint64_t depth,
               uint32_t box_rows) {
    EncodeTiledFn enc = get_encode_tiled();
    if (!enc) return false;
    cuuint64_t dims[3] = {inner, rows, depth};
    cuuint64_t strides[2] = {inner, inner * rows};
    cuuint32_t box[3] = {128, box_rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, dim, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Output map [depth][rows][cols]: boxes of 128 bytes by 32 rows, in the 128-byte swizzle.
bool out_map(CUtensorMap* m, void* base, bool f32, uint64_t cols, uint64_t rows, uint64_t depth) {
    EncodeTiledFn enc = get_encode_tiled();
    if (!enc) return false;
    const uint64_t el = f32 ? 4 : 2;
    cuuint64_t dims[3] = {cols, rows, depth};
    cuuint64_t strides[2] = {cols * el, cols * rows * el};
    cuuint32_t box[3] = {(cuuint32_t)(128 / el), 32, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides,
               box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
moe_status_t too_many_tiles(long long row_tiles, int cols) {
    return row_tiles * cdiv(cols, 64) > 0x3fffffffLL ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Forward product, or the input gradient, with `act` 0 or 1 + moe_act_t fused (forward).
moe_status_t run_rows_product(int kind, int act, const void* aq, const float* a_scales, int a_fp8, const void* wq,
                              const float* w_scales, int P, int N, int C, const int32_t* offsets, int E,
                              int out_dtype, int h_fp8, void* out, float* out_scales, void* stream) {
    const int Wn = act == 1 + MOE_ACT_SWIGLU ? 2 * N : N;  // weight rows of an expert
    if (P == 0) return MOE_OK;
    if (bad_ptr(aq) || bad_ptr(a_scales) || bad_ptr(wq) || bad_ptr(w_scales) || bad_ptr(out) ||
        (act && bad_ptr(out_scales)))
        return MOE_ERR_INVALID_ARG;
    const int depth = kind == PK_FORWARD ? C : N, cols = kind == PK_FORWARD ? N : C;
    const size_t out_bytes = (size_t)P * cols * (act ? 1 : dt_bytes(out_dtype));
    if (clash({{out, out_bytes}, {out_scales, scale_bytes(P, cols)}},
              {{aq, (size_t)P * depth},
               {a_scales, scale_bytes(P, depth)},
               {wq, (size_t)E * Wn * C},
               {w_scales, scale_bytes((size_t)E * cdiv(Wn, kQBlock), C)},
               {offsets, offset_bytes(E)}}))
        return MOE_ERR_INVALID_ARG;
    moe_status_t st = too_many_tiles(P / 32 + E, cols);
    if (st != MOE_OK) return st;
    ProductArgs a;
    std::memset(&a, 0, sizeof(a));
    a.cols = cols;
    a.P = P;
    a.E = E;
    a.nbl = cdiv(depth, kQBlock);
    a.wn = cdiv(Wn, kQBlock);
    a.wk = cdiv(C, kQBlock);
    a.offsets = offsets;
    a.sa = a_scales;
    a.sb = w_scales;
    a.a_e5m2 = a_fp8 == MOE_DT_E5M2;
    a.out_f32 = out_dtype == MOE_DT_FP32;
    a.up = N;
    a.h_e5m2 = h_fp8 == MOE_DT_E5M2;
    a.out = out;
    a.out_scales = out_scales;
    const int sms = sm_count();
    const int few = product_few_rows(act, a);
    const int w_box = few || kind == PK_INPUT_GRAD ? 128 : (act == 0 ? 256 : (act == 1 + MOE_ACT_SWIGLU ? 64 : 128));
    ProductMaps m;
    if (!bytes_map(&m.a, aq, 2, depth, P, 1, kRowBox) || !bytes_map(&m.b, wq, 3, C, Wn, E, w_box))
        return MOE_ERR_CUDA;
    if (few) return launched(launch_product_few(kind, act, few, a, m, sms, (cudaStream_t)stream));
    if (act) m.out = m.a;  // unused
    else if (!out_map(&m.out, out, a.out_f32, cols, P, 1)) return MOE_ERR_CUDA;
    return launched(launch_product(kind, act, a, m, sms, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

moe_status_t moe_dispatch(const void* x, int dtype, int M, int K, int H, const int32_t* inv, int P, void* xs,
                          void* stream) {
    const moe_status_t st = check_slots(dtype, M, K, H, P, 8);
    if (st != MOE_OK) return st;
    if (M == 0 || P == 0) return MOE_OK;
    if (bad_ptr(x) || bad_ptr(inv) || bad_ptr(xs)) return MOE_ERR_INVALID_ARG;
    const size_t el = dt_bytes(dtype);
    if (clash({{xs, (size_t)P * H * el}}, {{x, (size_t)M * H * el}, {inv, slot_bytes(M, K)}})) return MOE_ERR_INVALID_ARG;
    const RowsArgs a = {x, nullptr, inv, nullptr, xs, nullptr, M, K, H, P};
    return launched(launch_dispatch(a, dtype == MOE_DT_FP32, sm_count(), (cudaStream_t)stream));
}

moe_status_t moe_combine(const void* ys, int dtype, int M, int K, int H, const int32_t* inv, int P,
                         const float* weights, void* y, void* stream) {
    const moe_status_t st = check_slots(dtype, M, K, H, P, 8);
    if (st != MOE_OK) return st;
    if (M == 0) return MOE_OK;
    if ((P > 0 && bad_ptr(ys)) || bad_ptr(inv) || bad_opt(weights) || bad_ptr(y)) return MOE_ERR_INVALID_ARG;
    const size_t el = dt_bytes(dtype);
    if (clash({{y, (size_t)M * H * el}},
              {{ys, (size_t)P * H * el}, {inv, slot_bytes(M, K)}, {weights, slot_bytes(M, K)}}))
        return MOE_ERR_INVALID_ARG;
    const RowsArgs a = {ys, nullptr, inv, weights, y, nullptr, M, K, H, P};
    return launched(launch_combine(a, dtype == MOE_DT_FP32, sm_count(), (cudaStream_t)stream));
}

moe_status_t moe_combine_backward(const void* dy, const void* ys, int dtype, int M, int K, int H, const int32_t* inv,
                                  int P, const float* weights, void* dys, float* dweights, void* stream) {
    const moe_status_t st = check_slots(dtype, M, K, H, P, 8);
    if (st != MOE_OK) return st;
    if (M == 0) return MOE_OK;
    if (bad_ptr(dy) || (P > 0 && (bad_ptr(ys) || bad_ptr(dys))) || bad_ptr(inv) || bad_ptr(weights) ||
        bad_ptr(dweights))
        return MOE_ERR_INVALID_ARG;
    const size_t el = dt_bytes(dtype), rows = (size_t)P * H * el;
    if (clash({{dys, rows}, {dweights, slot_bytes(M, K)}},
              {{dy, (size_t)M * H * el}, {ys, rows}, {inv, slot_bytes(M, K)}, {weights, slot_bytes(M, K)}}))
        return MOE_ERR_INVALID_ARG;
    const RowsArgs a = {ys, dy, inv, weights, dys, dweights, M, K, H, P};
    return launched(launch_combine_backward(a, dtype == MOE_DT_FP32, sm_count(), (cudaStream_t)stream));
}

moe_status_t moe_quantize_rows(const void* x, int dtype, int R, int C, int fp8, void* q, float* scales,
                               void* stream) {
    if (bad_dtype(dtype) || bad_fp8(fp8) || R < 0) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_features(C, 16);
    if (st != MOE_OK) return st;
    if (R == 0) return MOE_OK;
    if (bad_ptr(x) || bad_ptr(q) || bad_ptr(scales)) return MOE_ERR_INVALID_ARG;
    const size_t n = (size_t)R * C;
    if (clash({{q, n}, {scales, scale_bytes(R, C)}}, {{x, n * dt_bytes(dtype)}})) return MOE_ERR_INVALID_ARG;
    const QuantArgs a = {x, nullptr, static_cast<uint8_t*>(q), scales, nullptr, R, 1, C, R, fp8 == MOE_DT_E5M2};
    return launched(launch_quantize_rows(a, QS_ROWS, dtype == MOE_DT_FP32, sm_count(), (cudaStream_t)stream));
}

moe_status_t moe_dispatch_quantize(const void* x, int dtype, int M, int K, int H, const int32_t* inv, int P, int fp8,
                                   void* q, float* scales, void* stream) {
    const moe_status_t st = check_slots(dtype, M, K, H, P, 16);
    if (st != MOE_OK) return st;
    if (bad_fp8(fp8)) return MOE_ERR_INVALID_ARG;
    if (M == 0 || P == 0) return MOE_OK;
    if (bad_ptr(x) || bad_ptr(inv) || bad_ptr(q) || bad_ptr(scales)) return MOE_ERR_INVALID_ARG;
    if (clash({{q, (size_t)P * H}, {scales, scale_bytes(P, H)}},
              {{x, (size_t)M * H * dt_bytes(dtype)}, {inv, slot_bytes(M, K)}}))
        return MOE_ERR_INVALID_ARG;
    const QuantArgs a = {x, inv, static_cast<uint8_t*>(q), scales, nullptr, M, K, H, P, fp8 == MOE_DT_E5M2};
    return launched(launch_quantize_rows(a, QS_ROWS, dtype == MOE_DT_FP32, sm_count(), (cudaStream_t)stream));
}

moe_status_t moe_quantize_blocks(const void* w, int dtype, int E, int N, int C, int fp8, void* q, float* scales,
                                 void* stream) {
    if (bad_dtype(dtype) || bad_fp8(fp8) || E < 0) return MOE_ERR_INVALID_ARG;
    moe_status_t st = check_features(N, 16);
    if (st == MOE_OK) st = check_features(C, 16);
    if (st != MOE_OK) return st;
    if ((long long)E * cdiv(N, kQBlock) * cdiv(C, kQBlock) > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
    if (E == 0) return MOE_OK;
    if (bad_ptr(w) || bad_ptr(q) || bad_ptr(scales)) return MOE_ERR_INVALID_ARG;
    const size_t n = (size_t)E * N * C;
    if (clash({{q, n}, {scales, scale_bytes((size_t)E * cdiv(N, kQBlock), C)}}, {{w, n * dt_bytes(dtype)}}))
        return MOE_ERR_INVALID_ARG;
    return launched(launch_quantize_blocks(w, dtype == MOE_DT_FP32, E, N, C, fp8 == MOE_DT_E5M2,
                                           static_cast<uint8_t*>(q), scales, (cudaStream_t)stream));
}

int moe_column_blocks(int P, int E) { return P < 0 || E < 1 ? 0 : P / kQBlock + std::min(P, E); }

moe_status_t moe_quantize_columns(const void* x, int dtype, int P, int C, const int32_t* offsets, int E, int fp8,
                                  void* q, float* scales, void* stream) {
    if (bad_dtype(dtype) || bad_fp8(fp8)) return MOE_ERR_INVALID_ARG;
    moe_status_t st = check_features(C, 16);
    if (st == MOE_OK) st = check_experts(P, offsets, E);
    if (st != MOE_OK) return st;
    if (P == 0) return MOE_OK;
    if (bad_ptr(x) || bad_ptr(q) || bad_ptr(scales)) return MOE_ERR_INVALID_ARG;
    const int blocks = moe_column_blocks(P, E);
    if (clash({{q, (size_t)blocks * kQBlock * C}, {scales, (size_t)blocks * C * sizeof(float)}},
              {{x, (size_t)P * C * dt_bytes(dtype)}, {offsets, offset_bytes(E)}}))
        return MOE_ERR_INVALID_ARG;
    return launched(launch_quantize_columns(x, dtype == MOE_DT_FP32, P, C, offsets, E, fp8 == MOE_DT_E5M2,
                                            static_cast<uint8_t*>(q), scales, blocks, sm_count(),
                                            (cudaStream_t)stream));
}

static moe_status_t check_activation(int dtype, int act, int P, int I, int multiple) {
    if (bad_dtype(dtype) || (act != MOE_ACT_SWIGLU && act != MOE_ACT_RELU2) || P < 0) return MOE_ERR_INVALID_ARG;
    return check_features(I, multiple);
}

moe_status_t moe_activation(const void* y, int dtype, int act, int P, int I, void* h, void* stream) {
    const moe_status_t st = check_activation(dtype, act, P, I, 8);
    if (st != MOE_OK) return st;
    if (P == 0) return MOE_OK;
    if (bad_ptr(y) || bad_ptr(h)) return MOE_ERR_INVALID_ARG;
    const bool swiglu = act == MOE_ACT_SWIGLU;
    const size_t n = (size_t)P * I * dt_bytes(dtype);
    if (clash({{h, n}}, {{y, swiglu ? 2 * n : n}})) return MOE_ERR_INVALID_ARG;
    const QuantArgs a = {y, nullptr, nullptr, nullptr, h, P, 1, I, P, 0};
    return launched(launch_quantize_rows(a, swiglu ? QS_SWIGLU : QS_RELU2, dtype == MOE_DT_FP32, sm_count(),
                                         (cudaStream_t)stream));
}

moe_status_t moe_activation_quantize(const void* y, int dtype, int act, int P, int I, int fp8, void* q, float* scales,
                                     void* stream) {
    const moe_status_t st = check_activation(dtype, act, P, I, 16);
    if (st != MOE_OK) return st;
    if (bad_fp8(fp8)) return MOE_ERR_INVALID_ARG;
    if (P == 0) return MOE_OK;
    if (bad_ptr(y) || bad_ptr(q) || bad_ptr(scales)) return MOE_ERR_INVALID_ARG;
    const bool swiglu = act == MOE_ACT_SWIGLU;
    const size_t n = (size_t)P * I;
    if (clash({{q, n}, {scales, scale_bytes(P, I)}}, {{y, n * dt_bytes(dtype) * (swiglu ? 2 : 1)}}))
        return MOE_ERR_INVALID_ARG;
    const QuantArgs a = {y, nullptr, static_cast<uint8_t*>(q), scales, nullptr, P, 1, I, P, fp8 == MOE_DT_E5M2};
    return launched(launch_quantize_rows(a, swiglu ? QS_SWIGLU : QS_RELU2, dtype == MOE_DT_FP32, sm_count(),
                                         (cudaStream_t)stream));
}

moe_status_t moe_activation_backward(const void* y, const void* dh, int dtype, int act, int P, int I, void* dy,
                                     void* stream) {
    const moe_status_t st = check_activation(dtype, act, P, I, 8);
    if (st != MOE_OK) return st;
    if (P == 0) return MOE_OK;
    if (bad_ptr(y) || bad_ptr(dh) || bad_ptr(dy)) return MOE_ERR_INVALID_ARG;
    const bool swiglu = act == MOE_ACT_SWIGLU;
    const size_t n = (size_t)P * I * dt_bytes(dtype), ny = swiglu ? 2 * n : n;
    if (clash({{dy, ny}}, {{y, ny}, {dh, n}})) return MOE_ERR_INVALID_ARG;
    return launched(launch_activation_backward(y, dh, dtype == MOE_DT_FP32, swiglu, P, I, dy, sm_count(),
                                               (cudaStream_t)stream));
}

static moe_status_t check_product(int P, int N, int C, const int32_t* offsets, int E) {
    moe_status_t st = check_experts(P, offsets, E);
    if (st == MOE_OK) st = check_features(N, 16);
    if (st == MOE_OK) st = check_features(C, 16);
    return st;
}

moe_status_t moe_product(const void* xq, const float* x_scales, int x_fp8, const void* wq, const float* w_scales,
                         int P, int N, int C, const int32_t* offsets, int E, int out_dtype, void* y, void* stream) {
    const moe_status_t st = check_product(P, N, C, offsets, E);
    if (st != MOE_OK) return st;
    if (bad_fp8(x_fp8) || bad_dtype(out_dtype)) return MOE_ERR_INVALID_ARG;
    return run_rows_product(PK_FORWARD, 0, xq, x_scales, x_fp8, wq, w_scales, P, N, C, offsets, E, out_dtype, 0, y,
                            nullptr, stream);
}

moe_status_t moe_product_activation(const void* xq, const float* x_scales, int x_fp8, const void* wq,
                                    const float* w_scales, int P, int I, int C, const int32_t* offsets, int E,
                                    int act, int h_fp8, void* hq, float* h_scales, void* stream) {
    const moe_status_t st = check_product(P, I, C, offsets, E);
    if (st != MOE_OK) return st;
    if (bad_fp8(x_fp8) || bad_fp8(h_fp8) || (act != MOE_ACT_SWIGLU && act != MOE_ACT_RELU2))
        return MOE_ERR_INVALID_ARG;
    return run_rows_product(PK_FORWARD, 1 + act, xq, x_scales, x_fp8, wq, w_scales, P, I, C, offsets, E, MOE_DT_BF16,
                            h_fp8, hq, h_scales, stream);
}

moe_status_t moe_product_input_grad(const void* dyq, const float* dy_scales, int dy_fp8, const void* wq,
                                    const float* w_scales, int P, int N, int C, const int32_t* offsets, int E,
                                    int out_dtype, void* dx, void* stream) {
    const moe_status_t st = check_product(P, N, C, offsets, E);
    if (st != MOE_OK) return st;
    if (bad_fp8(dy_fp8) || bad_dtype(out_dtype)) return MOE_ERR_INVALID_ARG;
    return run_rows_product(PK_INPUT_GRAD, 0, dyq, dy_scales, dy_fp8, wq, w_scales, P, N, C, offsets, E, out_dtype, 0,
                            dx, nullptr, stream);
}

moe_status_t moe_product_weight_grad(const void* dyq, const float* dy_scales, int dy_fp8, const void* xq,
                                     const float* x_scales, int x_fp8, int B, int N, int C, const int32_t* offsets,
                                     int E, int out_dtype, int accumulate, void* dw, void* stream) {
    moe_status_t st = check_product(0, N, C, offsets, E);
    if (st != MOE_OK) return st;
    if (B < 0) return MOE_ERR_INVALID_ARG;
    if (B > moe_column_blocks(MOE_MAX_ROWS, MOE_MAX_EXPERTS)) return MOE_ERR_UNSUPPORTED;
    if (bad_fp8(dy_fp8) || bad_fp8(x_fp8) || bad_dtype(out_dtype) || (accumulate != 0 && accumulate != 1))
        return MOE_ERR_INVALID_ARG;
    if (bad_ptr(dw)) return MOE_ERR_INVALID_ARG;
    st = too_many_tiles((long long)E * cdiv(N, 128), C);
    if (st != MOE_OK) return st;
    const size_t out_bytes = (size_t)E * N * C * dt_bytes(out_dtype);
    if (B == 0)  // no rows: zeros, or nothing to add
        return accumulate ? MOE_OK : launched(cudaMemsetAsync(dw, 0, out_bytes, (cudaStream_t)stream));
    if (bad_ptr(dyq) || bad_ptr(dy_scales) || bad_ptr(xq) || bad_ptr(x_scales)) return MOE_ERR_INVALID_ARG;
    const size_t rows = (size_t)B * kQBlock;
    if (clash({{dw, out_bytes}}, {{dyq, rows * N},
                                  {dy_scales, (size_t)B * N * sizeof(float)},
                                  {xq, rows * C},
                                  {x_scales, (size_t)B * C * sizeof(float)},
                                  {offsets, offset_bytes(E)}}))
        return MOE_ERR_INVALID_ARG;
    ProductArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = N;
    a.cols = C;
    a.P = (int)rows;
    a.E = E;
    a.offsets = offsets;
    a.sa = dy_scales;
    a.sb = x_scales;
    a.blocks = B;
    a.a_e5m2 = dy_fp8 == MOE_DT_E5M2;
    a.b_e5m2 = x_fp8 == MOE_DT_E5M2;
    a.out_f32 = out_dtype == MOE_DT_FP32;
    a.accumulate = accumulate;
    a.out = dw;
    const int sms = sm_count();
    ProductMaps m;
    if (!bytes_map(&m.a, dyq, 2, N, rows, 1, 128) || !bytes_map(&m.b, xq, 2, C, rows, 1, 128) ||
        !out_map(&m.out, dw, a.out_f32, C, N, E))
        return MOE_ERR_CUDA;
    return launched(launch_weight_grad(a, m, sms, (cudaStream_t)stream));
}

moe_status_t moe_product_get_error(int* code, void* stream) {
    if (!code) return MOE_ERR_INVALID_ARG;
    int v = 0;
    if (product_error(&v, (cudaStream_t)stream) != cudaSuccess) return MOE_ERR_CUDA;
    *code = v;
    return v ? MOE_ERR_DEVICE : MOE_OK;
}

}  // extern "C"
