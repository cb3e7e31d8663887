// product.cu -- grouped 8-bit products with one FP32 scale per block of 128 along the
// contraction, on the 5th-generation tensor cores (tcgen05.mma kind::f8f6f4).
//
//   forward          y[p, n]  = sum_b sx[p, b] sw[e, n/128, b] sum_{c in b} qx[p, c] qw[e, n, c]
//   input gradient   dx[p, c] = sum_b sdy[p, b] sw[e, b, c/128] sum_{n in b} qdy[p, n] qw[e, n, c]
//   weight gradient  dw[e, n, c] = sum over the 128-row blocks b of e of
//                                  sdy[b, n] sx[b, c] sum_{p in b} qdy[p, n] qx[p, c]
//   forward + activation: SwiGLU or ReLU^2 of the FP32 sums, rounded to 8 bits with one scale
//   per row and 128 features.
//
// One tile is 128 output rows (TMEM lanes) by BN output columns.  The scales change with
// every block of 128, so the tensor core sums one block at a time into one of several TMEM
// buffers, and the epilogue warps add buffer * scale to FP32 sums in registers while the
// next block's MMAs run.  Output rows are tokens, so a token's scale is one register per
// thread and a weight block's scale is one value for all 128 columns of a thread.
// The weights lie in memory once, [E, N, C]: the forward product reads them K-major
// (contraction over C), the input gradient MN-major (contraction over N), and the weight
// gradient reads both operands MN-major, so nothing is transposed.
//
// Warps: 0 TMA producer, 1 TMEM allocator and MMA issuer, 2-9 epilogue (warp w reads TMEM
// lanes of quarter w % 4 and one half of the columns).  One persistent CTA per SM; tiles go
// round-robin, inside an expert in bands of 16 row tiles, column tiles outer, so that the
// CTAs at work share weights and rows in L2.
#include "experts.cuh"

namespace moe {
namespace {

__device__ int g_product_error;  // MOE_DEVERR_* bits of the products on this device

constexpr int BM = 128, BKB = 128;  // tile rows; bytes (= values) of one block along the contraction
constexpr int kBand = 16;           // row tiles that share a pass over the weights
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int A_BYTES = BM * BKB;
constexpr int kStageOut = 2048;  // staging of one epilogue warp: 32 rows x 64 bytes

template <int BN>
struct Cfg {
    static constexpr int kBBytes = BN * BKB;
    static constexpr int kStageBytes = A_BYTES + kBBytes;
    static constexpr int kBufs = BN == 256 ? 2 : 4;
    static constexpr int kTmemCols = kBufs * BN;
    static constexpr size_t kMeta = 512 + (size_t)(MOE_MAX_EXPERTS + 1) * 8 + 256 + 4 * BM * 4;
    static constexpr int kFit = (int)((227 * 1024 - 1024 - kMeta - kEpiWarps * kStageOut) / kStageBytes);
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + kEpiWarps * kStageOut + kMeta;
    static constexpr int kCpt = BN / 2;  // columns of a tile per epilogue thread
    static_assert(kStages >= 3, "ring too shallow");
    static_assert(8 * (2 * kStages + 2 * kBufs + 4) + 8 <= 512, "barrier block");
};

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzle layout: rows of
// 128 bytes hold 128 values along M or N, one row per step of the contraction.  Eight-row
// groups are 1024 bytes apart (stride byte offset), 128-value chunks along M or N 128 rows
// apart (leading byte offset).
__device__ __forceinline__ uint64_t sdesc_sw128_mn(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((128u * 128u) >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}
// Instruction descriptor, kind::f8f6f4: D FP32; A and B e4m3 (0) or e5m2 (1), each K-major
// (0) or MN-major (1).
__device__ __forceinline__ uint32_t idesc_fp8(int a_e5m2, int b_e5m2, int a_mn, int b_mn, int N) {
    return (1u << 4) | ((uint32_t)a_e5m2 << 7) | ((uint32_t)b_e5m2 << 10) | ((uint32_t)a_mn << 15) |
           ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_fp8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

struct Tile {
    int e;      // expert
    int row0;   // first output row: of [P] (forward, input gradient) or of N (weight gradient)
    int n;      // valid rows
    int ct;     // column tile
    int nk;     // blocks along the contraction
    int blk0;   // weight gradient: first row block of the expert
};

template <int KIND>
__device__ __forceinline__ Tile decode(const ProductArgs& a, const int* off, const int* first, int nct, int tile) {
    Tile t;
    if (KIND == PK_WEIGHT_GRAD) {
        const int per = cdiv(a.rows, BM) * nct;
        t.e = tile / per;
        const int r = tile - t.e * per;
        t.row0 = (r / nct) * BM;
        t.ct = r - (r / nct) * nct;
        t.n = min(BM, a.rows - t.row0);
        t.blk0 = min(first[t.e], a.blocks);
        t.nk = min(first[t.e + 1], a.blocks) - t.blk0;
        return t;
    }
    t.e = expert_of(first, a.E, tile, nct);
    const int mts = first[t.e + 1] - first[t.e];
    int l = tile - first[t.e] * nct;
    const int band = l / (kBand * nct);
    l -= band * kBand * nct;
    const int mb = min(kBand, mts - band * kBand);
    t.ct = l / mb;
    const int mt = band * kBand + (l - t.ct * mb);
    t.row0 = off[t.e] + mt * BM;
    t.n = min(BM, off[t.e + 1] - t.row0);
    t.nk = a.nbl;
    t.blk0 = 0;
    return t;
}

// One 64-byte piece of the warp's 32 output rows: staged in shared memory with the 16-byte
// chunks of a row rotated, so that both the row-wise writes and the reads, four lanes to
// a row, are free of bank conflicts; then written 64 contiguous bytes per row.
template <typename F>
__device__ __forceinline__ void write_rows(uint8_t* stage, const uint4 (&v)[4], int lane, F&& store) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(stage + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = v[j];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2), j = lane & 3;
        store(r, j, *reinterpret_cast<const uint4*>(stage + r * 64 + ((j ^ ((r >> 1) & 3)) << 4)));
    }
    __syncwarp();
}

template <int KIND, int BN, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const ProductArgs a, const __grid_constant__ CUtensorMap tm_a,
                   const __grid_constant__ CUtensorMap tm_b, int a_rows) {
    using C = Cfg<BN>;
    constexpr bool kSwiglu = ACT == 1 + MOE_ACT_SWIGLU;
    constexpr bool kAmn = KIND == PK_WEIGHT_GRAD, kBmn = KIND != PK_FORWARD;
    constexpr int kColStep = kSwiglu ? BN / 2 : BN;  // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (base_u32 - raw_u32);
    uint8_t* staging = base + (size_t)C::kStages * C::kStageBytes;
    uint8_t* meta = staging + kEpiWarps * kStageOut;
    const uint32_t bar_u32 = smem_u32(meta);
    auto full_bar = [&](int s) { return bar_u32 + 8u * s; };
    auto empty_bar = [&](int s) { return bar_u32 + 8u * (C::kStages + s); };
    auto tfull_bar = [&](int b) { return bar_u32 + 8u * (2 * C::kStages + b); };
    auto tempty_bar = [&](int b) { return bar_u32 + 8u * (2 * C::kStages + C::kBufs + b); };
    auto amax_bar = [&](int q) { return bar_u32 + 8u * (2 * C::kStages + 2 * C::kBufs + q); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meta + 8 * (2 * C::kStages + 2 * C::kBufs + 4));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* s_off = reinterpret_cast<int*>(meta + 512);
    int* s_first = s_off + MOE_MAX_EXPERTS + 1;
    int* s_warp = s_first + MOE_MAX_EXPERTS + 1;
    uint32_t* s_amax = reinterpret_cast<uint32_t*>(s_warp + 34);  // [tile parity][half][128]
    int* err = &g_product_error;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < C::kBufs; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), kEpiWarps);
        }
        for (int q = 0; q < 4; ++q) mbar_init(amax_bar(q), 2);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    expert_blocks(a.offsets, a.E, a.P, s_off, s_first, s_warp);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int nct = cdiv(a.cols, kColStep);
    const int total = KIND == PK_WEIGHT_GRAD ? a.E * cdiv(a.rows, BM) * nct : s_first[a.E] * nct;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
                const Tile t = decode<KIND>(a, s_off, s_first, nct, tile);
                const int c0 = t.ct * kColStep;
                const int abox = KIND == PK_WEIGHT_GRAD ? 1 : cdiv(t.n, a_rows);
                const uint32_t bytes = (KIND == PK_WEIGHT_GRAD ? A_BYTES : abox * a_rows * BKB) + C::kBBytes;
                for (int kb = 0; kb < t.nk; ++kb, ++it) {
                    const int s = it % C::kStages;
                    if (!mbar_wait(empty_bar(s), ((uint32_t)(it / C::kStages) & 1u) ^ 1u, abort_flag, err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = base_u32 + (uint32_t)s * C::kStageBytes, sb = sa + A_BYTES;
                    const uint32_t bar = full_bar(s);
                    mbar_expect_tx(bar, bytes);
                    if (KIND == PK_WEIGHT_GRAD) {
                        const int r = (t.blk0 + kb) * BKB;
                        tma_load_2d(sa, &tm_a, bar, t.row0, r);
                        for (int j = 0; j < BN / 128; ++j) tma_load_2d(sb + j * 16384, &tm_b, bar, c0 + j * 128, r);
                    } else {
                        for (int j = 0; j < abox; ++j)
                            tma_load_2d(sa + j * a_rows * BKB, &tm_a, bar, kb * BKB, t.row0 + j * a_rows);
                        if (KIND == PK_INPUT_GRAD) {
                            for (int j = 0; j < BN / 128; ++j)
                                tma_load_3d(sb + j * 16384, &tm_b, bar, c0 + j * 128, kb * BKB, t.e);
                        } else if (kSwiglu) {
                            tma_load_3d(sb, &tm_b, bar, kb * BKB, c0, t.e);
                            tma_load_3d(sb + (BN / 2) * BKB, &tm_b, bar, kb * BKB, a.up + c0, t.e);
                        } else {
                            tma_load_3d(sb, &tm_b, bar, kb * BKB, c0, t.e);
                        }
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t idesc = idesc_fp8(a.a_e5m2, a.b_e5m2, kAmn, kBmn, BN);
            int it = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
                const Tile t = decode<KIND>(a, s_off, s_first, nct, tile);
                for (int kb = 0; kb < t.nk; ++kb, ++it) {
                    const int s = it % C::kStages, b = it % C::kBufs;
                    if (!mbar_wait(tempty_bar(b), ((uint32_t)(it / C::kBufs) & 1u) ^ 1u, abort_flag, err) ||
                        !mbar_wait(full_bar(s), (uint32_t)(it / C::kStages) & 1u, abort_flag, err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = base_u32 + (uint32_t)s * C::kStageBytes, sb = sa + A_BYTES;
                    const uint32_t d = tmem_base + (uint32_t)(b * BN);
#pragma unroll
                    for (int kk = 0; kk < BKB / 32; ++kk) {
                        const uint64_t ad = kAmn ? sdesc_sw128_mn(sa + kk * 4096) : sdesc_sw128(sa + kk * 32);
                        const uint64_t bd = kBmn ? sdesc_sw128_mn(sb + kk * 4096) : sdesc_sw128(sb + kk * 32);
                        tc_mma_fp8(d, ad, bd, idesc, kk > 0);
                    }
                    tc_commit(empty_bar(s));
                    tc_commit(tfull_bar(b));
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, half = (warp - 2) >> 2;
        const int r = q * 32 + lane;  // this thread's row of the tile
        uint8_t* stage = staging + (warp - 2) * kStageOut;
        const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16);
        int it = 0, ntile = 0;
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x, ++ntile) {
            const Tile t = decode<KIND>(a, s_off, s_first, nct, tile);
            const int c0 = t.ct * kColStep;
            const bool live = q * 32 < t.n;  // any row of this warp in the tile
            const bool mine = r < t.n;
            float acc[C::kCpt];
#pragma unroll
            for (int j = 0; j < C::kCpt; ++j) acc[j] = 0.0f;
            // Scales: sa of this thread's row; sb of the weight blocks of its columns.
            const float* sa = nullptr;
            const float* sb = nullptr;
            int sa_step = 1, sb_step = 1, up0 = 0, up_cut = 0;
            if (KIND == PK_WEIGHT_GRAD) {
                sa = a.sa + (size_t)t.blk0 * a.rows + t.row0 + (mine ? r : 0);
                sa_step = a.rows;
                sb = a.sb + (size_t)t.blk0 * a.cols;
                sb_step = a.cols;
            } else {
                sa = a.sa + (size_t)(t.row0 + (mine ? r : 0)) * a.nbl;
                if (KIND == PK_INPUT_GRAD) {
                    sb = a.sb + (size_t)t.e * a.wn * a.wk + min((c0 + half * C::kCpt) / 128, a.wk - 1);
                    sb_step = a.wk;
                } else {
                    const int nb = min((c0 + (kSwiglu ? half * (C::kCpt / 2) : half * C::kCpt)) / 128, a.wn - 1);
                    sb = a.sb + ((size_t)t.e * a.wn + nb) * a.wk;
                    if (kSwiglu) {  // up features start anywhere in a block: the first up_cut of them are in block up0
                        const int u = a.up + c0 + half * (C::kCpt / 2);
                        up0 = min(u / 128, a.wn - 1);
                        up_cut = (u / 128 + 1) * 128 - u;
                    }
                }
            }
            for (int kb = 0; kb < t.nk; ++kb, ++it) {
                const int b = it % C::kBufs;
                const float s0 = live ? __ldg(sa + (size_t)kb * sa_step) : 0.0f;
                float s1 = 0.0f, u1 = 0.0f, u2 = 0.0f;
                if (KIND != PK_WEIGHT_GRAD) s1 = s0 * __ldg(sb + (size_t)kb * sb_step);
                if (kSwiglu) {
                    const float* up = a.sb + ((size_t)t.e * a.wn + up0) * a.wk + kb;
                    u1 = s0 * __ldg(up);
                    u2 = up0 + 1 < a.wn ? s0 * __ldg(up + a.wk) : 0.0f;
                }
                if (!mbar_wait(tfull_bar(b), (uint32_t)(it / C::kBufs) & 1u, abort_flag, err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (live) {
#pragma unroll
                    for (int j0 = 0; j0 < C::kCpt; j0 += 32) {
                        const bool is_up = kSwiglu && j0 >= C::kCpt / 2;
                        const int col = kSwiglu ? (is_up ? BN / 2 + half * (C::kCpt / 2) + j0 - C::kCpt / 2
                                                         : half * (C::kCpt / 2) + j0)
                                                : half * C::kCpt + j0;
                        uint32_t v[32];
                        tmem_ld32(tq + (uint32_t)(b * BN + col), v);
                        tmem_ld_wait();
                        if (KIND == PK_WEIGHT_GRAD) {
                            const float* sc = sb + (size_t)kb * sb_step + c0 + col;
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (c0 + col + j < a.cols) w = __ldg(reinterpret_cast<const float4*>(sc + j));
                                acc[j0 + j] = fmaf(__uint_as_float(v[j]), s0 * w.x, acc[j0 + j]);
                                acc[j0 + j + 1] = fmaf(__uint_as_float(v[j + 1]), s0 * w.y, acc[j0 + j + 1]);
                                acc[j0 + j + 2] = fmaf(__uint_as_float(v[j + 2]), s0 * w.z, acc[j0 + j + 2]);
                                acc[j0 + j + 3] = fmaf(__uint_as_float(v[j + 3]), s0 * w.w, acc[j0 + j + 3]);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                // block boundaries fall on multiples of 16 columns
                                const float sc = is_up ? ((j0 - C::kCpt / 2 + (j & 16)) < up_cut ? u1 : u2) : s1;
                                acc[j0 + j] = fmaf(__uint_as_float(v[j]), sc, acc[j0 + j]);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(tempty_bar(b));
            }
            if (!ok) break;
            if (ACT == 0) {
                // ---- rows of the output, 64 bytes at a time
                const size_t out_row0 = (KIND == PK_WEIGHT_GRAD ? (size_t)t.e * a.rows : 0) + t.row0 + q * 32;
                if (live && (KIND != PK_WEIGHT_GRAD || t.nk > 0 || !a.accumulate)) {
                    // FP32 pieces also where BF16 values are added to: their sum is rounded once.
                    const bool add = KIND == PK_WEIGHT_GRAD && a.accumulate;
                    if (a.out_f32 || add) {
                        float* out = static_cast<float*>(a.out);
#pragma unroll
                        for (int j0 = 0; j0 < C::kCpt; j0 += 16) {
                            const int c = c0 + half * C::kCpt + j0;
                            if (c >= a.cols) break;
                            uint4 v[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                v[j] = make_uint4(__float_as_uint(acc[j0 + 4 * j]), __float_as_uint(acc[j0 + 4 * j + 1]),
                                                  __float_as_uint(acc[j0 + 4 * j + 2]),
                                                  __float_as_uint(acc[j0 + 4 * j + 3]));
                            write_rows(stage, v, lane, [&](int rr, int j, uint4 w) {
                                if (q * 32 + rr >= t.n) return;
                                const size_t at = (out_row0 + rr) * a.cols + c + 4 * j;
                                if (!a.out_f32) {
                                    uint2* p = reinterpret_cast<uint2*>(static_cast<bf16*>(a.out) + at);
                                    const uint2 o = *p;
                                    *p = make_uint2(f2bf_bits(__uint_as_float(w.x) + bf16lo(o.x)) |
                                                        ((uint32_t)f2bf_bits(__uint_as_float(w.y) + bf16hi(o.x)) << 16),
                                                    f2bf_bits(__uint_as_float(w.z) + bf16lo(o.y)) |
                                                        ((uint32_t)f2bf_bits(__uint_as_float(w.w) + bf16hi(o.y)) << 16));
                                    return;
                                }
                                float* p = out + at;
                                if (add) {
                                    const float4 o = *reinterpret_cast<const float4*>(p);
                                    w = make_uint4(__float_as_uint(__uint_as_float(w.x) + o.x),
                                                   __float_as_uint(__uint_as_float(w.y) + o.y),
                                                   __float_as_uint(__uint_as_float(w.z) + o.z),
                                                   __float_as_uint(__uint_as_float(w.w) + o.w));
                                }
                                *reinterpret_cast<uint4*>(p) = w;
                            });
                        }
                    } else {
                        bf16* out = static_cast<bf16*>(a.out);
#pragma unroll
                        for (int j0 = 0; j0 < C::kCpt; j0 += 32) {
                            const int c = c0 + half * C::kCpt + j0;
                            if (c >= a.cols) break;
                            uint4 v[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float f[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) f[i] = acc[j0 + 8 * j + i];
                                v[j] = Chunk<bf16>::pack(f);
                            }
                            write_rows(stage, v, lane, [&](int rr, int j, uint4 w) {
                                if (q * 32 + rr >= t.n || c + 8 * j >= a.cols) return;
                                *reinterpret_cast<uint4*>(out + (out_row0 + rr) * a.cols + c + 8 * j) = w;
                            });
                        }
                    }
                }
            } else {
                // ---- activation, the row's maximum over the tile's 128 features (two warps hold
                // 64 each), and 64 bytes of 8-bit values per row
                constexpr int kH = 64;
                float h[kH];
                uint32_t mx = 0;
                const int f0 = c0 + half * kH;
#pragma unroll
                for (int j = 0; j < kH; ++j) {
                    h[j] = kSwiglu ? act_swiglu(acc[j], acc[(kSwiglu ? kH : 0) + j]) : relu2_nan(acc[j]);
                    if (f0 + (j & ~15) < a.cols) mx = max(mx, abs_bits(h[j]));
                }
                // Two buffers by tile parity: a warp writes one again only after the other warp's
                // arrival for the tile between, which follows that warp's read.
                uint32_t* am = s_amax + (ntile & 1) * 2 * BM;
                am[half * BM + r] = mx;
                __syncwarp();
                if (lane == 0) mbar_arrive(amax_bar(q));
                if (!mbar_wait(amax_bar(q), (uint32_t)ntile & 1u, abort_flag, err)) break;
                mx = max(am[r], am[BM + r]);
                float scale, factor;
                block_scale(mx, fp8_max(a.h_e5m2), scale, factor);
                if (half == 0 && mine) a.out_scales[(size_t)(t.row0 + r) * cdiv(a.cols, kQBlock) + t.ct] = scale;
                if (live && f0 < a.cols) {
                    uint8_t* out = static_cast<uint8_t*>(a.out);
                    uint4 v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float f[8], g[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            f[i] = h[16 * j + i];
                            g[i] = h[16 * j + 8 + i];
                        }
                        const uint2 x = a.h_e5m2 ? pack8_fp8<true>(f, factor) : pack8_fp8<false>(f, factor);
                        const uint2 y = a.h_e5m2 ? pack8_fp8<true>(g, factor) : pack8_fp8<false>(g, factor);
                        v[j] = make_uint4(x.x, x.y, y.x, y.y);
                    }
                    write_rows(stage, v, lane, [&](int rr, int j, uint4 w) {
                        if (q * 32 + rr < t.n && f0 + 16 * j < a.cols)
                            *reinterpret_cast<uint4*>(out + (size_t)(t.row0 + q * 32 + rr) * a.cols + f0 + 16 * j) = w;
                    });
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag) {  // let in-flight bulk copies and MMAs land before the CTA retires
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 50000ull) {
        }
    }
    if (warp == 1) tmem_dealloc(tmem_base, C::kTmemCols);
}

template <int KIND, int BN, int ACT>
cudaError_t launch_t(const ProductArgs& a, const ProductMaps& m, int a_rows, int sms, cudaStream_t s) {
    auto kern = product_kernel<KIND, BN, ACT>;
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<BN>::kSmem);
    if (e != cudaSuccess) return e;
    const int step = ACT == 1 + MOE_ACT_SWIGLU ? BN / 2 : BN;
    const long long nct = cdiv(a.cols, step);
    const long long rts = KIND == PK_WEIGHT_GRAD ? (long long)a.E * cdiv(a.rows, BM)
                                                 : a.P / BM + std::min(a.E, a.P);
    const int grid = (int)std::max<long long>(1, std::min<long long>(nct * rts, sms));
    return launch_k(kern, dim3(grid), dim3(kThreads), Cfg<BN>::kSmem, s, false, a, m.a, m.b, a_rows);
}

}  // namespace

ProductTile product_tile(int kind, int act, const ProductArgs& a, int sms) {
    if (act == 1 + MOE_ACT_SWIGLU) return {256, 32};
    if (act) return {128, 32};
    if (kind == PK_WEIGHT_GRAD) return {256, 128};
    if ((long long)a.P >= 64LL * a.E) return {256, 128};
    return {128, 32};
}

cudaError_t launch_product(int kind, int act, const ProductTile& t, const ProductArgs& a, const ProductMaps& m,
                           int sms, cudaStream_t s) {
    if (act == 1 + MOE_ACT_SWIGLU) return launch_t<PK_FORWARD, 256, 1 + MOE_ACT_SWIGLU>(a, m, t.a_rows, sms, s);
    if (act == 1 + MOE_ACT_RELU2) return launch_t<PK_FORWARD, 128, 1 + MOE_ACT_RELU2>(a, m, t.a_rows, sms, s);
    switch (kind) {
        case PK_FORWARD:
            return t.bn == 256 ? launch_t<PK_FORWARD, 256, 0>(a, m, t.a_rows, sms, s)
                               : launch_t<PK_FORWARD, 128, 0>(a, m, t.a_rows, sms, s);
        case PK_INPUT_GRAD:
            return t.bn == 256 ? launch_t<PK_INPUT_GRAD, 256, 0>(a, m, t.a_rows, sms, s)
                               : launch_t<PK_INPUT_GRAD, 128, 0>(a, m, t.a_rows, sms, s);
        case PK_WEIGHT_GRAD: return launch_t<PK_WEIGHT_GRAD, 256, 0>(a, m, t.a_rows, sms, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t product_error(int* code, cudaStream_t s) {
    void* p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_product_error);
    if (e == cudaSuccess) e = cudaMemcpyAsync(code, p, sizeof(int), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(p, 0, sizeof(int), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return e;
}

}  // namespace moe
