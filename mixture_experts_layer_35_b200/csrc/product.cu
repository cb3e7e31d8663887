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
// Warps: 0 TMA producer, 1 TMEM allocator and MMA issuer, 4-11 epilogue (warp w reads TMEM
// lanes of quarter w % 4 and one half of the columns); 2 and 3 only fill the warpgroup.  One persistent CTA per SM; tiles go
// round-robin, inside an expert in bands of 16 row tiles, column tiles outer, so that the
// CTAs at work share weights and rows in L2.
#include "experts.cuh"

namespace moe {
namespace {

__device__ int g_product_error;  // MOE_DEVERR_* bits of the products on this device

constexpr int BM = 128, BKB = 128;  // tile rows; bytes (= values) of one block along the contraction
constexpr int kBand = 16;           // row tiles that share a pass over the weights
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
// With 128 sums a thread (BN = 256) the epilogue warpgroups take registers from the first
// one: 128 * 40 + 256 * 224 of the 384 * 168 that a block is launched with.
constexpr int kRegsIssue = 40, kRegsEpilogue = 224;
constexpr int kRegsLaunch = (128 * kRegsIssue + 256 * kRegsEpilogue + kThreads - 1) / kThreads;
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
    static constexpr bool kMoveRegs = BN == 256;
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

template <int N>
__device__ __forceinline__ void regs_set_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_set_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
// Waits for this thread's TMEM loads; the values loaded cannot be used before it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                   "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                   "+r"(v[30]), "+r"(v[31]));
}
// Two FP32 operations in one instruction, on register pairs.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    return pair(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ void unpair(uint64_t p, float& lo, float& hi) {
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(p));
    lo = __uint_as_float(a);
    hi = __uint_as_float(b);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
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

    if (warp < 4) {
        if (C::kMoveRegs) regs_set_down<kRegsIssue>();
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
        }
    } else {
        // ------------------------------------------------------------ epilogue
        if (C::kMoveRegs) regs_set_up<kRegsEpilogue>();
        const int q = warp & 3, half = (warp - 4) >> 2;
        const int r = q * 32 + lane;  // this thread's row of the tile
        uint8_t* stage = staging + (warp - 4) * kStageOut;
        const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16);
        int it = 0, ntile = 0;
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x, ++ntile) {
            const Tile t = decode<KIND>(a, s_off, s_first, nct, tile);
            const int c0 = t.ct * kColStep;
            const bool live = q * 32 < t.n;  // any row of this warp in the tile
            const bool mine = r < t.n;
            uint64_t acc2[C::kCpt / 2];  // the sums, in pairs of neighbouring columns
#pragma unroll
            for (int j = 0; j < C::kCpt / 2; ++j) acc2[j] = 0;
            // Scales of a block, loaded one block ahead: ra of this thread's row; rb of the weight
            // block of its columns.  SwiGLU's up features start anywhere in a weight block: the
            // first up_cut of them lie in block up0 (ru), the others in the next (rv).  Weight
            // gradient: each lane loads four of the warp's column scales (rc), and passes them
            // through shared memory.
            const float* sa = nullptr;
            const float* sb = nullptr;
            const float* su = nullptr;
            const float* sv = nullptr;
            int sa_step = 1, sb_step = 1, up_cut = 0;
            const bool cols_in = c0 + half * C::kCpt + 4 * lane < a.cols && 4 * lane < C::kCpt;
            if (KIND == PK_WEIGHT_GRAD) {
                sa = a.sa + (size_t)t.blk0 * a.rows + t.row0 + (mine ? r : 0);
                sa_step = a.rows;
                sb = a.sb + (size_t)t.blk0 * a.cols + (cols_in ? c0 + half * C::kCpt + 4 * lane : 0);
                sb_step = a.cols;
            } else {
                sa = a.sa + (size_t)(t.row0 + (mine ? r : 0)) * a.nbl;
                if (KIND == PK_INPUT_GRAD) {
                    sb = a.sb + (size_t)t.e * a.wn * a.wk + min((c0 + half * C::kCpt) / 128, a.wk - 1);
                    sb_step = a.wk;
                } else {
                    const int nb = min((c0 + (kSwiglu ? half * (C::kCpt / 2) : half * C::kCpt)) / 128, a.wn - 1);
                    sb = a.sb + ((size_t)t.e * a.wn + nb) * a.wk;
                    if (kSwiglu) {
                        const int u = a.up + c0 + half * (C::kCpt / 2);
                        const int up0 = min(u / 128, a.wn - 1);
                        up_cut = (u / 128 + 1) * 128 - u;
                        su = a.sb + ((size_t)t.e * a.wn + up0) * a.wk;
                        sv = a.sb + ((size_t)t.e * a.wn + min(up0 + 1, a.wn - 1)) * a.wk;
                    }
                }
            }
            float ra = 0.0f, rb = 0.0f, ru = 0.0f, rv = 0.0f;
            float4 rc = make_float4(0.f, 0.f, 0.f, 0.f);
            auto load_scales = [&](int kb) {
                if (!live) return;
                ra = __ldg(sa + (size_t)kb * sa_step);
                if (KIND == PK_WEIGHT_GRAD) {
                    if (cols_in) rc = __ldg(reinterpret_cast<const float4*>(sb + (size_t)kb * sb_step));
                } else {
                    rb = __ldg(sb + (size_t)kb * sb_step);
                    if (kSwiglu) {
                        ru = __ldg(su + kb);
                        rv = __ldg(sv + kb);
                    }
                }
            };
            if (t.nk > 0) load_scales(0);
            for (int kb = 0; kb < t.nk; ++kb, ++it) {
                const int b = it % C::kBufs;
                const float s0 = ra;
                const uint64_t s1 = KIND == PK_WEIGHT_GRAD ? pair(s0, s0) : pair(s0 * rb, s0 * rb);
                const uint64_t u1 = pair(s0 * ru, s0 * ru), u2 = pair(s0 * rv, s0 * rv);
                if (KIND == PK_WEIGHT_GRAD) {
                    __syncwarp();  // the last block's scales have been read
                    if (4 * lane < C::kCpt) reinterpret_cast<float4*>(stage)[lane] = rc;
                    __syncwarp();
                }
                if (kb + 1 < t.nk) load_scales(kb + 1);
                if (!mbar_wait(tfull_bar(b), (uint32_t)(it / C::kBufs) & 1u, abort_flag, err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (live) {
                    // 32 columns at a time, the next ones loading while these are added
                    uint32_t v[2][32];
                    auto column = [&](int j0) {  // first TMEM column of piece j0 of this thread
                        if (!kSwiglu) return half * C::kCpt + j0;
                        return (j0 >= C::kCpt / 2 ? BN / 2 - C::kCpt / 2 : 0) + half * (C::kCpt / 2) + j0;
                    };
                    const uint32_t tb = tq + (uint32_t)(b * BN);
                    tmem_ld32(tb + column(0), v[0]);
#pragma unroll
                    for (int j0 = 0; j0 < C::kCpt; j0 += 32) {
                        uint32_t(&w)[32] = v[(j0 / 32) & 1];
                        tmem_ld_wait_for(w);
                        if (j0 + 32 < C::kCpt) {
                            tmem_ld32(tb + column(j0 + 32), v[(j0 / 32 + 1) & 1]);
                        } else {  // the buffer has been read
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(tempty_bar(b));
                        }
                        const bool is_up = kSwiglu && j0 >= C::kCpt / 2;
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            uint64_t sc = s1;
                            if (KIND == PK_WEIGHT_GRAD)
                                sc = mul2(s1, *reinterpret_cast<const uint64_t*>(stage + (j0 + j) * 4));
                            else if (is_up)  // block boundaries fall on multiples of 16 columns
                                sc = (j0 - C::kCpt / 2 + (j & 16)) < up_cut ? u1 : u2;
                            acc2[(j0 + j) / 2] = fma2(pair(w[j], w[j + 1]), sc, acc2[(j0 + j) / 2]);
                        }
                    }
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tempty_bar(b));
                }
            }
            __syncwarp();
            float acc[C::kCpt];
#pragma unroll
            for (int j = 0; j < C::kCpt / 2; ++j) unpair(acc2[j], acc[2 * j], acc[2 * j + 1]);
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
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<BN>::kSmem);
    if (e != cudaSuccess) return e;
    if (Cfg<BN>::kMoveRegs) {  // the registers moved between warpgroups must be the block's own
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, kern);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
    }
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
