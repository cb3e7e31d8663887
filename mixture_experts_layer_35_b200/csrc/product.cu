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
// Warps: 0 TMA producer, 1 TMEM allocator and MMA issuer, 2 loads scales into
// a ring in shared memory, 4-11 epilogue (warp w reads TMEM lanes of quarter w % 4 and one half of
// the columns); 3 only fills the warpgroup.  One persistent CTA per SM; tiles go
// round-robin, inside an expert in bands of 16 row tiles, column tiles outer, so that the
// CTAs at work share weights and rows in L2.
#include "experts.cuh"

namespace moe {
namespace {

__device__ int g_product_error;  // MOE_DEVERR_* bits of the products on this device

constexpr int BM = 128, BKB = 128;  // rows of an MMA; bytes (= values) of one block along the contraction
constexpr int kBand = 16;           // row tiles that share a pass over the weights
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
// With 128 sums a thread (BN = 256) the epilogue warpgroups take registers from the first
// one: 128 * 40 + 256 * 224 of the 384 * 168 that a block is launched with.
constexpr int kRegsIssue = 40, kRegsEpilogue = 224;
constexpr int kRegsLaunch = (128 * kRegsIssue + 256 * kRegsEpilogue + kThreads - 1) / kThreads;

// HT: rows of a tile, 128, or 32 where experts have few rows.  A 32-row tile loads only its
// rows; the MMA's other 96 lanes read whatever follows them in shared memory, and nothing
// reads their sums.
template <int KIND, int BN, int HT, int ACT>
struct Cfg {
    static constexpr int kABytes = HT * BKB;
    static constexpr int kStageBytes = kABytes + BN * BKB;
    static constexpr int kBufs = BN == 256 ? 2 : 4;
    static constexpr int kTmemCols = kBufs * BN;
    static constexpr int kCpt = BN / 2;  // columns of a tile per epilogue thread
    // Epilogue warps with rows, and each one's staging: two boxes of 32 rows x 128 bytes for the
    // copy engine, or 32 rows x 64 bytes where a tile's rows are few or its values 8-bit.
    static constexpr int kRowWarps = HT == 32 ? 2 : kEpiWarps;
    static constexpr bool kBulkStore = HT == 128 && ACT == 0;
    static constexpr int kStageOut = kBulkStore ? 8192 : 2048;
    // Ring of scales, one slot per block along the contraction: the rows' 128, and the weight
    // blocks' (four for each half of the columns) or, for the weight gradient, the columns'.
    static constexpr int kSlots = 4;
    static constexpr int kSlotFloats = BM + (KIND == PK_WEIGHT_GRAD ? BN : 8);
    static constexpr size_t kTables = 512 + (size_t)(2 * (MOE_MAX_EXPERTS + 1) + 34) * 4;
    static constexpr size_t kScales = (kTables + 15) / 16 * 16;
    static constexpr size_t kAmax = kScales + (size_t)kSlots * kSlotFloats * 4;
    static constexpr size_t kMeta = kAmax + (ACT ? 4 * BM * 4 : 0);
    static constexpr int kFit =
        (int)((227 * 1024 - 1024 - kMeta - kRowWarps * kStageOut) / kStageBytes);
    static constexpr int kStages = kFit < 16 ? kFit : 16;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + kRowWarps * kStageOut + kMeta;
    static constexpr bool kMoveRegs = BN == 256;
    static_assert(kStages >= 3, "ring too shallow");
    static_assert(kABytes + BN * BKB + kRowWarps * kStageOut >= BM * BKB, "an MMA's rows must lie in shared memory");
    static_assert(8 * (2 * kStages + 2 * kBufs + 2 * kSlots + 4) + 8 <= 512, "barrier block");
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
// 32 lanes x 16 columns of 32-bit sums.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
// Waits for this thread's TMEM loads; the values loaded cannot be used before it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                   "+r"(v[15]));
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
// Four-byte asynchronous copy to shared memory, and an arrival on `bar` once this thread's
// copies so far have landed.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

struct Tile {
    int e;      // expert
    int row0;   // first output row: of [P] (forward, input gradient) or of N (weight gradient)
    int n;      // valid rows
    int c0;     // first output column
    int nk;     // blocks along the contraction
    int blk0;   // weight gradient: first row block of the expert
};

template <int KIND, int HT>
__device__ __forceinline__ Tile decode(const ProductArgs& a, const int* off, const int* first, int nct, int step,
                                       int tile) {
    Tile t;
    if (KIND == PK_WEIGHT_GRAD) {
        const int per = cdiv(a.rows, BM) * nct;
        t.e = tile / per;
        const int r = tile - t.e * per;
        t.row0 = (r / nct) * BM;
        t.c0 = (r - (r / nct) * nct) * step;
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
    const int ct = l / mb;
    t.c0 = ct * step;
    t.row0 = off[t.e] + (band * kBand + (l - ct * mb)) * HT;
    t.n = min(HT, off[t.e + 1] - t.row0);
    t.nk = a.nbl;
    t.blk0 = 0;
    return t;
}

// One 64-byte piece of the warp's 32 output rows: staged in shared memory with the 16-byte
// chunks of a row rotated, so that both the row-wise writes and the reads, four lanes to
// a row, are free of bank conflicts; then store(row, chunk, value) with 64 contiguous bytes
// per row.
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

// A box of 32 rows x 128 bytes from shared memory to global memory, what lies outside the tensor
// dropped, or added to what is there.
__device__ __forceinline__ void store_box(const CUtensorMap* tm, uint32_t src, int c0, int c1, int c2, bool add) {
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(tm)),
                     "r"(src), "r"(c0), "r"(c1), "r"(c2)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(tm)),
                     "r"(src), "r"(c0), "r"(c1), "r"(c2)
                     : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Waits until at most N of this thread's boxes are still being read from shared memory.
template <int N>
__device__ __forceinline__ void store_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int KIND, int BN, int HT, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const ProductArgs a, const __grid_constant__ CUtensorMap tm_a,
                   const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_out) {
    using C = Cfg<KIND, BN, HT, ACT>;
    constexpr bool kSwiglu = ACT == 1 + MOE_ACT_SWIGLU;
    constexpr bool kAmn = KIND == PK_WEIGHT_GRAD, kBmn = KIND != PK_FORWARD;
    constexpr int kColStep = kSwiglu ? BN / 2 : BN;  // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (base_u32 - raw_u32);
    uint8_t* staging = base + (size_t)C::kStages * C::kStageBytes;
    uint8_t* meta = staging + C::kRowWarps * C::kStageOut;
    const uint32_t bar_u32 = smem_u32(meta);
    auto full_bar = [&](int s) { return bar_u32 + 8u * s; };
    auto empty_bar = [&](int s) { return bar_u32 + 8u * (C::kStages + s); };
    auto tfull_bar = [&](int b) { return bar_u32 + 8u * (2 * C::kStages + b); };
    auto tempty_bar = [&](int b) { return bar_u32 + 8u * (2 * C::kStages + C::kBufs + b); };
    auto sfull_bar = [&](int i) { return bar_u32 + 8u * (2 * C::kStages + 2 * C::kBufs + i); };
    auto sempty_bar = [&](int i) { return bar_u32 + 8u * (2 * C::kStages + 2 * C::kBufs + C::kSlots + i); };
    auto amax_bar = [&](int q) { return bar_u32 + 8u * (2 * C::kStages + 2 * C::kBufs + 2 * C::kSlots + q); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meta + 8 * (2 * C::kStages + 2 * C::kBufs + 2 * C::kSlots + 4));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* s_off = reinterpret_cast<int*>(meta + 512);
    int* s_first = s_off + MOE_MAX_EXPERTS + 1;
    int* s_warp = s_first + MOE_MAX_EXPERTS + 1;
    float* s_scales = reinterpret_cast<float*>(meta + C::kScales);
    uint32_t* s_amax = reinterpret_cast<uint32_t*>(meta + C::kAmax);  // fused activation: [tile parity][half][128]
    int* err = &g_product_error;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < C::kBufs; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), C::kRowWarps);
        }
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(sfull_bar(i), 32);
            mbar_init(sempty_bar(i), C::kRowWarps);
        }
        for (int q = 0; q < 4; ++q) mbar_init(amax_bar(q), 2);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
        if (C::kBulkStore) tma_prefetch_desc(&tm_out);
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    expert_blocks<HT>(a.offsets, a.E, a.P, s_off, s_first, s_warp);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int nct = cdiv(a.cols, kColStep);
    const int total = KIND == PK_WEIGHT_GRAD ? a.E * cdiv(a.rows, BM) * nct : s_first[a.E] * nct;
    auto tile_at = [&](int tile) { return decode<KIND, HT>(a, s_off, s_first, nct, kColStep, tile); };

    if (warp < 4) {
        if (C::kMoveRegs) regs_set_down<kRegsIssue>();
        if (warp == 0) {
            // ------------------------------------------------------------ TMA producer
            if (lane == 0) {
                int it = 0;
                bool ok = true;
                for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
                    const Tile t = tile_at(tile);
                    for (int kb = 0; kb < t.nk; ++kb, ++it) {
                        const int s = it % C::kStages;
                        if (!mbar_wait(empty_bar(s), ((uint32_t)(it / C::kStages) & 1u) ^ 1u, abort_flag, err)) {
                            ok = false;
                            break;
                        }
                        const uint32_t sa = base_u32 + (uint32_t)s * C::kStageBytes, sb = sa + C::kABytes;
                        const uint32_t bar = full_bar(s);
                        mbar_expect_tx(bar, C::kStageBytes);
                        if (KIND == PK_WEIGHT_GRAD) {
                            const int r = (t.blk0 + kb) * BKB;
                            tma_load_2d(sa, &tm_a, bar, t.row0, r);
                            for (int j = 0; j < BN / 128; ++j) tma_load_2d(sb + j * 16384, &tm_b, bar, t.c0 + j * 128, r);
                            continue;
                        }
                        tma_load_2d(sa, &tm_a, bar, kb * BKB, t.row0);
                        if (KIND == PK_INPUT_GRAD) {
                            for (int j = 0; j < BN / 128; ++j)
                                tma_load_3d(sb + j * 16384, &tm_b, bar, t.c0 + j * 128, kb * BKB, t.e);
                        } else if (kSwiglu) {  // 64 gate rows, their up rows, and again
                            for (int j = 0; j < 2; ++j) {
                                tma_load_3d(sb + j * 16384, &tm_b, bar, kb * BKB, t.c0 + j * 64, t.e);
                                tma_load_3d(sb + j * 16384 + 8192, &tm_b, bar, kb * BKB, a.up + t.c0 + j * 64, t.e);
                            }
                        } else {
                            tma_load_3d(sb, &tm_b, bar, kb * BKB, t.c0, t.e);
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
                    const Tile t = tile_at(tile);
                    for (int kb = 0; kb < t.nk; ++kb, ++it) {
                        const int s = it % C::kStages, b = it % C::kBufs;
                        if (!mbar_wait(full_bar(s), (uint32_t)(it / C::kStages) & 1u, abort_flag, err)) {
                            ok = false;
                            break;
                        }
                        const uint32_t sa = base_u32 + (uint32_t)s * C::kStageBytes, sb = sa + C::kABytes;
                        if (!mbar_wait(tempty_bar(b), ((uint32_t)(it / C::kBufs) & 1u) ^ 1u, abort_flag, err)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tmem_base + (uint32_t)(b * BN);
#pragma unroll
                        for (int kk = 0; kk < BKB / 32; ++kk) {
                            const uint64_t ad = kAmn ? sdesc_sw128_mn(sa + kk * 4096) : sdesc_sw128(sa + kk * 32);
                            const uint64_t bd = kBmn ? sdesc_sw128_mn(sb + kk * 4096) : sdesc_sw128(sb + kk * 32);
                            tc_mma_fp8(d, ad, bd, idesc, kk > 0);
                        }
                        tc_commit(tfull_bar(b));
                        tc_commit(empty_bar(s));
                    }
                }
            }
        } else if (warp == 2) {
            // ------------------------------------------------------------ scales
            // Up to kSlots blocks ahead of the sums, so that no sum waits for memory.  SwiGLU's up
            // features start anywhere in a weight block: 64 of them lie in one or two blocks.
            int it = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
                const Tile t = tile_at(tile);
                const float* wsc = a.sb + (size_t)t.e * a.wn * a.wk;
                int w0 = 0, w_step = 1;  // this lane's weight scale (lanes 0-7: four for each half)
                if (KIND == PK_INPUT_GRAD) {
                    w0 = min((t.c0 + (lane >> 2) * C::kCpt) / 128, a.wk - 1);
                    w_step = a.wk;
                } else if (KIND == PK_FORWARD) {
                    const int c = t.c0 + (lane >> 2) * (kSwiglu ? 64 : C::kCpt);
                    int nb = (kSwiglu && (lane & 3) ? a.up + c : c) / 128;
                    if ((lane & 3) == 2) ++nb;
                    w0 = min(nb, a.wn - 1) * a.wk;
                }
                for (int kb = 0; kb < t.nk; ++kb, ++it) {
                    const int i = it % C::kSlots;
                    if (!mbar_wait(sempty_bar(i), ((uint32_t)(it / C::kSlots) & 1u) ^ 1u, abort_flag, err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = smem_u32(s_scales + (size_t)i * C::kSlotFloats);
                    if (KIND == PK_WEIGHT_GRAD) {
                        const size_t blk = t.blk0 + kb;
                        if (t.row0 + 4 * lane < a.rows) cp_async16(dst + 16 * lane, a.sa + blk * a.rows + t.row0 + 4 * lane, 16);
                        for (int j = lane; j < BN / 4; j += 32)
                            if (t.c0 + 4 * j < a.cols)
                                cp_async16(dst + (BM + 4 * j) * 4, a.sb + blk * a.cols + t.c0 + 4 * j, 16);
                    } else {
                        for (int r = lane; r < t.n; r += 32)
                            cp_async4(dst + 4 * r, a.sa + (size_t)(t.row0 + r) * a.nbl + kb);
                        if (lane < 8) cp_async4(dst + (BM + lane) * 4, wsc + w0 + (size_t)kb * w_step);
                    }
                    cp_async_arrive(sfull_bar(i));
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        if (C::kMoveRegs) regs_set_up<kRegsEpilogue>();
        const int q = warp & 3, half = (warp - 4) >> 2;
        const int r = q * 32 + lane;  // this thread's row of the tile
        uint8_t* stage = staging + (HT == 32 ? half : warp - 4) * C::kStageOut;
        const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * C::kCpt);
        int it = 0, ntile = 0, nbox = 0;
        bool ok = true;
        // (the warps without rows of a 32-row tile have nothing to do)
        for (int tile = HT == 32 && q != 0 ? total : blockIdx.x; tile < total; tile += gridDim.x, ++ntile) {
            const Tile t = tile_at(tile);
            const bool live = q * 32 < t.n, mine = r < t.n;
            const int up_cut = kSwiglu ? 128 - (a.up + t.c0 + half * 64) % 128 : 0;  // up features in the first block
            uint64_t acc2[C::kCpt / 2];  // the sums, in pairs of neighbouring columns
#pragma unroll
            for (int j = 0; j < C::kCpt / 2; ++j) acc2[j] = 0;
            for (int kb = 0; kb < t.nk; ++kb, ++it) {
                const int b = it % C::kBufs, i = it % C::kSlots;
                if (!mbar_wait(sfull_bar(i), (uint32_t)(it / C::kSlots) & 1u, abort_flag, err) ||
                    !mbar_wait(tfull_bar(b), (uint32_t)(it / C::kBufs) & 1u, abort_flag, err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (live) {
                    const float* sc = s_scales + (size_t)i * C::kSlotFloats;
                    const float* sw = sc + BM + (KIND == PK_WEIGHT_GRAD ? half * C::kCpt : 4 * half);
                    const uint32_t tb = tq + (uint32_t)(b * BN);
                    // Up to 64 columns are read in one go: with few rows two warps of one scheduler do all
                    // the sums, and each read's latency counts (product of 128 rows of 256 experts: 55 ->
                    // 50 us).  128 are read 16 at a time, the next ones loading while these are added:
                    // there are not the registers for more (with 32 the allocator copies the loaded values
                    // into pairs: 1014 -> 1435 us at 16384 x 8192 x 8192).  So are the weight gradient's 64
                    // (119 against 127 us for 64 experts x 256 rows x 1024 x 2048).
                    constexpr bool kAtOnce = C::kCpt <= 64 && KIND != PK_WEIGHT_GRAD;
                    constexpr int kVec = kAtOnce ? C::kCpt / 16 : 2;
                    uint32_t v[kVec][16];
#pragma unroll
                    for (int i16 = 0; i16 < (kAtOnce ? kVec : 1); ++i16) tmem_ld16(tb + 16 * i16, v[i16]);
                    const float s0 = sc[r];
                    const float s1 = KIND == PK_WEIGHT_GRAD ? s0 : s0 * sw[0];
                    const float u1 = kSwiglu ? s0 * sw[1] : 0.0f, u2 = kSwiglu ? s0 * sw[2] : 0.0f;
#pragma unroll
                    for (int j0 = 0; j0 < C::kCpt; j0 += 16) {
                        uint32_t(&w)[16] = v[(j0 / 16) % kVec];
                        tmem_ld_wait_for(w);
                        if (!kAtOnce && j0 + 16 < C::kCpt) tmem_ld16(tb + j0 + 16, v[(j0 / 16 + 1) % kVec]);
                        if (j0 == (kAtOnce ? 0 : C::kCpt - 16)) {  // the buffer has been read
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(tempty_bar(b));
                        }
                        const bool is_up = kSwiglu && j0 >= C::kCpt / 2;
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            uint64_t a0 = pair(s1, s1), a1 = a0;
                            if (KIND == PK_WEIGHT_GRAD) {
                                const float4 c4 = *reinterpret_cast<const float4*>(sw + j0 + j);
                                a1 = mul2(a0, pair(c4.z, c4.w));
                                a0 = mul2(a0, pair(c4.x, c4.y));
                            } else if (is_up) {  // block boundaries fall on multiples of 16 columns
                                const float u = (j0 - C::kCpt / 2) < up_cut ? u1 : u2;
                                a0 = a1 = pair(u, u);
                            }
                            acc2[(j0 + j) / 2] = fma2(pair(w[j], w[j + 1]), a0, acc2[(j0 + j) / 2]);
                            acc2[(j0 + j) / 2 + 1] = fma2(pair(w[j + 2], w[j + 3]), a1, acc2[(j0 + j) / 2 + 1]);
                        }
                    }
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tempty_bar(b));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sempty_bar(i));
            }
            if (!ok) break;
            float acc[C::kCpt];
#pragma unroll
            for (int j = 0; j < C::kCpt / 2; ++j) unpair(acc2[j], acc[2 * j], acc[2 * j + 1]);
            if (ACT == 0) {
                // ---- rows of the output, 64 bytes at a time
                const size_t out_row0 = (KIND == PK_WEIGHT_GRAD ? (size_t)t.e * a.rows : 0) + t.row0 + q * 32;
                const int c = t.c0 + half * C::kCpt, rows = t.n - q * 32;
                const bool add = KIND == PK_WEIGHT_GRAD && a.accumulate;
                if (C::kBulkStore && KIND != PK_WEIGHT_GRAD && rows < 32) {  // staged by hand below
                    if (lane == 0) store_wait_read<0>();
                    __syncwarp();
                }
                // Whole 32-row blocks go through the copy engine (rows past an expert's end must not be
                // written; past the tensor's end it drops them), two boxes at a time per warp, so that
                // they drain while the next tile is summed.
                const bool boxes = C::kBulkStore && (KIND == PK_WEIGHT_GRAD ? a.out_f32 || !add : rows >= 32);
                if (!live || (add && t.nk == 0)) {
                    // nothing to write
                } else if (boxes) {
                    const int row = t.row0 + q * 32, e = KIND == PK_WEIGHT_GRAD ? t.e : 0;
                    auto box = [&](int j0, auto chunk) {  // chunk(j): 16 bytes of this thread's row
                        if (lane == 0) store_wait_read<1>();
                        __syncwarp();
                        uint8_t* slot = stage + (nbox & 1) * 4096;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint4*>(slot + lane * 128 + ((j ^ (lane & 7)) << 4)) = chunk(j);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) store_box(&tm_out, smem_u32(slot), c + j0, row, e, add);
                        ++nbox;
                    };
                    if (a.out_f32) {
#pragma unroll
                        for (int j0 = 0; j0 < C::kCpt; j0 += 32) {
                            if (c + j0 >= a.cols) break;
                            box(j0, [&](int j) {
                                return make_uint4(__float_as_uint(acc[j0 + 4 * j]), __float_as_uint(acc[j0 + 4 * j + 1]),
                                                  __float_as_uint(acc[j0 + 4 * j + 2]),
                                                  __float_as_uint(acc[j0 + 4 * j + 3]));
                            });
                        }
                    } else {
#pragma unroll
                        for (int j0 = 0; j0 + 64 <= C::kCpt; j0 += 64) {
                            if (c + j0 >= a.cols) break;
                            box(j0, [&](int j) {
                                float f[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) f[i] = acc[j0 + 8 * j + i];
                                return Chunk<bf16>::pack(f);
                            });
                        }
                    }
                } else if (a.out_f32 || add) {  // FP32 pieces also where BF16 values are added to: rounded once
#pragma unroll
                    for (int j0 = 0; j0 < C::kCpt; j0 += 16) {
                        if (c + j0 >= a.cols) break;
                        uint4 v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            v[j] = make_uint4(__float_as_uint(acc[j0 + 4 * j]), __float_as_uint(acc[j0 + 4 * j + 1]),
                                              __float_as_uint(acc[j0 + 4 * j + 2]), __float_as_uint(acc[j0 + 4 * j + 3]));
                        write_rows(stage, v, lane, [&](int rr, int j, uint4 w) {
                            if (rr >= rows) return;
                            const size_t at = (out_row0 + rr) * a.cols + c + j0 + 4 * j;
                            float f[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z),
                                          __uint_as_float(w.w)};
                            if (a.out_f32) {
                                float* p = static_cast<float*>(a.out) + at;
                                if (add) {
                                    const float4 o = *reinterpret_cast<const float4*>(p);
                                    f[0] += o.x, f[1] += o.y, f[2] += o.z, f[3] += o.w;
                                }
                                *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
                            } else {
                                uint2* p = reinterpret_cast<uint2*>(static_cast<bf16*>(a.out) + at);
                                const uint2 o = *p;
                                *p = make_uint2(f2bf_bits(f[0] + bf16lo(o.x)) | ((uint32_t)f2bf_bits(f[1] + bf16hi(o.x)) << 16),
                                                f2bf_bits(f[2] + bf16lo(o.y)) | ((uint32_t)f2bf_bits(f[3] + bf16hi(o.y)) << 16));
                            }
                        });
                    }
                } else {
                    bf16* out = static_cast<bf16*>(a.out);
#pragma unroll
                    for (int j0 = 0; j0 < C::kCpt; j0 += 32) {
                        if (c + j0 >= a.cols) break;
                        uint4 v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float f[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) f[i] = acc[j0 + 8 * j + i];
                            v[j] = Chunk<bf16>::pack(f);
                        }
                        write_rows(stage, v, lane, [&](int rr, int j, uint4 w) {
                            if (rr < rows && c + j0 + 8 * j < a.cols)
                                *reinterpret_cast<uint4*>(out + (out_row0 + rr) * a.cols + c + j0 + 8 * j) = w;
                        });
                    }
                }
            } else {
                // ---- activation, the row's maximum over the tile's 128 features (two warps hold
                // 64 each), and 64 bytes of 8-bit values per row
                constexpr int kH = 64;
                float h[kH];
                uint32_t mx = 0;
                const int f0 = t.c0 + half * kH;
#pragma unroll
                for (int j = 0; j < kH; ++j) {
                    h[j] = kSwiglu ? quick_swiglu(acc[j], acc[(kSwiglu ? kH : 0) + j]) : relu2_nan(acc[j]);
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
                if (half == 0 && mine)
                    a.out_scales[(size_t)(t.row0 + r) * cdiv(a.cols, kQBlock) + t.c0 / kQBlock] = scale;
                if (live && f0 < a.cols) {
                    uint8_t* out = static_cast<uint8_t*>(a.out) + (size_t)(t.row0 + q * 32) * a.cols + f0;
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
                            *reinterpret_cast<uint4*>(out + (size_t)rr * a.cols + 16 * j) = w;
                    });
                }
            }
        }
        if (C::kBulkStore && lane == 0) store_wait();
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

template <int KIND, int BN, int HT, int ACT>
cudaError_t launch_t(const ProductArgs& a, const ProductMaps& m, int sms, cudaStream_t s) {
    using C = Cfg<KIND, BN, HT, ACT>;
    auto kern = product_kernel<KIND, BN, HT, ACT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    if (C::kMoveRegs) {  // the registers moved between warpgroups must be the block's own
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, kern);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
    }
    const int step = ACT == 1 + MOE_ACT_SWIGLU ? BN / 2 : BN;
    const long long nct = cdiv(a.cols, step);
    const long long rts = KIND == PK_WEIGHT_GRAD ? (long long)a.E * cdiv(a.rows, BM) : a.P / HT + std::min(a.E, a.P);
    const int grid = (int)std::max<long long>(1, std::min<long long>(nct * rts, sms));
    return launch_k(kern, dim3(grid), dim3(kThreads), C::kSmem, s, false, a, m.a, m.b, m.out);
}

}  // namespace

ProductTile product_tile(int kind, int act, const ProductArgs& a, int sms) {
    if (kind == PK_WEIGHT_GRAD) return {(long long)a.blocks >= 6LL * a.E ? 256 : 128, 128};
    const int ht = (long long)a.P >= 32LL * a.E ? 128 : 32;
    if (act) return {act == 1 + MOE_ACT_SWIGLU ? 256 : 128, ht};
    if (ht == 128) return {256, 128};
    const bool few = (long long)std::min(a.E, a.P) * cdiv(a.cols, 128) < sms;
    return {kind == PK_FORWARD && few ? 64 : 128, 32};
}

cudaError_t launch_product(int kind, int act, const ProductTile& t, const ProductArgs& a, const ProductMaps& m,
                           int sms, cudaStream_t s) {
    constexpr int kSw = 1 + MOE_ACT_SWIGLU, kRe = 1 + MOE_ACT_RELU2;
    const bool tall = t.rows == 128;
    if (act == kSw)
        return tall ? launch_t<PK_FORWARD, 256, 128, kSw>(a, m, sms, s) : launch_t<PK_FORWARD, 256, 32, kSw>(a, m, sms, s);
    if (act == kRe)
        return tall ? launch_t<PK_FORWARD, 128, 128, kRe>(a, m, sms, s) : launch_t<PK_FORWARD, 128, 32, kRe>(a, m, sms, s);
    if (kind == PK_WEIGHT_GRAD)
        return t.bn == 256 ? launch_t<PK_WEIGHT_GRAD, 256, 128, 0>(a, m, sms, s)
                           : launch_t<PK_WEIGHT_GRAD, 128, 128, 0>(a, m, sms, s);
    if (kind == PK_INPUT_GRAD)
        return tall ? launch_t<PK_INPUT_GRAD, 256, 128, 0>(a, m, sms, s)
                    : launch_t<PK_INPUT_GRAD, 128, 32, 0>(a, m, sms, s);
    if (tall) return launch_t<PK_FORWARD, 256, 128, 0>(a, m, sms, s);
    return t.bn == 64 ? launch_t<PK_FORWARD, 64, 32, 0>(a, m, sms, s) : launch_t<PK_FORWARD, 128, 32, 0>(a, m, sms, s);
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
