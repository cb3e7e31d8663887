// product.cu -- grouped 8-bit products with one FP32 scale per block of 128 along the
// contraction, on the 5th-generation tensor cores (tcgen05.mma kind::f8f6f4).
//
//   forward          y[p, n]  = sum_b sx[p, b] sw[e, n/128, b] sum_{c in b} qx[p, c] qw[e, n, c]
//   input gradient   dx[p, c] = sum_b sdy[p, b] sw[e, b, c/128] sum_{n in b} qdy[p, n] qw[e, n, c]
//   forward + activation: SwiGLU or ReLU^2 of the FP32 sums, rounded to 8 bits with one scale
//   per row and 128 features.
//
// One tile is 128 output rows (TMEM lanes) by BN output columns.  The scales change with
// every block of 128, so the tensor core sums one block at a time into one of several TMEM
// buffers, and the epilogue warps add buffer * scale to FP32 sums in registers while the
// next block's MMAs run.  Output rows are tokens, so a token's scale is one register per
// thread and a weight block's scale is one value for all 128 columns of a thread.
// The weights lie in memory once, [E, N, C]: the forward product reads them K-major
// (contraction over C), the input gradient MN-major (contraction over N), so nothing is
// transposed.
//
// One persistent CTA per SM; tiles go round-robin, inside an expert in bands of 16 row tiles,
// column tiles outer, so that the CTAs at work share weights and rows in L2.  At 16384 x 8192 x
// 8192 the MMAs alone (no loads, no sums) take 400 ns of a block of 128 x 256 x 128, loads and
// MMAs 500 (48 KB a block and SM, 14 TB/s out of L2: what bounds it), all of it 570, 2.1 PFLOP/s.
// 65536 rows of 256 experts x 1024 x 2048, unequal: 193 us cold, 232 to 247 in a run that lasts, where
// the 1000 W cap holds the clock at 1.4 GHz (1.1 PFLOP/s of the rows' own work); equal: 197.
#include "product.cuh"

namespace moe {
namespace {

__device__ int g_product_error;  // MOE_DEVERR_* bits of the products on this device

constexpr int BM = 128;    // rows of a tile
constexpr int kBand = 16;  // row tiles that share a pass over the weights

template <int BN, int ACT>
struct Cfg {
    static constexpr int kABytes = BM * BKB;
    static constexpr int kStageBytes = kABytes + BN * BKB;
    static constexpr int kBufs = BN == 256 ? 2 : 4;
    static constexpr int kTmemCols = kBufs * BN;
    static constexpr int kCpt = BN / 2;  // columns of a tile per epilogue thread
    // Staging of one epilogue warp: two boxes of 32 rows x 128 bytes for the copy engine, or 32
    // rows x 64 bytes of 8-bit values.
    static constexpr int kStageOut = ACT ? 2048 : 8192;
    // Ring of scales, one slot per block along the contraction: the rows' 128, and four for each half of
    // the columns (the weight block's; SwiGLU: the gate's and the two that the up half may lie in).
    static constexpr int kSlots = 4;
    static constexpr int kSlotFloats = BM + 8;
    static constexpr size_t kTables = 512 + (size_t)(2 * (MOE_MAX_EXPERTS + 1) + 34) * 4;
    static constexpr size_t kScales = (kTables + 15) / 16 * 16;
    static constexpr size_t kAmax = kScales + (size_t)kSlots * kSlotFloats * 4;
    static constexpr size_t kMeta = kAmax + (ACT ? 4 * BM * 4 : 0);
    static constexpr int kFit = (int)((227 * 1024 - 1024 - kMeta - kEpiWarps * kStageOut) / kStageBytes);
    static constexpr int kStages = kFit < 16 ? kFit : 16;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + kEpiWarps * kStageOut + kMeta;
    static constexpr bool kMoveRegs = BN == 256;
    static_assert(kStages >= 3, "ring too shallow");
    static_assert(8 * (2 * kStages + 2 * kBufs + 2 * kSlots + 4) + 8 <= 512, "barrier block");
};

struct Tile {
    int e;      // expert
    int row0;   // first row
    int n;      // rows
    int c0;     // first output column
};

__device__ __forceinline__ Tile decode(const ProductArgs& a, const int* off, const int* first, int nct, int step,
                                       int tile) {
    Tile t;
    t.e = expert_of(first, a.E, tile, nct);
    const int rts = first[t.e + 1] - first[t.e];
    int l = tile - first[t.e] * nct;
    const int band = l / (kBand * nct);
    l -= band * kBand * nct;
    const int rb = min(kBand, rts - band * kBand);
    const int ct = l / rb;
    t.c0 = ct * step;
    t.row0 = off[t.e] + (band * kBand + (l - ct * rb)) * BM;
    t.n = min(BM, off[t.e + 1] - t.row0);
    return t;
}

template <int KIND, int BN, int ACT>
__global__ void __launch_bounds__(kProductThreads, 1)
    product_kernel(const ProductArgs a, const __grid_constant__ CUtensorMap tm_a,
                   const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_out) {
    using C = Cfg<BN, ACT>;
    constexpr bool kSwiglu = ACT == 1 + MOE_ACT_SWIGLU;
    constexpr bool kBmn = KIND == PK_INPUT_GRAD;
    constexpr int kColStep = kSwiglu ? BN / 2 : BN;  // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (base_u32 - raw_u32);
    uint8_t* staging = base + (size_t)C::kStages * C::kStageBytes;
    uint8_t* meta = staging + kEpiWarps * C::kStageOut;
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
            mbar_init(tempty_bar(b), kEpiWarps);
        }
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(sfull_bar(i), 32);
            mbar_init(sempty_bar(i), kEpiWarps);
        }
        for (int q = 0; q < 4; ++q) mbar_init(amax_bar(q), 2);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
        if (ACT == 0) tma_prefetch_desc(&tm_out);
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    chain();
    expert_blocks<BM>(a.offsets, a.E, a.P, s_off, s_first, s_warp);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int nct = cdiv(a.cols, kColStep), nk = a.nbl;
    const int total = s_first[a.E] * nct;
    auto tile_at = [&](int tile) { return decode(a, s_off, s_first, nct, kColStep, tile); };

    if (warp < 4) {
        if (C::kMoveRegs) regs_set_down<kRegsIssue>();
        if (warp == 0) {
            // ------------------------------------------------------------ TMA producer
            if (lane == 0) {
                int it = 0;
                bool ok = true;
                for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
                    const Tile t = tile_at(tile);
                    for (int kb = 0; kb < nk; ++kb, ++it) {
                        const int s = it % C::kStages;
                        if (!mbar_wait(empty_bar(s), ((uint32_t)(it / C::kStages) & 1u) ^ 1u, abort_flag, err)) {
                            ok = false;
                            break;
                        }
                        const uint32_t sa = base_u32 + (uint32_t)s * C::kStageBytes, sb = sa + C::kABytes;
                        const uint32_t bar = full_bar(s);
                        mbar_expect_tx(bar, C::kStageBytes);
                        // Boxes of 32 rows; those past the expert's rows are zeros from behind the tensor's
                        // end, which move no bytes (266 -> 264 us, 24576 rows of 128 experts x 1856 x 2688).
                        for (int j = 0; j < BM / 32; ++j)
                            tma_load_2d(sa + (uint32_t)(32 * j * BKB), &tm_a, bar, kb * BKB,
                                        32 * j < t.n ? t.row0 + 32 * j : a.P);
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
                const uint32_t idesc = idesc_fp8(a.a_e5m2, 0, 0, kBmn, BN);
                int it = 0;
                bool ok = true;
                for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
                    const Tile t = tile_at(tile);
                    for (int kb = 0; kb < nk; ++kb, ++it) {
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
                            const uint64_t bd = kBmn ? sdesc_sw128_mn(sb + kk * 4096) : sdesc_sw128(sb + kk * 32);
                            tc_mma_fp8(d, sdesc_sw128(sa + kk * 32), bd, idesc, kk > 0);
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
                } else {
                    const int c = t.c0 + (lane >> 2) * (kSwiglu ? 64 : C::kCpt);
                    int nb = (kSwiglu && (lane & 3) ? a.up + c : c) / 128;
                    if ((lane & 3) == 2) ++nb;
                    w0 = min(nb, a.wn - 1) * a.wk;
                }
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const int i = it % C::kSlots;
                    if (!mbar_wait(sempty_bar(i), ((uint32_t)(it / C::kSlots) & 1u) ^ 1u, abort_flag, err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = smem_u32(s_scales + (size_t)i * C::kSlotFloats);
                    for (int r = lane; r < t.n; r += 32) cp_async4(dst + 4 * r, a.sa + (size_t)(t.row0 + r) * a.nbl + kb);
                    if (lane < 8) cp_async4(dst + (BM + lane) * 4, wsc + w0 + (size_t)kb * w_step);
                    cp_async_arrive(sfull_bar(i));
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        if (C::kMoveRegs) regs_set_up<kRegsEpilogue>();
        const int q = warp & 3, half = (warp - 4) >> 2;
        const int r = q * 32 + lane;  // this thread's row of the tile
        uint8_t* stage = staging + (warp - 4) * C::kStageOut;
        const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * C::kCpt);
        int it = 0, ntile = 0, nbox = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < total; tile += gridDim.x, ++ntile) {
            const Tile t = tile_at(tile);
            const bool live = q * 32 < t.n, mine = r < t.n;
            const int up_cut = kSwiglu ? 128 - (a.up + t.c0 + half * 64) % 128 : 0;  // up features in the first block
            uint64_t acc2[C::kCpt / 2];  // the sums, in pairs of neighbouring columns
#pragma unroll
            for (int j = 0; j < C::kCpt / 2; ++j) acc2[j] = 0;
            for (int kb = 0; kb < nk; ++kb, ++it) {
                const int b = it % C::kBufs, i = it % C::kSlots;
                if (!mbar_wait(sfull_bar(i), (uint32_t)(it / C::kSlots) & 1u, abort_flag, err) ||
                    !mbar_wait(tfull_bar(b), (uint32_t)(it / C::kBufs) & 1u, abort_flag, err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (live) {
                    const float* sc = s_scales + (size_t)i * C::kSlotFloats;
                    const float* sw = sc + BM + 4 * half;
                    const uint32_t tb = tq + (uint32_t)(b * BN);
                    // 64 columns are read in one go.  128 are read 16 at a time, the next ones loading while
                    // these are added: there are not the registers for more (with 32 the allocator copies
                    // the loaded values into pairs: 1014 -> 1435 us at 16384 x 8192 x 8192).
                    constexpr bool kAtOnce = C::kCpt <= 64;
                    constexpr int kVec = kAtOnce ? C::kCpt / 16 : 2;
                    uint32_t v[kVec][16];
#pragma unroll
                    for (int i16 = 0; i16 < (kAtOnce ? kVec : 1); ++i16) tmem_ld16(tb + 16 * i16, v[i16]);
                    const float s0 = sc[r];
                    const float s1 = s0 * sw[0];
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
                            float u = s1;  // block boundaries fall on multiples of 16 columns
                            if (is_up) u = (j0 - C::kCpt / 2) < up_cut ? u1 : u2;
                            const uint64_t a0 = pair(u, u);
                            acc2[(j0 + j) / 2] = fma2(pair(w[j], w[j + 1]), a0, acc2[(j0 + j) / 2]);
                            acc2[(j0 + j) / 2 + 1] = fma2(pair(w[j + 2], w[j + 3]), a0, acc2[(j0 + j) / 2 + 1]);
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
                // ---- whole 32-row blocks go through the copy engine, two boxes at a time per warp, so that
                // they drain while the next tile is summed; a shorter one by hand, 64 bytes of a row
                // at a time, since rows past the expert's end must not be written.
                const int c = t.c0 + half * C::kCpt, row = t.row0 + q * 32, rows = t.n - q * 32;
                auto f32_chunk = [&](int j) {
                    return make_uint4(__float_as_uint(acc[j]), __float_as_uint(acc[j + 1]), __float_as_uint(acc[j + 2]),
                                      __float_as_uint(acc[j + 3]));
                };
                auto bf16_chunk = [&](int j) {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = acc[j + i];
                    return Chunk<bf16>::pack(f);
                };
                if (rows >= 32) {
                    auto box = [&](int j0, auto chunk) {  // chunk(j): 16 bytes of this thread's row
                        if (lane == 0) store_wait_read<1>();
                        __syncwarp();
                        uint8_t* slot = stage + (nbox & 1) * 4096;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint4*>(slot + lane * 128 + ((j ^ (lane & 7)) << 4)) = chunk(j);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) store_box(&tm_out, smem_u32(slot), c + j0, row, 0, false);
                        ++nbox;
                    };
                    if (a.out_f32) {
#pragma unroll
                        for (int j0 = 0; j0 < C::kCpt; j0 += 32) {
                            if (c + j0 >= a.cols) break;
                            box(j0, [&](int j) { return f32_chunk(j0 + 4 * j); });
                        }
                    } else {
#pragma unroll
                        for (int j0 = 0; j0 < C::kCpt; j0 += 64) {
                            if (c + j0 >= a.cols) break;
                            box(j0, [&](int j) { return bf16_chunk(j0 + 8 * j); });
                        }
                    }
                } else if (rows > 0) {
                    if (lane == 0) store_wait_read<0>();
                    __syncwarp();
                    uint8_t* out = static_cast<uint8_t*>(a.out) + ((size_t)row * a.cols + c) * (a.out_f32 ? 4 : 2);
                    const size_t pitch = (size_t)a.cols * (a.out_f32 ? 4 : 2);
                    auto piece = [&](int j0, int width, const uint4(&v)[4]) {  // 64 bytes from column j0 on
                        write_rows(stage, v, lane, [&](int rr, int j, uint4 x) {
                            if (rr < rows && c + j0 + width * j < a.cols)
                                *reinterpret_cast<uint4*>(out + rr * pitch + (size_t)(j0 / width) * 16 + 16 * j) = x;
                        });
                    };
                    if (a.out_f32) {
#pragma unroll
                        for (int j0 = 0; j0 < C::kCpt; j0 += 16) {
                            if (c + j0 >= a.cols) break;
                            const uint4 v[4] = {f32_chunk(j0), f32_chunk(j0 + 4), f32_chunk(j0 + 8), f32_chunk(j0 + 12)};
                            piece(j0, 4, v);
                        }
                    } else {
#pragma unroll
                        for (int j0 = 0; j0 < C::kCpt; j0 += 32) {
                            if (c + j0 >= a.cols) break;
                            const uint4 v[4] = {bf16_chunk(j0), bf16_chunk(j0 + 8), bf16_chunk(j0 + 16), bf16_chunk(j0 + 24)};
                            piece(j0, 8, v);
                        }
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
        if (ACT == 0 && lane == 0) store_wait();
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
cudaError_t launch_t(const ProductArgs& a, const ProductMaps& m, int sms, cudaStream_t s) {
    using C = Cfg<BN, ACT>;
    const cudaError_t e = prepare_product(product_kernel<KIND, BN, ACT>, C::kSmem, C::kMoveRegs);
    if (e != cudaSuccess) return e;
    // (without the overlap with the kernel before that the other operators have: 270 against 264 us for
    // the input gradient of 24576 rows of 128 experts x 1856 x 2688)
    const int step = ACT == 1 + MOE_ACT_SWIGLU ? BN / 2 : BN;
    const long long tiles = (long long)cdiv(a.cols, step) * (a.P / BM + std::min(a.E, a.P));
    return launch_k(product_kernel<KIND, BN, ACT>, dim3((unsigned)std::min<long long>(tiles, sms)),
                    dim3(kProductThreads), C::kSmem, s, false, a, m.a, m.b, m.out);
}

}  // namespace

// By the rows an expert has on average, which is all that the host knows.  Measured on 128 experts
// of 1280 x 2560, us of a run that lasts, product_few.cu against product.cu, with equal experts:
//   rows            8        16        24        32        40        48        56        64
//   forward     77 / 87   81 / 91   83 / 91   85 / 92   92 / 93   92 / 96   99 / 96  100 / 96
//   input grad  88 / 93   86 / 93   93 / 94   94 / 91  101 / 98  105 / 98  109 / 99  111 / 96
//   SwiGLU      74 / 91   75 / 92   76 / 93   77 / 93   82 / 96   83 / 96   89 / 97   92 / 97
// (SwiGLU's two tiles of weights share a row tile.)  The borders lie below the crossovers because
// experts are seldom equal, and crowded rows cost product_few.cu more: 16 rows on average, forward,
// 46 / 52 with all of them on 64 of the experts, 46 / 37 on 32, 45 / 21 on 16, 45 / 18 on 8; 32 rows
// 52 / 55, 51 / 39, 49 / 33, 49 / 31.  Tiles of 32 rows while most experts fit one, else of 64.
int product_few_rows(int act, const ProductArgs& a) {
    const long long rows = a.P, e = a.E;
    if (rows >= (act == 1 + MOE_ACT_SWIGLU ? 56 : 36) * e) return 0;
    return rows <= 22 * e ? 32 : 64;
}

cudaError_t launch_product(int kind, int act, const ProductArgs& a, const ProductMaps& m, int sms, cudaStream_t s) {
    if (act == 1 + MOE_ACT_SWIGLU) return launch_t<PK_FORWARD, 256, 1 + MOE_ACT_SWIGLU>(a, m, sms, s);
    if (act == 1 + MOE_ACT_RELU2) return launch_t<PK_FORWARD, 128, 1 + MOE_ACT_RELU2>(a, m, sms, s);
    if (kind == PK_INPUT_GRAD) return launch_t<PK_INPUT_GRAD, 256, 0>(a, m, sms, s);
    return launch_t<PK_FORWARD, 256, 0>(a, m, sms, s);
}

cudaError_t product_error_word(int** p) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_product_error);
}

}  // namespace moe
