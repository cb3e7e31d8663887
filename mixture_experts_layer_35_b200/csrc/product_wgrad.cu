// product_wgrad.cu -- the grouped 8-bit product's weight gradient on the tensor cores (tcgen05.mma
// kind::f8f6f4):
//
//   dw[e, n, c] = sum over the 128-row blocks b of expert e of
//                 sdy[b, n] sx[b, c] sum_{p in b} qdy[p, n] qx[p, c]
//
// One tile is 128 rows n (TMEM lanes) by BN columns c.  Both operands are read MN-major as they
// lie, 128 rows p a step, so nothing is transposed.  The scales change with every block, so the
// tensor core sums one block at a time into one of several TMEM buffers, and the epilogue
// warps add buffer * sdy * sx to FP32 sums in registers while the next block's MMAs run.
// With few rows per expert the output's bytes bound it: its boxes, two per warp, drain through
// the copy engine while the next tile is summed (64 experts x 256 rows x 1024 x 2048, FP32, 128-column
// tiles: 162 us with stores by the warps, 119 to 125 so).
// 512 experts x 2560 x 640 are written at 4.6 TB/s; a plain kernel that stores the same boxes of
// 128 bytes x 32 rows reaches 5.2 to 5.6, whole rows 6.1.  (Rows of 512 bytes as copies of their own:
// 757 -> 848 us; boxes of eight rows, a row's four close together: 1141.)
#include "product.cuh"

namespace moe {
namespace {

__device__ int g_wgrad_error;  // MOE_DEVERR_* bits of the weight gradients on this device

constexpr int BM = 128;  // rows of a tile

template <int BN>
struct Cfg {
    static constexpr int kABytes = BM * BKB;
    static constexpr int kStageBytes = kABytes + BN * BKB;
    static constexpr int kBufs = BN == 256 ? 2 : 4;
    static constexpr int kTmemCols = kBufs * BN;
    static constexpr int kCpt = BN / 2;       // columns of a tile per epilogue thread
    static constexpr int kStageOut = 8192;    // per epilogue warp: two boxes of 32 rows x 128 bytes
    // Ring of scales, one slot per block: the rows' 128 and the columns'.
    static constexpr int kSlots = 4;
    static constexpr int kSlotFloats = BM + BN;
    static constexpr size_t kTables = 512 + (size_t)(2 * (MOE_MAX_EXPERTS + 1) + 34) * 4;
    static constexpr size_t kScales = (kTables + 15) / 16 * 16;
    static constexpr size_t kMeta = kScales + (size_t)kSlots * kSlotFloats * 4;
    static constexpr int kStages = (int)((227 * 1024 - 1024 - kMeta - kEpiWarps * kStageOut) / kStageBytes);
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + kEpiWarps * kStageOut + kMeta;
    static constexpr bool kMoveRegs = BN == 256;
    static_assert(kStages >= 3, "ring too shallow");
    static_assert(8 * (2 * kStages + 2 * kBufs + 2 * kSlots) + 8 <= 512, "barrier block");
};

struct Tile {
    int e;      // expert
    int row0;   // first output row
    int n;      // valid rows
    int c0;     // first output column
    int nk;     // blocks of rows of the expert
    int blk0;   // the first of them
};

__device__ __forceinline__ Tile decode(const ProductArgs& a, const int* first, int nct, int step, int tile) {
    Tile t;
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

template <int BN>
__global__ void __launch_bounds__(kProductThreads, 1)
    wgrad_kernel(const ProductArgs a, const __grid_constant__ CUtensorMap tm_a,
                   const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_out) {
    using C = Cfg<BN>;
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
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meta + 8 * (2 * C::kStages + 2 * C::kBufs + 2 * C::kSlots));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* s_off = reinterpret_cast<int*>(meta + 512);
    int* s_first = s_off + MOE_MAX_EXPERTS + 1;
    int* s_warp = s_first + MOE_MAX_EXPERTS + 1;
    float* s_scales = reinterpret_cast<float*>(meta + C::kScales);
    int* err = &g_wgrad_error;

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
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
        tma_prefetch_desc(&tm_out);
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    chain();
    // Offsets clamped to the room for rows, a.P = 128 * blocks, as the column quantiser lays its blocks out.
    expert_blocks<kQBlock>(a.offsets, a.E, a.P, s_off, s_first, s_warp);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int nct = cdiv(a.cols, BN);
    const int total = a.E * cdiv(a.rows, BM) * nct;
    auto tile_at = [&](int tile) { return decode(a, s_first, nct, BN, tile); };

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
                        const int r = (t.blk0 + kb) * BKB;
                        tma_load_2d(sa, &tm_a, bar, t.row0, r);
                        for (int j = 0; j < BN / 128; ++j) tma_load_2d(sb + j * 16384, &tm_b, bar, t.c0 + j * 128, r);
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            if (lane == 0) {
                const uint32_t idesc = idesc_fp8(a.a_e5m2, a.b_e5m2, 1, 1, BN);
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
                        for (int kk = 0; kk < BKB / 32; ++kk)
                            tc_mma_fp8(d, sdesc_sw128_mn(sa + kk * 4096), sdesc_sw128_mn(sb + kk * 4096), idesc, kk > 0);
                        tc_commit(tfull_bar(b));
                        tc_commit(empty_bar(s));
                    }
                }
            }
        } else if (warp == 2) {
            // ------------------------------------------------------------ scales
            // Up to kSlots blocks ahead of the sums, so that no sum waits for memory.
            int it = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
                const Tile t = tile_at(tile);
                for (int kb = 0; kb < t.nk; ++kb, ++it) {
                    const int i = it % C::kSlots;
                    if (!mbar_wait(sempty_bar(i), ((uint32_t)(it / C::kSlots) & 1u) ^ 1u, abort_flag, err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = smem_u32(s_scales + (size_t)i * C::kSlotFloats);
                    const size_t blk = t.blk0 + kb;
                    if (t.row0 + 4 * lane < a.rows) cp_async16(dst + 16 * lane, a.sa + blk * a.rows + t.row0 + 4 * lane, 16);
                    for (int j = lane; j < BN / 4; j += 32)
                        if (t.c0 + 4 * j < a.cols)
                            cp_async16(dst + (BM + 4 * j) * 4, a.sb + blk * a.cols + t.c0 + 4 * j, 16);
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
        int it = 0, nbox = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
            const Tile t = tile_at(tile);
            const bool live = q * 32 < t.n;  // any row of this warp in the tile
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
                    const float* sw = sc + BM + half * C::kCpt;
                    const uint32_t tb = tq + (uint32_t)(b * BN);
                    // 16 columns at a time, the next ones loading while these are added: there are not
                    // the registers for more (with 32 the allocator copies the loaded values into pairs).
                    uint32_t v[2][16];
                    tmem_ld16(tb, v[0]);
                    const uint64_t s0 = pair(sc[r], sc[r]);
#pragma unroll
                    for (int j0 = 0; j0 < C::kCpt; j0 += 16) {
                        uint32_t(&w)[16] = v[(j0 / 16) & 1];
                        tmem_ld_wait_for(w);
                        if (j0 + 16 < C::kCpt) {
                            tmem_ld16(tb + j0 + 16, v[(j0 / 16 + 1) & 1]);
                        } else {  // the buffer has been read
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(tempty_bar(b));
                        }
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 c4 = *reinterpret_cast<const float4*>(sw + j0 + j);
                            const uint64_t a0 = mul2(s0, pair(c4.x, c4.y)), a1 = mul2(s0, pair(c4.z, c4.w));
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
            // ---- the output: boxes through the copy engine, which drops what lies past the tensor's
            // end, two at a time per warp, so that they drain while the next tile is summed; or, where
            // BF16 values are added to, FP32 pieces by hand, so that the sum is rounded once.
            const int c = t.c0 + half * C::kCpt, row = t.row0 + q * 32, rows = t.n - q * 32, e = t.e;
            const bool add = a.accumulate;
            if (!live || (add && t.nk == 0)) continue;
            if (a.out_f32 || !add) {
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
            } else {
                bf16* out = static_cast<bf16*>(a.out) + ((size_t)e * a.rows + row) * a.cols + c;
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
                        uint2* p = reinterpret_cast<uint2*>(out + (size_t)rr * a.cols + j0 + 4 * j);
                        const uint2 o = *p;
                        *p = make_uint2(f2bf_bits(__uint_as_float(w.x) + bf16lo(o.x)) |
                                            ((uint32_t)f2bf_bits(__uint_as_float(w.y) + bf16hi(o.x)) << 16),
                                        f2bf_bits(__uint_as_float(w.z) + bf16lo(o.y)) |
                                            ((uint32_t)f2bf_bits(__uint_as_float(w.w) + bf16hi(o.y)) << 16));
                    });
                }
            }
        }
        if (lane == 0) store_wait();
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

template <int BN>
cudaError_t launch_t(const ProductArgs& a, const ProductMaps& m, int sms, cudaStream_t s) {
    using C = Cfg<BN>;
    const cudaError_t e = prepare_product(wgrad_kernel<BN>, C::kSmem, C::kMoveRegs);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)a.E * cdiv(a.rows, BM) * cdiv(a.cols, BN);
    return launch_k(wgrad_kernel<BN>, dim3((unsigned)std::min<long long>(tiles, sms)), dim3(kProductThreads), C::kSmem, s, true, a, m.a, m.b, m.out);
}

}  // namespace

// By the output and by the blocks that there is room for, rows / 128 + 1 an expert.  Measured, us of
// a run that lasts, 128- against 256-column tiles, at 128, 384, 640, 1024 and 2048 rows an expert of
// 64 experts x 1024 x 2048:
//   FP32           115 / 114, 157 / 164, 215 / 219, 306 / 301, 543 / 523
//   BF16            94 /  86, 157 / 144, 218 / 200, 307 / 284, 546 / 506
// (128 experts x 1856 x 2688, 512 x 2560 x 640 and 8 x 4096 x 4096 the same way: FP32 within 4 % below
// 300 rows, 128 columns up to 8 % faster from 384 to 640, 256 from 1024 on; BF16 256 throughout.)
// BF16 values that are added to are read and written by the warps: 389 / 395 at 64 rows, 412 / 413
// at 256, 465 / 461 at 512, 578 / 564 at 1024 (512 x 2560 x 640 with 64 rows: 2387 / 2842).  FP32 added
// by the copy engine: within 2 % everywhere.
cudaError_t launch_weight_grad(const ProductArgs& a, const ProductMaps& m, int sms, cudaStream_t s) {
    if ((a.out_f32 || a.accumulate) && a.blocks < 6LL * a.E) return launch_t<128>(a, m, sms, s);
    return launch_t<256>(a, m, sms, s);
}

cudaError_t weight_grad_error_word(int** p) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_wgrad_error);
}

}  // namespace moe
