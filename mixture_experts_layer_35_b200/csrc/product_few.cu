// product_few.cu -- the grouped 8-bit products of product.cu where experts have few rows (decode,
// and prefill spread over many experts): there the weights' bytes bound them.
//
// The MMA's M side is 128 output features of one expert's weights, its N side up to NT of that
// expert's rows, rounded up to 16: what is loaded besides the weights, computed and summed follows
// the rows an expert really has, and the shared memory left holds more weights in flight.  A
// thread holds one feature of every row.  Two warps of their own multiply the rows' scales with the
// weight block's into a ring in shared memory, ahead of the sums, and the epilogue's threads
// read them as broadcasts.  Those reads compete with the tensor cores' for shared memory: at 256 rows per
// expert this orientation takes 416 us where product.cu's takes 197 (256 experts x 1024 x 2048).
// At 8 rows it takes 51 us where product.cu's takes 60 (128 experts; 5.3 TB/s of weights).
//
// A call with fewer tiles than half of the SMs (one token, a few experts) splits the contraction
// over a cluster of two CTAs: each sums its half of the blocks, the second writes its FP32 sums into
// the first one's shared memory, and that one adds them.  One token of top-8, H 2048, I 512,
// captured: forward 10.9 -> 9.9 us, SwiGLU 13.7 -> 11.7.
#include "product.cuh"

namespace moe {
namespace {

__device__ int g_few_error;  // MOE_DEVERR_* bits of these products on this device

constexpr int BF = 128;  // features of a tile
constexpr int A_BYTES = BF * BKB;
constexpr int kSplit = 2;  // CTAs that share a tile's contraction

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of every CTA of the cluster, whatever has happened in it: no wait can stay open.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// Address of `addr` in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void peer_store(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// mbar_wait for arrivals and data of other CTAs of the cluster; bounded in the same way.
__device__ __forceinline__ bool cluster_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
    const uint64_t t0 = globaltimer_ns();
    uint32_t n = 0;
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((++n & 255u) == 0) {
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                *abort_flag = 1;
                set_dev_error(err, MOE_DEVERR_WAIT_TIMEOUT);
                return false;
            }
        }
    }
}

template <int NT, int ACT, bool SPLIT>
struct Cfg {
    static constexpr bool kSwiglu = ACT == 1 + MOE_ACT_SWIGLU;
    static constexpr int kNA = kSwiglu ? 2 : 1;  // weight tiles: gate and up
    static constexpr int kStageBytes = kNA * A_BYTES + NT * BKB;
    static constexpr int kAccCols = kNA * NT;
    static constexpr int kBufs = 4;
    static constexpr int kTmemCols = kBufs * kAccCols;
    // Each half of the epilogue warps takes every other group of 16 rows.
    static constexpr int kGroups = NT / 32;
    static constexpr int kHalf = NT / 2;
    // Ring of scales, one slot per block along the contraction: the rows' times the weight block's.
    // SwiGLU: times the gate's; the up block's; and the next up block's, since 128 up features may
    // start anywhere in a block.
    static constexpr int kSlots = 4;
    static constexpr int kSlotFloats = kSwiglu ? 3 * NT : NT;
    static constexpr size_t kTables = 512 + (size_t)(2 * (MOE_MAX_EXPERTS + 1) + 34) * 4;
    static constexpr size_t kScales = (kTables + 15) / 16 * 16;
    static constexpr size_t kAmax = kScales + (size_t)kSlots * kSlotFloats * 4;  // [tile parity][quarter][NT]
    static constexpr size_t kFactor = kAmax + (ACT ? 8 * NT * 4 : 0);            // [warp][kHalf]
    static constexpr size_t kMeta = kFactor + (ACT ? kEpiWarps * kHalf * 4 : 0);
    // The second CTA's sums: [value][epilogue thread].
    static constexpr int kValues = kNA * kGroups * 16;
    static constexpr int kPartBytes = SPLIT ? kValues * 32 * kEpiWarps * 4 : 0;
    static constexpr int kFit = (int)((227 * 1024 - 1024 - kMeta - kPartBytes) / kStageBytes);
    static constexpr int kStages = kFit < 16 ? kFit : 16;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + kPartBytes + kMeta;
    static_assert(NT == 32 || NT == 64, "a scale warp's lane has one row; a lane keeps one row's maximum");
    static_assert(kTmemCols <= 512, "the accumulator buffers must fit");
    static_assert(kStages >= 3, "ring too shallow");
    static_assert(8 * (2 * kStages + 2 * kBufs + 2 * kSlots + 3) + 8 <= 512, "barrier block");
};

struct Tile {
    int e;      // expert
    int row0;   // first row
    int n;      // rows
    int f0;     // first feature
    int alone;  // the expert's only tile of rows: its weights are read once
};

template <int NT>
__device__ __forceinline__ Tile decode(const ProductArgs& a, const int* off, const int* first, int nft, int tile) {
    Tile t;
    t.e = expert_of(first, a.E, tile, nft);
    const int rts = first[t.e + 1] - first[t.e];
    const int l = tile - first[t.e] * nft, ft = l / rts;
    t.f0 = ft * BF;
    t.row0 = off[t.e] + (l - ft * rts) * NT;
    t.n = min(NT, off[t.e + 1] - t.row0);
    t.alone = rts == 1;
    return t;
}

template <int KIND, int NT, int ACT, bool SPLIT>
__global__ void __launch_bounds__(kProductThreads, 1)
    few_kernel(const ProductArgs a, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_x) {
    using C = Cfg<NT, ACT, SPLIT>;
    constexpr bool kSwiglu = C::kSwiglu;
    constexpr bool kAmn = KIND == PK_INPUT_GRAD;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
    float* parts = reinterpret_cast<float*>(smem_raw + (base_u32 - raw_u32) + (size_t)C::kStages * C::kStageBytes);
    uint8_t* meta = reinterpret_cast<uint8_t*>(parts) + C::kPartBytes;
    const uint32_t bar_u32 = smem_u32(meta);
    auto full_bar = [&](int s) { return bar_u32 + 8u * s; };
    auto empty_bar = [&](int s) { return bar_u32 + 8u * (C::kStages + s); };
    auto tfull_bar = [&](int b) { return bar_u32 + 8u * (2 * C::kStages + b); };
    auto tempty_bar = [&](int b) { return bar_u32 + 8u * (2 * C::kStages + C::kBufs + b); };
    auto sfull_bar = [&](int i) { return bar_u32 + 8u * (2 * C::kStages + 2 * C::kBufs + i); };
    auto sempty_bar = [&](int i) { return bar_u32 + 8u * (2 * C::kStages + 2 * C::kBufs + C::kSlots + i); };
    auto amax_bar = [&](int h) { return bar_u32 + 8u * (2 * C::kStages + 2 * C::kBufs + 2 * C::kSlots + h); };
    const uint32_t part_bar = amax_bar(2);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meta + 8 * (2 * C::kStages + 2 * C::kBufs + 2 * C::kSlots + 3));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* s_off = reinterpret_cast<int*>(meta + 512);
    int* s_first = s_off + MOE_MAX_EXPERTS + 1;
    int* s_warp = s_first + MOE_MAX_EXPERTS + 1;
    float* s_scales = reinterpret_cast<float*>(meta + C::kScales);
    int* err = &g_few_error;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = SPLIT ? (int)cluster_rank() : 0;
    constexpr int split = SPLIT ? kSplit : 1;
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
            mbar_init(sfull_bar(i), 2);
            mbar_init(sempty_bar(i), kEpiWarps);
        }
        for (int h = 0; h < 2; ++h) mbar_init(amax_bar(h), 4);
        if (SPLIT) mbar_init(part_bar, 32 * kEpiWarps);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_x);
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    chain();
    expert_blocks<NT>(a.offsets, a.E, a.P, s_off, s_first, s_warp);
    tc_fence_before();
    __syncthreads();
    if (SPLIT) cluster_sync();  // every CTA of the cluster has its barriers
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int nft = cdiv(a.cols, BF), nk = a.nbl;
    // This CTA's blocks of the contraction, its first tile, and the one after a tile.  (A split call
    // has at least as many clusters as tiles: one tile each.  Read where they are used: held in
    // registers from here on, they cost 128 rows of 256 experts 47 us instead of 43.5.)
    const int kb0 = SPLIT ? nk * rank / split : 0, kb1 = SPLIT ? nk * (rank + 1) / split : nk;
    auto first_tile = [] { return SPLIT ? (int)blockIdx.x / split : (int)blockIdx.x; };
    auto tile_after = [](int tile) { return SPLIT ? tile + (int)gridDim.x / split : tile + (int)gridDim.x; };
    const int total = s_first[a.E] * nft;
    auto tile_at = [&](int tile) { return decode<NT>(a, s_off, s_first, nft, tile); };

    if (warp < 4) {
        if (warp == 0) {
            // ------------------------------------------------------------ TMA producer
            if (lane == 0) {
                const uint64_t once = l2_policy_evict_first();
                int it = 0;
                bool ok = true;
                for (int tile = first_tile(); ok && tile < total; tile = tile_after(tile)) {
                    const Tile t = tile_at(tile);
                    const int boxes = cdiv(t.n, kRowBox);
                    auto load_w = [&](uint32_t dst, uint32_t bar, int c0, int c1) {
                        if (t.alone) tma_load_3d_hint(dst, &tm_w, bar, c0, c1, t.e, once);
                        else tma_load_3d(dst, &tm_w, bar, c0, c1, t.e);
                    };
                    for (int kb = kb0; kb < kb1; ++kb, ++it) {
                        const int s = it % C::kStages;
                        if (!mbar_wait(empty_bar(s), ((uint32_t)(it / C::kStages) & 1u) ^ 1u, abort_flag, err)) {
                            ok = false;
                            break;
                        }
                        const uint32_t sw = base_u32 + (uint32_t)s * C::kStageBytes, sx = sw + C::kNA * A_BYTES;
                        const uint32_t bar = full_bar(s);
                        mbar_expect_tx(bar, (uint32_t)(C::kNA * A_BYTES + boxes * kRowBox * BKB));
                        if (KIND == PK_INPUT_GRAD) {
                            load_w(sw, bar, t.f0, kb * BKB);
                        } else {
                            load_w(sw, bar, kb * BKB, t.f0);
                            if (kSwiglu) load_w(sw + A_BYTES, bar, kb * BKB, a.up + t.f0);
                        }
                        for (int j = 0; j < boxes; ++j)
                            tma_load_2d(sx + (uint32_t)(j * kRowBox * BKB), &tm_x, bar, kb * BKB,
                                        t.row0 + j * kRowBox);
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            if (lane == 0) {
                int it = 0;
                bool ok = true;
                for (int tile = first_tile(); ok && tile < total; tile = tile_after(tile)) {
                    const Tile t = tile_at(tile);
                    const uint32_t idesc = idesc_fp8(0, a.a_e5m2, kAmn, 0, cdiv(t.n, 16) * 16);
                    for (int kb = kb0; kb < kb1; ++kb, ++it) {
                        const int s = it % C::kStages, b = it % C::kBufs;
                        if (!mbar_wait(full_bar(s), (uint32_t)(it / C::kStages) & 1u, abort_flag, err) ||
                            !mbar_wait(tempty_bar(b), ((uint32_t)(it / C::kBufs) & 1u) ^ 1u, abort_flag, err)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sw = base_u32 + (uint32_t)s * C::kStageBytes, sx = sw + C::kNA * A_BYTES;
                        const uint32_t d = tmem_base + (uint32_t)(b * C::kAccCols);
#pragma unroll
                        for (int kk = 0; kk < BKB / 32; ++kk) {
                            const uint64_t xd = sdesc_sw128(sx + kk * 32);
#pragma unroll
                            for (int h = 0; h < C::kNA; ++h) {
                                const uint32_t wa = sw + h * A_BYTES;
                                const uint64_t wd = kAmn ? sdesc_sw128_mn(wa + kk * 4096) : sdesc_sw128(wa + kk * 32);
                                tc_mma_fp8(d + h * NT, wd, xd, idesc, kk > 0);
                            }
                        }
                        tc_commit(tfull_bar(b));
                        tc_commit(empty_bar(s));
                    }
                }
            }
        } else {
            // ------------------------------------------------------------ scales (warps 2 and 3)
            // Row r of the tile.  Each block's scales are loaded while the block before is written, up to
            // kSlots blocks ahead of the sums.
            const int r = 32 * (warp - 2) + lane;
            float x = 0.0f, w[3];
            const float *xp = nullptr, *wp = nullptr, *up0 = nullptr, *up1 = nullptr;
            int n = 0, w_step = 1;
            auto load = [&](int kb) {
                x = r < n ? __ldg(xp + kb) : 0.0f;
                w[0] = __ldg(wp + (size_t)kb * w_step);
                if (kSwiglu) {
                    w[1] = __ldg(up0 + kb);
                    w[2] = __ldg(up1 + kb);
                }
            };
            auto begin_tile = [&](int tile) {
                const Tile t = tile_at(tile);
                n = t.n;
                xp = a.sa + (size_t)(t.row0 + (r < n ? r : 0)) * a.nbl;
                const float* we = a.sb + (size_t)t.e * a.wn * a.wk;
                if (KIND == PK_INPUT_GRAD) {
                    wp = we + t.f0 / BF;
                    w_step = a.wk;
                } else {
                    wp = we + (size_t)(t.f0 / BF) * a.wk;
                    const int u = (a.up + t.f0) / BF;
                    up0 = we + (size_t)min(u, a.wn - 1) * a.wk;
                    up1 = we + (size_t)min(u + 1, a.wn - 1) * a.wk;
                }
                load(kb0);
            };
            int it = 0;
            bool ok = true;
            if (first_tile() < total) begin_tile(first_tile());
            for (int tile = first_tile(); ok && tile < total; tile = tile_after(tile)) {
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int i = it % C::kSlots;
                    const float now = x, wn[3] = {w[0], w[1], w[2]};
                    if (kb + 1 < kb1) load(kb + 1);
                    else if (tile_after(tile) < total) begin_tile(tile_after(tile));
                    if (!mbar_wait(sempty_bar(i), ((uint32_t)(it / C::kSlots) & 1u) ^ 1u, abort_flag, err)) {
                        ok = false;
                        break;
                    }
                    float* dst = s_scales + (size_t)i * C::kSlotFloats + r;
                    if (r < NT) {
                        dst[0] = now * wn[0];
                        if (kSwiglu) {
                            dst[NT] = now * wn[1];
                            dst[2 * NT] = now * wn[2];
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sfull_bar(i));
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(16 * half);
        int it = 0, ntile = 0;
        bool ok = true;
        for (int tile = first_tile(); tile < total; tile = tile_after(tile), ++ntile) {
            const Tile t = tile_at(tile);
            const int f = t.f0 + q * 32 + lane;  // this thread's feature
            const bool live = t.f0 + q * 32 < a.cols;
            // groups of 16 rows of this warp: rows 32 g + 16 half + 0..15
            const int groups = live ? min(C::kGroups, (t.n - 16 * half + 31) / 32) : 0;
            const int up_block = kSwiglu ? (a.up + f) / 128 - (a.up + t.f0) / 128 : 0;
            uint64_t acc2[C::kNA * C::kGroups][8];  // the sums, in pairs of neighbouring rows
#pragma unroll
            for (int p = 0; p < C::kNA * C::kGroups; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc2[p][j] = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int b = it % C::kBufs, i = it % C::kSlots;
                if (!mbar_wait(sfull_bar(i), (uint32_t)(it / C::kSlots) & 1u, abort_flag, err) ||
                    !mbar_wait(tfull_bar(b), (uint32_t)(it / C::kBufs) & 1u, abort_flag, err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float* sx = s_scales + (size_t)i * C::kSlotFloats + 16 * half;
                const uint32_t tb = tq + (uint32_t)(b * C::kAccCols);
                // Piece p: group p / kNA of the first (gate) or second (up) sums; all are read at once.
                constexpr int kPieces = C::kNA * C::kGroups;
                const int pieces = C::kNA * groups;
                auto column = [&](int p) { return (uint32_t)((p % C::kNA) * NT + 32 * (p / C::kNA)); };
                uint32_t v[kPieces][16];
#pragma unroll
                for (int p = 0; p < kPieces; ++p)
                    if (p < pieces) tmem_ld16(tb + column(p), v[p]);
                if (pieces == 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tempty_bar(b));
                }
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
                    if (p >= pieces) break;
                    uint32_t(&w)[16] = v[p];
                    tmem_ld_wait_for(w);
                    if (p == 0) {  // this warp has read the buffer
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(tempty_bar(b));
                    }
                    const float4* s4 =
                        reinterpret_cast<const float4*>(sx + (p % C::kNA ? NT * (1 + up_block) : 0) + 32 * (p / C::kNA));
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 x = s4[j / 4];
                        acc2[p][j / 2] = fma2(pair(w[j], w[j + 1]), pair(x.x, x.y), acc2[p][j / 2]);
                        acc2[p][j / 2 + 1] = fma2(pair(w[j + 2], w[j + 3]), pair(x.z, x.w), acc2[p][j / 2 + 1]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sempty_bar(i));
            }
            if (!ok) break;
            if (SPLIT && rank > 0) {  // this CTA's sums to the first one's shared memory
                const uint32_t mine = smem_u32(parts + threadIdx.x - 128);
                const uint32_t dst = peer_smem(mine, 0);
#pragma unroll
                for (int p = 0; p < C::kNA * C::kGroups; ++p)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float x, y;
                        unpair(acc2[p][j], x, y);
                        peer_store(dst + (16 * p + 2 * j) * (32 * kEpiWarps * 4), x);
                        peer_store(dst + (16 * p + 2 * j + 1) * (32 * kEpiWarps * 4), y);
                    }
                peer_arrive(peer_smem(part_bar, 0));
                continue;
            }
            if (SPLIT) {  // the second CTA's sums
                if (!cluster_wait(part_bar, (uint32_t)ntile & 1u, abort_flag, err)) break;
                const float* from = parts + threadIdx.x - 128;
#pragma unroll
                for (int p = 0; p < C::kNA * C::kGroups; ++p)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float x, y;
                        unpair(acc2[p][j], x, y);
                        x += from[(16 * p + 2 * j) * 32 * kEpiWarps];
                        y += from[(16 * p + 2 * j + 1) * 32 * kEpiWarps];
                        acc2[p][j] = pair(x, y);
                    }
            }
            if (ACT == 0) {
                // ---- a warp holds 32 neighbouring features of each row: FP32 rows are written as they
                // are, 128 bytes each; for BF16 two lanes swap halves of two rows, so that each
                // writes two features of one row (64 bytes of a row per warp).
#pragma unroll
                for (int g = 0; g < C::kGroups; ++g) {
                    if (g >= groups) break;
                    const int r0 = 32 * g + 16 * half;
                    if (a.out_f32) {
                        float* out = static_cast<float*>(a.out) + (size_t)(t.row0 + r0) * a.cols + f;
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            float x, y;
                            unpair(acc2[g][j / 2], x, y);
                            if (f < a.cols && r0 + j < t.n) out[(size_t)j * a.cols] = x;
                            if (f < a.cols && r0 + j + 1 < t.n) out[(size_t)(j + 1) * a.cols] = y;
                        }
                    } else {
                        const int odd = lane & 1;
                        bf16* out = static_cast<bf16*>(a.out) + (size_t)(t.row0 + r0 + odd) * a.cols + (f - odd);
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            float x, y;  // this feature's values of rows j and j + 1
                            unpair(acc2[g][j / 2], x, y);
                            const float got = __shfl_xor_sync(0xffffffffu, odd ? x : y, 1);
                            const float lo = odd ? got : x, hi = odd ? y : got;
                            if (f < a.cols && r0 + j + odd < t.n)
                                *reinterpret_cast<uint32_t*>(out + (size_t)j * a.cols) =
                                    (uint32_t)f2bf_bits(lo) | ((uint32_t)f2bf_bits(hi) << 16);
                        }
                    }
                }
            } else {
                // ---- activation; each row's maximum over the tile's 128 features (one reduction per
                // warp, then the four warps of the same rows through shared memory); and four
                // neighbouring features of a row per lane, by swapping bytes among four lanes.
                float h[C::kHalf];
#pragma unroll
                for (int i = 0; i < C::kHalf; i += 2) {
                    float x, y;
                    unpair(acc2[C::kNA * (i / 16)][(i % 16) / 2], x, y);
                    if (kSwiglu) {
                        float ux, uy;
                        unpair(acc2[C::kNA * (i / 16) + (kSwiglu ? 1 : 0)][(i % 16) / 2], ux, uy);
                        h[i] = quick_swiglu(x, ux);
                        h[i + 1] = quick_swiglu(y, uy);
                    } else {
                        h[i] = relu2_nan(x);
                        h[i + 1] = relu2_nan(y);
                    }
                }
                uint32_t keep = 0;  // lane i: of row i
#pragma unroll
                for (int i = 0; i < C::kHalf; ++i) {
                    const uint32_t m = __reduce_max_sync(0xffffffffu, f < a.cols ? abs_bits(h[i]) : 0u);
                    if (i == lane) keep = m;
                }
                // Two buffers by tile parity: a warp writes one again only after the other warps'
                // arrivals for the tile between, which follow their reads.
                uint32_t* am = reinterpret_cast<uint32_t*>(meta + C::kAmax) + (ntile & 1) * 4 * NT + half * C::kHalf;
                if (lane < C::kHalf) am[q * NT + lane] = keep;
                __syncwarp();
                if (lane == 0) mbar_arrive(amax_bar(half));
                if (!mbar_wait(amax_bar(half), (uint32_t)ntile & 1u, abort_flag, err)) break;
                float* factors = reinterpret_cast<float*>(meta + C::kFactor) + (warp - 4) * C::kHalf;
                if (lane < C::kHalf) {
                    float scale, factor;
                    block_scale(max(max(am[lane], am[NT + lane]), max(am[2 * NT + lane], am[3 * NT + lane])),
                                fp8_max(a.h_e5m2), scale, factor);
                    factors[lane] = factor;
                    const int row = 32 * (lane / 16) + 16 * half + lane % 16;
                    if (q == 0 && row < t.n)
                        a.out_scales[(size_t)(t.row0 + row) * cdiv(a.cols, kQBlock) + t.f0 / kQBlock] = scale;
                }
                __syncwarp();
                uint8_t* out = static_cast<uint8_t*>(a.out) + (size_t)t.row0 * a.cols + (f & ~3);
#pragma unroll
                for (int i = 0; i < C::kHalf; i += 4) {
                    if (i / 16 >= groups) break;
                    const float4 s = *reinterpret_cast<const float4*>(factors + i);
                    const __nv_fp8_interpretation_t kind = a.h_e5m2 ? __NV_E5M2 : __NV_E4M3;
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                        make_float2(__fmul_rn(h[i], s.x), __fmul_rn(h[i + 1], s.y)), __NV_SATFINITE, kind);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                        make_float2(__fmul_rn(h[i + 2], s.z), __fmul_rn(h[i + 3], s.w)), __NV_SATFINITE, kind);
                    const uint32_t x = lo | (hi << 16);  // this feature's bytes of rows i .. i + 3
                    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, 2);
                    const uint32_t m = lane & 2 ? __byte_perm(y, x, 0x7632) : __byte_perm(x, y, 0x5410);
                    const uint32_t z = __shfl_xor_sync(0xffffffffu, m, 1);
                    const uint32_t o = __byte_perm(m, z, lane & 1 ? 0x3715 : 0x6240);
                    const int row = 32 * (i / 16) + 16 * half + i % 16 + (lane & 3);
                    if (row < t.n && f < a.cols) *reinterpret_cast<uint32_t*>(out + (size_t)row * a.cols) = o;
                }
                __syncwarp();  // the factors have been read
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
    if (SPLIT) cluster_sync();  // no CTA leaves while another may still write to it
}

template <int KIND, int NT, int ACT, bool SPLIT>
cudaError_t launch_t(const ProductArgs& a, const ProductMaps& m, int sms, cudaStream_t s) {
    using C = Cfg<NT, ACT, SPLIT>;
    auto kern = few_kernel<KIND, NT, ACT, SPLIT>;
    const cudaError_t e = prepare_product(kern, C::kSmem, false);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)cdiv(a.cols, BF) * (a.P / NT + std::min(a.E, a.P));
    if constexpr (!SPLIT)
        return launch_k(kern, dim3((unsigned)std::min<long long>(tiles, sms)), dim3(kProductThreads), C::kSmem, s, true, a,
                        m.b, m.a);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles * kSplit);
    cfg.blockDim = dim3(kProductThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kSplit;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a, m.b, m.a);
}
template <int KIND, int ACT>
cudaError_t launch_rows(const ProductArgs& a, const ProductMaps& m, int rows, int sms, cudaStream_t s) {
    if (rows != 32) return launch_t<KIND, 64, ACT, false>(a, m, sms, s);
    const long long tiles = (long long)cdiv(a.cols, BF) * (a.P / 32 + std::min(a.E, a.P));
    if (kSplit * tiles <= sms && a.nbl >= 2 * kSplit) return launch_t<KIND, 32, ACT, true>(a, m, sms, s);
    return launch_t<KIND, 32, ACT, false>(a, m, sms, s);
}

}  // namespace

cudaError_t launch_product_few(int kind, int act, int rows, const ProductArgs& a, const ProductMaps& m, int sms,
                               cudaStream_t s) {
    if (act == 1 + MOE_ACT_SWIGLU) return launch_rows<PK_FORWARD, 1 + MOE_ACT_SWIGLU>(a, m, rows, sms, s);
    if (act == 1 + MOE_ACT_RELU2) return launch_rows<PK_FORWARD, 1 + MOE_ACT_RELU2>(a, m, rows, sms, s);
    if (kind == PK_INPUT_GRAD) return launch_rows<PK_INPUT_GRAD, 0>(a, m, rows, sms, s);
    return launch_rows<PK_FORWARD, 0>(a, m, rows, sms, s);
}

cudaError_t product_few_error_word(int** p) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_few_error);
}

}  // namespace moe
