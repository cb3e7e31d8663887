// product.cuh -- what the grouped 8-bit products share: tcgen05 kind::f8f6f4 with operands in the
// 128-byte swizzle, TMEM reads, paired FP32 arithmetic, register moves between warpgroups.
#pragma once
#include "experts.cuh"

namespace moe {

constexpr int BKB = 128;  // bytes (= values) of one block along the contraction
// Warps of a product kernel: 0 TMA producer, 1 TMEM allocator and MMA issuer, 2 scales, 3 fills the
// warpgroup, 4-11 epilogue (warp w reads TMEM lanes of quarter w % 4).
constexpr int kEpiWarps = 8;
constexpr int kProductThreads = 128 + 32 * kEpiWarps;
// With 128 sums a thread the epilogue warpgroups take registers from the first one:
// 128 * 40 + 256 * 224 of the 384 * 168 that a block is launched with.
constexpr int kRegsIssue = 40, kRegsEpilogue = 224;
constexpr int kRegsLaunch = (128 * kRegsIssue + 256 * kRegsEpilogue + kProductThreads - 1) / kProductThreads;

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
// (0) or MN-major (1); M 128.
__device__ __forceinline__ uint32_t idesc_fp8(int a_e5m2, int b_e5m2, int a_mn, int b_mn, int N) {
    return (1u << 4) | ((uint32_t)a_e5m2 << 7) | ((uint32_t)b_e5m2 << 10) | ((uint32_t)a_mn << 15) |
           ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
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

// Sets a kernel's shared memory, and checks that the registers it moves between warpgroups are
// the block's own.
template <typename Kern>
cudaError_t prepare_product(Kern kern, size_t smem, bool moves_registers) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess || !moves_registers) return e;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    return fa.numRegs < kRegsLaunch ? cudaErrorInvalidConfiguration : cudaSuccess;
}

}  // namespace moe
