// Inline PTX of the fifth-generation tensor cores: tensor memory, its matrix instruction with the A
// operand in tensor memory and B in shared memory, and tiled copies by a tensor map.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace lmloss {

// ---------------------------------------------------------- tensor memory
// `columns`: a power of two from 32 to 512.  By one whole warp, which frees them too.
__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}

// A warp's 32 lanes (its quarter of the 128, lane << 16 in the address) by 32 or 16 columns of 32 bits.
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&f)[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(r[i]);
}
// The values that the loads before it put into f: nothing uses them before this.
__device__ __forceinline__ void tmem_wait_load(float (&f)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(f[0]), "+f"(f[1]), "+f"(f[2]), "+f"(f[3]), "+f"(f[4]), "+f"(f[5]), "+f"(f[6]), "+f"(f[7]), "+f"(f[8]),
                   "+f"(f[9]), "+f"(f[10]), "+f"(f[11]), "+f"(f[12]), "+f"(f[13]), "+f"(f[14]), "+f"(f[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Order of tensor-memory accesses across threads, around a barrier.
__device__ __forceinline__ void tcgen05_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 1 in one thread of a whole warp, 0 in the others.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one;
}

// ------------------------------------------------------------ the product
// D [128 x n] fp32 (+)= A [128 x 16] B [n x 16]^T, both fp16: A in tensor memory, row i in lane i, two
// neighbouring k to a column; B in shared memory by a descriptor.  A whole warp goes along, with uniform
// operands, and the thread with `leader` issues: predicated, since in a branch of that thread alone the
// operands' arithmetic leaves the uniform registers (8 products and a commit, n = 16: 200 clocks so, 250 there).
template <bool ACCUMULATE>
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %4, 0;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(leader), "n"(ACCUMULATE ? 1 : 0)
        : "memory");
}
// Arrives at a barrier of this block when every product that the thread has issued is done.
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}
// fp16 by fp16 into fp32, 128 rows, n columns (a multiple of 16), both operands along k.
__host__ __device__ constexpr uint32_t mma_f16_idesc(int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
// Rows of 128 bytes (64 fp16 along k) whose 16-byte parts lie at place (part ^ row % 8), eight rows
// after another: the 128-byte swizzle.  The address is a multiple of 1024; +32 bytes steps 16 along k.
__device__ __forceinline__ uint64_t mma_desc_128b(uint32_t addr)
{
    return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
           (uint64_t(2) << 61);
}

// ---------------------------------------------------------------- waiting
__device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(100000u)
        : "memory");
    return done != 0;
}
// (few instructions between tries: a dozen waiting warps share the issue slots and the
// instruction cache with those that work)
__device__ __forceinline__ bool mbar_sleep_slowly(uint32_t bar, uint32_t parity, long long limit_cycles, volatile int* failed)
{
    const long long start = clock64();
#pragma unroll 1
    for (uint32_t tries = 1;; ++tries) {
        if (mbar_sleep(bar, parity)) return true;
        __nanosleep(20);
        if ((tries & 63u) == 0) {
            if (*failed) return true;
            if (clock64() - start > limit_cycles) {
                *failed = 1;
                return false;
            }
        }
    }
}
// Waits for a phase.  After `limit_cycles` it sets *failed, which ends every other such wait of the block at once: all
// go on, to a clean end with results that mean nothing, and never wait for one another in vain.  False where it
// gave up itself.
__device__ __forceinline__ bool mbar_sleep_bounded(uint32_t bar, uint32_t parity, long long limit_cycles, volatile int* failed)
{
    return mbar_sleep(bar, parity) || mbar_sleep_slowly(bar, parity, limit_cycles, failed);
}

// ------------------------------------------------------------ tiled copies
__device__ __forceinline__ void tile_load_2d(uint32_t dst, const void* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

}  // namespace lmloss
