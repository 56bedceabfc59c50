// The fifth-generation tensor core's instructions that the expert products
// use, one inline function each (sm_103a).
//
// Operands lie in shared memory in the K-major layout with a 128-byte swizzle
// that a tensor-map copy writes; their E8M0 scales and the binary32
// accumulators lie in tensor memory (TMEM, 128 lanes of 512 32-bit columns).
#pragma once

#include "fp8q_device.cuh"

namespace fp8q {

// Tensor memory of one CTA: `columns` (a power of two, at least 32) are
// allocated by one whole warp, which also frees them; the address is written
// to shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t* smem_addr_out, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(smem_addr_out)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}

// Order tcgen05 work around barriers that other threads wait on.
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// One thread of a warp, chosen by the hardware.  Inside a branch on it the
// compiler knows that a single thread runs, and keeps addresses and
// descriptors in the uniform registers that the tensor core's instructions
// read; in a branch on the lane number it moves every operand of every
// instruction there in a loop over the active lanes (134 cycles between two
// products on a GB300, whatever their size, against 39 to 112 by size).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Descriptors are 64 bits: the address and the offset that a swizzled K-major
// operand ignores in the lower half, the layout in the upper half.
// An operand: rows of 128 bytes, groups of 8 rows 1024 bytes apart, 128-byte
// swizzle (code 2 in bits 61..63).
constexpr uint32_t kOperandLayout = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t operand_desc(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
// A 512-byte scale tile: 32 rows of 16 bytes, groups of 8 rows 128 bytes
// apart, no swizzle.
constexpr uint32_t kScaleLayout = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t scale_desc(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4; }

// A scale tile of 128 rows x 4 scales: shared memory -> 4 TMEM columns, to
// the 32 lanes of each of the four warps' quarters.
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint32_t desc) {
    asm volatile(
        "{\n\t.reg .b64 s;\n\tmov.b64 s, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], s;\n\t}" ::"r"(taddr),
        "r"(desc), "n"(kScaleLayout)
        : "memory");
}

// Instruction descriptor of an e4m3 x e4m3 product with E8M0 scales: M = m
// (128, or 256 for a pair of CTAs), N = n (a multiple of 16), and which byte of
// the scale words this K step of 32 uses.
__device__ __forceinline__ uint32_t mx_instr_desc(uint32_t m, int n) {
    return ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((m >> 4) << 24);
}
__device__ __forceinline__ uint32_t mx_instr_step(uint32_t idesc, uint32_t step) {
    return idesc | (step << 4) | (step << 29);
}

// D[128, n] (+)= A[128, 32] * B[n, 32]^T with one scale per row and 32 columns.
__device__ __forceinline__ void tc_mma_mx(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                          bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)accumulate), "n"(kOperandLayout)
        : "memory");
}

// Arrives on `bar` once everything this thread issued to the tensor core is done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// 16 lanes x 16 columns in the fragment order of the 8 x 8 matrix stores:
// r[4 * h + 2 * i + j] = TMEM[lane / 4 + 8 * i, taddr + 8 * h + 2 * (lane % 4) + j].
__device__ __forceinline__ void tmem_load_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
// The loads are asynchronous: their registers are defined only behind this
// wait, which therefore names them.
__device__ __forceinline__ void tmem_load_wait(uint32_t (&a)[8], uint32_t (&b)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                   "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7])
                 :
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Barrier `id` (1 to 15) of the block's `threads` threads that call it.
__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Four 8 x 8 matrices of 16-bit elements, stored transposed: lane l gives the
// address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix_x4_trans(void* smem_row, const uint32_t (&m)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_addr(smem_row)),
                 "r"(m[0]), "r"(m[1]), "r"(m[2]), "r"(m[3])
                 : "memory");
}

// Asynchronous copy of 4 bytes to shared memory (`bytes` of them read, the rest zero).
__device__ __forceinline__ void cp_async4(void* smem_dst, const void* gmem_src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(smem_dst)), "l"(gmem_src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async16(void* smem_dst, const void* gmem_src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem_dst)), "l"(gmem_src) : "memory");
}
// Arrives on `bar` (one of its counted arrivals) once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ------------------------------------------------------- pairs of CTAs ----
// Two CTAs of a cluster may work on one product of M = 256 (cta_group::2): each
// holds 128 rows of A, half of the rows of B and the accumulators of its own
// 128 rows.  One thread of the CTA of rank 0 issues for both; descriptors and
// TMEM addresses name the same places in both.
constexpr uint16_t kPairMask = 3;
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_addr_out, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(smem_addr_out)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}
__device__ __forceinline__ void tc_copy_scales_pair(uint32_t taddr, uint32_t desc) {
    asm volatile(
        "{\n\t.reg .b64 s;\n\tmov.b64 s, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], s;\n\t}" ::"r"(taddr),
        "r"(desc), "n"(kScaleLayout)
        : "memory");
}
__device__ __forceinline__ void tc_mma_mx_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                               bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)accumulate), "n"(kOperandLayout)
        : "memory");
}
// Arrives on the barriers at this offset of both CTAs.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(kPairMask)
        : "memory");
}
// Arrives on the barrier at this offset of the CTA of rank 0, and releases to
// the cluster what this CTA has stored in its shared memory, for a wait that
// acquires it (an arrival without a scope orders its own CTA only).  The fence
// is for shared memory alone: with mbarrier.arrive.release.cluster, which
// releases global memory too, gate/up of 65,536 rows takes 419 us instead of 160.
__device__ __forceinline__ void mbar_arrive_first(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
        "fence.release.sync_restrict::shared::cta.cluster;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [r];\n\t}" ::"r"(smem_addr(bar))
        : "memory");
}

// Fetches a tensor map (a kernel parameter) ahead of its first copy.
__device__ __forceinline__ void prefetch_tmap(const void* tmap) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(tmap) : "memory");
}

// 3D tiled bulk copy of the box at (x, y, z); x * element size must be a
// multiple of 16 bytes, out-of-range elements read as zero.
__device__ __forceinline__ void tma_3d_g2s(void* smem_dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_addr(smem_dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

}  // namespace fp8q
