// q4_tcgen05.cuh -- 5th-generation tensor core (tcgen05) building blocks for
// sm_100a: tensor-memory allocation, register <-> tensor-memory copies, the
// shared-memory matrix descriptor of a 128-byte-swizzled K-major tile, the
// instruction descriptor of a 16-bit MMA with fp32 accumulation, the MMA with
// its A operand in tensor memory, and completion tracking through mbarriers.
//
// Tensor memory (TMEM) is 128 lanes x 512 columns of 32 bits per SM.  An
// address is (lane << 16) | column; warp w of a CTA may touch only lanes
// [32 (w % 4), 32 (w % 4) + 32).  An M = 128 accumulator holds row m in lane m;
// a 16-bit A operand holds row m in lane m with elements k, k+1 packed in one
// column (k even in the low half).
#pragma once

#include <stdint.h>

#include "q4_device.cuh"

namespace q4dev {

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Whole-warp TMEM allocation of `ncols` columns (a power of two >= 32); the
// base address is written to shared memory at `dst`.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(dst)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}

// Eight consecutive columns of this thread's lane from / to registers.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}
// Sixteen lanes (taddr's and the 15 after it) x 16 columns in the layout of MMA
// accumulators: of the i-th 8 columns, v[4 i], v[4 i + 1] are columns 2 (lane % 4),
// + 1 of lane lane / 4, and v[4 i + 2], v[4 i + 3] the same of lane lane / 4 + 8.
// No memory clobber: the values are tied to the wait by tmem_wait_ld_for instead, so that
// the compiler may schedule other loads around both.
__device__ __forceinline__ void tmem_ld_frag16(uint32_t taddr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld_for(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
                   "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]),
                   "+r"(v[13]), "+r"(v[14]), "+r"(v[15]));
}
__device__ __forceinline__ void tmem_st_frag16w(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
}
// Sixteen lanes x 8 columns of packed pairs in the same layout: v[2 i] is column
// 4 i + lane % 4 of lane lane / 4, v[2 i + 1] of lane lane / 4 + 8.
__device__ __forceinline__ void tmem_st_pairs8(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Shared-memory descriptor of a K-major operand tile stored with the 128-byte
// swizzle, as a TMA load with CU_TENSOR_MAP_SWIZZLE_128B writes it: rows of
// 128 bytes, groups of 8 rows 1024 bytes apart, the atom 1024-byte aligned.
// `saddr` is the shared address of the first row's 16-element (32-byte) K
// slice; slices further along K inside the 128-byte row are addressed by
// adding their byte offset to the start address.
__device__ __forceinline__ uint64_t umma_desc_sw128_kmajor(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);  // start address, 16-byte units
    d |= static_cast<uint64_t>(16 >> 4) << 16;           // leading offset (unused by SW128 K-major)
    d |= static_cast<uint64_t>(1024 >> 4) << 32;         // stride between 8-row groups
    d |= static_cast<uint64_t>(1) << 46;                 // descriptor version of sm_100
    d |= static_cast<uint64_t>(2) << 61;                 // layout: 128-byte swizzle
    return d;
}

// Shared-memory descriptor of a B operand [K, N] stored with N contiguous
// (N-major), 128-byte swizzle: blocks of 64 N elements `block_bytes` apart, in a
// block one 128-byte row per K index, groups of 8 rows 1024 bytes apart, each
// row's 16-byte chunks XOR-ed with its index in the group.  `saddr` is the
// address of the K slice's first row (1024-byte aligned).
__device__ __forceinline__ uint64_t umma_desc_sw128_nmajor(uint32_t saddr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((block_bytes >> 4) & 0x3FFFu) << 16;  // between blocks of 64 along N
    d |= static_cast<uint64_t>(1024 >> 4) << 32;                     // between groups of 8 along K
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
// Bit of the instruction descriptor for such a B.
constexpr uint32_t kIdescNMajorB = 1u << 16;

// Instruction descriptor: D fp32, A and B bf16 (or fp16), both K-major,
// M x N with M in {64, 128} and N a multiple of 16 (M = 128).
template <bool BF16, int M, int N>
__host__ __device__ constexpr uint32_t umma_idesc_f16() {
    return (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A[tmem] * B[smem]^T for one K = 16 step; `accumulate` = 0
// overwrites D.  Issued by one thread.
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n\t}" ::"r"(
            tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(0u), "r"(0u), "r"(0u), "r"(0u)
        : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T for one K = 16 step, both operands
// described by shared-memory descriptors.  Issued by one thread.
__device__ __forceinline__ void umma_f16_ss(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive (once) on `bar` when every MMA this thread issued so far completes.
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_u32(bar))
        : "memory");
}

// Generic-proxy writes to shared memory before this are visible to the tensor
// core's reads that are ordered after it.
__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

}  // namespace q4dev
