// sv_tc.cuh — the tensor-core instructions of sm_103a that sv_kv_attend's kernels use: tcgen05.mma with operands in shared or
// tensor memory, its completion barriers, and the moves between registers and tensor memory.
#pragma once

#include <cuda.h>

#include "sv_device.cuh"

namespace sv {

// A box of the tensor that `map` describes, to shared memory; completes its bytes on `bar`.
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// Shared-memory operand of tcgen05.mma in the 128-byte swizzle: rows of 128 bytes, 16-byte chunk c of row r at
// chunk c ^ (r & 7), groups of 8 rows `stride` bytes apart.  `lead` is the distance of the next 64 elements of an operand
// whose contiguous axis is not the one summed over (unused otherwise).
__device__ __forceinline__ uint64_t smem_operand(uint32_t addr, uint32_t lead, uint32_t stride) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)((lead >> 4) & 0x3FFF) << 16 | (uint64_t)((stride >> 4) & 0x3FFF) << 32 |
           1ull << 46 | 2ull << 61;
}

// bf16 operands, float32 accumulation, M = 128 rows by N columns.  a_t, b_t: the operand's contiguous axis in shared memory is not
// the one summed over; a_neg, b_neg: the operand enters negated.
__host__ __device__ constexpr uint32_t mma_shape(int N, bool a_t, bool b_t, bool a_neg, bool b_neg) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (a_neg ? 1u << 13 : 0u) | (b_neg ? 1u << 14 : 0u) | (a_t ? 1u << 15 : 0u) |
           (b_t ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 | (128u >> 4) << 24;
}

// The same with binary16 operands.
__host__ __device__ constexpr uint32_t mma_shape_f16(int N, bool a_t, bool b_t, bool a_neg, bool b_neg) {
    return mma_shape(N, a_t, b_t, a_neg, b_neg) & ~(1u << 7 | 1u << 10);
}

// One thread of the warp, the same one every time.  Products are issued inside `if (elect_one())` in code that the whole
// warp runs with uniform operands: they then cost 13 (A in tensor memory) to 33 cycles each to issue, against 75 to 100 when
// the thread is picked by its number, and the tensor cores take 64 for 128 x 128 x 16.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
    return p != 0;
}

// D (tensor memory) = or += A B, both from shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(shape), "r"(accumulate)
        : "memory");
}
// A from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t shape, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(shape), "r"(accumulate)
        : "memory");
}
// The barrier completes once every tcgen05 operation this thread issued before has finished.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Writes to shared memory become visible to the tensor cores' reads.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tmem_alloc(uint32_t *where, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}

#define SV_R4(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3])
#define SV_R16(x, i) SV_R4(x, i), SV_R4(x, i + 4), SV_R4(x, i + 8), SV_R4(x, i + 12)
#define SV_W4(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3])
#define SV_W16(x, i) SV_W4(x, i), SV_W4(x, i + 4), SV_W4(x, i + 8), SV_W4(x, i + 12)

// 32 columns of the warp's 32 rows: a thread gets its row's 32 words.  Complete after tc_wait_ld.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *x) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : SV_R16(x, 0), SV_R16(x, 16)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *x) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : SV_R16(x, 0)
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *x) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
        ::SV_W16(x, 0), SV_W16(x, 16), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *x) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::SV_W16(x, 0),
                 "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld4(uint32_t at, uint32_t (&x)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at));
}
__device__ __forceinline__ void tmem_ld8(uint32_t at, uint32_t (&x)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : SV_R4(x, 0), SV_R4(x, 4) : "r"(at));
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&x)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::SV_W4(x, 0), SV_W4(x, 4), "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t addr) {
    uint32_t x;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(addr));
    return x;
}

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace sv
