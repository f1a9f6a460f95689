// Fifth-generation tensor core (tcgen05) building blocks for sm_100a, kind::f16 with
// fp16 operands and fp32 accumulators (tensor memory and barriers: stepq_tc.cuh).
//
// Shared-memory operands use the 128-byte swizzle: rows of 128 bytes (64
// values), 8-row groups of 1,024 bytes, the 16-byte chunk c of row r at chunk
// position c ^ (r % 8); tiles start on 1,024-byte boundaries.  Such a tile serves as
// a K-major operand (row = M or N index, its values along K) and, since K may be the
// row index just as well, as an MN-major one.  An A operand in tensor memory holds
// two consecutive K values in a 32-bit column, row m in lane m.
#pragma once

#include <cuda_fp16.h>

#include "stepq_tc.cuh"

namespace stepq {
namespace tc16 {

// Byte offset of (row, col) in a tile of 128-byte rows of 16-bit values, col < 64.
__host__ __device__ constexpr uint32_t sw_off(int row, int col) {
    return (uint32_t)(row * 128 + (((col >> 3) ^ (row & 7)) << 4) + (col & 7) * 2);
}

// Descriptor: 128-byte swizzle (2 at bit 61), version 1 at bit 46.  K-major: groups of 8 rows SBO
// apart (the other stride is not used).  MN-major: 64-value columns blocks LBO apart, groups of 8 K rows SBO apart.
__device__ __forceinline__ uint64_t desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFF) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t kmajor(uint32_t saddr) { return desc(saddr, 16, 1024); }

// Instruction descriptor: D f32, A and B f16, A K-major, B K-major or MN-major, M x N.
__host__ __device__ constexpr uint32_t idesc(int m, int n, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

// True in one lane of the (whole) warp, always the same one.
__device__ __forceinline__ bool elect() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}

// D (tmem) [+]= A B for one K step of 16: A from shared memory / from tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
}

#define STEPQ_W8(b) "r"(v[b]), "r"(v[b + 1]), "r"(v[b + 2]), "r"(v[b + 3]), "r"(v[b + 4]), "r"(v[b + 5]), \
                    "r"(v[b + 6]), "r"(v[b + 7])
// Twice 16 consecutive columns of this warp's lanes; waits for both loads.
__device__ __forceinline__ void ld16x2(uint32_t ta, uint32_t (&v)[16], uint32_t tb, uint32_t (&w)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]), "=r"(w[8]), "=r"(w[9]), "=r"(w[10]), "=r"(w[11]), "=r"(w[12]), "=r"(w[13]), "=r"(w[14]), "=r"(w[15])
        : "r"(ta), "r"(tb)
        : "memory");
}
// Stores of 16 / 32 columns of this warp's lanes; st_wait() before anything reads them.
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
                     taddr),
                 STEPQ_W8(0), STEPQ_W8(8)
                 : "memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        STEPQ_W8(0), STEPQ_W8(8), STEPQ_W8(16), STEPQ_W8(24)
        : "memory");
}
#undef STEPQ_W8
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// (x0, x1) as the sum of two fp16 pairs: hi the nearest, lo the nearest to the rest.
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __float22half2_rn(x);
    const float2 back = __half22float2(h);
    const __half2 l = __floats2half2_rn(x.x - back.x, x.y - back.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
__device__ __forceinline__ uint32_t pack2(float2 x) {
    const __half2 h = __float22half2_rn(x);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// One warp's 16 x 8 += 16 x 16 times 16 x 8 (the warp-level instruction, for products too small for the others).
__device__ __forceinline__ void mma_sync(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Barrier `id` of n threads; true where every thread's ok was.
__device__ __forceinline__ bool group_and(int id, int n, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n barrier.cta.red.and.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(r)
        : "r"(id), "r"(n), "r"((uint32_t)ok)
        : "memory");
    return r != 0;
}

}  // namespace tc16
}  // namespace stepq
