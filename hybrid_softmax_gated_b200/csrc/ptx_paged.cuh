// Inline-PTX wrappers that only the kernels over the paged cache use: e4m3
// products, 16-byte asynchronous copies, 16-column TMEM stores.  Each wrapper is
// one PTX instruction, or an issue sequence of one kind.
#pragma once

#include "ptx.cuh"

namespace arl2 {
namespace ptx {

// Asynchronous copy of 16 bytes into shared memory (src_bytes = 0: zeros), and an
// arrival on bar when the thread's copies so far have landed (it counts as one
// of the barrier's expected arrivals).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(__cvta_generic_to_global(src))), "r"(src_bytes)
                 : "memory");
}

__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// D[tmem] (+)= A[smem desc] * B[smem desc] with e4m3 operands, 32 deep (the
// whole warp; one elected lane issues).
__device__ __forceinline__ void umma_e4m3_ss_w(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

// Instruction descriptor for kind::f8f6f4 with e4m3 A and B, both K-major, fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4)                      // D format fp32 (A and B formats 0: e4m3)
           | ((uint32_t)(N >> 3) << 17)   // N / 8
           | ((uint32_t)(M >> 4) << 24);  // M / 16
}

// D = A_0 B + A_1 B with e4m3 operands, 128 deep (four k-steps of 32 bytes
// each): A_0 and A_1 are two K-major tiles of 128 rows x 128 bytes, 16 KB
// apart, B one such tile.
__device__ __forceinline__ void umma_e4m3_two_terms(uint32_t d_tmem, uint64_t a0, uint64_t b0, uint32_t idesc) {
    const uint32_t alo = (uint32_t)a0, ahi = (uint32_t)(a0 >> 32);
    const uint32_t blo = (uint32_t)b0, bhi = (uint32_t)(b0 >> 32);
    asm volatile(
        "{\n\t.reg .pred e, p, one;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t"
        "setp.ne.b32 p, %5, %5;\n\t"
        "setp.eq.b32 one, %5, %5;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t"
        "add.u32 x, %1, 2;\n\tadd.u32 y, %3, 2;\n\tmov.b64 a, {x, %2};\n\tmov.b64 b, {y, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, one;\n\t"
        "add.u32 x, %1, 4;\n\tadd.u32 y, %3, 4;\n\tmov.b64 a, {x, %2};\n\tmov.b64 b, {y, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, one;\n\t"
        "add.u32 x, %1, 6;\n\tadd.u32 y, %3, 6;\n\tmov.b64 a, {x, %2};\n\tmov.b64 b, {y, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, one;\n\t"
        "add.u32 x, %1, 1024;\n\tmov.b64 a, {x, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, one;\n\t"
        "add.u32 x, %1, 1026;\n\tadd.u32 y, %3, 2;\n\tmov.b64 a, {x, %2};\n\tmov.b64 b, {y, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, one;\n\t"
        "add.u32 x, %1, 1028;\n\tadd.u32 y, %3, 4;\n\tmov.b64 a, {x, %2};\n\tmov.b64 b, {y, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, one;\n\t"
        "add.u32 x, %1, 1030;\n\tadd.u32 y, %3, 6;\n\tmov.b64 a, {x, %2};\n\tmov.b64 b, {y, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, one;\n\t}" ::"r"(d_tmem),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc)
        : "memory");
}

}  // namespace ptx
}  // namespace arl2
