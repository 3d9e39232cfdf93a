// attention_tc.cuh -- what the tcgen05 attention kernels share: operand and
// instruction descriptors, TMA loads of caches and queries, the MMAs of a product.
#pragma once
#include <cstdint>

#include "common.cuh"
#include "tc.cuh"

namespace dtm {

// B operand, MN-major, 128-byte swizzle: 64 elements of N contiguous, the
// next 64 `lbo` bytes on; 8 rows of K 128 bytes apart, the next 8 1024 on.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t lbo) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

template <bool F16>
__host__ __device__ constexpr uint32_t pa_idesc(uint32_t N, bool mn_major_b) {
    return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | (mn_major_b ? 1u << 16 : 0u) |
           ((N >> 3) << 17) | ((128u >> 4) << 24);
}

// Called by the whole warp; an elected lane issues.
__device__ __forceinline__ void tma_load_4d_elect(uint32_t dst, const void *tmap, int x, int y, int z,
                                            int w, uint32_t bar) {
    asm volatile(
        "{ .reg .pred p; elect.sync _|p, 0xffffffff;\n"
        "@p cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4, %5}], [%6]; }" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int x, int y, int z,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4}], [%5];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void ld_32x32b_x32(uint32_t taddr, float *r) {
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
          "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
          "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr)
        : "memory");
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (F16) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    return bf16x2_rn(lo, hi);
}

// The MMAs of one product, issued by an elected lane of the whole warp, in one
// block with one election: 4 (D = 64) or 8 steps of 16 along the scores' inner
// dimension, 8 along a tile's keys.  Operands advance in the descriptors'
// 16-byte units, the A operand in TMEM in columns.
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    if (D == 64) {
        asm volatile(
            "{ .reg .pred p, f, t; .reg .b64 a1, a2, a3, b1, b2, b3;\n"
            "setp.ne.u32 f, 0, 0; setp.eq.u32 t, 0, 0; elect.sync _|p, 0xffffffff;\n"
            "add.s64 a1, %1, 2; add.s64 a2, %1, 4; add.s64 a3, %1, 6;\n"
            "add.s64 b1, %2, 2; add.s64 b2, %2, 4; add.s64 b3, %2, 6;\n"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t; }" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc)
            : "memory");
    } else {
        asm volatile(
            "{ .reg .pred p, f, t; .reg .b64 a1, a2, a3, a4, a5, a6, a7, b1, b2, b3, b4, b5, b6, b7;\n"
            "setp.ne.u32 f, 0, 0; setp.eq.u32 t, 0, 0; elect.sync _|p, 0xffffffff;\n"
            "add.s64 a1, %1, 2; add.s64 a2, %1, 4; add.s64 a3, %1, 6; add.s64 a4, %1, 1024;\n"
            "add.s64 a5, %1, 1026; add.s64 a6, %1, 1028; add.s64 a7, %1, 1030;\n"
            "add.s64 b1, %2, 2; add.s64 b2, %2, 4; add.s64 b3, %2, 6; add.s64 b4, %2, 1024;\n"
            "add.s64 b5, %2, 1026; add.s64 b6, %2, 1028; add.s64 b7, %2, 1030;\n"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a4, b4, %3, t;\n"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a5, b5, %3, t;\n"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a6, b6, %3, t;\n"
            "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a7, b7, %3, t; }" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc)
            : "memory");
    }
}
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p, q, t; .reg .b32 a1, a2, a3, a4, a5, a6, a7; .reg .b64 b1, b2, b3, b4, b5, b6, b7;\n"
        "setp.ne.u32 q, %4, 0; setp.eq.u32 t, 0, 0; elect.sync _|p, 0xffffffff;\n"
        "add.s32 a1, %1, 8; add.s32 a2, %1, 16; add.s32 a3, %1, 24; add.s32 a4, %1, 32;\n"
        "add.s32 a5, %1, 40; add.s32 a6, %1, 48; add.s32 a7, %1, 56;\n"
        "add.s64 b1, %2, 128; add.s64 b2, %2, 256; add.s64 b3, %2, 384; add.s64 b4, %2, 512;\n"
        "add.s64 b5, %2, 640; add.s64 b6, %2, 768; add.s64 b7, %2, 896;\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a4], b4, %3, t;\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a5], b5, %3, t;\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a6], b6, %3, t;\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a7], b7, %3, t; }" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The lowest n bits (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t ones(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

}  // namespace dtm
