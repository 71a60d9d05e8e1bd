// tcgen05 instructions issued by a warp, a group of products at a time.
#pragma once

#include <stdint.h>

namespace rx {

// ---------------------------------------------------------------- tensor core instructions of a warp
// The whole warp runs the issuing code, so that addresses and descriptors stay warp-uniform, and
// one elected lane issues a group of products.  (Issued under `if (lane == 0)`, one product at a
// time, they took 75 clocks each where the tensor core needs 64.)  Descriptors (sdesc_sw128) come as
// their low word (start address in 16-byte units, leading offset); the high word (stride offset 1024
// bytes, version, 128-byte swizzle) is the same for all.
constexpr uint32_t PT_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);

#define PT_SS(DA, DB, ACC)                                                     \
    "add.u32 a, %1, " #DA ";\n\tadd.u32 b, %2, " #DB ";\n\t"                   \
    "mov.b64 da, {a, %4};\n\tmov.b64 db, {b, %4};\n\t"                         \
    "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, " #ACC ";\n\t"
#define PT_TS(TA, DB, ACC)                                                     \
    "add.u32 a, %1, " #TA ";\n\tadd.u32 b, %2, " #DB ";\n\t"                   \
    "mov.b64 db, {b, %4};\n\t"                                                 \
    "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, " #ACC ";\n\t"
#define PT_GROUP "{\n\t.reg .pred e, t, f;\n\t.reg .b32 a, b;\n\t.reg .b64 da, db;\n\telect.sync _|e, 0xffffffff;\n\t"

// S[128 x 128] = Q K^T over D channels: 16 channels (32 bytes) an instruction, 64 a 16 KB half tile.
template <int D>
__device__ __forceinline__ void pt_mma_s(uint32_t s, uint32_t q, uint32_t k, uint32_t idesc) {
    if constexpr (D == 128)
        asm volatile(PT_GROUP "setp.eq.u32 t, 0, 0;\n\tsetp.ne.u32 f, 0, 0;\n\t" PT_SS(0, 0, f) PT_SS(2, 2, t) PT_SS(4, 4, t)
                         PT_SS(6, 6, t) PT_SS(1024, 1024, t) PT_SS(1026, 1026, t) PT_SS(1028, 1028, t) PT_SS(1030, 1030, t) "}" ::"r"(s),
                     "r"(q), "r"(k), "r"(idesc), "r"(PT_DESC_HI)
                     : "memory");
    else
        asm volatile(PT_GROUP "setp.eq.u32 t, 0, 0;\n\tsetp.ne.u32 f, 0, 0;\n\t" PT_SS(0, 0, f) PT_SS(2, 2, t) PT_SS(4, 4, t)
                         PT_SS(6, 6, t) "}" ::"r"(s),
                     "r"(q), "r"(k), "r"(idesc), "r"(PT_DESC_HI)
                     : "memory");
}

// O[128 x D] += P V over 64 keys: 16 keys (8 TMEM columns of P, 2 KB of V) an instruction; with
// `fresh` the first of them overwrites O.
__device__ __forceinline__ void pt_mma_pv(uint32_t o, uint32_t pt, uint32_t v, uint32_t idesc, bool fresh) {
    asm volatile(PT_GROUP "setp.eq.u32 t, 0, 0;\n\tsetp.eq.u32 f, %5, 0;\n\t" PT_TS(0, 0, f) PT_TS(8, 128, t) PT_TS(16, 256, t)
                     PT_TS(24, 384, t) "}" ::"r"(o),
                 "r"(pt), "r"(v), "r"(idesc), "r"(PT_DESC_HI), "r"(fresh ? 1u : 0u)
                 : "memory");
}
#undef PT_SS
#undef PT_TS
#undef PT_GROUP

__device__ __forceinline__ void pt_commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

}  // namespace rx
