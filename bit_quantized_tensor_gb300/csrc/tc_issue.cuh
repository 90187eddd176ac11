// tcgen05.mma of fp16 operands issued by a whole warp under an elected lane's predicate, with
// shared-memory descriptors whose high word is fixed: in convergent code their words stay in
// uniform registers.
#pragma once
#include "qg_ptx.cuh"

namespace qg {

// 128-byte swizzle, 1024 bytes between groups of 8 rows; the low word has the address and, for an
// MN-major operand, the distance of the next 64 columns (K-major: 16).
constexpr uint32_t kTileHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t tile_lo(uint32_t addr, uint32_t next) {
    return ((addr & 0x3FFFFu) >> 4) | ((next >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t accumulate,
                                       uint32_t elected) {
    asm volatile(
        "{\n.reg .pred p, q;\n.reg .b64 da, db;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "mov.b64 da, {%1, %6};\nmov.b64 db, {%2, %6};\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "r"(elected), "r"(kTileHi)
        : "memory");
}

}  // namespace qg
