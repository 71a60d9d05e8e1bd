// 8-bit codes of the KV pools: where a value's scale is, and the codes' conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "radix_attn.h"
#include "rx_common.h"

namespace rx {

// The pools of one layer.
struct Q8Pools {
    const uint8_t* k;
    const uint8_t* v;
    const float2* scales;      // [blocks][hkv]: K's, V's
    int32_t shift;             // log2 of the slots per scale
};

// The scales of a slot's kv head.
__device__ __forceinline__ float2 q8_scales(const Q8Pools& p, int32_t slot, int hkv, int g) {
    return p.scales[(int64_t)(slot >> p.shift) * hkv + g];
}

inline int q8_shift(const rx_q8_desc* q) {
    int s = 0;
    while ((1 << s) < q->block) ++s;
    return s;
}

// The checks that all entry points share.
inline int q8_check(const char* fn, const rx_attn_desc* d, const rx_q8_desc* q, bool attention) {
    RX_REQUIRE(d && q, "%s: bad arguments", fn);
    RX_REQUIRE(d->dtype == RX_F32 || d->dtype == RX_BF16, "%s: unknown dtype %d", fn, d->dtype);
    RX_REQUIRE(d->head_dim == 64 || d->head_dim == 128, "%s: head_dim must be 64 or 128", fn);
    RX_REQUIRE(d->hkv > 0 && d->hkv <= 4096 && d->num_slots > 0 && d->num_slots <= INT32_MAX, "%s: bad shape", fn);
    RX_REQUIRE(!attention || (d->hq > 0 && d->hq <= 4096 && d->hq % d->hkv == 0), "%s: bad head counts", fn);
    RX_REQUIRE(q->format == RX_Q8_INT8 || q->format == RX_Q8_E4M3, "%s: unknown format %d", fn, q->format);
    RX_REQUIRE(q->block >= 1 && q->block <= (1 << 30) && (q->block & (q->block - 1)) == 0,
               "%s: a scale's block of %d slots is not a power of two up to 2^30", fn, q->block);
    RX_REQUIRE(q->fixed == 0 || q->fixed == 1, "%s: fixed must be 0 or 1", fn);
    RX_REQUIRE(q->fixed || q->block == 1, "%s: scales of blocks of %d slots have to be given (fixed)", fn, q->block);
    return RX_OK;
}

// Four codes, as 32-bit numbers.
template <int FMT>
__device__ __forceinline__ void q8_to_f32(uint32_t w, float* f) {
    if (FMT == RX_Q8_INT8) {
        // the code plus 128 as the last bits of 2^23, and that taken off: exact, without an integer conversion
        const uint32_t u = w ^ 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)) - 8388736.f;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3));
            const float2 x = __half22float2(h);
            f[2 * i] = x.x;
            f[2 * i + 1] = x.y;
        }
    }
}

}  // namespace rx
