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

// Four codes as two pairs of f16, exact: bytes (0, 1) and (2, 3), or, TRANSPOSED, (0, 2) and (1, 3) -- the codes of two keys at
// one channel each, where the word holds two neighbouring channels of two keys.
template <int FMT, bool TRANSPOSED>
__device__ __forceinline__ void q8_to_f16(uint32_t w, uint32_t& a, uint32_t& b) {
    if (FMT == RX_Q8_INT8) {
        // the code plus 128 as the last bits of 1024, and 1152 taken off
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t x = __byte_perm(u, 0x64646464u, TRANSPOSED ? 0x4240 : 0x4140);
        const uint32_t y = __byte_perm(u, 0x64646464u, TRANSPOSED ? 0x4341 : 0x4342);
        const uint32_t off = 0x64806480u;                   // 1152, twice
        const __half2 p = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&off));
        const __half2 q = __hsub2(*reinterpret_cast<const __half2*>(&y), *reinterpret_cast<const __half2*>(&off));
        a = *reinterpret_cast<const uint32_t*>(&p);
        b = *reinterpret_cast<const uint32_t*>(&q);
    } else {
        if (TRANSPOSED) w = __byte_perm(w, 0, 0x3120);
        const __half2_raw p = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
        const __half2_raw q = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
        a = *reinterpret_cast<const uint32_t*>(&p);
        b = *reinterpret_cast<const uint32_t*>(&q);
    }
}

// Four codes as two pairs of bf16, exact.
template <int FMT>
__device__ __forceinline__ void q8_to_bf16(uint32_t w, uint32_t& a, uint32_t& b) {
    const uint32_t low = w & 0x7f7f7f7fu, top = w & 0x80808080u;
    if (FMT == RX_Q8_INT8) {
        // 128 + the code's low seven bits, less 128 or, where its top bit is set, 256
        const uint32_t x = __byte_perm(low, 0x43434343u, 0x4140), y = __byte_perm(low, 0x43434343u, 0x4342);
        const uint32_t u = __byte_perm(top, 0x43434343u, 0x4140), v = __byte_perm(top, 0x43434343u, 0x4342);
        const __nv_bfloat162 p = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&u));
        const __nv_bfloat162 q = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&y), *reinterpret_cast<const __nv_bfloat162*>(&v));
        a = *reinterpret_cast<const uint32_t*>(&p);
        b = *reinterpret_cast<const uint32_t*>(&q);
    } else {
        // exponent and mantissa at bf16's places make 2^-120 of the value (the smallest ones bf16 numbers below
        // 2^-126, which the product takes as they are); 0x7f, e4m3's NaN, which no computed code is, reads as 480
        const uint32_t x = __byte_perm(low, 0, 0x4140) * 16 + __byte_perm(top, 0, 0x1404);
        const uint32_t y = __byte_perm(low, 0, 0x4342) * 16 + __byte_perm(top, 0, 0x3424);
        const uint32_t scale = 0x7b807b80u;                  // 2^120, twice
        const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&scale));
        const __nv_bfloat162 q = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&y), *reinterpret_cast<const __nv_bfloat162*>(&scale));
        a = *reinterpret_cast<const uint32_t*>(&p);
        b = *reinterpret_cast<const uint32_t*>(&q);
    }
}

}  // namespace rx
