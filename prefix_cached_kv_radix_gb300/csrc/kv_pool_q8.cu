// kv_pool_write_q8 and kv_pool_read_q8: K/V rows into pools of 8-bit codes, and back.
//
// A written row (one token, one kv head, K or V) becomes d codes and a scale: a = max |x|, s = a / 127 (int8) or the
// smallest power of two with a <= 448 s (e4m3), code = x / s rounded to nearest.  A group of d / 8 lanes
// holds one token's K row and V row of one head in registers, 8 elements a lane, so a is a reduction over 3 or 4
// shuffles, each element is read once and its code written once, and both scales leave in one
// 8-byte store.  Bound by HBM: d * (size + 1) + 4 bytes a row.  Measured: 24 ragged prompts of up to 2049 (bf16, 8 heads x 128,
// e4m3) 31.8 us, 5.0 TB/s or 75 % of a copy, with the arithmetic pipes beside it; 64 decode tokens 3.0 us, a launch; 40001 slots
// read (int8) 39.4 us, 94 % of a copy.
//
// The codes are those of the real quotient.  For e4m3 1 / s is a power of two and the product exact.  For int8 (and given
// scales) q = x * (1 / s) is off by a few 2^-24 of itself, which matters only next to a half: there the
// sign of x - t s, t the half, decides (one fused multiply-add, whose sign is that of the exact difference).
#include <cuda_runtime.h>

#include <algorithm>

#include "kv_pool_table.cuh"
#include "kv_q8.cuh"
#include "radix_attn.h"
#include "rx_common.h"
#include "rx_device.cuh"
#include "rx_launch.h"

namespace rx {

constexpr int Q8_THREADS = 256;
constexpr int Q8_TILE = Q8_THREADS * 4;            // slot-table entries per block
constexpr float Q8_LEAST = 0x1p-126f;              // no scale is smaller

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Eight elements of a row.  Magnitudes are compared as integers: a NaN is above all others.
template <typename T>
struct Row8;
template <>
struct Row8<float> {
    uint4 u[2];
    __device__ __forceinline__ void load(const float* p) {
        u[0] = reinterpret_cast<const uint4*>(p)[0];
        u[1] = reinterpret_cast<const uint4*>(p)[1];
    }
    __device__ __forceinline__ void get(float* f) const {
        const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
        return m;
    }
    // the largest magnitudes of two rows, each spread over LANES lanes, as bits of float
    template <int LANES>
    static __device__ __forceinline__ void tops(const Row8& k, const Row8& v, uint32_t* t) {
        t[0] = k.top(), t[1] = v.top();
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) {
            t[0] = max(t[0], __shfl_xor_sync(0xffffffffu, t[0], o));
            t[1] = max(t[1], __shfl_xor_sync(0xffffffffu, t[1], o));
        }
    }
    static __device__ __forceinline__ void store(float* p, const float* f) {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};
template <>
struct Row8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float* f) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // of the even and of the odd elements, in the two halves
    __device__ __forceinline__ uint32_t top() const {
        return max_u16x2(max_u16x2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), max_u16x2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
    }
    template <int LANES>
    static __device__ __forceinline__ void tops(const Row8& k, const Row8& v, uint32_t* t) {
        const uint32_t a = k.top(), b = v.top();
        uint32_t m = max_u16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));      // K's low, V's high
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
        t[0] = m << 16, t[1] = m & 0xffff0000u;
    }
    // rounded once, from the 32-bit product
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};

// The scale of a row whose largest magnitude has these bits.
template <int FMT>
__device__ __forceinline__ float scale_of(uint32_t bits) {
    if (bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);        // an infinity or NaN
    if (FMT == RX_Q8_INT8) return fmaxf(__fdiv_rn(__uint_as_float(bits), 127.f), Q8_LEAST);
    // 448 = 1.75 * 2^8: the exponent less 8, and one more where the mantissa is above 1.75
    const int e = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// q = x / s but for a few units of its last place, as the nearest whole number to the real quotient.
__device__ __forceinline__ float nearest_whole(float q, float x, float s) {
    const float n = rintf(q), d = q - n;
    if (fabsf(d) < 0.4999f) return n;
    const float t = n + copysignf(0.5f, d), r = fmaf(-t, s, x);
    return r > 0.f ? t + 0.5f : r < 0.f ? t - 0.5f : rintf(t);
}

template <bool FIXED>
__device__ __forceinline__ uint2 codes_int8(const float* x, float s, float inv) {
    // 1.5 * 2^23 + q: its last bits are q = x / s rounded to a whole number n; x - n s, which is exact, tells how near a half q was
    constexpr float MAGIC = 12582912.f;
    float n[8], off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float y = x[i];
        if (FIXED) y = y == y ? fminf(fmaxf(y, -127.f * s), 127.f * s) : 0.f;
        n[i] = fmaf(y, inv, MAGIC);
        off = fmaxf(off, fabsf(fmaf(MAGIC - n[i], s, y)));
    }
    // some quotient is next to a half, or 127 s is no number that an infinity could be cut to
    if (off >= 0.4999f * s || (FIXED && s > 0x1p121f)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float q = x[i] * inv;
            if (FIXED) q = q == q ? q : 0.f;
            n[i] = fminf(fmaxf(fabsf(q) < 128.f ? nearest_whole(q, x[i], s) : q, -127.f), 127.f) + MAGIC;
        }
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = __byte_perm(__byte_perm(__float_as_uint(n[4 * i]), __float_as_uint(n[4 * i + 1]), 0x0040),
                           __byte_perm(__float_as_uint(n[4 * i + 2]), __float_as_uint(n[4 * i + 3]), 0x0040), 0x5410);
    return make_uint2(w[0], w[1]);
}

template <bool FIXED>
__device__ __forceinline__ uint2 codes_e4m3(const float* x, float s, float inv) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = x[i] * inv;
        if (FIXED) {
            if (y[i] != y[i]) y[i] = 0.f;          // a NaN
            // Steps of e4m3 at y: an eighth of its power of two, 2^-9 at least.  Next to the middle between two
            // codes the exact difference decides, by moving y off that middle.
            const int e = min(max((int)((__float_as_uint(y[i]) >> 23) & 0xffu), 121), 136) - 3;
            const float step = __uint_as_float((uint32_t)e << 23), z = y[i] * __uint_as_float((uint32_t)(254 - e) << 23);
            const float n = rintf(z), d = z - n;
            if (fabsf(z) < 32.f && fabsf(d) > 0.4999f) {
                const float t = (n + copysignf(0.5f, d)) * step, r = fmaf(-t, s, x[i]);
                y[i] = r == 0.f ? t : __uint_as_float(__float_as_uint(t) + ((r > 0.f) == (t > 0.f) ? 1 : -1));
            }
        }
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i], y[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2], y[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

struct WriteQ8Params {
    int32_t batch, tiles;
    const int32_t* prefix_slots;
    const int64_t* prefix_indptr;
    const int32_t* new_slots;
    const int64_t* qo_indptr;
    const void* k;
    const void* v;
    int64_t k_stride, v_stride;
    uint8_t* k_pool;
    uint8_t* v_pool;
    float2* scales;
    int32_t shift, hkv, step_rows, step_heads;     // a block's lane groups: so many rows and heads from a group's unit to its next
    int32_t* r2t;
    int64_t r2t_stride, num_slots, total;
    int32_t* status;
};

// Blocks [0, batch * tiles): the slot table.  The others: Q8_UNITS * (Q8_THREADS / (D / 8)) (token, head) pairs each, Q8_UNITS in flight
// per lane group.
template <typename T, int D, int FMT, bool FIXED, int Q8_UNITS>
__global__ void __launch_bounds__(Q8_THREADS) kv_pool_write_q8_kernel(const __grid_constant__ WriteQ8Params p) {
    constexpr int LANES = D / 8;                   // lanes of a row
    constexpr int ROWS = Q8_THREADS / LANES;       // pairs a block has in hand at a time
    pdl_launch_dependents();
    pdl_wait();
    const int64_t table_blocks = (int64_t)p.batch * p.tiles;
    if ((int64_t)blockIdx.x < table_blocks) {
        kpw_table_tile<Q8_THREADS>((int)(blockIdx.x / p.tiles), blockIdx.x % p.tiles, p.prefix_slots, p.prefix_indptr, p.new_slots,
                                   p.qo_indptr, p.r2t, p.r2t_stride, p.num_slots, 0, p.total, p.status);
        return;
    }
    const int64_t block = blockIdx.x - table_blocks;
    const int lane = threadIdx.x % LANES;
    const int64_t b0 = block * (ROWS * Q8_UNITS), tb = b0 / p.hkv;
    const uint32_t u0 = (uint32_t)(b0 - tb * p.hkv) + threadIdx.x / LANES, r0 = u0 / (uint32_t)p.hkv;
    Row8<T> k[Q8_UNITS], v[Q8_UNITS];
    int32_t slot[Q8_UNITS];
    int64_t t = tb + r0;
    int h = (int)(u0 - r0 * p.hkv);
    // the rows (total of them there are) and their slots beside the batch's boundaries, not after them
#pragma unroll
    for (int i = 0; i < Q8_UNITS; ++i) {
        slot[i] = -1;
        if (t < p.total) {
            slot[i] = p.new_slots[t];
            k[i].load((const T*)p.k + t * p.k_stride + h * D + lane * 8);
            v[i].load((const T*)p.v + t * p.v_stride + h * D + lane * 8);
        }
        t += p.step_rows;
        h += p.step_heads;
        if (h >= p.hkv) h -= p.hkv, ++t;
    }
    // rows of the batch only: what lies before its first and behind its last request is not written
    const int64_t first = p.qo_indptr[0], end = p.qo_indptr[p.batch];
    if (block == 0 && threadIdx.x == 0 && (end > p.total || first < 0 || end < first)) report(p.status, RX_DEV_BAD_LENGTH);
    t = tb + r0;
    h = (int)(u0 - r0 * p.hkv);
#pragma unroll
    for (int i = 0; i < Q8_UNITS; ++i) {
        const int head = h;
        const bool inside = t >= first && t < end && t < p.total;
        if (inside && (slot[i] < 0 || slot[i] >= p.num_slots) && head == 0 && lane == 0) report(p.status, RX_DEV_BAD_SLOT);
        const bool in = inside && slot[i] >= 0 && slot[i] < p.num_slots;      // the same in all lanes of a row
        t += p.step_rows;
        h += p.step_heads;
        if (h >= p.hkv) h -= p.hkv, ++t;
        const int64_t row = in ? (int64_t)slot[i] * p.hkv + head : 0;
        uint32_t top[2] = {0, 0};
        float s[2];
        if (FIXED) {
            const float2 given = p.scales[in ? (int64_t)(slot[i] >> p.shift) * p.hkv + head : 0];
            s[0] = given.x, s[1] = given.y;
        } else {
            Row8<T>::template tops<LANES>(k[i], v[i], top);                   // (rows that are not there: anything, and not used)
            s[0] = scale_of<FMT>(top[0]), s[1] = scale_of<FMT>(top[1]);
        }
        if (!in) continue;
        float x[2][8];
        k[i].get(x[0]);
        v[i].get(x[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint2 c = make_uint2(0u, 0u);
            if (FIXED || top[j] < 0x7f800000u) {
                const float inv = __frcp_rn(s[j]);
                c = FMT == RX_Q8_INT8 ? codes_int8<FIXED>(x[j], s[j], inv) : codes_e4m3<FIXED>(x[j], s[j], inv);
            }
            reinterpret_cast<uint2*>((j == 0 ? p.k_pool : p.v_pool) + row * D)[lane] = c;
        }
        if (!FIXED && lane == 0) p.scales[row] = make_float2(s[0], s[1]);
    }
}

struct ReadQ8Params {
    Q8Pools pools;
    const int32_t* slots;
    int64_t n, num_slots;
    int32_t hkv;
    void* k_out;
    void* v_out;
    int64_t k_stride, v_stride;
    int32_t* status;
};

// One (slot, head) pair per lane group and step, Q8_UNITS in flight.
template <typename T, int D, int FMT, int Q8_UNITS>
__global__ void __launch_bounds__(Q8_THREADS) kv_pool_read_q8_kernel(const __grid_constant__ ReadQ8Params p) {
    constexpr int LANES = D / 8;
    constexpr int ROWS = Q8_THREADS / LANES;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x % LANES;
    const int64_t b0 = (int64_t)blockIdx.x * (ROWS * Q8_UNITS), rb = b0 / p.hkv;
    const uint32_t u0 = (uint32_t)(b0 - rb * p.hkv) + threadIdx.x / LANES;
    uint2 c[Q8_UNITS][2];
    float2 s[Q8_UNITS];
    int64_t at[Q8_UNITS];
    int head[Q8_UNITS];
#pragma unroll
    for (int i = 0; i < Q8_UNITS; ++i) {
        const uint32_t u = u0 + i * ROWS, ur = u / (uint32_t)p.hkv;
        const int64_t r = rb + ur;
        head[i] = (int)(u - ur * p.hkv);
        at[i] = -1;
        if (r >= p.n) continue;
        const int32_t slot = p.slots[r];
        if (slot < 0 || slot >= p.num_slots) {
            if (head[i] == 0 && lane == 0) report(p.status, RX_DEV_BAD_SLOT);
            continue;
        }
        at[i] = r;
        const int64_t row = (int64_t)slot * p.hkv + head[i];
        s[i] = q8_scales(p.pools, slot, p.hkv, head[i]);
        if (p.k_out) c[i][0] = reinterpret_cast<const uint2*>(p.pools.k + row * D)[lane];
        if (p.v_out) c[i][1] = reinterpret_cast<const uint2*>(p.pools.v + row * D)[lane];
    }
#pragma unroll
    for (int i = 0; i < Q8_UNITS; ++i) {
        if (at[i] < 0) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            T* out = (T*)(j == 0 ? p.k_out : p.v_out);
            if (!out) continue;
            float f[8];
            q8_to_f32<FMT>(c[i][j].x, f);
            q8_to_f32<FMT>(c[i][j].y, f + 4);
            const float sc = j == 0 ? s[i].x : s[i].y;
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= sc;
            Row8<T>::store(out + at[i] * (j == 0 ? p.k_stride : p.v_stride) + head[i] * D + lane * 8, f);
        }
    }
}

// (token, head) pairs per lane group: one where that leaves few blocks (64 decode tokens: 3.0 us, and 6.1 with four), else
// four (24 ragged prompts: 31.8 us, with two 37.3), or two of the twice as wide f32 rows (7 x 1500: 17.0 us, with four 19.9).
static int q8_units(int64_t pairs, const rx_attn_desc* d) {
    const int64_t rows = Q8_THREADS / (d->head_dim / 8);
    const int most = d->dtype == RX_F32 ? 2 : 4;
    return pairs < rows * most * 152 * 4 ? 1 : most;
}

template <typename T, int D, int FMT, bool FIXED>
static void launch_write(const WriteQ8Params& p, int units, unsigned grid, cudaStream_t s) {
    constexpr int MOST = sizeof(T) == 4 ? 2 : 4;
    units == 1 ? launch_pdl(kv_pool_write_q8_kernel<T, D, FMT, FIXED, 1>, grid, Q8_THREADS, 0, s, p)
               : launch_pdl(kv_pool_write_q8_kernel<T, D, FMT, FIXED, MOST>, grid, Q8_THREADS, 0, s, p);
}

template <typename T, int D>
static void launch_write(const WriteQ8Params& p, const rx_q8_desc* q8, int units, unsigned grid, cudaStream_t s) {
    if (q8->format == RX_Q8_INT8)
        q8->fixed ? launch_write<T, D, RX_Q8_INT8, true>(p, units, grid, s) : launch_write<T, D, RX_Q8_INT8, false>(p, units, grid, s);
    else
        q8->fixed ? launch_write<T, D, RX_Q8_E4M3, true>(p, units, grid, s) : launch_write<T, D, RX_Q8_E4M3, false>(p, units, grid, s);
}

template <typename T, int D, int FMT>
static void launch_read(const ReadQ8Params& p, int units, unsigned grid, cudaStream_t s) {
    constexpr int MOST = sizeof(T) == 4 ? 2 : 4;
    units == 1 ? launch_pdl(kv_pool_read_q8_kernel<T, D, FMT, 1>, grid, Q8_THREADS, 0, s, p)
               : launch_pdl(kv_pool_read_q8_kernel<T, D, FMT, MOST>, grid, Q8_THREADS, 0, s, p);
}

template <typename T, int D>
static void launch_read(const ReadQ8Params& p, int format, int units, unsigned grid, cudaStream_t s) {
    format == RX_Q8_INT8 ? launch_read<T, D, RX_Q8_INT8>(p, units, grid, s) : launch_read<T, D, RX_Q8_E4M3>(p, units, grid, s);
}

static int q8_launched(const char* fn) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("%s: launch failed: %s", fn, cudaGetErrorString(e));
        return RX_ECUDA;
    }
    return RX_OK;
}

}  // namespace rx

using namespace rx;

extern "C" int kv_pool_write_q8(const rx_attn_desc* desc, const rx_q8_desc* q8, int32_t batch, const int32_t* d_prefix_slots,
                                const int64_t* d_prefix_indptr, const int32_t* d_new_slots, const int64_t* d_qo_indptr,
                                const void* d_k_new, int64_t k_stride, const void* d_v_new, int64_t v_stride, void* d_k_pool,
                                void* d_v_pool, float* d_scales, int32_t* d_req_to_token, int64_t r2t_stride, int64_t total_new,
                                int32_t* d_status, void* stream) {
    RX_TRACE("kv_pool_write_q8");
    const int rc = q8_check("kv_pool_write_q8", desc, q8, false);
    if (rc != RX_OK) return rc;
    RX_REQUIRE(batch >= 0 && total_new >= 0 && total_new <= INT32_MAX && r2t_stride >= 0, "kv_pool_write_q8: bad arguments");
    if (batch == 0 || (total_new == 0 && !d_req_to_token)) return RX_OK;
    RX_REQUIRE(d_qo_indptr && (!d_req_to_token || d_prefix_indptr), "kv_pool_write_q8: null device pointer");
    RX_REQUIRE(total_new == 0 || (d_new_slots && d_k_new && d_v_new && d_k_pool && d_v_pool && d_scales),
               "kv_pool_write_q8: null device pointer");
    const int64_t elt = desc->dtype == RX_F32 ? 4 : 2, row = (int64_t)desc->hkv * desc->head_dim;
    const struct {
        const void* p;
        int64_t stride;
    } rows[] = {{d_k_new, k_stride}, {d_v_new, v_stride}};
    for (const auto& r : rows)
        RX_REQUIRE(!r.p || (((uintptr_t)r.p & 15) == 0 && r.stride * elt % 16 == 0 && r.stride >= row),
                   "kv_pool_write_q8: rows must be 16-byte aligned and at least a row apart");
    RX_REQUIRE(((uintptr_t)d_k_pool & 15) == 0 && ((uintptr_t)d_v_pool & 15) == 0 && ((uintptr_t)d_scales & 7) == 0,
               "kv_pool_write_q8: pools must be 16-byte aligned, scales 8-byte");
    const int64_t tiles = d_req_to_token ? std::max<int64_t>(1, (r2t_stride + Q8_TILE - 1) / Q8_TILE) : 0;
    const int units = q8_units(total_new * desc->hkv, desc);
    const int64_t per = (int64_t)units * (Q8_THREADS / (desc->head_dim / 8));
    const int64_t grid = batch * tiles + (total_new * desc->hkv + per - 1) / per;
    RX_REQUIRE(grid < (1ll << 31) && tiles < (1ll << 31), "kv_pool_write_q8: batch, stride or rows too large");
    WriteQ8Params p{};
    p.batch = batch;
    p.tiles = (int32_t)tiles;
    p.prefix_slots = d_prefix_slots;
    p.prefix_indptr = d_prefix_indptr;
    p.new_slots = d_new_slots;
    p.qo_indptr = d_qo_indptr;
    p.k = d_k_new;
    p.v = d_v_new;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.k_pool = (uint8_t*)d_k_pool;
    p.v_pool = (uint8_t*)d_v_pool;
    p.scales = (float2*)d_scales;
    p.shift = q8_shift(q8);
    p.hkv = desc->hkv;
    p.step_rows = Q8_THREADS / (desc->head_dim / 8) / desc->hkv;
    p.step_heads = Q8_THREADS / (desc->head_dim / 8) % desc->hkv;
    p.r2t = d_req_to_token;
    p.r2t_stride = r2t_stride;
    p.num_slots = desc->num_slots;
    p.total = total_new;
    p.status = d_status;
    cudaStream_t s = (cudaStream_t)stream;
    if (desc->dtype == RX_F32)
        desc->head_dim == 128 ? launch_write<float, 128>(p, q8, units, (unsigned)grid, s) : launch_write<float, 64>(p, q8, units, (unsigned)grid, s);
    else
        desc->head_dim == 128 ? launch_write<__nv_bfloat16, 128>(p, q8, units, (unsigned)grid, s)
                              : launch_write<__nv_bfloat16, 64>(p, q8, units, (unsigned)grid, s);
    return q8_launched("kv_pool_write_q8");
}

extern "C" int kv_pool_read_q8(const rx_attn_desc* desc, const rx_q8_desc* q8, int64_t n, const int32_t* d_slots,
                               const void* d_k_pool, const void* d_v_pool, const float* d_scales, void* d_k_out, int64_t k_stride,
                               void* d_v_out, int64_t v_stride, int32_t* d_status, void* stream) {
    RX_TRACE("kv_pool_read_q8");
    const int rc = q8_check("kv_pool_read_q8", desc, q8, false);
    if (rc != RX_OK) return rc;
    RX_REQUIRE(n >= 0 && n <= INT32_MAX, "kv_pool_read_q8: bad count");
    if (n == 0 || (!d_k_out && !d_v_out)) return RX_OK;
    RX_REQUIRE(d_slots && d_scales && (!d_k_out || d_k_pool) && (!d_v_out || d_v_pool), "kv_pool_read_q8: null device pointer");
    const int64_t elt = desc->dtype == RX_F32 ? 4 : 2, row = (int64_t)desc->hkv * desc->head_dim;
    const struct {
        const void* p;
        int64_t stride;
    } rows[] = {{d_k_out, k_stride}, {d_v_out, v_stride}};
    for (const auto& r : rows)
        RX_REQUIRE(!r.p || (((uintptr_t)r.p & 15) == 0 && r.stride * elt % 16 == 0 && r.stride >= row),
                   "kv_pool_read_q8: rows must be 16-byte aligned and at least a row apart");
    RX_REQUIRE(((uintptr_t)d_k_pool & 15) == 0 && ((uintptr_t)d_v_pool & 15) == 0 && ((uintptr_t)d_scales & 7) == 0,
               "kv_pool_read_q8: pools must be 16-byte aligned, scales 8-byte");
    const int units = q8_units(n * desc->hkv, desc);
    const int64_t per = (int64_t)units * (Q8_THREADS / (desc->head_dim / 8));
    const int64_t grid = (n * desc->hkv + per - 1) / per;
    RX_REQUIRE(grid < (1ll << 31), "kv_pool_read_q8: too many rows");
    ReadQ8Params p{};
    p.pools = {(const uint8_t*)d_k_pool, (const uint8_t*)d_v_pool, (const float2*)d_scales, q8_shift(q8)};
    p.slots = d_slots;
    p.n = n;
    p.num_slots = desc->num_slots;
    p.hkv = desc->hkv;
    p.k_out = d_k_out;
    p.v_out = d_v_out;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.status = d_status;
    cudaStream_t s = (cudaStream_t)stream;
    if (desc->dtype == RX_F32)
        desc->head_dim == 128 ? launch_read<float, 128>(p, q8->format, units, (unsigned)grid, s)
                              : launch_read<float, 64>(p, q8->format, units, (unsigned)grid, s);
    else
        desc->head_dim == 128 ? launch_read<__nv_bfloat16, 128>(p, q8->format, units, (unsigned)grid, s)
                              : launch_read<__nv_bfloat16, 64>(p, q8->format, units, (unsigned)grid, s);
    return q8_launched("kv_pool_read_q8");
}
