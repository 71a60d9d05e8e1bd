// Attention of few rows over 8-bit pools, split over the keys: decode, and prompts of few new tokens.
//
// The rows are (token, query head) pairs of one request and kv head, the head fastest, in tiles of 8 NT; decode is a
// request's one token at position L - 1.  With codes kc, vc and scales ks, vs of a key j,
//   x_j = c ks_j (q . kc_j),  y_j = x_j + log2 vs_j     (c = scale log2 e)
//   o = sum_j 2^y_j vc_j / sum_j 2^x_j,
// each sum over its own running maximum: vs enters the exponent, so that what is weighed and rounded to 16 bits is 2^(y_j - max y)
// next to the largest term of o, however far apart the rows' scales are.
//
// One CTA per (request, chunk of keys, row tile, kv head); 16-byte cp.async gathers of 64-key stages of codes, 3 deep,
// and of their scales.  Each warp takes 16 keys of a stage: S^T = K Q^T with the keys in M of m16n8k16, then
// O^T += V^T P^T.  Codes become f16 in registers, where they are exact (int8 and e4m3 both): K fragments by ldmatrix over 16-byte
// rows, four neighbouring channels a lane, which the query fragments follow; V by ldmatrix.trans over byte
// pairs, whose two channels are parted by the byte permutation that widens them.  Queries are f16 after a
// power of two per row that brings the row's largest to 2^14 (bf16 is exact in that down to 2^-29 of the largest); f32 rows
// and f32 rows' weights are two f16 parts each, 22 bits.
// Bound by HBM: 2 d + 8 bytes a key and kv head, read once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "kv_q8.cuh"
#include "radix_attn.h"
#include "rx_common.h"
#include "rx_device.cuh"
#include "rx_launch.h"
#include "rx_q8.h"

namespace rx {

constexpr int RQ_THREADS = 128;
constexpr int RQ_STAGE = 64;          // keys per stage, 16 a warp
constexpr int RQ_NS = 3;              // stages
constexpr int RQ_CHUNK = 1024;        // most keys per CTA (their slots are staged in shared memory)
constexpr float RQ_LOG2E = 1.4426950408889634f, RQ_LN2 = 0.6931471805599453f;
constexpr float RQ_TOP = 15.f;        // a row's largest weight is 2^15 in f16

template <int D>
struct RowsLayout {
    static constexpr int CODES = RQ_STAGE * D;                         // one pool's codes of a stage
    static constexpr int STAGE = 2 * CODES + RQ_STAGE * 8;             // K, V, scales
    static constexpr int SLOTS = RQ_NS * STAGE;
    static constexpr int BYTES = SLOTS + RQ_CHUNK * 4;
    static constexpr int RS = D + 4;                                   // floats between merged rows
};

// 16-byte chunk c of key row `key`: rows of 128 bytes, or two of 64 to a line, so that 8 rows' chunks lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t code_at(int key, int c) {
    return D == 128 ? (uint32_t)(key * 128 + ((c ^ (key & 7)) << 4)) : (uint32_t)(key * 64 + ((c ^ ((key >> 1) & 3)) << 4));
}

__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

// D(16x8 fp32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// What is left of a pair after its f16 part.
__device__ __forceinline__ uint32_t pack_rest_f16x2(float lo, float hi, uint32_t part) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&part));
    return pack_f16x2(lo - p.x, hi - p.y);
}

__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// cells of the grid, kv head fastest, so that neighbouring CTAs share the lines of scales
struct RowsParams {
    const void* q;
    const int64_t* qo_indptr;         // extend only
    const int32_t* prefix_lens;       // extend only
    const int32_t* kv_lens;           // decode only
    const int32_t* r2t;
    int64_t stride, num_slots;
    Q8Pools pools;
    int32_t batch, hq, hkv, group;
    int32_t max_qo_len, max_kv_len;
    int32_t tiles, chunks, chunk;     // row tiles, splits of the keys, keys of a split (a multiple of RQ_STAGE)
    float scale_log2;
    void* out;
    float* lse;
    float* part_o;                    // [batch * max_qo_len * hq][chunks][D], where chunks > 1
    float* part_lse;
    int32_t* status;
};

// A request's rows: where its first is, how many tokens, and how many keys lie before them; false where there is none to do.
__device__ __forceinline__ bool rows_of(const RowsParams& p, int b, bool tell, int64_t& q0, int& n, int& before) {
    if (p.kv_lens) {
        const int32_t L = p.kv_lens[b];
        q0 = b, n = 1, before = L - 1;
        if (L >= 0 && L <= p.max_kv_len && L <= p.stride) return true;
    } else {
        q0 = p.qo_indptr[b];
        const int64_t m = p.qo_indptr[b + 1] - q0, P = p.prefix_lens[b];
        if (m == 0) return false;
        n = (int)m, before = (int)P;
        if (q0 >= 0 && m > 0 && m <= p.max_qo_len && P >= 0 && P + m <= p.stride && P + m <= p.max_kv_len) return true;
    }
    if (tell) report(p.status, RX_DEV_BAD_LENGTH);
    return false;
}

template <typename T>
__device__ __forceinline__ void store_row2(T* p, float a, float b);
template <>
__device__ __forceinline__ void store_row2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
template <>
__device__ __forceinline__ void store_row2(__nv_bfloat16* p, float a, float b) { *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(a, b); }

template <typename T, int D, int FMT, int NT>
__global__ void __launch_bounds__(RQ_THREADS) rows_q8_kernel(const __grid_constant__ RowsParams p) {
    using LY = RowsLayout<D>;
    constexpr bool TWO = std::is_same<T, float>::value;     // two f16 parts
    constexpr int KS = D / 16;                              // 16-byte chunks of a row: steps of K, and of V's M
    constexpr int CPT = RQ_STAGE * KS / RQ_THREADS;         // copies per thread, stage and pool
    extern __shared__ __align__(1024) unsigned char smem[];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, t4 = lane & 3, r8 = lane >> 2;
    int cell = blockIdx.x;
    const int g = cell % p.hkv;
    cell /= p.hkv;
    const int tile = cell % p.tiles;
    cell /= p.tiles;
    const int c = cell % p.chunks, b = cell / p.chunks;
    int64_t q0;
    int n, before;
    if (!rows_of(p, b, tid == 0 && g == 0 && tile == 0 && c == 0, q0, n, before)) return;
    const int G = p.group, rows = n * G, R0 = tile * 8 * NT;
    if (R0 >= rows) return;
    const int last = min(R0 + 8 * NT, rows) - 1;
    const int k_begin = c * p.chunk;
    const int nk = min(before + last / G + 1 - k_begin, p.chunk);      // keys of this CTA
    if (nk <= 0 && c > 0) return;                                      // chunk 0 writes the row of no keys
    int32_t* slot_s = reinterpret_cast<int32_t*>(smem + LY::SLOTS);
    const int nstages = max(nk + RQ_STAGE - 1, 0) / RQ_STAGE;
    bool bad = false;
    {
        const int32_t* row = p.r2t + (int64_t)b * p.stride + k_begin;
        for (int i = tid; i < nstages * RQ_STAGE; i += RQ_THREADS) {
            int32_t s = i < nk ? row[i] : -1;
            if (i < nk && (s < 0 || s >= p.num_slots)) {
                report(p.status, RX_DEV_BAD_SLOT);
                s = -1;
                bad = true;
            }
            slot_s[i] = s;
        }
    }
    // query fragments: columns of the B operand, row R0 + 8 t + r8, channels 16 s + 4 t4 ..+3; and each accumulator
    // column's factor, scale log2(e) over the row's power of two
    uint32_t qb[NT][TWO ? 2 : 1][KS][2];
    float f[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int R = R0 + 8 * t + r8;
        const bool in = R < rows;
        const T* qr = (const T*)p.q + (in ? ((q0 + R / G) * p.hq + g * G + R % G) * D : 0);
        float x[KS][4];
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if (TWO) {
                const float4 v = in ? *reinterpret_cast<const float4*>((const float*)qr + 16 * s + 4 * t4) : make_float4(0, 0, 0, 0);
                x[s][0] = v.x, x[s][1] = v.y, x[s][2] = v.z, x[s][3] = v.w;
            } else {
                const uint2 v = in ? *reinterpret_cast<const uint2*>((const __nv_bfloat16*)qr + 16 * s + 4 * t4) : make_uint2(0, 0);
                x[s][0] = __uint_as_float(v.x << 16), x[s][1] = __uint_as_float(v.x & 0xffff0000u);
                x[s][2] = __uint_as_float(v.y << 16), x[s][3] = __uint_as_float(v.y & 0xffff0000u);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(x[s][e]) & 0x7fffffffu);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the power of two that brings the largest to [2^14, 2^15), at most 2^126; none for a row that is not finite
        const uint32_t up = top >= 0x7f800000u ? 127u : (uint32_t)min(268 - max((int)(top >> 23), 1), 253);
        const float mul = __uint_as_float(up << 23), undo = __uint_as_float((254u - up) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float a0 = x[s][2 * h] * mul, a1 = x[s][2 * h + 1] * mul;
                qb[t][0][s][h] = pack_f16x2(a0, a1);
                if (TWO) qb[t][TWO ? 1 : 0][s][h] = pack_rest_f16x2(a0, a1, qb[t][0][s][h]);
            }
        const float mine = p.scale_log2 * undo;            // of row r8; the accumulators' columns are rows 2 t4, 2 t4 + 1
        f[t][0] = __shfl_sync(0xffffffffu, mine, 8 * t4);
        f[t][1] = __shfl_sync(0xffffffffu, mine, 8 * t4 + 4);
    }
    const bool any_bad = __syncthreads_or(bad);
    // the first key that each of this lane's columns may not see, relative to the chunk
    int end[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) end[t][e] = min(before + (R0 + 8 * t + 2 * t4 + e) / G + 1 - k_begin, nk);
    const int least = min(before + R0 / G + 1 - k_begin, nk);           // every row sees the keys before this

    const uint32_t sbase = smem_u32(smem);
    const int64_t pitch = (int64_t)p.hkv * D;
    const uint8_t* kcol = p.pools.k + (int64_t)g * D + (tid % KS) * 16;
    const uint8_t* vcol = p.pools.v + (int64_t)g * D + (tid % KS) * 16;
    auto load_stage = [&](int st) {
        const uint32_t kb = sbase + (uint32_t)((st % RQ_NS) * LY::STAGE), vb = kb + LY::CODES;
#pragma unroll
        for (int x = 0; x < CPT; ++x) {
            const int key = tid / KS + x * (RQ_THREADS / KS);
            const int32_t s = slot_s[st * RQ_STAGE + key];
            const int64_t off = (int64_t)max(s, 0) * pitch;
            const uint32_t so = code_at<D>(key, tid % KS), bytes = s >= 0 ? 16u : 0u;
            cp_async_16(kb + so, kcol + off, bytes);
            cp_async_16(vb + so, vcol + off, bytes);
        }
        if (tid < RQ_STAGE) {
            const int32_t s = slot_s[st * RQ_STAGE + tid];
            cp_async_8(vb + LY::CODES + tid * 8, p.pools.scales + (int64_t)(max(s, 0) >> p.pools.shift) * p.hkv + g, s >= 0 ? 8u : 0u);
        }
    };
    float o[NT][KS][4];
    float mx[NT][2], l[NT][2], my[NT][2];      // of x in this lane, the sum, and of y in the warp
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < KS; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
        mx[t][0] = mx[t][1] = my[t][0] = my[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.f;
    }
#pragma unroll
    for (int s = 0; s < RQ_NS - 1; ++s) {
        if (s < nstages) load_stage(s);
        cp_async_commit();
    }
    for (int it = 0; it < nstages; ++it) {
        cp_async_wait<RQ_NS - 2>();
        __syncthreads();                       // stage it is here, and every warp is done with stage it - 1
        if (it + RQ_NS - 1 < nstages) load_stage(it + RQ_NS - 1);
        cp_async_commit();
        const int key0 = it * RQ_STAGE + warp * 16;
        if (key0 >= nk) continue;
        const uint32_t kb = sbase + (uint32_t)((it % RQ_NS) * LY::STAGE), vb = kb + LY::CODES;
        const int mi = lane >> 3, lrow = warp * 16 + (mi & 1) * 8 + (lane & 7);
        float sacc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) sacc[t][0] = sacc[t][1] = sacc[t][2] = sacc[t][3] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; s += 2) {
            uint32_t w[4];                     // keys r8, r8 + 8 of chunk s, then of chunk s + 1
            ldmatrix_x4(kb + code_at<D>(lrow, s + (mi >> 1)), w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t a[4];
                q8_to_f16<FMT, false>(w[2 * j], a[0], a[2]);
                q8_to_f16<FMT, false>(w[2 * j + 1], a[1], a[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int u = 0; u < (TWO ? 2 : 1); ++u) mma_f16_16816(sacc[t], a, qb[t][u][s + j][0], qb[t][u][s + j][1]);
            }
        }
        const float2* sc = reinterpret_cast<const float2*>(smem + (it % RQ_NS) * LY::STAGE + 2 * LY::CODES) + warp * 16;
        const float2 sa = sc[r8], sb = sc[r8 + 8];
        const float la = fast_log2(sa.y), lb = fast_log2(sb.y);
        const bool whole = key0 + 16 <= least && !any_bad;     // no key of these is hidden from any row
        const bool oka = !any_bad || slot_s[key0 + r8] >= 0, okb = !any_bad || slot_s[key0 + r8 + 8] >= 0;
        uint32_t pb[NT][TWO ? 2 : 1][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float x[4] = {sacc[t][0] * (f[t][0] * sa.x), sacc[t][1] * (f[t][1] * sa.x), sacc[t][2] * (f[t][0] * sb.x),
                          sacc[t][3] * (f[t][1] * sb.x)};
            float y[4] = {x[0] + la, x[1] + la, x[2] + lb, x[3] + lb};
            if (!whole) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (key0 + r8 + (e >> 1) * 8 >= end[t][e & 1] || !(e < 2 ? oka : okb)) x[e] = y[e] = -INFINITY;
            }
            float w[4];
            bool moved = false;
            float up[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float a = fmaxf(mx[t][e], fmaxf(x[e], x[e + 2])), ra = a == -INFINITY ? 0.f : a;
                l[t][e] = l[t][e] * fast_exp2(mx[t][e] - ra) + fast_exp2(x[e] - ra) + fast_exp2(x[e + 2] - ra);
                mx[t][e] = a;
                float m = fmaxf(y[e], y[e + 2]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                m = fmaxf(m, my[t][e]);
                const float rm = m == -INFINITY ? 0.f : m;
                up[e] = fast_exp2(my[t][e] - rm);
                moved |= m != my[t][e];
                my[t][e] = m;
                w[e] = fast_exp2(y[e] - (rm - RQ_TOP));
                w[e + 2] = fast_exp2(y[e + 2] - (rm - RQ_TOP));
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    o[t][i][0] *= up[0];
                    o[t][i][1] *= up[1];
                    o[t][i][2] *= up[0];
                    o[t][i][3] *= up[1];
                }
            }
            const uint32_t h0 = pack_f16x2(w[0], w[1]), h1 = pack_f16x2(w[2], w[3]);
            pb[t][0][0] = movmatrix_trans(h0);
            pb[t][0][1] = movmatrix_trans(h1);
            if (TWO) {
                pb[t][TWO ? 1 : 0][0] = movmatrix_trans(pack_rest_f16x2(w[0], w[1], h0));
                pb[t][TWO ? 1 : 0][1] = movmatrix_trans(pack_rest_f16x2(w[2], w[3], h1));
            }
        }
#pragma unroll
        for (int i = 0; i < KS; i += 2) {
            uint32_t w[4];                     // byte pairs of channels 2 r8, 2 r8 + 1: keys 2 t4, 2 t4 + 1, then those + 8; two chunks
            ldmatrix_x4_trans(vb + code_at<D>(lrow, i + (mi >> 1)), w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t a[4];                 // rows r8: channel 2 r8, rows r8 + 8: channel 2 r8 + 1
                q8_to_f16<FMT, true>(w[2 * j], a[0], a[1]);
                q8_to_f16<FMT, true>(w[2 * j + 1], a[2], a[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int u = 0; u < (TWO ? 2 : 1); ++u) mma_f16_16816(o[t][i + j], a, pb[t][u][0], pb[t][u][1]);
            }
        }
    }
    cp_async_wait<0>();

    // One row's parts of the four warps: O relative to 2^(my - 15), l relative to 2^mx.
    constexpr int RS = LY::RS;
    float* red_o = reinterpret_cast<float*>(smem);             // [4 warps][8 rows][RS]
    float* red_m = red_o + 4 * 8 * RS;                         // [4][8]: mx, then l, then my
    float* red_w = red_m + 3 * 32;                             // [4][8] weights
    float* red_lse = red_w + 32;                               // [8]
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (R0 + 8 * t >= rows) break;                         // the same for the block
        __syncthreads();                                       // the ring, or the tile before, is done with
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float m = mx[t][e];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            float s = l[t][e] * fast_exp2(mx[t][e] - (m == -INFINITY ? 0.f : m));
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            if (r8 == 0) {
                red_m[warp * 8 + 2 * t4 + e] = m;
                red_m[32 + warp * 8 + 2 * t4 + e] = s;
                red_m[64 + warp * 8 + 2 * t4 + e] = my[t][e];
            }
#pragma unroll
            for (int i = 0; i < KS; ++i)
                *reinterpret_cast<float2*>(red_o + (warp * 8 + 2 * t4 + e) * RS + 16 * i + 2 * r8) =
                    make_float2(o[t][i][e], o[t][i][e + 2]);
        }
        __syncthreads();
        if (tid < 8) {
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) M = fmaxf(M, red_m[w * 8 + tid]);
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < 4; ++w) L += red_m[32 + w * 8 + tid] * exp2f(red_m[w * 8 + tid] - ref);
            const float inv = L == 0.f ? 0.f : 1.f / L;        // no key: zeros
#pragma unroll
            for (int w = 0; w < 4; ++w) red_w[w * 8 + tid] = exp2f(red_m[64 + w * 8 + tid] - RQ_TOP - ref) * inv;
            red_lse[tid] = L == 0.f ? -INFINITY : M + log2f(L);
        }
        __syncthreads();
        constexpr int HALF = D / 2;
        const int nr = min(8, rows - R0 - 8 * t);
        for (int idx = tid; idx < nr * HALF; idx += RQ_THREADS) {
            const int r = idx / HALF, d = 2 * (idx % HALF), R = R0 + 8 * t + r, tok = R / G, h = g * G + R % G;
            float a0 = 0.f, a1 = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float wt = red_w[w * 8 + r];
                const float2 v = *reinterpret_cast<const float2*>(red_o + (w * 8 + r) * RS + d);
                a0 += wt * v.x;
                a1 += wt * v.y;
            }
            if (p.chunks == 1) {
                const int64_t at = (q0 + tok) * p.hq + h;
                store_row2((T*)p.out + at * D + d, a0, a1);
                if (d == 0 && p.lse) p.lse[at] = red_lse[r] * RQ_LN2;
            } else {
                const int64_t at = (((int64_t)b * p.max_qo_len + tok) * p.hq + h) * p.chunks + c;
                *reinterpret_cast<float2*>(p.part_o + at * D + d) = make_float2(a0, a1);
                if (d == 0) p.part_lse[at] = red_lse[r];
            }
        }
    }
}

// The chunks' parts of a row: one warp a (token, query head).
template <typename T, int D>
__global__ void __launch_bounds__(128) rows_q8_merge_kernel(const __grid_constant__ RowsParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t per = (int64_t)p.max_qo_len * p.hq;
    const int b = (int)(item / per);
    if (b >= p.batch) return;
    const int rest = (int)(item - b * per), tok = rest / p.hq, h = rest - tok * p.hq;
    int64_t q0;
    int n, before;
    if (!rows_of(p, b, false, q0, n, before) || tok >= n) return;
    // the chunks that the tile of this row went through (a chunk behind the row's own keys, of a tile with later rows, has no weight)
    const int parts = max((before + tok + 1 + p.chunk - 1) / p.chunk, 1);
    const float* pl = p.part_lse + item * p.chunks;
    const float* po = p.part_o + item * p.chunks * D;
    float M = -INFINITY;
    for (int s = lane; s < parts; s += 32) M = fmaxf(M, pl[s]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    const float ref = M == -INFINITY ? 0.f : M;
    constexpr int E = D / 32;
    float acc[E], W = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
        const float w = exp2f(pl[s] - ref);
        W += w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += w * po[(int64_t)s * D + lane * E + e];
    }
    const float inv = W == 0.f ? 0.f : 1.f / W;
    const int64_t at = (q0 + tok) * p.hq + h;
    T* row = (T*)p.out + at * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) store_row2(row + e, acc[e] * inv, acc[e + 1] * inv);
    if (p.lse && lane == 0) p.lse[at] = W == 0.f ? -INFINITY : (M + log2f(W)) * RQ_LN2;
}

template <typename T, int D, int FMT, int NT>
static int launch_tile(const char* fn, const RowsParams& p, unsigned grid, cudaStream_t s) {
    constexpr int smem = RowsLayout<D>::BYTES;
    static PerDeviceOnce attr;
    const int rc = per_device_once(attr, [&] {
        auto* k = rows_q8_kernel<T, D, FMT, NT>;
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) (void)cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) {
            set_error("%s: cannot set shared memory size: %s", fn, cudaGetErrorString(e));
            return (int)RX_ECUDA;
        }
        return (int)RX_OK;
    });
    if (rc != RX_OK) return rc;
    launch_pdl(rows_q8_kernel<T, D, FMT, NT>, grid, RQ_THREADS, smem, s, p);
    if (p.chunks > 1) {
        const int64_t items = (int64_t)p.batch * p.max_qo_len * p.hq;
        launch_pdl(rows_q8_merge_kernel<T, D>, (unsigned)((items + 3) / 4), 128, 0, s, p);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("%s: launch failed: %s", fn, cudaGetErrorString(e));
        return RX_ECUDA;
    }
    return RX_OK;
}

template <typename T, int D, int FMT>
static int launch_fmt(const char* fn, const RowsParams& p, int nt, unsigned grid, cudaStream_t s) {
    if (nt == 1) return launch_tile<T, D, FMT, 1>(fn, p, grid, s);
    if constexpr (std::is_same<T, float>::value) return launch_tile<T, D, FMT, 2>(fn, p, grid, s);
    else return nt == 2 ? launch_tile<T, D, FMT, 2>(fn, p, grid, s) : launch_tile<T, D, FMT, 4>(fn, p, grid, s);
}

template <typename T, int D>
static int launch_rows(const char* fn, const RowsParams& p, int nt, int format, unsigned grid, cudaStream_t s) {
    return format == RX_Q8_INT8 ? launch_fmt<T, D, RX_Q8_INT8>(fn, p, nt, grid, s) : launch_fmt<T, D, RX_Q8_E4M3>(fn, p, nt, grid, s);
}

// 8-row tiles that a CTA takes: as many as the rows fill, up to four (f32 rows, with two parts each, two: registers).
static int rows_nt(int64_t rows, int dtype) { return rows <= 8 ? 1 : rows <= 16 || dtype == RX_F32 ? 2 : 4; }

RowsPlan rows_q8_plan(const rx_attn_desc* d, int32_t batch, int32_t max_qo_len, int32_t max_kv_len) {
    RowsPlan L{};
    const int64_t rows = (int64_t)max_qo_len * (d->hq / d->hkv);
    L.nt = rows_nt(rows, d->dtype);
    L.tiles = (rows + 8 * L.nt - 1) / (8 * L.nt);
    // Long chunks amortise a CTA's start and end over more keys; short ones keep enough CTAs to fill 152 SMs.
    const int64_t units = L.tiles * d->hkv * batch;
    auto chunks = [&](int c) { return std::max<int64_t>(((int64_t)max_kv_len + c - 1) / c, 1); };
    L.chunk = RQ_CHUNK;
    while (L.chunk > 256 && units * chunks(L.chunk) < 152 * 8) L.chunk /= 2;
    if (max_kv_len <= 512 && units >= 152) L.chunk = 512;
    L.chunks = chunks(L.chunk);
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    if (L.chunks > 1) {
        const size_t parts = (size_t)batch * max_qo_len * d->hq * L.chunks;
        L.o_bytes = up(parts * d->head_dim * sizeof(float));
        L.bytes = L.o_bytes + up(parts * sizeof(float));
    }
    return L;
}

int rows_q8_launch(const char* fn, const RowsQ8Args& a, const rx_attn_desc* d, const rx_q8_desc* q8, void* ws, size_t ws_bytes,
                   cudaStream_t stream) {
    const RowsPlan L = rows_q8_plan(d, a.batch, a.max_qo_len, a.max_kv_len);
    const int64_t grid = (int64_t)a.batch * L.chunks * L.tiles * d->hkv, items = (int64_t)a.batch * a.max_qo_len * d->hq;
    RX_REQUIRE(grid < (1ll << 31) && (items + 3) / 4 < (1ll << 31), "%s: too many rows or chunks (split the batch)", fn);
    RX_REQUIRE(L.bytes == 0 || (ws && ws_bytes >= L.bytes && ((uintptr_t)ws & 255) == 0),
               "%s: a 256-byte aligned workspace of %zu bytes is needed (got %zu)", fn, L.bytes, ws_bytes);
    RowsParams p{};
    p.q = a.q;
    p.qo_indptr = a.qo_indptr;
    p.prefix_lens = a.prefix_lens;
    p.kv_lens = a.kv_lens;
    p.r2t = a.r2t;
    p.stride = a.stride;
    p.num_slots = d->num_slots;
    p.pools = {a.k_pool, a.v_pool, a.scales, q8_shift(q8)};
    p.batch = a.batch;
    p.hq = d->hq;
    p.hkv = d->hkv;
    p.group = d->hq / d->hkv;
    p.max_qo_len = a.max_qo_len;
    p.max_kv_len = a.max_kv_len;
    p.tiles = (int32_t)L.tiles;
    p.chunks = (int32_t)L.chunks;
    p.chunk = L.chunk;
    p.scale_log2 = d->scale * RQ_LOG2E;
    p.out = a.out;
    p.lse = a.lse;
    p.part_o = (float*)ws;
    p.part_lse = (float*)((unsigned char*)ws + L.o_bytes);
    p.status = a.status;
    if (d->dtype == RX_F32)
        return d->head_dim == 128 ? launch_rows<float, 128>(fn, p, L.nt, q8->format, (unsigned)grid, stream)
                                  : launch_rows<float, 64>(fn, p, L.nt, q8->format, (unsigned)grid, stream);
    return d->head_dim == 128 ? launch_rows<__nv_bfloat16, 128>(fn, p, L.nt, q8->format, (unsigned)grid, stream)
                              : launch_rows<__nv_bfloat16, 64>(fn, p, L.nt, q8->format, (unsigned)grid, stream);
}

}  // namespace rx
