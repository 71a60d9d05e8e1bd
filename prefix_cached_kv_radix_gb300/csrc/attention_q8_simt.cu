// Attention over 8-bit pools on CUDA cores, one warp per (row, query head): the plain kernel.
//
// o = sum_j 2^(x_j - m) vs_j vc_j / sum_j 2^(x_j - m), x_j = scale log2(e) ks_j (q . kc_j), with codes kc, vc
// and scales ks, vs; lanes split the head dimension.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_q8.cuh"
#include "radix_attn.h"
#include "rx_common.h"
#include "rx_device.cuh"
#include "rx_kernels.h"
#include "rx_launch.h"

namespace rx {

// p's own pools are not used.
struct Q8SimtParams {
    SimtParams p;
    Q8Pools pools;
    int32_t max_kv_len;           // extend: host bound of a request's keys
};

template <int FMT, int E>
__device__ __forceinline__ void load_codes(const uint8_t* p, float* f) {
    float t[4];
    q8_to_f32<FMT>(E == 4 ? *reinterpret_cast<const uint32_t*>(p) : (uint32_t)*reinterpret_cast<const uint16_t*>(p), t);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = t[e];
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(128) attn_q8_simt_kernel(const __grid_constant__ Q8SimtParams a) {
    constexpr int E = D / 32, KG = 8;
    constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
    const SimtParams& p = a.p;
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 4 + warp;
    if (item >= p.total_rows * p.hq) return;
    int64_t row = item / p.hq;
    const int h = (int)(item - row * p.hq), g = h / (p.hq / p.hkv);
    int b;
    int64_t nkeys;
    if (p.kv_lens) {
        b = (int)row;
        const int32_t L = p.kv_lens[b];
        if (L < 0 || L > p.max_len || L > p.stride) {
            if (lane == 0 && h == 0) report(p.status, RX_DEV_BAD_LENGTH);
            return;
        }
        nkeys = L;
    } else {
        b = (int)(row / p.max_len);
        const int64_t i = row - (int64_t)b * p.max_len, q0 = p.qo_indptr[b], n = p.qo_indptr[b + 1] - q0, P = p.prefix_lens[b];
        if (n == 0) return;
        if (q0 < 0 || n < 0 || n > p.max_len || P < 0 || P + n > p.stride || P + n > a.max_kv_len) {
            if (lane == 0 && h == 0 && i == 0) report(p.status, RX_DEV_BAD_LENGTH);
            return;
        }
        if (i >= n) return;
        row = q0 + i;
        nkeys = P + i + 1;
    }
    const T* qr = (const T*)p.q + (row * p.hq + h) * D + lane * E;
    float qv[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qv[e] = (float)qr[e];
        acc[e] = 0.f;
    }
    const int32_t* slots = p.r2t + (int64_t)b * p.stride;
    float m = -INFINITY, l = 0.f;
    for (int64_t j0 = 0; j0 < nkeys; j0 += 32) {
        const int cnt = (int)(nkeys - j0 < 32 ? nkeys - j0 : 32);
        int32_t s_lane = lane < cnt ? slots[j0 + lane] : -1;
        if (s_lane < 0 || s_lane >= p.num_slots) {
            if (lane < cnt) report(p.status, RX_DEV_BAD_SLOT);
            s_lane = -1;
        }
        const float2 sc_lane = s_lane >= 0 ? q8_scales(a.pools, s_lane, p.hkv, g) : make_float2(0.f, 0.f);
        for (int k0 = 0; k0 < cnt; k0 += KG) {
            float kv[KG][E], vv[KG][E];
            int32_t sl[KG];
#pragma unroll
            for (int u = 0; u < KG; ++u) {
                sl[u] = __shfl_sync(0xffffffffu, s_lane, (k0 + u) & 31);     // -1 past the row's last key
                const int64_t base = ((int64_t)max(sl[u], 0) * p.hkv + g) * D + lane * E;
                load_codes<FMT, E>(a.pools.k + base, kv[u]);
                load_codes<FMT, E>(a.pools.v + base, vv[u]);
            }
#pragma unroll
            for (int u = 0; u < KG; ++u) {
                const float ks = __shfl_sync(0xffffffffu, sc_lane.x, (k0 + u) & 31);
                const float vs = __shfl_sync(0xffffffffu, sc_lane.y, (k0 + u) & 31);
                if (sl[u] < 0) continue;
                float dot = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) dot += qv[e] * kv[u][e];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                const float x = dot * (p.scale * LOG2E) * ks;
                const float mn = fmaxf(m, x), ref = mn == -INFINITY ? 0.f : mn;
                const float corr = exp2f(m - ref), w = exp2f(x - ref);
                l = l * corr + w;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = acc[e] * corr + w * vs * vv[u][e];
                m = mn;
            }
        }
    }
    T* orow = (T*)p.out + (row * p.hq + h) * D + lane * E;
    const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) orow[e] = (T)(acc[e] * inv);
    if (p.lse && lane == 0) p.lse[row * p.hq + h] = l != 0.f ? (m + log2f(l)) * LN2 : -INFINITY;
}

template <typename T, int D>
static void launch_fmt(const Q8SimtParams& a, int format, unsigned blocks, cudaStream_t s) {
    format == RX_Q8_INT8 ? launch_pdl(attn_q8_simt_kernel<T, D, RX_Q8_INT8>, blocks, 128, 0, s, a)
                         : launch_pdl(attn_q8_simt_kernel<T, D, RX_Q8_E4M3>, blocks, 128, 0, s, a);
}

static int launch_q8_simt(const char* fn, const Q8SimtParams& a, const rx_attn_desc* d, int format, cudaStream_t s) {
    const int64_t blocks = (a.p.total_rows * a.p.hq + 3) / 4;
    RX_REQUIRE(blocks < (1ll << 31), "%s: too many rows", fn);
    if (d->dtype == RX_F32)
        d->head_dim == 128 ? launch_fmt<float, 128>(a, format, (unsigned)blocks, s) : launch_fmt<float, 64>(a, format, (unsigned)blocks, s);
    else
        d->head_dim == 128 ? launch_fmt<__nv_bfloat16, 128>(a, format, (unsigned)blocks, s)
                           : launch_fmt<__nv_bfloat16, 64>(a, format, (unsigned)blocks, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("%s: launch failed: %s", fn, cudaGetErrorString(e));
        return RX_ECUDA;
    }
    return RX_OK;
}

}  // namespace rx

using namespace rx;

static int q8_attention_args(const char* fn, const rx_attn_desc* desc, const rx_q8_desc* q8, const void* d_q, const void* d_k_pool,
                             const void* d_v_pool, const void* d_scales, const void* d_out) {
    RX_REQUIRE(d_q && d_k_pool && d_v_pool && d_scales && d_out, "%s: null device pointer", fn);
    for (const void* x : {d_q, d_k_pool, d_v_pool, d_out}) RX_REQUIRE(((uintptr_t)x & 15) == 0, "%s: rows and pools must be 16-byte aligned", fn);
    RX_REQUIRE(((uintptr_t)d_scales & 7) == 0, "%s: scales must be 8-byte aligned", fn);
    return RX_OK;
}

extern "C" size_t decode_q8_workspace_bytes(const rx_attn_desc*, int32_t, int32_t, const rx_shared_groups*) { return 0; }

extern "C" size_t extend_q8_workspace_bytes(const rx_attn_desc*, int32_t, int32_t, int32_t) { return 0; }

extern "C" int decode_attention_q8(const rx_attn_desc* desc, const rx_q8_desc* q8, int32_t batch, const void* d_q,
                                   const int32_t* d_req_to_token, int64_t r2t_stride, const int32_t* d_kv_lens,
                                   const rx_shared_groups* groups, const void* d_k_pool, const void* d_v_pool, const float* d_scales,
                                   void* d_out, float* d_lse, int32_t max_kv_len, void* d_workspace, size_t ws_bytes,
                                   int32_t* d_status, void* stream) {
    RX_TRACE("decode_attention_q8");
    int rc = q8_check("decode_attention_q8", desc, q8, true);
    if (rc != RX_OK) return rc;
    RX_REQUIRE(batch >= 0 && max_kv_len >= 0 && r2t_stride >= 0, "decode_attention_q8: bad arguments");
    if (batch == 0) return RX_OK;
    rc = q8_attention_args("decode_attention_q8", desc, q8, d_q, d_k_pool, d_v_pool, d_scales, d_out);
    if (rc != RX_OK) return rc;
    RX_REQUIRE(d_req_to_token && d_kv_lens, "decode_attention_q8: null device pointer");
    Q8SimtParams a{};
    a.pools = {(const uint8_t*)d_k_pool, (const uint8_t*)d_v_pool, (const float2*)d_scales, q8_shift(q8)};
    SimtParams& p = a.p;
    p.batch = batch;
    p.hq = desc->hq;
    p.hkv = desc->hkv;
    p.total_rows = batch;
    p.q = d_q;
    p.kv_lens = d_kv_lens;
    p.r2t = d_req_to_token;
    p.stride = r2t_stride;
    p.num_slots = desc->num_slots;
    p.out = d_out;
    p.lse = d_lse;
    p.scale = desc->scale;
    p.max_len = max_kv_len;
    p.status = d_status;
    return launch_q8_simt("decode_attention_q8", a, desc, q8->format, (cudaStream_t)stream);
}

extern "C" int prefix_extend_attention_q8(const rx_attn_desc* desc, const rx_q8_desc* q8, int32_t batch, const void* d_q,
                                          const int64_t* d_qo_indptr, const int32_t* d_prefix_lens, const int32_t* d_req_to_token,
                                          int64_t r2t_stride, const void* d_k_pool, const void* d_v_pool, const float* d_scales,
                                          void* d_out, float* d_lse, int32_t max_qo_len, int32_t max_kv_len, void* d_workspace,
                                          size_t ws_bytes, int32_t* d_status, void* stream) {
    RX_TRACE("prefix_extend_attention_q8");
    int rc = q8_check("prefix_extend_attention_q8", desc, q8, true);
    if (rc != RX_OK) return rc;
    RX_REQUIRE(batch >= 0 && max_qo_len >= 0 && max_kv_len >= 0 && r2t_stride >= 0, "prefix_extend_attention_q8: bad arguments");
    if (batch == 0 || max_qo_len == 0) return RX_OK;
    rc = q8_attention_args("prefix_extend_attention_q8", desc, q8, d_q, d_k_pool, d_v_pool, d_scales, d_out);
    if (rc != RX_OK) return rc;
    RX_REQUIRE(d_qo_indptr && d_prefix_lens && d_req_to_token, "prefix_extend_attention_q8: null device pointer");
    Q8SimtParams a{};
    a.pools = {(const uint8_t*)d_k_pool, (const uint8_t*)d_v_pool, (const float2*)d_scales, q8_shift(q8)};
    a.max_kv_len = max_kv_len;
    SimtParams& p = a.p;
    p.batch = batch;
    p.hq = desc->hq;
    p.hkv = desc->hkv;
    p.total_rows = (int64_t)batch * max_qo_len;
    p.q = d_q;
    p.qo_indptr = d_qo_indptr;
    p.prefix_lens = d_prefix_lens;
    p.r2t = d_req_to_token;
    p.stride = r2t_stride;
    p.num_slots = desc->num_slots;
    p.out = d_out;
    p.lse = d_lse;
    p.scale = desc->scale;
    p.max_len = max_qo_len;
    p.status = d_status;
    return launch_q8_simt("prefix_extend_attention_q8", a, desc, q8->format, (cudaStream_t)stream);
}
