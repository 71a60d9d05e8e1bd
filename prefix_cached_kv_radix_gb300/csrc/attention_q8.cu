// The entry points of attention over 8-bit pools: argument checks, and which kernel takes a call.
#include <algorithm>
#include <cmath>

#include "kv_q8.cuh"
#include "radix_attn.h"
#include "rx_common.h"
#include "rx_q8.h"

using namespace rx;

static int attention_q8_check(const char* fn, const rx_attn_desc* desc, const rx_q8_desc* q8, int32_t batch, int64_t r2t_stride,
                              int32_t max_qo_len, int32_t max_kv_len) {
    const int rc = q8_check(fn, desc, q8, true);
    if (rc != RX_OK) return rc;
    RX_REQUIRE(batch >= 0 && max_qo_len >= 0 && max_kv_len >= 0 && r2t_stride >= 0, "%s: bad arguments", fn);
    RX_REQUIRE(std::isfinite(desc->scale * 1.4426950408889634f), "%s: the scale must be finite", fn);
    return RX_OK;
}

static int attention_q8_pointers(const char* fn, const RowsQ8Args& a) {
    RX_REQUIRE(a.q && a.r2t && a.k_pool && a.v_pool && a.scales && a.out && (a.kv_lens || (a.qo_indptr && a.prefix_lens)),
               "%s: null device pointer", fn);
    for (const void* x : {a.q, (const void*)a.k_pool, (const void*)a.v_pool, (const void*)a.out})
        RX_REQUIRE(((uintptr_t)x & 15) == 0, "%s: rows and pools must be 16-byte aligned", fn);
    RX_REQUIRE(((uintptr_t)a.scales & 7) == 0, "%s: scales must be 8-byte aligned", fn);
    return RX_OK;
}

// The most keys of a request: the kernels count keys in 32 bits, and up to two stages' past the last.
constexpr int32_t Q8_MOST_KEYS = INT32_MAX - 65535;

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// f32 rows read each request's own keys.
static bool uses_groups(const rx_attn_desc* d, const rx_shared_groups* g) { return g && g->num_groups > 0 && d->dtype == RX_BF16; }

static bool workspace_shape(const rx_attn_desc* d, int32_t batch, int32_t max_qo_len, int32_t max_kv_len) {
    return d && batch > 0 && max_qo_len > 0 && max_kv_len >= 0 && d->hkv > 0 && d->hkv <= 4096 && d->hq > 0 && d->hq <= 4096 &&
           d->hq % d->hkv == 0 && (d->head_dim == 64 || d->head_dim == 128);
}

// bf16 rows that fill a tile of 128 at least in part go to the tcgen05 kernel; f32 rows keep 32-bit results on mma.sync.
static bool many_rows(const rx_attn_desc* d, int32_t max_qo_len) {
    return d->dtype == RX_BF16 && (int64_t)max_qo_len * (d->hq / d->hkv) > ROWS_Q8_MOST;
}

extern "C" size_t decode_q8_workspace_bytes(const rx_attn_desc* desc, int32_t batch, int32_t max_kv_len,
                                            const rx_shared_groups* groups) {
    if (!workspace_shape(desc, batch, 1, max_kv_len)) return 0;
    const size_t own = up256(rows_q8_plan(desc, batch, 1, max_kv_len).room);
    return uses_groups(desc, groups) ? own + shared_q8_bytes(desc, batch, groups->num_groups) : own;
}

extern "C" size_t extend_q8_workspace_bytes(const rx_attn_desc* desc, int32_t batch, int32_t max_qo_len, int32_t max_kv_len) {
    if (!workspace_shape(desc, batch, max_qo_len, max_kv_len)) return 0;
    if (many_rows(desc, max_qo_len)) return extend_q8_bytes(desc);
    return rows_q8_plan(desc, batch, max_qo_len, max_kv_len).room;
}

extern "C" int decode_attention_q8(const rx_attn_desc* desc, const rx_q8_desc* q8, int32_t batch, const void* d_q,
                                   const int32_t* d_req_to_token, int64_t r2t_stride, const int32_t* d_kv_lens,
                                   const rx_shared_groups* groups, const void* d_k_pool, const void* d_v_pool, const float* d_scales,
                                   void* d_out, float* d_lse, int32_t max_kv_len, void* d_workspace, size_t ws_bytes,
                                   int32_t* d_status, void* stream) {
    static const char* fn = "decode_attention_q8";
    RX_TRACE("decode_attention_q8");
    int rc = attention_q8_check(fn, desc, q8, batch, r2t_stride, 1, max_kv_len);
    if (rc != RX_OK || batch == 0) return rc;
    RX_REQUIRE(d_kv_lens, "%s: null device pointer", fn);
    RowsQ8Args a{d_q,  nullptr, nullptr, d_kv_lens, d_req_to_token, r2t_stride, (const uint8_t*)d_k_pool, (const uint8_t*)d_v_pool,
                 (const float2*)d_scales, d_out, d_lse, batch, 1, std::min(max_kv_len, Q8_MOST_KEYS), d_status};
    rc = attention_q8_pointers(fn, a);
    if (rc != RX_OK) return rc;
    if (uses_groups(desc, groups)) {
        RX_REQUIRE(groups->d_group_indptr && groups->d_group_members && groups->d_group_len && groups->max_group_size >= 1 &&
                       groups->max_group_len >= 1,
                   "%s: incomplete shared groups", fn);
        const size_t own = up256(rows_q8_plan(desc, batch, 1, a.max_kv_len).bytes), need = own + shared_q8_bytes(desc, batch, groups->num_groups);
        RX_REQUIRE(d_workspace && ws_bytes >= need && ((uintptr_t)d_workspace & 255) == 0,
                   "%s: a 256-byte aligned workspace of %zu bytes is needed (got %zu)", fn, need, ws_bytes);
        rc = shared_q8_launch(fn, a, desc, q8, groups, (unsigned char*)d_workspace + own, (cudaStream_t)stream);
        if (rc != RX_OK) return rc;
    }
    return rows_q8_launch(fn, a, desc, q8, d_workspace, ws_bytes, (cudaStream_t)stream);
}

extern "C" int prefix_extend_attention_q8(const rx_attn_desc* desc, const rx_q8_desc* q8, int32_t batch, const void* d_q,
                                          const int64_t* d_qo_indptr, const int32_t* d_prefix_lens, const int32_t* d_req_to_token,
                                          int64_t r2t_stride, const void* d_k_pool, const void* d_v_pool, const float* d_scales,
                                          void* d_out, float* d_lse, int32_t max_qo_len, int32_t max_kv_len, void* d_workspace,
                                          size_t ws_bytes, int32_t* d_status, void* stream) {
    static const char* fn = "prefix_extend_attention_q8";
    RX_TRACE("prefix_extend_attention_q8");
    int rc = attention_q8_check(fn, desc, q8, batch, r2t_stride, max_qo_len, max_kv_len);
    if (rc != RX_OK || batch == 0 || max_qo_len == 0) return rc;
    const RowsQ8Args a{d_q,  d_qo_indptr, d_prefix_lens, nullptr, d_req_to_token, r2t_stride, (const uint8_t*)d_k_pool,
                       (const uint8_t*)d_v_pool, (const float2*)d_scales, d_out, d_lse, batch, max_qo_len, std::min(max_kv_len, Q8_MOST_KEYS),
                       d_status};
    rc = attention_q8_pointers(fn, a);
    if (rc != RX_OK) return rc;
    if (many_rows(desc, max_qo_len)) return extend_q8_launch(fn, a, desc, q8, d_workspace, ws_bytes, (cudaStream_t)stream);
    return rows_q8_launch(fn, a, desc, q8, d_workspace, ws_bytes, (cudaStream_t)stream);
}
