// Internal launch interfaces of the attention over 8-bit pools.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kv_q8.cuh"
#include "radix_attn.h"
#include "rx_kernels.h"

namespace rx {

// What both entry points hand on.  kv_lens non-null selects decode (one token a request, max_qo_len 1).
struct RowsQ8Args {
    const void* q;
    const int64_t* qo_indptr;
    const int32_t* prefix_lens;
    const int32_t* kv_lens;
    const int32_t* r2t;
    int64_t stride;
    const uint8_t* k_pool;
    const uint8_t* v_pool;
    const float2* scales;
    void* out;
    float* lse;
    int32_t batch, max_qo_len, max_kv_len;
    int32_t* status;
    // decode with shared runs: the keys that each request leaves to its group's run (0: none), and that run's part of its rows
    const int32_t* shared_of;
    const float* shared_o;
    const float* shared_lse;
};

// A group of requests of a decode batch with a shared run of keys.
struct SharedGroup {
    int32_t first, count;        // members
    int32_t len;                 // keys
    int32_t src;                 // a member, whose slot-table row has them
};

// How rows_q8.cu shares out a call, and the workspace it needs for parts of rows (0: none).  room: what calls of any smaller
// batch and lengths need at most, which is not always less: long contexts of few requests are shared out, of many not.
struct RowsPlan {
    int nt, hb;                  // 8-row tiles of a CTA, log2 of its heads
    bool shared;
    int64_t tiles, ctas;
    size_t lse_at, meta_at, bytes, room;
};
RowsPlan rows_q8_plan(const rx_attn_desc* d, int32_t batch, int32_t max_qo_len, int32_t max_kv_len);
int rows_q8_launch(const char* fn, const RowsQ8Args& a, const rx_attn_desc* d, const rx_q8_desc* q8, void* ws, size_t ws_bytes,
                   cudaStream_t stream);

// bf16 rows past what a tile of rows_q8.cu takes: the tensor-core kernel of extend_q8.cu and its workspace.
constexpr int64_t ROWS_Q8_MOST = 16;
size_t extend_q8_bytes(const rx_attn_desc* d);
int extend_q8_launch(const char* fn, const RowsQ8Args& a, const rx_attn_desc* d, const rx_q8_desc* q8, void* ws, size_t ws_bytes,
                     cudaStream_t stream);

// The shared runs of a decode batch's groups on that kernel; sets a's shared_* for the call of rows_q8_launch that does the rest.
size_t shared_q8_bytes(const rx_attn_desc* d, int32_t batch, int32_t num_groups);
int shared_q8_launch(const char* fn, RowsQ8Args& a, const rx_attn_desc* d, const rx_q8_desc* q8, const rx_shared_groups* g, void* ws,
                     cudaStream_t stream);

}  // namespace rx
