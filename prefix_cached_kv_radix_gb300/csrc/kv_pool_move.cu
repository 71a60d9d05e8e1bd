// kv_pool_copy and kv_pool_fork: rows of the KV pools moved to other slots of the same pools.
//
// A cached token's keys and values sit at one slot of every layer's K pool and V pool; moving the
// token moves that row of each.  kv_pool_copy takes a list of pages (runs of page_size slots, a
// slot where it is 1) and their destinations, as compaction makes it; kv_pool_fork makes the slot
// tables of sequences that continue others, sharing the slots of the tokens they keep and copying
// the K/V of the rest.
//
// Both are bound by HBM: each byte is read once and written once, and nothing is computed.  A warp
// moves a segment of up to MOVE_SEG 16-byte vectors of one page in one pool, all its loads in
// flight before its first store (4 KB a warp, 32 warps an SM: more than the latency of HBM times
// its rate needs), so the rows' order in the pool does not matter as long as a row is some hundred
// bytes.  The pool addresses travel as a kernel argument, so one launch moves a token's rows of
// every layer.  Measured: 3001 pages of 16 tokens in 4 layers (8 kv heads x 128, bf16), 1.57 GB read and
// written, 240 us, 6.56 TB/s (97 % of the measured copy rate); 64 forked rows with 10,000 copied tokens of
// 2 layers in f32 48 us, 7.2 TB/s (part of it from the L2); 700 slots of 2 layers 2.8 us, the launch.
#include <cuda_runtime.h>

#include <algorithm>

#include "radix_attn.h"
#include "rx_common.h"
#include "rx_device.cuh"
#include "rx_launch.h"

namespace rx {

constexpr int MOVE_THREADS = 256;
constexpr int MOVE_WARPS = MOVE_THREADS / 32;
constexpr int MOVE_PER = 8;                        // vectors in flight per lane
constexpr int MOVE_SEG = 32 * MOVE_PER;            // vectors per warp and step
constexpr int MOVE_POOLS = 256;                    // pool addresses per launch (2 KB of arguments)
constexpr int FORK_TILE = MOVE_THREADS * 4;        // table entries per block (4 per thread)

struct PoolList {
    uint4* p[MOVE_POOLS];
};

// `cnt` vectors from src to dst by one warp.
__device__ __forceinline__ void warp_copy(uint4* dst, const uint4* src, int cnt, int lane) {
    uint4 x[MOVE_PER];
#pragma unroll
    for (int i = 0; i < MOVE_PER; ++i)
        if (lane + 32 * i < cnt) x[i] = src[lane + 32 * i];
#pragma unroll
    for (int i = 0; i < MOVE_PER; ++i)
        if (lane + 32 * i < cnt) dst[lane + 32 * i] = x[i];
}

struct CopyParams {
    const int32_t* src;
    const int32_t* dst;
    int64_t n, pages, page_vecs;   // pages moved, pages in a pool, vectors per page
    int64_t segs, items;           // segments per page; pools * n * segs
    int32_t* status;
};

// Item = (pool, page, segment), segment fastest.
__global__ void __launch_bounds__(MOVE_THREADS) kv_pool_copy_kernel(const __grid_constant__ CopyParams p,
                                                                   const __grid_constant__ PoolList pools) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * MOVE_WARPS;
    for (int64_t it = (int64_t)blockIdx.x * MOVE_WARPS + (threadIdx.x >> 5); it < p.items; it += step) {
        const int64_t row = it / p.segs, seg = it - row * p.segs;
        const int64_t pool = row / p.n, i = row - pool * p.n;
        const int32_t s = p.src[i], d = p.dst[i];
        if (s < 0 || s >= p.pages || d < 0 || d >= p.pages) {
            if (lane == 0) report(p.status, RX_DEV_BAD_SLOT);
            continue;
        }
        if (s == d) continue;
        uint4* base = pools.p[pool] + seg * MOVE_SEG;
        warp_copy(base + d * p.page_vecs, base + s * p.page_vecs, (int)min((int64_t)MOVE_SEG, p.page_vecs - seg * MOVE_SEG),
                  lane);
    }
}

struct ForkParams {
    int32_t rows, tiles, in_rows;
    const int32_t* parents;        // [rows] row of the table read
    const int32_t* keep;           // [rows] leading tokens that keep the parent's slots
    const int32_t* lens;           // [rows] tokens in all
    const int64_t* tail_indptr;    // [rows + 1] into tail_slots
    const int32_t* tail_slots;
    const int32_t* r2t_in;
    int64_t in_stride;
    int32_t* r2t_out;
    int64_t out_stride, num_slots, total_tail, row_vecs;
    int64_t segs;                  // segments per K/V row
    int32_t n_pools;
    int32_t* status;
};

// Whether output row f can be made: its lengths fit the tables and its tail list.
__device__ __forceinline__ bool fork_row_ok(const ForkParams& p, int f) {
    const int32_t parent = p.parents[f], keep = p.keep[f], len = p.lens[f];
    const int64_t a = p.tail_indptr[f], b = p.tail_indptr[f + 1];
    return parent >= 0 && parent < p.in_rows && keep >= 0 && keep <= len && len <= p.in_stride && len <= p.out_stride &&
           a >= 0 && b <= p.total_tail && b - a == len - keep;
}

// Whether no tail offset is below the one before it, by a warp.
__device__ __noinline__ int offsets_ordered(const ForkParams& p, int lane) {
    bool down = false;
    for (int f = lane; f < p.rows; f += 32) down |= p.tail_indptr[f + 1] < p.tail_indptr[f];
    return !__any_sync(0xffffffffu, down);
}

// The first row that can be made and that tail token i is of, by a warp; -1: none.
__device__ __noinline__ int row_of_token(const ForkParams& p, int64_t i, int lane) {
    for (int f0 = 0; f0 < p.rows; f0 += 32) {
        const int f = f0 + lane;
        const unsigned m = __ballot_sync(0xffffffffu, f < p.rows && p.tail_indptr[f] <= i && i < p.tail_indptr[f + 1] && fork_row_ok(p, f));
        if (m) return f0 + __ffs(m) - 1;
    }
    return -1;
}

// Blocks [0, rows * tiles): the output table, one tile of FORK_TILE entries of a row each.  The
// others: one (tail token, pool, segment) per warp and step.
__global__ void __launch_bounds__(MOVE_THREADS) kv_pool_fork_kernel(const __grid_constant__ ForkParams p,
                                                                   const __grid_constant__ PoolList pools) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t table_blocks = (int64_t)p.rows * p.tiles;
    if ((int64_t)blockIdx.x < table_blocks) {
        const int f = (int)(blockIdx.x / p.tiles);
        const int64_t j0 = (int64_t)(blockIdx.x % p.tiles) * FORK_TILE + threadIdx.x;
        const bool ok = fork_row_ok(p, f);
        if (!ok && j0 == 0) report(p.status, RX_DEV_BAD_LENGTH);
        const int32_t* from = p.r2t_in + (ok ? (int64_t)p.parents[f] * p.in_stride : 0);
        const int64_t keep = ok ? p.keep[f] : 0, len = ok ? p.lens[f] : 0, tail = p.tail_indptr[f] - keep;
        int32_t s[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t j = j0 + u * MOVE_THREADS;
            s[u] = j < keep ? from[j] : j < len ? p.tail_slots[tail + j] : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t j = j0 + u * MOVE_THREADS;
            if (j >= p.out_stride) break;
            if (j < len && (s[u] < 0 || s[u] >= p.num_slots)) {
                report(p.status, RX_DEV_BAD_SLOT);
                s[u] = -1;
            }
            p.r2t_out[(int64_t)f * p.out_stride + j] = s[u];
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t step = (gridDim.x - table_blocks) * MOVE_WARPS;
    const int64_t items = p.total_tail * p.n_pools * p.segs;
    int ordered = -1;                                      // whether the tail offsets nowhere decrease (-1: not looked at)
    for (int64_t it = (blockIdx.x - table_blocks) * MOVE_WARPS + (threadIdx.x >> 5); it < items; it += step) {
        const int64_t q = it / p.segs, seg = it - q * p.segs;
        const int64_t i = q / p.n_pools;                   // tail token, of the last row that starts at or before it
        const int pool = (int)(q - i * p.n_pools);
        // the lanes look at 32 evenly spaced rows of the range left at a time
        int lo = 0, hi = p.rows;                           // tail_indptr[lo] <= i (or lo = 0), tail_indptr[hi] > i (or hi = rows)
        while (hi - lo > 1) {
            const int w = (hi - lo + 31) / 32, at = lo + lane * w;
            const unsigned m = __ballot_sync(0xffffffffu, at < hi && (lane == 0 || p.tail_indptr[at] <= i));
            const int last = 31 - __clz(m);
            lo += last * w;
            hi = min(hi, lo + w);
        }
        int f = lo;
        if (i < p.tail_indptr[f] || i >= p.tail_indptr[f + 1] || !fork_row_ok(p, f)) {
            // No row's token, or a bad row's (reported above), or the search was led astray by offsets that
            // decrease at some bad row: then each row is looked at, so that a good one gets its copies.
            if (ordered < 0) ordered = offsets_ordered(p, lane);
            if (ordered || (f = row_of_token(p, i, lane)) < 0) continue;
        }
        const int64_t j = p.keep[f] + (i - p.tail_indptr[f]);
        const int32_t s = p.r2t_in[(int64_t)p.parents[f] * p.in_stride + j], d = p.tail_slots[i];
        if (s < 0 || s >= p.num_slots || d < 0 || d >= p.num_slots) {
            if (lane == 0) report(p.status, RX_DEV_BAD_SLOT);
            continue;
        }
        if (s == d) continue;
        uint4* base = pools.p[pool] + seg * MOVE_SEG;
        warp_copy(base + d * p.row_vecs, base + s * p.row_vecs, (int)min((int64_t)MOVE_SEG, p.row_vecs - seg * MOVE_SEG), lane);
    }
}

// The checks both share; *vecs: 16-byte vectors of a slot's row.
static int move_shape(const char* fn, const rx_attn_desc* desc, int32_t n_pools, void* const* pools, int64_t* vecs) {
    RX_REQUIRE(desc && n_pools >= 0 && (n_pools == 0 || pools), "%s: bad arguments", fn);
    RX_REQUIRE(desc->dtype == RX_F32 || desc->dtype == RX_BF16, "%s: unknown dtype %d", fn, desc->dtype);
    RX_REQUIRE(desc->hkv > 0 && desc->head_dim > 0 && desc->num_slots > 0 && desc->num_slots <= INT32_MAX, "%s: bad shape", fn);
    const int64_t bytes = (int64_t)desc->hkv * desc->head_dim * (desc->dtype == RX_F32 ? 4 : 2);
    RX_REQUIRE(bytes % 16 == 0, "%s: K/V row of %lld bytes is not a multiple of 16", fn, (long long)bytes);
    for (int32_t i = 0; i < n_pools; ++i) {
        RX_REQUIRE(pools[i] && ((uintptr_t)pools[i] & 15) == 0, "%s: pool %d is null or not 16-byte aligned", fn, i);
        // a pool given twice would be moved twice at once
        for (int32_t j = 0; j < i; ++j) RX_REQUIRE(pools[i] != pools[j], "%s: pools %d and %d are the same", fn, j, i);
    }
    *vecs = bytes / 16;
    return RX_OK;
}

static int move_launched(const char* fn) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("%s: launch failed: %s", fn, cudaGetErrorString(e));
        return RX_ECUDA;
    }
    return RX_OK;
}

// Blocks of a grid-stride launch over `items` warps' work: a block for each eight, up to eight blocks an
// SM, twice what is resident, so that SMs that finish early take from the second half.
static int64_t move_blocks(int64_t items) { return std::min<int64_t>((items + MOVE_WARPS - 1) / MOVE_WARPS, 152 * 8); }

}  // namespace rx

using namespace rx;

extern "C" int kv_pool_copy(const rx_attn_desc* desc, int32_t n_pools, void* const* pools, int64_t page_size, int64_t n,
                            const int32_t* d_src, const int32_t* d_dst, int32_t* d_status, void* stream) {
    RX_TRACE("kv_pool_copy");
    int64_t vecs = 0;
    const int rc = move_shape("kv_pool_copy", desc, n_pools, pools, &vecs);
    if (rc != RX_OK) return rc;
    RX_REQUIRE(n >= 0 && n <= INT32_MAX && page_size >= 1 && page_size <= desc->num_slots, "kv_pool_copy: bad page size or count");
    if (n == 0 || n_pools == 0) return RX_OK;
    RX_REQUIRE(d_src && d_dst, "kv_pool_copy: null device pointer");
    CopyParams p{};
    p.src = d_src;
    p.dst = d_dst;
    p.n = n;
    p.pages = desc->num_slots / page_size;
    p.page_vecs = page_size * vecs;
    p.segs = (p.page_vecs + MOVE_SEG - 1) / MOVE_SEG;
    p.status = d_status;
    for (int32_t at = 0; at < n_pools; at += MOVE_POOLS) {
        PoolList list{};
        const int32_t k = std::min(MOVE_POOLS, n_pools - at);
        for (int32_t i = 0; i < k; ++i) list.p[i] = (uint4*)pools[at + i];
        p.items = n * k * p.segs;
        launch_pdl(kv_pool_copy_kernel, (unsigned)move_blocks(p.items), MOVE_THREADS, 0, (cudaStream_t)stream, p, list);
    }
    return move_launched("kv_pool_copy");
}

extern "C" int kv_pool_fork(const rx_attn_desc* desc, int32_t n_pools, void* const* pools, int32_t n_rows,
                            const int32_t* d_parents, const int32_t* d_keep_lens, const int32_t* d_kv_lens,
                            const int64_t* d_tail_indptr, const int32_t* d_tail_slots, const int32_t* d_r2t_in, int32_t in_rows,
                            int64_t in_stride, int32_t* d_r2t_out, int64_t out_stride, int64_t total_tail, int32_t* d_status,
                            void* stream) {
    RX_TRACE("kv_pool_fork");
    int64_t vecs = 0;
    const int rc = move_shape("kv_pool_fork", desc, n_pools, pools, &vecs);
    if (rc != RX_OK) return rc;
    RX_REQUIRE(n_rows >= 0 && in_rows >= 0 && in_stride >= 0 && out_stride >= 0 && total_tail >= 0 && total_tail <= INT32_MAX,
               "kv_pool_fork: bad arguments");
    if (n_rows == 0) return RX_OK;
    RX_REQUIRE(d_parents && d_keep_lens && d_kv_lens && d_tail_indptr && d_r2t_in && d_r2t_out && (total_tail == 0 || d_tail_slots),
               "kv_pool_fork: null device pointer");
    const int32_t *in_end = d_r2t_in + in_rows * in_stride, *out_end = d_r2t_out + n_rows * out_stride;
    RX_REQUIRE(in_end <= d_r2t_out || out_end <= d_r2t_in, "kv_pool_fork: the tables read and written overlap");
    const int64_t tiles = std::max<int64_t>(1, (out_stride + FORK_TILE - 1) / FORK_TILE);
    RX_REQUIRE(n_rows * tiles + 152 * 8 < (1ll << 31), "kv_pool_fork: rows or stride too large");
    ForkParams p{};
    p.rows = n_rows;
    p.in_rows = in_rows;
    p.parents = d_parents;
    p.keep = d_keep_lens;
    p.lens = d_kv_lens;
    p.tail_indptr = d_tail_indptr;
    p.tail_slots = d_tail_slots;
    p.r2t_in = d_r2t_in;
    p.in_stride = in_stride;
    p.r2t_out = d_r2t_out;
    p.out_stride = out_stride;
    p.num_slots = desc->num_slots;
    p.total_tail = total_tail;
    p.row_vecs = vecs;
    p.segs = (vecs + MOVE_SEG - 1) / MOVE_SEG;
    p.status = d_status;
    for (int32_t at = 0; at == 0 || at < n_pools; at += MOVE_POOLS) {   // the first launch makes the table too
        PoolList list{};
        p.n_pools = std::min(MOVE_POOLS, n_pools - at);
        for (int32_t i = 0; i < p.n_pools; ++i) list.p[i] = (uint4*)pools[at + i];
        p.tiles = at == 0 ? (int32_t)tiles : 0;
        const int64_t blocks = n_rows * (int64_t)p.tiles + move_blocks(total_tail * p.n_pools * p.segs);
        if (blocks > 0) launch_pdl(kv_pool_fork_kernel, (unsigned)blocks, MOVE_THREADS, 0, (cudaStream_t)stream, p, list);
    }
    return move_launched("kv_pool_fork");
}
