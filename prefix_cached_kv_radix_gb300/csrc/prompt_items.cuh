// The arguments of prompt_attention's kernels, and their work items: row tiles of the packed
// sequences, found from the sequence boundaries on the device.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "radix_attn.h"
#include "rx_device.cuh"

namespace rx {

// Causal attention over packed prompts (prompt_attention): sequence b's rows are
// indptr[b] .. indptr[b+1]-1 of q, k, v and out, strides in elements between rows.
struct PromptParams {
    int32_t batch, hq, hkv;
    int64_t total;                // rows of the buffers
    const void* q;
    const void* k;
    const void* v;
    void* out;
    int64_t q_stride, k_stride, v_stride, out_stride;
    const int64_t* indptr;
    float* lse;                   // natural log, [total, hq], optional
    float scale;
    int32_t by_level;             // order of the items
    int32_t* status;
};
int launch_prompt_simt(PromptParams p, int head_dim, cudaStream_t stream);

// A sequence [s, e) gets the tile places from floor(s / R) + b to floor(e / R) + b, b its number
// and R the tokens of a tile: enough for ceil((e - s) / R) tiles (at most one place is left over),
// in order and without overlap, so that a place's sequence is found by bisection and no prefix
// sum over the sequences' tiles is needed.  The host, which does not know the boundaries, launches
// all places up to those of the last possible sequence end.
__host__ __device__ inline int64_t prompt_items(int64_t total, int32_t batch, int tile_tokens) {
    return total / tile_tokens + batch;
}

// Division of a number below 2^31 by one fixed for the launch, as a product: with 2^(s-1) < d <= 2^s and
// m = ceil(2^(31+s) / d) < 2^32 + 1, floor(x / d) = floor(x m / 2^(31+s)) for every 0 <= x < 2^31, since
// m d - 2^(31+s) < d <= 2^s (Granlund and Montgomery 1994, theorem 4.2).
struct PromptDiv {
    int d = 1;
    uint64_t m = 1ull << 31;
    int s = 0;
    PromptDiv() = default;
    explicit PromptDiv(int divisor) : d(divisor) {
        while ((1ll << s) < divisor) ++s;
        m = ((1ull << (31 + s)) + (uint64_t)divisor - 1) / (uint64_t)divisor;
    }
    __host__ __device__ __forceinline__ int operator()(int x) const { return (int)(((uint64_t)(uint32_t)x * m) >> (31 + s)); }
};

// Whether the items are better taken by tile index, of all sequences together and from the highest
// down, than sequence by sequence: row tile x has about x tiles of keys, so the longest items come first
// and the launch ends on the shortest, whatever the order of the sequences (by sequence and by tile index,
// on rows that change from call to call: 48 ragged bf16 prompts 113 and 106 us; 12 heads x 64, one of 2000
// tokens 18.8 and 16.0, four of 4096 126 and 107, one of 16384 431 and 375; 8 ragged f32 prompts 622 and
// 425).  Not where all items run at once anyway, nor with more sequences than a warp's lanes hold at two each
// (searched in memory, 250 prompts of 64 tokens took 239 us and not 73), nor where the keys and values of all
// sequences are more than the L2 holds beside the rest (of 129 MB): each tile index reads them again (32
// prompts of 1024 tokens, 134 MB, the same rows in each call: 222 and 258 us; at 67 MB, 32/8 heads x 128, both are
// alike: one of 16384 1332 and 1335, four of 4096 370 and 369).
constexpr int PROMPT_LEVEL_SEQS = 64;    // two a lane
inline bool prompt_by_level(int64_t items, int resident, int32_t batch, int64_t kv_bytes) {
    return items > resident && batch <= PROMPT_LEVEL_SEQS && kv_bytes <= 80ll << 20;
}

// The longest sequence: the waits of the bf16 kernel, of which the longest is for one item, give up after 2 s;
// an item at the end of 2^26 rows takes about 0.7 s.
constexpr int PROMPT_MAX_ROWS = 1 << 26;

struct PromptItem {
    int start, n, head, tile;   // first row and rows of the sequence, head, row tile
};

// Finds the items' sequences.  A warp keeps 32 consecutive boundaries in its lanes: the items a
// block takes one after another lie close together, so most are found without a memory access, and
// the others in two or three rounds of loads.  32-bit arithmetic throughout: rows are below 2^31,
// and a boundary that is not is clamped.
struct PromptFinder {
    int w0 = -1;             // first boundary of the window (-1: none loaded)
    int mine = 0;            // boundary w0 + lane, clamped; beyond the last one: the last.  By level: tiles of sequence `lane`,
    int more = 0;            // and of sequence 32 + lane
    bool good = false;       // it lies in [0, total]

    // Whether a sequence's boundaries are in order and in [0, total], and it is not too long.
    static __device__ __forceinline__ bool sound(const PromptParams& p, int64_t s, int64_t e) {
        return s >= 0 && e >= s && e <= p.total && e - s <= PROMPT_MAX_ROWS;
    }

    // Reports sequence i's boundaries on item i: there are no fewer items than sequences and every item is
    // taken once, so each sequence is looked at, also where boundaries out of order keep its items from
    // finding it.  One lane of a block calls it, where no one waits for it.
    static __device__ __forceinline__ void check(const PromptParams& p, int i) {
        if (i < p.batch && !sound(p, p.indptr[i], p.indptr[i + 1])) report(p.status, RX_DEV_BAD_LENGTH);
    }

    __device__ __forceinline__ int load(const PromptParams& p, int b, bool& ok) const {
        const int64_t x = p.indptr[b];
        ok = x >= 0 && x <= p.total;
        return (int)min(max(x, (int64_t)0), p.total);
    }

    // Item `i` by tile index from the highest down, then sequence, then head.  There are f(x) = sum over the
    // sequences of max(0, tiles - x) tiles of index x and up; item place q has index x where
    // f(x + 1) <= q < f(x).  A sequence that is not sound has no tiles.
    __device__ __forceinline__ bool find_by_level(const PromptParams& p, int i, const PromptDiv& tile_tokens, const PromptDiv& heads,
                                                  PromptItem& it) {
        const int lane = threadIdx.x & 31;
        const int q = heads(i);
        if (w0 < 0) {
            w0 = 0;
            mine = tiles(p, lane, tile_tokens);
            more = tiles(p, 32 + lane, tile_tokens);
        }
        // q < f(lo), or lo = -1; q >= f(hi) = f_hi
        int lo = -1, hi = tile_tokens((int)p.total) + 2, f_hi = 0;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            const int f = (int)__reduce_add_sync(0xffffffffu, (unsigned)(max(0, mine - mid) + max(0, more - mid)));
            if (q < f) lo = mid;
            else hi = mid, f_hi = f;
        }
        if (lo < 0) return false;
        int r = q - f_hi;                    // which of the sequences that have a tile `lo`
#pragma unroll 1
        for (int m = 0; m < PROMPT_LEVEL_SEQS / 32; ++m) {
            const unsigned has = __ballot_sync(0xffffffffu, (m == 0 ? mine : more) > lo);
            const bool me = ((has >> lane) & 1u) && __popc(has & ((1u << lane) - 1u)) == r;
            const unsigned one = __ballot_sync(0xffffffffu, me);
            if (one) {
                const int b = 32 * m + __ffs(one) - 1;
                it.start = (int)p.indptr[b];
                it.n = (int)(p.indptr[b + 1] - p.indptr[b]);
                it.tile = lo;
                it.head = i - q * heads.d;
                return true;
            }
            r -= __popc(has);
        }
        return false;
    }

    // Row tiles of sequence b (0 beyond the batch, and where its boundaries are not sound).
    __device__ __forceinline__ int tiles(const PromptParams& p, int b, const PromptDiv& tile_tokens) {
        if (b >= p.batch) return 0;
        const int64_t s = p.indptr[b], e = p.indptr[b + 1];
        return sound(p, s, e) ? tile_tokens((int)(e - s) + tile_tokens.d - 1) : 0;
    }

    // Item `i` of the places x heads: within a sequence the heads one after another, and within a
    // head the tiles from the last, which has the most keys, to the first, so that the items that
    // end a launch are short ones.  False for a place left over, and for a sequence that is not sound.
    __device__ __forceinline__ bool find_by_place(const PromptParams& p, int i, const PromptDiv& tile_tokens, const PromptDiv& heads,
                                                  PromptItem& it) {
        const int lane = threadIdx.x & 31;
        const int place = heads(i);      // place-major bound of the sequence: base(b) <= place
        // the last sequence whose places start at or before this one
        unsigned m = 0;
        if (w0 >= 0) m = __ballot_sync(0xffffffffu, tile_tokens(mine) + w0 + lane <= place);
        if (m == 0 || (m >> 31)) {                            // not inside the window
            int lo = 0, hi = p.batch;
            bool ok;
            while (hi - lo > 1) {                             // 32 evenly spaced sequences at a time
                const int w = (hi - lo + 31) / 32, at = lo + lane * w;
                const bool before = at < hi && (lane == 0 || tile_tokens(load(p, at, ok)) + at <= place);
                const int last = 31 - __clz(__ballot_sync(0xffffffffu, before));
                lo += last * w;
                hi = min(hi, lo + w);
            }
            w0 = lo;
            mine = load(p, min(lo + lane, p.batch), good);
            m = 1;
        }
        int l = 31 - __clz(m);
        // beyond the last boundary every lane holds the last: the sequence is the last one
        l = min(l, p.batch - 1 - w0);
        const int b = w0 + l, s = __shfl_sync(0xffffffffu, mine, l), e = __shfl_sync(0xffffffffu, mine, l + 1);
        const unsigned in = __ballot_sync(0xffffffffu, good);
        if (((in >> l) & 3u) != 3u || e < s || e - s > PROMPT_MAX_ROWS) return false;
        const int first = tile_tokens(s);
        const int places = tile_tokens(e) - first + 1;
        const int64_t at = i - (int64_t)(first + b) * heads.d;
        if (at < 0 || at >= (int64_t)places * heads.d) return false;
        it.head = (int)((unsigned)at / (unsigned)places);
        it.tile = places - 1 - ((int)at - it.head * places);
        it.start = s;
        it.n = e - s;
        return (int64_t)it.tile * tile_tokens.d < it.n;
    }

    // Every thread of a warp calls it with the same item.
    __device__ __forceinline__ bool find(const PromptParams& p, int i, const PromptDiv& tile_tokens, const PromptDiv& heads,
                                         PromptItem& it) {
        return p.by_level ? find_by_level(p, i, tile_tokens, heads, it) : find_by_place(p, i, tile_tokens, heads, it);
    }
};

}  // namespace rx
