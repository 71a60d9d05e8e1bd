// The work items of prompt_attention: row tiles of the packed sequences, found from the sequence
// boundaries on the device.
#pragma once

#include <stdint.h>

#include "radix_attn.h"
#include "rx_device.cuh"
#include "rx_kernels.h"

namespace rx {

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

struct PromptItem {
    int start, n, head, tile;   // first row and rows of the sequence, head, row tile
};

// Finds the items' sequences.  A warp keeps 32 consecutive boundaries in its lanes: the items a
// block takes one after another lie close together, so most are found without a memory access, and
// the others in two or three rounds of loads.  32-bit arithmetic throughout: rows are below 2^31,
// and a boundary that is not (the sequence is reported) is clamped.
struct PromptFinder {
    int w0 = -1;             // first boundary of the window (-1: none loaded)
    int mine = 0;            // boundary w0 + lane, clamped; beyond the last one: the last
    bool good = false;       // it lies in [0, total]

    __device__ __forceinline__ int load(const PromptParams& p, int b, bool& ok) const {
        const int64_t x = p.indptr[b];
        ok = x >= 0 && x <= p.total;
        return (int)min(max(x, (int64_t)0), p.total);
    }

    // Item `i` of the places x heads: within a sequence the heads one after another, and within a
    // head the tiles from the last, which has the most keys, to the first, so that the items that
    // end a launch are short ones.  False for a place left over, and for a sequence whose boundaries
    // do not lie in order in [0, total] (reported).  Every thread of a warp calls it with the same item.
    __device__ __forceinline__ bool find(const PromptParams& p, int i, const PromptDiv& tile_tokens, const PromptDiv& heads, PromptItem& it) {
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
        const unsigned sound = __ballot_sync(0xffffffffu, good);
        if (((sound >> l) & 3u) != 3u || e < s) {
            if (lane == 0) report(p.status, RX_DEV_BAD_LENGTH);
            return false;
        }
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
};

}  // namespace rx
