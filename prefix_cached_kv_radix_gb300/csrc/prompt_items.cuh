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

struct PromptItem {
    int64_t start;   // first row of the sequence
    int n, head, tile;
};

// Item `i` of the places x heads: within a sequence the heads one after another, and within a head
// the tiles from the last, which has the most keys, to the first, so that the items that end a
// launch are short ones.  False for a place left over, and for a sequence whose boundaries do not
// lie in order in [0, total] (reported).  Every thread of a warp calls it with the same item.
__device__ __forceinline__ bool prompt_item(const PromptParams& p, int64_t i, int tile_tokens, int heads, PromptItem& it) {
    const int lane = threadIdx.x & 31;
    auto base = [&](int b) { return p.indptr[b] / tile_tokens + b; };
    int lo = 0, hi = p.batch;                        // base(lo) * heads <= i < base(hi) * heads, where they hold
    while (hi - lo > 1) {                            // 32 evenly spaced sequences at a time
        const int w = (hi - lo + 31) / 32, at = lo + lane * w;
        const unsigned m = __ballot_sync(0xffffffffu, at < hi && (lane == 0 || base(at) * heads <= i));
        const int last = 31 - __clz(m);
        lo += last * w;
        hi = min(hi, lo + w);
    }
    const int64_t s = p.indptr[lo], e = p.indptr[lo + 1];
    if (s < 0 || e < s || e > p.total || e - s > INT32_MAX) {
        if (lane == 0) report(p.status, RX_DEV_BAD_LENGTH);
        return false;
    }
    const int64_t places = e / tile_tokens - s / tile_tokens + 1;
    const int64_t at = i - (s / tile_tokens + lo) * heads;
    if (at < 0 || at >= places * heads) return false;
    it.head = (int)(at / places);
    it.tile = (int)(places - 1 - (at - it.head * places));
    it.start = s;
    it.n = (int)(e - s);
    return (int64_t)it.tile * tile_tokens < it.n;
}

}  // namespace rx
