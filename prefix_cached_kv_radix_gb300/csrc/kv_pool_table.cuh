// The slot-table part of the kernels that write new tokens into the KV pools.
#pragma once

#include <stdint.h>

#include "radix_attn.h"
#include "rx_device.cuh"

namespace rx {

// One tile of NT * PER entries of request b's slot-table row: its matched (prefix) slots, then
// its new slots, then -1 up to the row's stride.  All loads are issued before the first store
// (each thread has PER independent loads in flight).  Bad lengths (matched slots without a list of
// them are one) and slots are reported; a bad entry is written as -1.
template <int NT, int PER = 4>
__device__ __forceinline__ void kpw_table_tile(int b, int64_t tile, const int32_t* __restrict__ prefix_slots,
                                               const int64_t* __restrict__ prefix_indptr,
                                               const int32_t* __restrict__ new_slots,
                                               const int64_t* __restrict__ qo_indptr, int32_t* __restrict__ r2t,
                                               int64_t stride, int64_t num_slots, int64_t t_begin, int64_t t_end,
                                               int32_t* status) {
    const int64_t j0 = tile * NT * PER;
    const int64_t p0 = prefix_indptr[b], P = prefix_indptr[b + 1] - p0;
    const int64_t q0 = qo_indptr[b], n = qo_indptr[b + 1] - q0;
    int32_t* row = r2t + (int64_t)b * stride;
    // without sums: boundaries may be any numbers, and one that wrapped would pass
    const bool bad_len = P < 0 || n < 0 || P > stride || n > stride - P || q0 < t_begin || q0 > t_end || n > t_end - q0 ||
                         (P > 0 && !prefix_slots);
    if (bad_len && j0 == 0 && threadIdx.x == 0) report(status, RX_DEV_BAD_LENGTH);
    int32_t s[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) {          // the loads first, all in flight together
        const int64_t j = j0 + threadIdx.x + (int64_t)u * NT;
        s[u] = -1;
        if (!bad_len && j < P)
            s[u] = prefix_slots[p0 + j];
        else if (!bad_len && j < P + n)
            s[u] = new_slots[q0 + (j - P)];
    }
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int64_t j = j0 + threadIdx.x + (int64_t)u * NT;
        if (j >= stride) break;
        if (s[u] < -1 || s[u] >= num_slots || (s[u] == -1 && !bad_len && j < P + n)) {
            report(status, RX_DEV_BAD_SLOT);
            s[u] = -1;
        }
        row[j] = s[u];
    }
}

}  // namespace rx
