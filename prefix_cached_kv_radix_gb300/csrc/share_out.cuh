// Work of requests of different lengths shared out evenly over a grid of CTAs, without counters in memory.
#pragma once

#include <stdint.h>

#include "rx_device.cuh"

namespace rx {

// CTA blockIdx.x's part of the units of all requests, one after another: units(b) of request b, parts of at least `least`
// units.  A border that lies inside a request may move: snap(b, at, near) gives the place of the border at the
// request's unit `at`, moved by less than `near` (a sixteenth of a part), the same for both CTAs that share the border.
// Every thread of the block calls it; after a __syncthreads out[0], out[1] are the first unit of the part and of the next one, out[2] the
// request that the first lay in before it moved, out[3] the units before that request.  sums: one per warp.
template <int THREADS, class Units, class Snap>
__device__ __forceinline__ void share_out(int batch, int64_t least, int64_t* sums, int64_t* out, const Units& units, const Snap& snap) {
    constexpr int WARPS = THREADS / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t v = 0, mine = 0;             // this thread's request's units (of the last round), and those of all its requests
    for (int b = tid; b < batch; b += THREADS) {
        v = units(b, blockIdx.x == 0);
        mine += v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) sums[warp] = mine;
    if (tid < 4) out[tid] = 0;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) total += sums[w];
    const int64_t parts = max(min((int64_t)gridDim.x, total / least), (int64_t)1);
    const int64_t near = 1 + total / parts / 16;
    const int64_t want[2] = {min((int64_t)blockIdx.x, parts) * total / parts, min((int64_t)blockIdx.x + 1, parts) * total / parts};
    int64_t before = 0;                  // units of the rounds so far
    for (int b0 = 0; b0 < batch; b0 += THREADS) {
        const int b = b0 + tid;
        if (batch > THREADS) v = b < batch ? units(b, false) : 0;
        else if (b >= batch) v = 0;
        int64_t inc = v;                 // inclusive scan
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        __syncthreads();                 // the sums of the round before are read
        if (lane == 31) sums[warp] = inc;
        __syncthreads();
        int64_t at = before + inc - v;
        for (int w = 0; w < warp; ++w) at += sums[w];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (want[e] >= at && want[e] < at + v) {
                out[e] = at + snap(b, want[e] - at, near);
                if (e == 0) out[2] = b, out[3] = at;
            }
        for (int w = 0; w < WARPS; ++w) before += sums[w];
    }
    if (tid == 0) {                      // past the last unit
        if (want[0] >= total) out[0] = total;
        if (want[1] >= total) out[1] = total;
    }
}

// The parts of something that one CTA began and another one ended, for a block of 128 threads that merges them.  meta: [CTAs][2], entry 1
// what the CTA began and did not end, entry 0 what it went on with; x < 0: nothing, w != 0: ended here.  All call it: the parts of
// the `which`-th begun thing, list[i] = CTA * 2 + entry; returns their number, 0 where there are not that many things.
// room: MOST words.
template <int MOST>
__device__ __forceinline__ int parts_of(const int4* meta, int which, int ctas, int* list, uint32_t* room) {
    constexpr int PER = (MOST + 127) / 128;
    __shared__ int count;
    const int lane = threadIdx.x & 31;
    int4 m[PER][2];                      // all on their way together
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = threadIdx.x + 128 * i;
#pragma unroll
        for (int e = 0; e < 2; ++e) m[i][e] = c < ctas ? meta[c * 2 + e] : make_int4(-1, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {      // bit 0: begun here; 1: went on; 2: ended
        const int c = threadIdx.x + 128 * i;
        if (c < MOST) room[c] = (m[i][1].x >= 0 ? 1u : 0u) | (m[i][0].x >= 0 ? (m[i][0].w ? 6u : 2u) : 0u);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int first = -1, parts = 0;
        for (int c0 = 0; c0 < ctas && first < 0; c0 += 32) {
            const unsigned is = __ballot_sync(0xffffffffu, c0 + lane < ctas && (room[c0 + lane] & 1u));
            const int here = __popc(is);
            if (which >= here) which -= here;
            else first = c0 + (int)__fns(is, 0, which + 1);
        }
        if (first >= 0) {
            parts = 1;
            if (lane == 0) list[0] = first * 2 + 1;
            bool done = false;
            for (int c0 = first + 1; c0 < ctas && !done; c0 += 32) {
                const uint32_t f = c0 + lane < ctas ? room[c0 + lane] : 0u;
                const unsigned ends = __ballot_sync(0xffffffffu, f & 4u);
                const unsigned upto = ends ? (2u << (__ffs(ends) - 1)) - 1u : 0xffffffffu;      // to the part that ends it
                const unsigned is = __ballot_sync(0xffffffffu, f & 2u) & upto;
                if ((is >> lane) & 1u) list[parts + __popc(is & ((1u << lane) - 1u))] = (c0 + lane) * 2;
                parts += __popc(is);
                done = ends != 0;
            }
        }
        if (lane == 0) count = parts;
    }
    __syncthreads();
    return count;
}

// A row of D channels from its parts, list[0 .. parts - 1] (MOST at most), by a whole block of 128 threads.  Part i's row is row `r` of `rows`
// (normalised, its log-sum-exp to base 2).  Afterwards the first warp has the row, channels lane * D / 32 .., in acc; returns its
// log-sum-exp (-infinity: no key, and acc is zeros).  A warp takes every fourth part; the rows travel by cp.async, eight a
// warp at a time, twice (as loads, the compiler put each next to its use, and 256 parts took 38 us).
template <int D, int MOST>
__device__ __forceinline__ float merge_many(const int* list, int parts, const float* part_o, const float* part_lse, int rows, int r,
                                            float* acc) {
    constexpr int E = D / 32, AT = 8, PER = (MOST + 127) / 128, LANES = D / 4;
    __shared__ float lse_s[PER * 128], w_s[4];
    __shared__ __align__(16) float row_s[4][2][AT][D];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, mine = (parts - warp + 3) / 4;
    auto fetch = [&](int i0) {           // this warp's parts i0 .. i0 + 7
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            const int s = (i0 + i) * 4 + warp;
            if (s < parts && lane < LANES)
                cp_async_16(smem_u32(&row_s[warp][(i0 / AT) & 1][i][lane * 4]), part_o + ((int64_t)list[s] * rows + r) * D + lane * 4, 16);
        }
        cp_async_commit();
    };
    fetch(0);
    fetch(AT);
    float x[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = tid + 128 * i < parts ? part_lse[(int64_t)list[tid + 128 * i] * rows + r] : -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) lse_s[tid + 128 * i] = x[i];
    __syncthreads();
    float M = -INFINITY;
    for (int s = lane; s < parts; s += 32) M = fmaxf(M, lse_s[s]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == -INFINITY ? 0.f : M;
    float W = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int i0 = 0; i0 < mine; i0 += AT) {
        cp_async_wait<1>();
        __syncwarp();
        for (int i = i0; i < min(i0 + AT, mine); ++i) {
            const float w = exp2f(lse_s[i * 4 + warp] - ref);
            W += w;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += w * row_s[warp][(i0 / AT) & 1][i - i0][lane * E + e];
        }
        __syncwarp();
        fetch(i0 + 2 * AT);
    }
    cp_async_wait<0>();
    __syncthreads();                     // row_s has been read: it takes the warps' sums
#pragma unroll
    for (int e = 0; e < E; ++e) row_s[warp][0][0][lane * E + e] = acc[e];
    if (lane == 0) w_s[warp] = W;
    __syncthreads();
    W = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int o = 0; o < 4; ++o) {
        W += w_s[o];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += row_s[o][0][0][lane * E + e];
    }
    const float inv = W == 0.f ? 0.f : 1.f / W;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= inv;
    return W == 0.f ? -INFINITY : M + log2f(W);
}

// The same by a warp, for a few parts.
template <int D>
__device__ __forceinline__ float merge_few(const int* list, int parts, const float* part_o, const float* part_lse, int rows, int r,
                                           float* acc) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float M = -INFINITY;
    for (int s = lane; s < parts; s += 32) M = fmaxf(M, part_lse[(int64_t)list[s] * rows + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == -INFINITY ? 0.f : M;
    float W = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
        const int64_t at = (int64_t)list[s] * rows + r;
        const float w = exp2f(part_lse[at] - ref);
        W += w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += w * part_o[at * D + lane * E + e];
    }
    const float inv = W == 0.f ? 0.f : 1.f / W;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= inv;
    return W == 0.f ? -INFINITY : M + log2f(W);
}

}  // namespace rx
