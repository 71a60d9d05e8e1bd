// kv_pool_write_rope: kv_pool_write for rows that still need their rotary positions.
//
// A pair of channels (a, b) of a query or key row at position p turns by the angle p * w, w the
// pair's frequency:  (a cos - b sin, b cos + a sin).  With several position axes (time, height,
// width) each pair takes its position from one axis.  One launch turns the queries, turns the new
// keys on their way into their pool slots, copies the new values into theirs and fills the slot
// table, so that a token's rows cross HBM once: apart from the table the bytes are one read and
// one write of T * (hq + 2 hkv) * head_dim elements.
//
// The angle is exact for every 32-bit position: w / 2pi is kept as a 64-bit binary fraction of a
// turn (host), the product with the integer position wraps modulo one turn by itself, and the
// remaining fraction of a turn, in [-1/2, 1/2), goes to sincospif.  What is left is the rounding
// of w / 2pi to double, 2^-52 of the angle, and of the fraction to float, 2^-25 turn; 32-bit
// arithmetic from the start would be off by p * 2^-24 radians, a whole turn at p = 1e8, and
// 64-bit floating point runs at a small fraction of the 32-bit rate here.
//
// The angles of a block's tokens are computed once, into shared memory, and used by all their
// heads.  A thread moves two 16-byte vectors at a time, the two whose channels pair up (half a
// rotated width apart, or neighbours), ROPE_UNITS such pairs in flight before the block waits
// for its angles.
//
// Bound by HBM for prompts (24 image prompts, 64/8 heads x 128: 309 MB in 49.5 us, 6.2 TB/s, 92 % of the
// measured copy rate; 1550 f32 rows, 76 MB, in 15.5 us, where a plain copy of as many bytes takes 14.4), by
// the launch for decode steps (64 rows of 12 heads x 64: 3.5 us a call).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kv_pool_table.cuh"
#include "radix_attn.h"
#include "rx_common.h"
#include "rx_device.cuh"
#include "rx_launch.h"

namespace rx {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_PER = 16;                     // table entries per thread
constexpr int ROPE_TILE = ROPE_THREADS * ROPE_PER;   // and per block
constexpr int ROPE_MAX_PAIRS = 64;               // head_dim <= 128
constexpr int ROPE_MAX_TOKENS = 2;               // tokens per block
constexpr int ROPE_UNITS = 2;                    // vector pairs in flight per thread

struct RopeParams {
    int32_t batch, tiles;         // tiles: table blocks per request (0: no table)
    const int32_t* prefix_slots;
    const int64_t* prefix_indptr;
    const int32_t* new_slots;
    const int64_t* qo_indptr;
    const int32_t* positions;     // [axes, pos_stride]
    int64_t pos_stride;
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    void* k_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;   // elements between rows
    void* k_pool;
    void* v_pool;
    int32_t* r2t;
    int64_t r2t_stride, num_slots, total;
    int32_t hq, hkv, pairs, interleaved, tokens;   // tokens: rows per block
    int32_t* status;
    uint64_t turns[ROPE_MAX_PAIRS];                // frequency / 2pi as a 64-bit fraction of a turn
    uint8_t axis[ROPE_MAX_PAIRS];                  // position axis of each pair
};

// cos and sin of position * frequency.
__device__ __forceinline__ float2 rope_angle(int32_t pos, uint64_t turn) {
    const int64_t x = (int64_t)((uint64_t)(int64_t)pos * turn);       // modulo one turn
    const float t = (float)(int32_t)(x >> 32) * 0x1p-31f;             // in half turns
    float2 r;
    sincospif(t, &r.y, &r.x);
    return r;
}

template <typename T>
struct RopeVec;
template <>
struct RopeVec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const uint4& u, float* f) {
        f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 store(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <>
struct RopeVec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const uint4& u, float* f) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // rounded once, from the 32-bit result
    static __device__ __forceinline__ uint4 store(const float* f) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};

// Where pair i's angle lies in shared memory: the angles that one instruction of a warp reads (the same
// element of neighbouring vectors) side by side.  PV: pairs of a vector.
template <int PV>
__device__ __forceinline__ int rope_slot(int i) {
    return i % PV * (ROPE_MAX_PAIRS / PV) + i / PV;
}

template <typename T, int D>
__global__ void __launch_bounds__(ROPE_THREADS) kv_pool_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int VE = RopeVec<T>::N;          // elements per 16-byte vector
    constexpr int NU = D / VE / 2;             // vector pairs per head
    __shared__ float2 cs[ROPE_MAX_TOKENS][ROPE_MAX_PAIRS];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t table_blocks = (int64_t)p.batch * p.tiles;
    if ((int64_t)blockIdx.x < table_blocks) {
        kpw_table_tile<ROPE_THREADS, ROPE_PER>((int)(blockIdx.x / p.tiles), blockIdx.x % p.tiles, p.prefix_slots, p.prefix_indptr,
                                     p.new_slots, p.qo_indptr, p.r2t, p.r2t_stride, p.num_slots, 0, p.total, p.status);
        return;
    }
    const int64_t block = blockIdx.x - table_blocks;
    // rows of the batch only: what lies before its first and behind its last request is left alone
    const int64_t first = p.qo_indptr[0], end = p.qo_indptr[p.batch];
    const int64_t lo = max(first, (int64_t)0), hi = min(end, p.total);
    if (block == 0 && threadIdx.x == 0 && (end > p.total || first < 0 || end < first)) report(p.status, RX_DEV_BAD_LENGTH);
    const int64_t t0 = block * p.tokens;
    if (t0 >= hi) return;                                         // in 64 bits: `end` may be any number
    const int nt = (int)min((int64_t)p.tokens, hi - t0);          // hi - t0 is in [1, total]
    if (t0 + nt <= lo) return;
    const int qu = p.q ? p.hq * NU : 0;                           // units of a token's queries,
    const int ku = p.hkv * NU;                                    // of its keys, and of its values
    const int per = qu + ku + (p.new_slots ? ku : 0);
    const int units = per * nt;
    const int half = p.pairs / VE;                                // vectors in half the rotated width

    for (int u0 = threadIdx.x; u0 - (int)threadIdx.x < units; u0 += ROPE_THREADS * ROPE_UNITS) {
        uint4 x[ROPE_UNITS][2];
        int tok[ROPE_UNITS], rest[ROPE_UNITS], va[ROPE_UNITS], vb[ROPE_UNITS];
#pragma unroll
        for (int i = 0; i < ROPE_UNITS; ++i) {
            const int u = u0 + i * ROPE_THREADS;
            int t = 0, r = u;
#pragma unroll
            for (int j = 1; j < ROPE_MAX_TOKENS; ++j)
                if (u >= j * per) t = j, r = u - j * per;
            tok[i] = u < units && t0 + t >= lo ? t : -1;
            rest[i] = r;
            const int j = r & (NU - 1);
            if (p.interleaved || j >= half)
                va[i] = 2 * j, vb[i] = 2 * j + 1;
            else
                va[i] = j, vb[i] = j + half;
            if (tok[i] < 0) continue;
            const int64_t row = t0 + t;
            const T* src = r < qu        ? (const T*)p.q + row * p.q_stride + (r / NU) * D
                           : r < qu + ku ? (const T*)p.k + row * p.k_stride + ((r - qu) / NU) * D
                                         : (const T*)p.v + row * p.v_stride + ((r - qu - ku) / NU) * D;
            x[i][0] = reinterpret_cast<const uint4*>(src)[va[i]];
            x[i][1] = reinterpret_cast<const uint4*>(src)[vb[i]];
        }
        if (u0 == (int)threadIdx.x) {       // once, under the first loads
            for (int a = threadIdx.x; a < nt * p.pairs; a += ROPE_THREADS) {
                const int t = a / p.pairs, i = a - t * p.pairs;
                if (t0 + t >= lo)
                    cs[t][p.interleaved ? rope_slot<VE / 2>(i) : rope_slot<VE>(i)] = rope_angle(p.positions[p.axis[i] * p.pos_stride + t0 + t], p.turns[i]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < ROPE_UNITS; ++i) {
            if (tok[i] < 0) continue;
            const int r = rest[i];
            const int64_t row = t0 + tok[i];
            if (r < qu + ku && (p.interleaved ? va[i] * VE < 2 * p.pairs : va[i] < half)) {
                float a[VE], b[VE];
                RopeVec<T>::load(x[i][0], a);
                RopeVec<T>::load(x[i][1], b);
                const float2* c = cs[tok[i]];
                if (p.interleaved) {        // neighbouring channels: both vectors hold whole pairs
#pragma unroll
                    for (int e = 0; e < VE; e += 2) {
                        const float2 ca = c[rope_slot<VE / 2>((va[i] * VE + e) / 2)], cb = c[rope_slot<VE / 2>((vb[i] * VE + e) / 2)];
                        const float a0 = a[e], b0 = b[e];
                        a[e] = a0 * ca.x - a[e + 1] * ca.y;
                        a[e + 1] = a[e + 1] * ca.x + a0 * ca.y;
                        b[e] = b0 * cb.x - b[e + 1] * cb.y;
                        b[e + 1] = b[e + 1] * cb.x + b0 * cb.y;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float2 ce = c[rope_slot<VE>(va[i] * VE + e)];
                        const float a0 = a[e];
                        a[e] = a0 * ce.x - b[e] * ce.y;
                        b[e] = b[e] * ce.x + a0 * ce.y;
                    }
                }
                x[i][0] = RopeVec<T>::store(a);
                x[i][1] = RopeVec<T>::store(b);
            }
            if (r < qu) {
                uint4* o = reinterpret_cast<uint4*>((T*)p.q_out + row * p.q_out_stride + (r / NU) * D);
                o[va[i]] = x[i][0];
                o[vb[i]] = x[i][1];
                continue;
            }
            const bool key = r < qu + ku;
            const int h = key ? (r - qu) / NU : (r - qu - ku) / NU;
            if (key && p.k_out) {
                uint4* o = reinterpret_cast<uint4*>((T*)p.k_out + row * p.k_out_stride + h * D);
                o[va[i]] = x[i][0];
                o[vb[i]] = x[i][1];
            }
            if (p.new_slots) {
                const int32_t s = p.new_slots[row];
                if (s < 0 || s >= p.num_slots) {
                    if (r == qu) report(p.status, RX_DEV_BAD_SLOT);
                    continue;
                }
                uint4* o = reinterpret_cast<uint4*>((T*)(key ? p.k_pool : p.v_pool) + ((int64_t)s * p.hkv + h) * D);
                o[va[i]] = x[i][0];
                o[vb[i]] = x[i][1];
            }
        }
    }
}

// The frequencies as fractions of a turn, and the axis of each pair.
static int rope_table(const rx_rope_desc* r, int head_dim, RopeParams& p) {
    RX_REQUIRE(r->n_axes >= 1 && r->n_axes <= RX_ROPE_MAX_AXES, "kv_pool_write_rope: %d position axes (1 to %d)", r->n_axes,
               RX_ROPE_MAX_AXES);
    RX_REQUIRE(r->rot_dim >= 16 && r->rot_dim <= head_dim && r->rot_dim % 16 == 0,
               "kv_pool_write_rope: rot_dim %d is not a multiple of 16 up to head_dim", r->rot_dim);
    const int pairs = r->rot_dim / 2;
    int64_t sum = 0;
    int left[RX_ROPE_MAX_AXES] = {};
    for (int a = 0; a < r->n_axes; ++a) {
        RX_REQUIRE(r->sections[a] >= 0, "kv_pool_write_rope: negative section");
        sum += left[a] = r->sections[a];
    }
    RX_REQUIRE(sum == pairs, "kv_pool_write_rope: sections hold %lld pairs, rot_dim %d has %d", (long long)sum, r->rot_dim, pairs);
    RX_REQUIRE(r->inv_freq || (std::isfinite(r->base) && r->base > 0), "kv_pool_write_rope: base must be positive and finite");
    p.pairs = pairs;
    p.interleaved = r->interleaved ? 1 : 0;
    for (int i = 0, a = 0; i < pairs; ++i) {
        while (left[a] == 0) a = (a + 1) % r->n_axes;     // blocks: the next axis; in turn: one that has its share drops out
        p.axis[i] = (uint8_t)a;
        --left[a];
        if (r->cyclic) a = (a + 1) % r->n_axes;
        const double w = r->inv_freq ? r->inv_freq[i] : std::pow(r->base, -2.0 * i / r->rot_dim);
        RX_REQUIRE(std::isfinite(w), "kv_pool_write_rope: frequency %d is not finite", i);
        // Turns per position; whole turns do not matter.  Of the magnitude, the sign by the integers' wrap:
        // 1 - f would round a small f away.
        double f = std::fabs(w) / 6.283185307179586476925287;
        f -= std::floor(f);
        const uint64_t turn = (uint64_t)std::ldexp(f, 64);
        p.turns[i] = w < 0 ? 0 - turn : turn;
    }
    return RX_OK;
}

template <typename T, int D>
static void launch_rope(const RopeParams& p, unsigned grid, cudaStream_t stream) {
    launch_pdl(kv_pool_rope_kernel<T, D>, grid, ROPE_THREADS, 0, stream, p);   // an error shows in cudaGetLastError
}

}  // namespace rx

using namespace rx;

extern "C" int kv_pool_write_rope(const rx_attn_desc* desc, const rx_rope_desc* rope, int32_t batch,
                                  const int32_t* d_prefix_slots, const int64_t* d_prefix_indptr, const int32_t* d_new_slots,
                                  const int64_t* d_qo_indptr, const int32_t* d_positions, int64_t pos_stride, const void* d_q,
                                  int64_t q_stride, const void* d_k_new, int64_t k_stride, const void* d_v_new, int64_t v_stride,
                                  void* d_q_out, int64_t q_out_stride, void* d_k_out, int64_t k_out_stride, void* d_k_pool,
                                  void* d_v_pool, int32_t* d_req_to_token, int64_t r2t_stride, int64_t total_new,
                                  int32_t* d_status, void* stream) {
    RX_TRACE("kv_pool_write_rope");
    RX_REQUIRE(desc && rope && batch >= 0 && total_new >= 0 && r2t_stride >= 0, "kv_pool_write_rope: bad arguments");
    RX_REQUIRE(desc->dtype == RX_F32 || desc->dtype == RX_BF16, "kv_pool_write_rope: unknown dtype %d", desc->dtype);
    RX_REQUIRE(desc->head_dim == 64 || desc->head_dim == 128, "kv_pool_write_rope: head_dim must be 64 or 128");
    RX_REQUIRE(desc->hkv > 0 && desc->hkv <= 4096 && desc->num_slots > 0 && (!d_q || (desc->hq > 0 && desc->hq <= 4096)),
               "kv_pool_write_rope: bad shape");
    RopeParams p{};
    const int rc = rope_table(rope, desc->head_dim, p);
    if (rc != RX_OK) return rc;
    if (batch == 0 || (total_new == 0 && !d_req_to_token)) return RX_OK;
    const int64_t elt = desc->dtype == RX_F32 ? 4 : 2, kv_row = (int64_t)desc->hkv * desc->head_dim,
                  q_row = (int64_t)desc->hq * desc->head_dim;
    RX_REQUIRE(d_qo_indptr, "kv_pool_write_rope: null device pointer");
    RX_REQUIRE(!d_req_to_token || (d_prefix_indptr && d_new_slots), "kv_pool_write_rope: a slot table needs the slot lists");
    RX_REQUIRE(total_new == 0 || (d_positions && d_k_new && pos_stride >= total_new),
               "kv_pool_write_rope: null device pointer or too short a row of positions");
    RX_REQUIRE(total_new == 0 || !d_new_slots || (d_v_new && d_k_pool && d_v_pool), "kv_pool_write_rope: null device pointer");
    RX_REQUIRE(total_new == 0 || !d_q == !d_q_out, "kv_pool_write_rope: q and q_out go together");
    RX_REQUIRE(total_new == 0 || d_new_slots || d_k_out, "kv_pool_write_rope: neither slots nor k_out to write the keys to");
    const struct {
        const void* p;
        int64_t stride, row;
    } rows[] = {{d_q, q_stride, q_row},       {d_k_new, k_stride, kv_row},   {d_v_new, v_stride, kv_row},
                {d_q_out, q_out_stride, q_row}, {d_k_out, k_out_stride, kv_row}, {d_k_pool, kv_row, kv_row},
                {d_v_pool, kv_row, kv_row}};
    for (const auto& r : rows)
        RX_REQUIRE(!r.p || (((uintptr_t)r.p & 15) == 0 && r.stride * elt % 16 == 0 && r.stride >= r.row),
                   "kv_pool_write_rope: rows must be 16-byte aligned and at least a row apart");
    // turned in place, or into another buffer: rows of one that lie across rows of the other would be read after they change
    RX_REQUIRE((d_q != d_q_out || q_stride == q_out_stride) && (d_k_new != d_k_out || k_stride == k_out_stride),
               "kv_pool_write_rope: in place needs the same row stride");
    const int64_t tiles = d_req_to_token ? std::max<int64_t>(1, (r2t_stride + ROPE_TILE - 1) / ROPE_TILE) : 0;
    // Two tokens a block share the block's set-up (24 image prompts: 49.7 us; one a block 60, four 51.6);
    // one a block while that leaves fewer than two blocks an SM.
    p.tokens = total_new >= 2 * 152 * ROPE_MAX_TOKENS ? ROPE_MAX_TOKENS : 1;
    const int64_t grid = (int64_t)batch * tiles + (total_new + p.tokens - 1) / p.tokens;
    RX_REQUIRE(grid < (1ll << 31) && tiles < (1ll << 31), "kv_pool_write_rope: batch, stride or rows too large");
    p.batch = batch;
    p.tiles = (int32_t)tiles;
    p.prefix_slots = d_prefix_slots;
    p.prefix_indptr = d_prefix_indptr;
    p.new_slots = d_new_slots;
    p.qo_indptr = d_qo_indptr;
    p.positions = d_positions;
    p.pos_stride = pos_stride;
    p.q = d_q;
    p.k = d_k_new;
    p.v = d_v_new;
    p.q_out = d_q_out;
    p.k_out = d_k_out;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.k_pool = d_k_pool;
    p.v_pool = d_v_pool;
    p.r2t = d_req_to_token;
    p.r2t_stride = r2t_stride;
    p.num_slots = desc->num_slots;
    p.total = total_new;
    p.hq = desc->hq;
    p.hkv = desc->hkv;
    p.status = d_status;
    cudaStream_t s = (cudaStream_t)stream;
    if (desc->dtype == RX_F32)
        desc->head_dim == 128 ? launch_rope<float, 128>(p, (unsigned)grid, s) : launch_rope<float, 64>(p, (unsigned)grid, s);
    else
        desc->head_dim == 128 ? launch_rope<__nv_bfloat16, 128>(p, (unsigned)grid, s)
                              : launch_rope<__nv_bfloat16, 64>(p, (unsigned)grid, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("kv_pool_write_rope: launch failed: %s", cudaGetErrorString(e));
        return RX_ECUDA;
    }
    return RX_OK;
}
