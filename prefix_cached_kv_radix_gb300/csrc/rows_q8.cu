// Attention of few rows over 8-bit pools, split over the keys: decode, and prompts of few new tokens.
//
// The rows are (token, query head) pairs of one request and kv head, the head fastest, in tiles of 8 NT; decode is a
// request's one token at position L - 1.  With codes kc, vc and scales ks, vs of a key j,
//   x_j = c ks_j (q . kc_j),  y_j = x_j + log2 vs_j     (c = scale log2 e)
//   o = sum_j 2^y_j vc_j / sum_j 2^x_j,
// each sum over its own running maximum: vs enters the exponent, so that what is weighed and rounded to 16 bits is 2^(y_j - max y)
// next to the largest term of o, however far apart the rows' scales are.  For f32 rows only the exponent of vs = v 2^e does,
// 1/2 <= v < 1: a logarithm of 32 bits is off by up to 2^-18.  The sums' references are then the maxima rounded up to whole
// numbers, so that x_j - (max y - e_j) loses nothing of x_j (errors of 3e-7 to 5e-7 of the norm; with the logarithm
// 5e-7 to 1.1e-6, and 3e-6 at scales of 2^-110).
//
// A CTA of eight warps takes a run of a request's keys, a row tile and 1, 2, 4 or 8 neighbouring kv heads: a warp a head, or 8, 4, 2
// warps sharing one, 16 keys of a stage each.  The heads of a slot lie side by side in the pools, so a stage is
// gathered (16-byte cp.async, three stages deep) in pieces of up to 1 KB: slots are scattered, and pieces of 128 bytes, a head
// a CTA, cost a quarter of the bandwidth.  Short contexts are a CTA's each, whole.  Else the stages of all requests, one
// after another, are shared out evenly over the CTAs that are resident at a time (with chunks of one size, the last round
// of CTAs left SMs idle for a third of the time), and rows that a border cuts are merged from normalised parts by a second kernel.
// S^T = K Q^T with the keys in M of m16n8k16, then O^T += V^T P^T.  Codes become f16 in registers, where they are exact
// (int8 and e4m3 both): K fragments by ldmatrix over 16-byte rows, four neighbouring channels a lane, which the query
// fragments follow; V by ldmatrix.trans over byte pairs, whose two channels are parted by the byte permutation that
// widens them.  Queries are f16 after a power of two per row that brings the row's largest to 2^14 (bf16 is exact in that
// down to 2^-29 of the largest); f32 rows' queries and weights are two f16 parts each, 22 bits.
// Bound by HBM: 2 d + 8 bytes a key and kv head, read once.  Measured: 256 requests of 1024-8192 keys (32/8 heads x 128,
// e4m3) 389 us, 91 % of the copy rate; two of 131071 (64/8) 102.5 us, 73 %: the launch, the first loads and the merge
// (10 us) are a fifth of it; 64 of 441 (12 heads x 64, int8) 19.5 us, of which a CTA's one chain of length, slots, codes
// and joining is most.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "kv_q8.cuh"
#include "radix_attn.h"
#include "rx_common.h"
#include "rx_device.cuh"
#include "rx_launch.h"
#include "rx_q8.h"
#include "share_out.cuh"

namespace rx {

constexpr int RQ_THREADS = 256;
constexpr int RQ_WARPS = RQ_THREADS / 32;
constexpr int RQ_NS = 3;              // stages
constexpr int RQ_RUN = 512;           // keys whose slots are read at a time: two stages at least
constexpr int RQ_CTAS = 152 * 2;      // most CTAs that stages are shared out to
constexpr float RQ_LOG2E = 1.4426950408889634f, RQ_LN2 = 0.6931471805599453f;
constexpr float RQ_TOP = 15.f;        // a row's largest weight is at most 2^15 in f16

template <int D>
struct RowsLayout {
    static constexpr int SUB = 128 / D, KEYS = 16 * SUB;               // tiles of 16 keys, and keys, of a warp's stage
    static constexpr int CODES = KEYS * D;                             // one pool's codes of it
    static constexpr int WARP = 2 * CODES + KEYS * 8;                  // K, V, scales
    static constexpr int STAGE = RQ_WARPS * WARP;
    static constexpr int LIST = RQ_NS * STAGE;                         // slots of two runs of RQ_RUN keys
    static constexpr int BYTES = LIST + 2 * RQ_RUN * 4;
    static constexpr int RS = D + 4;                                   // floats between rows that are joined
    // eight warps' 8 rows, their statistics, weights and each row's lse
    static constexpr int JOIN = RQ_WARPS * 8 * (RS + 5) * 4;
    static_assert(JOIN <= LIST, "the ring holds what is joined");
};

// CTAs an SM holds: registers.
constexpr int rows_a_sm(bool f32, int D, int nt) { return nt > 1 || (f32 && D == 128) ? 1 : 2; }
template <typename T, int D, int NT>
constexpr int rows_a_sm() { return rows_a_sm(sizeof(T) == 4, D, NT); }

// 16-byte chunk c of key row `key`: rows of 128 bytes, or two of 64 to a line, so that 8 rows' chunks lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t code_at(int key, int c) {
    return D == 128 ? (uint32_t)(key * 128 + ((c ^ (key & 7)) << 4)) : (uint32_t)(key * 64 + ((c ^ ((key >> 1) & 3)) << 4));
}

// With the neighbouring 32-byte sector: scales of a slot's other heads, which other warps want at about the same time.
__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global.L2::64B [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// D(16x8 fp32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// What is left of a pair after its f16 part.
__device__ __forceinline__ uint32_t pack_rest_f16x2(float lo, float hi, uint32_t part) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&part));
    return pack_f16x2(lo - p.x, hi - p.y);
}

// Off by 2^-22 of itself, 2^-15 at most: bf16 rows' weights are rounded by 2^-11.
__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x = part 2^power, part in [1/2, 1); what is no positive normal number is its own part, of power 0.
__device__ __forceinline__ void split_scale(float x, float& part, float& power) {
    const uint32_t bits = __float_as_uint(x), e = bits >> 23;
    const bool normal = e - 1u < 254u;
    part = normal ? __uint_as_float((bits & 0x7fffffu) | 0x3f000000u) : x;
    power = normal ? (float)((int)e - 126) : 0.f;
}

struct RowsParams {
    const void* q;
    const int64_t* qo_indptr;         // extend only
    const int32_t* prefix_lens;       // extend only
    const int32_t* kv_lens;           // decode only
    const int32_t* r2t;
    int64_t stride, num_slots;
    Q8Pools pools;
    int32_t batch, hq, hkv, group;
    int32_t max_qo_len, max_kv_len;
    int32_t tiles;                    // row tiles
    int32_t shared;                   // 1: stages shared out over the CTAs; 0: a CTA a (request, row tile, group of heads)
    int32_t hb;                       // log2 of the kv heads a CTA takes
    float scale_log2;
    void* out;
    float* lse;
    float* part_o;                    // [CTAs][2][heads of a CTA][rows of a tile][D], normalised
    float* part_lse;                  // base 2
    const int32_t* shared_of;         // decode with shared runs: leading keys that are not read here (null: none),
    const float* shared_o;            // and their part of the rows [batch * hq][D], normalised
    const float* shared_lse;          // base 2
    int4* meta;                       // [CTAs][2]: request (-1: no part), row tile, first head, whether its keys end here
    int32_t* status;
};

// A row's part from a shared run, if it has one, joined to its own: two factors, of the row's own and of the run's, and
// the log-sum-exp of both.
__device__ __forceinline__ float2 join_shared(const RowsParams& p, int64_t at, int64_t request, float& lse) {
    if (p.shared_of[request] == 0) return make_float2(1.f, 0.f);
    const float other = p.shared_lse[at], M = fmaxf(lse, other), ref = M == -INFINITY ? 0.f : M;
    const float a = exp2f(lse - ref), b = exp2f(other - ref), sum = a + b;
    if (sum == 0.f) return make_float2(1.f, 0.f);
    lse = M + log2f(sum);
    return make_float2(a / sum, b / sum);
}

// A request's rows: where its first is, how many tokens, and how many keys lie before them; false where there is none to do.
template <bool RUNS>
__device__ __forceinline__ bool rows_of(const RowsParams& p, int b, bool tell, int64_t& q0, int& n, int& before) {
    if (p.kv_lens) {
        const int32_t L = p.kv_lens[b];
        q0 = b, n = 1, before = L - 1 - (RUNS ? p.shared_of[b] : 0);
        if (L >= 0 && L <= p.max_kv_len && L <= p.stride) return true;
    } else {
        q0 = p.qo_indptr[b];
        const int64_t m = p.qo_indptr[b + 1] - q0, P = p.prefix_lens[b];
        if (m == 0) return false;
        n = (int)m, before = (int)P;
        if (q0 >= 0 && m > 0 && m <= p.max_qo_len && P >= 0 && P + m <= p.stride && P + m <= p.max_kv_len) return true;
    }
    if (tell) report(p.status, RX_DEV_BAD_LENGTH);
    return false;
}

// Stages of a row tile (one at least: a row of no keys is written too), and of all tiles and groups of heads of a request.
__device__ __forceinline__ int tile_stages(const RowsParams& p, int n, int before, int tile, int rows_a_tile, int span) {
    const int last = min((tile + 1) * rows_a_tile, n * p.group) - 1;
    return max(before + last / p.group + span, span) / span;
}

template <bool RUNS>
__device__ __forceinline__ int64_t request_stages(const RowsParams& p, int b, bool tell, int rows_a_tile, int span) {
    int64_t q0, sum = 0;
    int n, before;
    if (!rows_of<RUNS>(p, b, tell, q0, n, before)) return 0;
    for (int t = 0; t * rows_a_tile < n * p.group; ++t) sum += tile_stages(p, n, before, t, rows_a_tile, span);
    return sum * (p.hkv >> p.hb);
}

template <typename T>
__device__ __forceinline__ void store_row2(T* p, float a, float b);
template <>
__device__ __forceinline__ void store_row2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
template <>
__device__ __forceinline__ void store_row2(__nv_bfloat16* p, float a, float b) { *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(a, b); }

// RUNS: some requests' leading keys are shared runs, not read here.
template <typename T, int D, int FMT, int NT, bool RUNS>
__global__ void __launch_bounds__(RQ_THREADS, rows_a_sm<T, D, NT>()) rows_q8_kernel(const __grid_constant__ RowsParams p) {
    using LY = RowsLayout<D>;
    constexpr bool TWO = std::is_same<T, float>::value;     // two f16 parts
    constexpr int KS = D / 16;                              // 16-byte chunks of a row: steps of K, and of V's M
    constexpr int SUB = LY::SUB, KEYS = LY::KEYS;
    constexpr int CPT = RQ_WARPS * KEYS * KS / RQ_THREADS;    // copies per thread, stage and pool
    constexpr int WPI = RQ_THREADS / 32;
    extern __shared__ __align__(1024) unsigned char smem[];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, t4 = lane & 3, r8 = lane >> 2;
    const int HB = 1 << p.hb, ways = WPI >> p.hb, way = warp >> p.hb, span = KEYS * ways;      // span: keys of a stage
    constexpr int RT = 8 * NT;                                         // rows of a tile
    const int G = p.group, groups = p.hkv >> p.hb;
    __shared__ int64_t share[RQ_WARPS + 4];
    int b, tile, gi, s0 = 0;             // the piece: request, row tile, group of heads, first stage
    int64_t left = 1;                    // stages of this CTA's part
    if (p.shared) {
        auto locate = [&](int r, int64_t at, int& t, int& gr, int& stages) {       // stage `at` of request r's; returns the tile's
            int64_t q;
            int m, bf;
            rows_of<RUNS>(p, r, false, q, m, bf);
            for (t = 0;; ++t) {
                stages = tile_stages(p, m, bf, t, RT, span);
                if (at < (int64_t)stages * groups) break;
                at -= (int64_t)stages * groups;
            }
            gr = (int)(at / stages);
            return (int)(at - (int64_t)gr * stages);
        };
        share_out<RQ_THREADS>(
            p.batch, 4, share, share + RQ_WARPS, [&](int r, bool tell) { return request_stages<RUNS>(p, r, tell, RT, span); },
            [&](int r, int64_t at, int64_t near) {
                int t, gr, stages;
                const int j = locate(r, at, t, gr, stages);
                return at + (j < near ? -j : stages - j < near ? stages - j : 0);
            });
        __syncthreads();
        int64_t at = share[RQ_WARPS] - share[RQ_WARPS + 3];
        left = share[RQ_WARPS + 1] - share[RQ_WARPS];
        b = (int)share[RQ_WARPS + 2];
        if (left > 0) {                  // the border may have moved past the end of its request
            for (int64_t all; b + 1 < p.batch && at >= (all = request_stages<RUNS>(p, b, false, RT, span)); ++b) at -= all;
            int stages;
            s0 = locate(b, at, tile, gi, stages);
        }
    } else {
        uint32_t cell = blockIdx.x;
        gi = (int)(cell % (uint32_t)groups);
        cell /= (uint32_t)groups;
        tile = (int)(cell % (uint32_t)p.tiles);
        b = (int)(cell / (uint32_t)p.tiles);
    }
    int4 told[2] = {make_int4(-1, 0, 0, 0), make_int4(-1, 0, 0, 0)};
    for (; left > 0;) {
    const int g0 = gi << p.hb, g = g0 + (warp & (HB - 1)), R0 = tile * RT, k_begin = s0 * span;
    // What this thread copies of a stage: 16-byte chunk `col` of the heads' HB * D bytes of every key it handles, and one key's scales
    // of one head.
    const int cols = KS << p.hb, col = tid & (cols - 1), row0 = tid / cols, rstep = RQ_THREADS / cols;
    const int skey = tid >> p.hb, shead = tid & (HB - 1);              // scales: key of the stage, head
    // Slots: runs of RQ_RUN keys in shared memory, two in turn.  The first ones are loaded, up to the table's stride, beside the
    // request's lengths, not after them; a later one while the one before it is used.
    const int64_t skip = (RUNS ? p.shared_of[b] : 0) + (int64_t)k_begin;      // keys of the request before this piece's
    const int32_t* table = p.r2t + (int64_t)b * p.stride + skip;
    const int64_t width = p.stride - skip;
    int32_t* list = reinterpret_cast<int32_t*>(smem + LY::LIST);
    int32_t run[2];                      // two keys a thread, of a run on its way to the list
    auto load_run = [&](int i) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int key = i * RQ_RUN + tid + x * RQ_THREADS;
            run[x] = key < width ? table[key] : -1;
        }
    };
    auto keep_run = [&](int i) {
#pragma unroll
        for (int x = 0; x < 2; ++x) list[(i & 1) * RQ_RUN + tid + x * RQ_THREADS] = run[x];
    };
    load_run(0);
    int64_t q0;
    int n, before;
    const bool there = rows_of<RUNS>(p, b, !p.shared && tid == 0 && gi == 0 && tile == 0, q0, n, before);
    const int rows = there ? n * G : 0;
    if (R0 >= rows) break;                                             // no rows of this cell (not shared)
    const int last = min(R0 + RT, rows) - 1, stages = tile_stages(p, n, before, tile, RT, span);
    const int s1 = p.shared ? (int)min((int64_t)stages, s0 + left) : stages;
    const bool whole = s0 == 0 && s1 == stages;
    const int slot = s0 == 0 ? 1 : 0;
    if (!whole) told[slot] = make_int4(b, tile, g0, s1 == stages ? 1 : 0);
    const int nk = min(before + last / G + 1, s1 * span) - k_begin;    // keys of this piece
    const int nstages = max(nk + span - 1, 0) / span;
    const uint32_t ring = smem_u32(smem);
    const int64_t pitch = (int64_t)p.hkv * D;
    const uint8_t* kcol = p.pools.k + (int64_t)g0 * D + col * 16;
    const uint8_t* vcol = p.pools.v + (int64_t)g0 * D + col * 16;
    const float2* scol = p.pools.scales + g0 + shead;
    // Copies stage i, whose slots are in the list; a key behind the last or at a bad slot is zeros, its scales marked (0, -1).
    auto load_stage = [&](int i) {
        const uint32_t buf = ring + (uint32_t)(i % RQ_NS * LY::STAGE);
        const int32_t* slots = list + i * span % (2 * RQ_RUN);
#pragma unroll
        for (int x = 0; x < CPT; ++x) {
            const int key = row0 + x * rstep;
            const int32_t s = slots[key];
            const bool in = i * span + key < nk && s >= 0 && s < p.num_slots;
            const int64_t off = in ? (int64_t)s * pitch : 0;
            const uint32_t to = buf + (uint32_t)(((key / KEYS << p.hb) + col / KS) * LY::WARP) + code_at<D>(key % KEYS, col % KS);
            cp_async_16(to, kcol + off, in ? 16u : 0u);
            cp_async_16(to + LY::CODES, vcol + off, in ? 16u : 0u);
        }
        if (skey < span) {
            const uint32_t to = buf + (uint32_t)(((skey / KEYS << p.hb) + shead) * LY::WARP + 2 * LY::CODES + skey % KEYS * 8);
            const int32_t s = slots[skey];
            const bool in = i * span + skey < nk, good = in && s >= 0 && s < p.num_slots;
            if (in && !good) report(p.status, RX_DEV_BAD_SLOT);
            if (good) cp_async_8(to, scol + (int64_t)(s >> p.pools.shift) * p.hkv);
            else asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(0.f), "f"(-1.f) : "memory");
        }
    };
    const int a_run = RQ_RUN / span;     // stages of a run
    keep_run(0);
    load_run(1);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RQ_NS - 1; ++i) {
        if (i < nstages) load_stage(i);
        cp_async_commit();
    }
    // query fragments: columns of the B operand, row R0 + 8 t + r8, channels 16 s + 4 t4 ..+3; and each accumulator
    // column's factor, scale log2(e) over the row's power of two
    uint32_t qb[NT][TWO ? 2 : 1][KS][2];
    float f[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int R = R0 + 8 * t + r8;
        const bool in = R < rows;
        const T* qr = (const T*)p.q + (in ? ((q0 + R / G) * p.hq + g * G + R % G) * D : 0);
        float x[KS][4];
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if (TWO) {
                const float4 v = in ? *reinterpret_cast<const float4*>((const float*)qr + 16 * s + 4 * t4) : make_float4(0, 0, 0, 0);
                x[s][0] = v.x, x[s][1] = v.y, x[s][2] = v.z, x[s][3] = v.w;
            } else {
                const uint2 v = in ? *reinterpret_cast<const uint2*>((const __nv_bfloat16*)qr + 16 * s + 4 * t4) : make_uint2(0, 0);
                x[s][0] = __uint_as_float(v.x << 16), x[s][1] = __uint_as_float(v.x & 0xffff0000u);
                x[s][2] = __uint_as_float(v.y << 16), x[s][3] = __uint_as_float(v.y & 0xffff0000u);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(x[s][e]) & 0x7fffffffu);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the power of two that brings the largest to [2^14, 2^15), at most 2^126; none for a row that is not finite
        const uint32_t up = top >= 0x7f800000u ? 127u : (uint32_t)min(268 - max((int)(top >> 23), 1), 253);
        const float mul = __uint_as_float(up << 23), undo = __uint_as_float((254u - up) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float a0 = x[s][2 * h] * mul, a1 = x[s][2 * h + 1] * mul;
                qb[t][0][s][h] = pack_f16x2(a0, a1);
                if (TWO) qb[t][TWO ? 1 : 0][s][h] = pack_rest_f16x2(a0, a1, qb[t][0][s][h]);
            }
        const float mine = p.scale_log2 * undo;            // of row r8; the accumulators' columns are rows 2 t4, 2 t4 + 1
        f[t][0] = __shfl_sync(0xffffffffu, mine, 8 * t4);
        f[t][1] = __shfl_sync(0xffffffffu, mine, 8 * t4 + 4);
    }
    // the first key that each of this lane's columns may not see, relative to the chunk
    int end[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) end[t][e] = before + (R0 + 8 * t + 2 * t4 + e) / G + 1 - k_begin;
    const int least = before + R0 / G + 1 - k_begin;                   // every row sees the keys before this

    float o[NT][KS][4];
    float mx[NT][2], l[NT][2], my[NT][2];      // references of x in this lane, the sum, and of y in the warp
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < KS; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
        mx[t][0] = mx[t][1] = my[t][0] = my[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.f;
    }
    keep_run(1);                         // seen after the next barrier; its first stage is copied after that
    for (int it = 0; it < nstages; ++it) {
        cp_async_wait<RQ_NS - 2>();
        __syncthreads();                       // stage `it` is here, of all threads, and the one before it has been read
        const int nx = it + RQ_NS - 1;         // the stage to be copied; the first of a run brings the run after it
        if (nx < nstages) load_stage(nx);
        cp_async_commit();
        if (nx >= a_run) {
            if (nx % a_run == 0) load_run(nx / a_run + 1);
            else if (nx % a_run == 1) keep_run(nx / a_run + 1);
        }
        const int key0 = it * span + way * KEYS;
        if (key0 >= nk) continue;
        const uint32_t kb = ring + (uint32_t)(it % RQ_NS * LY::STAGE + warp * LY::WARP), vb = kb + LY::CODES;
        const int mi = lane >> 3, lrow = (mi & 1) * 8 + (lane & 7);
        float sacc[SUB][NT][4];
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            float sodd[NT][4];                 // of odd chunks: two chains of products
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) sacc[u][t][e] = sodd[t][e] = 0.f;
#pragma unroll
            for (int s = 0; s < KS; s += 2) {
                uint32_t w[4];                 // keys r8, r8 + 8 of chunk s, then of chunk s + 1
                ldmatrix_x4(kb + code_at<D>(16 * u + lrow, s + (mi >> 1)), w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t a[4];
                    q8_to_f16<FMT, false>(w[2 * j], a[0], a[2]);
                    q8_to_f16<FMT, false>(w[2 * j + 1], a[1], a[3]);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < (TWO ? 2 : 1); ++i)
                            mma_f16_16816(j ? sodd[t] : sacc[u][t], a, qb[t][i][s + j][0], qb[t][i][s + j][1]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) sacc[u][t][e] += sodd[t][e];
        }
        float ks[2 * SUB], vp[2 * SUB], lv[2 * SUB];       // of keys 8 i + r8: K's scale, log2 of V's, or its part and exponent
        bool ok[2 * SUB], all_ok = true;
#pragma unroll
        for (int i = 0; i < 2 * SUB; ++i) {
            float vs;
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks[i]), "=f"(vs) : "r"(vb + LY::CODES + r8 * 8 + 64 * i) : "memory");
            ok[i] = vs != -1.f;
            all_ok &= ok[i];
            if (TWO) split_scale(vs, vp[i], lv[i]);
            else lv[i] = fast_log2(vs);
        }
        const bool whole = key0 + KEYS <= least && __all_sync(0xffffffffu, all_ok);     // no key of these is hidden from any row
        uint32_t pb[SUB][NT][TWO ? 2 : 1][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            // (Two forms of one step: with f32's second half after the branch it is 2 % faster, with bf16's there 1 % slower.)
            float x[2 * SUB][2], w[2 * SUB][2], up[2];
            bool moved = false;
            if constexpr (TWO) {
                float m[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float a = mx[t][e];
                    m[e] = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 2 * SUB; ++i) {
                        x[i][e] = sacc[i / 2][t][2 * (i & 1) + e] * (f[t][e] * ks[i]);
                        if (!whole && (key0 + 8 * i + r8 >= end[t][e] || !ok[i])) x[i][e] = -INFINITY;
                        a = fmaxf(a, x[i][e]);
                        m[e] = fmaxf(m[e], x[i][e] + lv[i]);
                    }
                    a = ceilf(a);
                    const float ra = a == -INFINITY ? 0.f : a;
                    l[t][e] *= fast_exp2(mx[t][e] - ra);
#pragma unroll
                    for (int i = 0; i < 2 * SUB; ++i) l[t][e] += fast_exp2(x[i][e] - ra);
                    mx[t][e] = a;
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], off));
                    moved |= m[e] > my[t][e];
                }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float to = fmaxf(ceilf(m[e]), my[t][e]);
                        up[e] = fast_exp2(my[t][e] - (to == -INFINITY ? 0.f : to));
                        my[t][e] = to;
                    }
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[t][i][0] *= up[0];
                        o[t][i][1] *= up[1];
                        o[t][i][2] *= up[0];
                        o[t][i][3] *= up[1];
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float top = (my[t][e] == -INFINITY ? 0.f : my[t][e]) - RQ_TOP;
#pragma unroll
                    for (int i = 0; i < 2 * SUB; ++i) {
                        w[i][e] = fast_exp2(x[i][e] - (top - lv[i])) * vp[i];
                        if (!whole && x[i][e] == -INFINITY) w[i][e] = 0.f;       // hidden, whatever its scale
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float a = mx[t][e], m = -INFINITY, y[2 * SUB];
#pragma unroll
                    for (int i = 0; i < 2 * SUB; ++i) {
                        x[i][e] = sacc[i / 2][t][2 * (i & 1) + e] * (f[t][e] * ks[i]);
                        y[i] = x[i][e] + lv[i];
                        if (!whole && (key0 + 8 * i + r8 >= end[t][e] || !ok[i])) x[i][e] = y[i] = -INFINITY;
                        a = fmaxf(a, x[i][e]);
                        m = fmaxf(m, y[i]);
                    }
                    const float ra = a == -INFINITY ? 0.f : a;
                    l[t][e] *= fast_exp2(mx[t][e] - ra);
#pragma unroll
                    for (int i = 0; i < 2 * SUB; ++i) l[t][e] += fast_exp2(x[i][e] - ra);
                    mx[t][e] = a;
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                    m = fmaxf(m, my[t][e]);
                    const float rm = m == -INFINITY ? 0.f : m;
                    up[e] = fast_exp2(my[t][e] - rm);
                    moved |= m != my[t][e];
                    my[t][e] = m;
#pragma unroll
                    for (int i = 0; i < 2 * SUB; ++i) w[i][e] = fast_exp2(y[i] - (rm - RQ_TOP));
                }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[t][i][0] *= up[0];
                        o[t][i][1] *= up[1];
                        o[t][i][2] *= up[0];
                        o[t][i][3] *= up[1];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2 * SUB; ++i) {
                const uint32_t h = pack_f16x2(w[i][0], w[i][1]);
                pb[i / 2][t][0][i & 1] = movmatrix_trans(h);
                if (TWO) pb[i / 2][t][TWO ? 1 : 0][i & 1] = movmatrix_trans(pack_rest_f16x2(w[i][0], w[i][1], h));
            }
        }
        // f32 rows: a stage's products in accumulators of their own, added to the sum with rounding.  The tensor core cuts
        // its sums off, which over up to 1302 keys cost the outputs 6e-7 of their norm; 4e-7 are left, for 3 % of the time.
#pragma unroll
        for (int i = 0; i < KS; i += 2) {
            float part[TWO ? 2 : 1][NT][4];
            if (TWO)
#pragma unroll
                for (int j = 0; j < (TWO ? 2 : 1); ++j)
#pragma unroll
                    for (int t = 0; t < NT; ++t) part[j][t][0] = part[j][t][1] = part[j][t][2] = part[j][t][3] = 0.f;
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t w[4];                 // byte pairs of channels 2 r8, 2 r8 + 1: keys 2 t4, 2 t4 + 1, then those + 8; two chunks
                ldmatrix_x4_trans(vb + code_at<D>(16 * u + lrow, i + (mi >> 1)), w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t a[4];             // rows r8: channel 2 r8, rows r8 + 8: channel 2 r8 + 1
                    q8_to_f16<FMT, true>(w[2 * j], a[0], a[1]);
                    q8_to_f16<FMT, true>(w[2 * j + 1], a[2], a[3]);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int n = 0; n < (TWO ? 2 : 1); ++n)
                            mma_f16_16816(TWO ? part[TWO ? j : 0][t] : o[t][i + j], a, pb[u][t][n][0], pb[u][t][n][1]);
                }
            }
            if (TWO)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[t][i + j][e] += part[TWO ? j : 0][t][e];
        }
    }
    cp_async_wait<0>();

    // A row's channels 2 x, 2 x + 1 to where they belong: the output, or this part.
    auto put = [&](int r, int head, int d, float a0, float a1, float lse, bool with_lse) {
        if (whole) {
            const int R = R0 + r, tok = R / G;
            const int64_t at = (q0 + tok) * p.hq + (g0 + head) * G + R % G;
            if (RUNS) {
                const float2 f = join_shared(p, at, q0, lse);
                if (f.y != 0.f) {
                    const float2 s = *reinterpret_cast<const float2*>(p.shared_o + at * D + d);
                    a0 = a0 * f.x + s.x * f.y, a1 = a1 * f.x + s.y * f.y;
                }
            }
            store_row2((T*)p.out + at * D + d, a0, a1);
            if (with_lse && p.lse) p.lse[at] = lse * RQ_LN2;
        } else {
            const int64_t at = (((int64_t)blockIdx.x * 2 + slot) * HB + head) * RT + r;
            *reinterpret_cast<float2*>(p.part_o + at * D + d) = make_float2(a0, a1);
            if (with_lse) p.part_lse[at] = lse;
        }
    };
    // O is relative to 2^(my - 15), l to 2^mx of its lane.
    float* red_o = reinterpret_cast<float*>(smem);             // warps that share a head: [8 warps][8 rows][RS]
    float* red_m = red_o + RQ_WARPS * 8 * LY::RS;              // mx (then the row's factor), l, my, weight, lse of [8 warps][8 rows]
    constexpr int M = RQ_WARPS * 8;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (R0 + 8 * t >= rows) break;                         // the same for the block
        if (ways > 1) __syncthreads();                         // the ring, or the tile before, is done with
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float m = mx[t][e];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            const float ref = m == -INFINITY ? 0.f : m;
            float s = l[t][e] * fast_exp2(mx[t][e] - ref);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            if (ways == 1) {
                const int r = 8 * t + 2 * t4 + e;
                // two factors, -127 < my - ref <= 128: their product may be below the normal numbers, where the row is not
                const float w = s == 0.f ? 0.f : 0x1p-13f / s, f = exp2f((my[t][e] == -INFINITY ? ref : my[t][e]) - ref - (RQ_TOP - 13.f));
                const float lse = s == 0.f ? -INFINITY : m + log2f(s);
                if (R0 + r < rows)
#pragma unroll
                    for (int i = 0; i < KS; ++i) put(r, warp & (HB - 1), 16 * i + 2 * r8, o[t][i][e] * w * f, o[t][i][e + 2] * w * f, lse, i == 0 && r8 == 0);
                continue;
            }
            if (r8 == 0) {
                red_m[warp * 8 + 2 * t4 + e] = m;
                red_m[M + warp * 8 + 2 * t4 + e] = s;
                red_m[2 * M + warp * 8 + 2 * t4 + e] = my[t][e];
            }
#pragma unroll
            for (int i = 0; i < KS; ++i)
                *reinterpret_cast<float2*>(red_o + (warp * 8 + 2 * t4 + e) * LY::RS + 16 * i + 2 * r8) =
                    make_float2(o[t][i][e], o[t][i][e + 2]);
        }
        if (ways == 1) continue;
        __syncthreads();
        if (tid < 8 * HB) {                                    // a row of a head: entry tid + 8 HB w of warp w
            const int step = 8 * HB;
            float top = -INFINITY, L = 0.f;
            for (int w = 0; w < ways; ++w) top = fmaxf(top, red_m[tid + step * w]);
            const float ref = top == -INFINITY ? 0.f : top;
            for (int w = 0; w < ways; ++w) L += red_m[M + tid + step * w] * exp2f(red_m[tid + step * w] - ref);
            const float inv = L == 0.f ? 0.f : 1.f / L;
            for (int w = 0; w < ways; ++w) red_m[3 * M + tid + step * w] = exp2f(red_m[2 * M + tid + step * w] - ref - (RQ_TOP - 13.f));
            red_m[4 * M + tid] = L == 0.f ? -INFINITY : top + log2f(L);
            red_m[tid] = 0x1p-13f * inv;                       // two factors, as above
        }
        __syncthreads();
        constexpr int HALF = D / 2;
        for (int idx = tid; idx < HB * 8 * HALF; idx += RQ_THREADS) {
            const int hr = idx / HALF, d = 2 * (idx % HALF), r = 8 * t + (hr & 7);
            if (R0 + r >= rows) continue;
            const float f = red_m[hr];
            float a0 = 0.f, a1 = 0.f;
            for (int w = 0; w < ways; ++w) {
                const int at = hr + 8 * HB * w;
                const float wt = red_m[3 * M + at];
                const float2 v = *reinterpret_cast<const float2*>(red_o + at * LY::RS + d);
                a0 += wt * (f * v.x);
                a1 += wt * (f * v.y);
            }
            put(r, hr >> 3, d, a0, a1, red_m[4 * M + hr], d == 0);
        }
    }
    // on to the next group of heads, row tile, request
    left -= p.shared ? s1 - s0 : 1;
    if (left <= 0) break;
    s0 = 0;
    if (++gi == groups) {
        gi = 0;
        if (++tile * RT >= rows) {
            tile = 0;
            do ++b;
            while (b < p.batch && !rows_of<RUNS>(p, b, false, q0, n, before));
            if (b >= p.batch) break;
        }
    }
    __syncthreads();                     // the ring has been read
    }
    if (p.shared && tid < 2) p.meta[blockIdx.x * 2 + tid] = tid == 0 ? told[0] : told[1];
}

// Rows from their parts: blockIdx.x the begun and not ended item, four rows a block with a warp each (WAYS 1), or one row a block
// with all its warps.
template <typename T, int D, int WAYS, bool RUNS>
__global__ void __launch_bounds__(128) rows_q8_merge_kernel(const __grid_constant__ RowsParams p, int rows_a_tile, int ctas) {
    constexpr int E = D / 32;
    __shared__ int list[RQ_CTAS];
    __shared__ uint32_t room[RQ_CTAS];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int count = parts_of<RQ_CTAS>(p.meta, blockIdx.x, ctas, list, room);
    if (count == 0) return;
    const int4 what = p.meta[list[0]];
    int64_t q0;
    int n, before;
    rows_of<RUNS>(p, what.x, false, q0, n, before);
    const int r = blockIdx.y * (4 / WAYS) + (WAYS == 1 ? warp : 0);      // rows of a head, then the next head's
    const int R = what.y * rows_a_tile + r % rows_a_tile;
    if (R >= n * p.group) return;                                        // the same for all who share the row
    float acc[E];
    float lse;
    if constexpr (WAYS == 1) lse = merge_few<D>(list, count, p.part_o, p.part_lse, rows_a_tile << p.hb, r, acc);
    else lse = merge_many<D, RQ_CTAS>(list, count, p.part_o, p.part_lse, rows_a_tile << p.hb, r, acc);
    if (WAYS > 1 && warp != 0) return;
    const int64_t at = (q0 + R / p.group) * p.hq + (what.z + r / rows_a_tile) * p.group + R % p.group;
    const float2 f = RUNS ? join_shared(p, at, q0, lse) : make_float2(1.f, 0.f);
    if (f.y != 0.f)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f.x + p.shared_o[at * D + lane * E + e] * f.y;
    T* row = (T*)p.out + at * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) store_row2(row + e, acc[e], acc[e + 1]);
    if (p.lse && lane == 0) p.lse[at] = lse * RQ_LN2;
}

template <typename T, int D, int FMT, int NT, bool RUNS>
static int launch_tile(const char* fn, const RowsParams& p, unsigned grid, cudaStream_t s) {
    constexpr int smem = RowsLayout<D>::BYTES;
    static PerDeviceOnce attr;
    const int rc = per_device_once(attr, [&] {
        auto* k = rows_q8_kernel<T, D, FMT, NT, RUNS>;
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) (void)cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) {
            set_error("%s: cannot set shared memory size: %s", fn, cudaGetErrorString(e));
            return (int)RX_ECUDA;
        }
        return (int)RX_OK;
    });
    if (rc != RX_OK) return rc;
    launch_pdl(rows_q8_kernel<T, D, FMT, NT, RUNS>, grid, RQ_THREADS, smem, s, p);
    if (p.shared) {
        // few items: each in many parts, so a block a row; many items: a few parts each, a warp a row
        const int64_t items = (int64_t)p.batch * p.tiles * (p.hkv >> p.hb), rows = 8 * NT << p.hb;
        const bool few = items <= 64;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)std::min<int64_t>(items, grid), (unsigned)(few ? rows : rows / 4));
        cfg.blockDim = dim3(128);
        cfg.stream = s;
        cudaLaunchAttribute pdl[1];
        pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        pdl[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = pdl;
        cfg.numAttrs = 1;
        if (few) cudaLaunchKernelEx(&cfg, rows_q8_merge_kernel<T, D, 4, RUNS>, p, 8 * NT, (int)grid);
        else cudaLaunchKernelEx(&cfg, rows_q8_merge_kernel<T, D, 1, RUNS>, p, 8 * NT, (int)grid);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("%s: launch failed: %s", fn, cudaGetErrorString(e));
        return RX_ECUDA;
    }
    return RX_OK;
}

template <typename T, int D, int FMT>
static int launch_fmt(const char* fn, const RowsParams& p, int nt, unsigned grid, cudaStream_t s) {
    if constexpr (!std::is_same<T, float>::value)
        if (p.shared_of) return nt == 1 ? launch_tile<T, D, FMT, 1, true>(fn, p, grid, s) : launch_tile<T, D, FMT, 2, true>(fn, p, grid, s);
    return nt == 1 ? launch_tile<T, D, FMT, 1, false>(fn, p, grid, s) : launch_tile<T, D, FMT, 2, false>(fn, p, grid, s);
}

template <typename T, int D>
static int launch_rows(const char* fn, const RowsParams& p, int nt, int format, unsigned grid, cudaStream_t s) {
    return format == RX_Q8_INT8 ? launch_fmt<T, D, RX_Q8_INT8>(fn, p, nt, grid, s) : launch_fmt<T, D, RX_Q8_E4M3>(fn, p, nt, grid, s);
}

// 8-row tiles that a CTA takes.  Not more than two: four take 255 registers and spill (64 requests with 32 heads to a kv head: 127
// us; by two tiles of two, 70).
static int rows_nt(int64_t rows) { return rows <= 8 ? 1 : 2; }

RowsPlan rows_q8_plan(const rx_attn_desc* d, int32_t batch, int32_t max_qo_len, int32_t max_kv_len) {
    RowsPlan L{};
    const int64_t rows = (int64_t)max_qo_len * (d->hq / d->hkv);
    L.nt = rows_nt(rows);
    L.tiles = (rows + 8 * L.nt - 1) / (8 * L.nt);
    const int a_sm = rows_a_sm(d->dtype == RX_F32, d->head_dim, L.nt);
    int most = 3;
    while (most > 0 && d->hkv % (1 << most) != 0) --most;
    const int64_t slots = 152 * a_sm;
    const size_t parts = (size_t)slots * 2 * (8 * L.nt << most);       // rows
    L.lse_at = parts * d->head_dim * sizeof(float);
    L.meta_at = L.lse_at + parts * sizeof(float);
    L.room = L.meta_at + (size_t)RQ_CTAS * 2 * sizeof(int4);
    L.ctas = INT64_MAX;                  // what the launch refuses; the products below stay within 63 bits
    if ((double)L.tiles * batch > 0x1p40) return L;
    // Stages shared out evenly, as many neighbouring heads a CTA as there are, up to eight; or a request's whole context to a CTA, with as
    // many heads as take the least time.  In microseconds: a CTA's start and end four, a stage 1.1, or 1.7 with its twice as
    // many keys at 64 channels, a quarter more with two CTAs an SM; sharing out and merging nine, or 26 with two tiles, which
    // are a CTA an SM and more rows a part.  On 136 sizes that it was not fitted to, with a cold L2, it costs ten more than a
    // twentieth over the better of the two, at most a third.  Shared out and whole: decode of 4 requests of up to 1000 keys, 64 heads on 8, 20.5 and 14.9
    // us, of 4 of up to 3000 23.6 and 33.6; 9 f32 prompts of up to 101 over up to 1201 48.8 and 35.6; 40 of up to 9 over up
    // to 5000 74 and 146.
    const double stage = d->head_dim == 64 ? 1.7 : 1.1, both = 1.25 * stage, joining = L.nt == 1 ? 9 : 26;
    const int64_t units = L.tiles * batch;
    auto stages = [&](int hb) { return ((int64_t)max_kv_len << hb) / (16 * (128 / d->head_dim) * RQ_WARPS) + 1; };
    auto whole = [&](int hb) {
        const int64_t ctas = units * (d->hkv >> hb);
        return (double)((ctas + slots - 1) / slots) * (4 + (a_sm > 1 && ctas > 152 ? both : stage) * stages(hb));
    };
    L.hb = most;
    for (int hb = most - 1; hb >= 0; --hb)
        if (whole(hb) < whole(L.hb)) L.hb = hb;
    L.shared = whole(L.hb) > 4 + joining + (a_sm > 1 ? both : stage) * units * (d->hkv >> most) * stages(most) / slots;
    L.ctas = L.shared ? slots : units * (d->hkv >> L.hb);
    if (L.shared) L.hb = most, L.bytes = L.room;
    return L;
}

int rows_q8_launch(const char* fn, const RowsQ8Args& a, const rx_attn_desc* d, const rx_q8_desc* q8, void* ws, size_t ws_bytes,
                   cudaStream_t stream) {
    const RowsPlan L = rows_q8_plan(d, a.batch, a.max_qo_len, a.max_kv_len);
    RX_REQUIRE(L.ctas < (1ll << 31), "%s: too many rows (split the batch)", fn);
    RX_REQUIRE((int64_t)a.max_qo_len * (d->hq / d->hkv) < INT32_MAX - 64, "%s: too many rows in a request", fn);
    RX_REQUIRE(L.bytes == 0 || (ws && ws_bytes >= L.bytes && ((uintptr_t)ws & 255) == 0),
               "%s: a 256-byte aligned workspace of %zu bytes is needed (got %zu)", fn, L.bytes, ws_bytes);
    RowsParams p{};
    p.q = a.q;
    p.qo_indptr = a.qo_indptr;
    p.prefix_lens = a.prefix_lens;
    p.kv_lens = a.kv_lens;
    p.r2t = a.r2t;
    p.stride = a.stride;
    p.num_slots = d->num_slots;
    p.pools = {a.k_pool, a.v_pool, a.scales, q8_shift(q8)};
    p.batch = a.batch;
    p.hq = d->hq;
    p.hkv = d->hkv;
    p.group = d->hq / d->hkv;
    p.max_qo_len = a.max_qo_len;
    p.max_kv_len = a.max_kv_len;
    p.tiles = (int32_t)L.tiles;
    p.shared = L.shared ? 1 : 0;
    p.hb = L.hb;
    p.scale_log2 = d->scale * RQ_LOG2E;
    p.out = a.out;
    p.lse = a.lse;
    p.part_o = (float*)ws;
    p.part_lse = (float*)((unsigned char*)ws + L.lse_at);
    p.meta = (int4*)((unsigned char*)ws + L.meta_at);
    p.shared_of = a.shared_of;
    p.shared_o = a.shared_o;
    p.shared_lse = a.shared_lse;
    p.status = a.status;
    if (d->dtype == RX_F32)
        return d->head_dim == 128 ? launch_rows<float, 128>(fn, p, L.nt, q8->format, (unsigned)L.ctas, stream)
                                  : launch_rows<float, 64>(fn, p, L.nt, q8->format, (unsigned)L.ctas, stream);
    return d->head_dim == 128 ? launch_rows<__nv_bfloat16, 128>(fn, p, L.nt, q8->format, (unsigned)L.ctas, stream)
                              : launch_rows<__nv_bfloat16, 64>(fn, p, L.nt, q8->format, (unsigned)L.ctas, stream);
}

}  // namespace rx
