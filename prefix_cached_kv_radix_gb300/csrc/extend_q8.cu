// Extend attention over 8-bit pools on tcgen05 tensor cores: prompts of many new tokens (bf16 rows).
//
// Row i of request b attends keys 0 .. P_b + i, codes kc, vc with scales ks, vs:
//   x_j = scale log2(e) ks_j (q . kc_j),  P_j = 2^(x_j - m),  l += P_j,  O += bf16(P_j vs_j) vc_j,  o = O / l,
// m the row's running reference (moved when the maximum grows by more than 2^8).  Codes are exact in bf16, so the products
// are those of bf16 rows and the scales stay in 32 bits; P_j vs_j is rounded to bf16 for the tensor core (at
// most 2^-8 of it, as the bf16 kernel rounds P_j), l sums the unrounded P_j, o is rounded once.
//
// A work item is a request's kv head and 256 packed rows (row = token * G + query head of the group) in two Q tiles that share
// each K/V tile of 128 keys.  What is shared out is not items but the K/V tiles of all items, one after
// another: CTA i of 152 takes the i-th equal part of them, so that long and short requests, and few rows over a long
// context, fill the GPU alike without a counter in memory.  An item that a border cuts is finished from normalised
// parts in the workspace by a second kernel.  (Borders close to an item's end move there.)  Roles (512 threads):
//   warp 0       items in order, handed on through a ring in shared memory, and their Q tiles
//   warp 1       issues the tcgen05.mma: O_t += P_t(j) V(j) in two halves, then at once S_t(j+1) = Q_t K(j+1)^T
//   warps 2, 3, 12-15  K/V tiles: codes by 16-byte loads through the slot table, a tile ahead (K's by cp.async, V's in
//                registers), widened to bf16 and stored in the 128B-swizzled layout that tcgen05 reads; the keys' scales beside
//                the V tile
//   warps 4-7, 8-11  softmax of Q tile 0 and 1, in the tensor core's fragment layout, and the item's output
// Bound by the tensor core and the softmax taking turns.  4 prompts of 512 over 16384 (64/8 heads x 128): int8 1205 us, 927
// TFLOP/s.  A pair of Q tiles and a K/V tile take some 4900 clocks: the products 2150 of them, either Q tile's softmax
// 2700 from its scores to its last weights (both together, they use half the issue slots), and the next scores wait for
// both.  Without widening and storing the codes at all it would be 971 TFLOP/s (e4m3, of 909), so that is not what bounds it.  Tried and
// slower: scores and weights in halves of 64 keys with columns of their own (700: products of 64 columns keep the tensor core
// waiting for their rows), softmax warpgroups in strict turns (800), pairs of CTAs that widen half a tile each and copy it
// to the other (567), V's products without waiting for the next K tile (840).
// TMEM columns: S0/P0 [0,128) S1/P1 [128,256) O0 [256,256+D) O1 after.  Every wait is bounded; on time-out the kernel
// records RX_DEV_TIMEOUT, waits for its copies, frees TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "kv_q8.cuh"
#include "prompt_wait.cuh"
#include "radix_attn.h"
#include "rx_common.h"
#include "rx_device.cuh"
#include "rx_launch.h"
#include "rx_q8.h"
#include "share_out.cuh"
#include "tc_issue.cuh"

namespace rx {

constexpr int EQ_BN = 128;             // keys per K/V tile
constexpr int EQ_THREADS = 512;
constexpr int EQ_ROWS = 256;           // packed rows of an item
constexpr int EQ_CTAS = 152;
constexpr int EQ_RING = 4;             // items in flight between the roles
constexpr int EQ_CONSUMERS = 15;       // MMA warp, six converter warps, eight softmax warps
constexpr int EQ_CONV = 192;           // converter threads
// 168 / 88 registers: 16 prompts of 1024 over 1000, 12 heads x 64, 188 us, 178 so; 184 / 72 1427 us instead of 1205 above (spills)
constexpr uint32_t EQ_REGS_SOFTMAX = 176, EQ_REGS_OTHER = 80, EQ_REGS_LAUNCH = 128;   // 2*128*80 + 2*128*176 = 512*128
constexpr float EQ_LOG2E = 1.4426950408889634f, EQ_LN2 = 0.6931471805599453f;
constexpr float EQ_RESCALE = 8.0f;     // log2 units

struct ExtendQ8Params {
    const __nv_bfloat16* q;
    const int64_t* qo_indptr;
    const int32_t* prefix_lens;
    const int32_t* r2t;
    int64_t stride, num_slots;
    Q8Pools pools;
    __nv_bfloat16* out;
    float* lse;
    int32_t batch, hq, hkv, group;
    int32_t max_qo_len, max_kv_len;
    float scale_log2;
    int32_t* status;
    float* part_o;                     // [CTAs][2][EQ_ROWS][D], normalised
    float* part_lse;                   // [CTAs][2][EQ_ROWS], base 2
    int4* meta;                        // [CTAs][2]: request (-1: no part), kv head, first row, whether the item ends here
    // Shared runs of a decode batch (groups non-null): the "requests" are groups, a group's rows the heads of its members' one
    // token each, its keys the first len slots of a member's table row, all of them seen by every row.  A row's result goes,
    // normalised and in 32 bits, to shared_o [requests * hq][D], its log-sum-exp (base 2) to shared_lse.
    const SharedGroup* groups;
    const int32_t* members;            // request, or -1
    float* shared_o;
    float* shared_lse;
    int32_t q_map_ok;
    CUtensorMap q_map;
};

template <int D>
struct EqLayout {
    static constexpr int NK = D == 128 ? 2 : 4;    // K ring depth
    static constexpr int NV = D == 128 ? 2 : 4;    // V ring depth
    static constexpr int Q_TILE = 128 * D * 2;
    static constexpr int KV_TILE = EQ_BN * D * 2;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + 2 * Q_TILE;
    static constexpr int OFF_V = OFF_K + NK * KV_TILE;
    static constexpr int OFF_KS = OFF_V + NV * KV_TILE;              // [NV][128] K scales times scale log2(e)
    static constexpr int OFF_VS = OFF_KS + NV * EQ_BN * 4;           // [NV][128] V scales, -1 for a key at a bad slot
    static constexpr int OFF_FLAG = OFF_VS + NV * EQ_BN * 4;         // [NV] int4: some key of the tile is at a bad slot or has a scale that is not finite
    static constexpr int OFF_RING = OFF_FLAG + NV * 16;              // 3 int4 an entry
    static constexpr int OFF_SCAN = OFF_RING + EQ_RING * 48;         // int64 per warp, and four results
    static constexpr int CPR = D / 16;                               // 16-byte chunks of a row's codes
    static constexpr int NX = (EQ_BN * CPR + EQ_CONV - 1) / EQ_CONV; // chunks per converter thread, tile and pool
    static constexpr int OFF_CODES = OFF_SCAN + 20 * 8;              // [NX][EQ_CONV] 16-byte chunks of the coming K tile's codes
    static constexpr int OFF_BAR = OFF_CODES + NX * EQ_CONV * 16;
    static constexpr int BAR_Q = 0, BAR_KF = 1, BAR_KE = BAR_KF + NK, BAR_VF = BAR_KE + NK, BAR_VE = BAR_VF + NV, BAR_S = BAR_VE + NV,
                         BAR_P = BAR_S + 2, BAR_QE = BAR_P + 4, BAR_OR = BAR_QE + 2, BAR_IF = BAR_OR + 2, BAR_IE = BAR_IF + EQ_RING,
                         BAR_DONE = BAR_IE + EQ_RING, NBAR = BAR_DONE + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;              // TMEM address, abort flag
    static constexpr int ALLOC = OFF_MISC + 8 + 1024;                // room to align the base to 1024 B
    static constexpr uint32_t TMEM_COLS = 512, COL_O0 = 256;
    static_assert(ALLOC <= 232448, "shared memory budget");
};

// A piece of an item: K/V tiles j0 .. j1 - 1 of its rows.
struct EqItem {
    int b, g, row0, ntiles, n, before, j0, j1, kv_end, whole, slot;
    int64_t q0;
};

// A request's rows and keys; n = 0 where there is none to do.
__device__ __forceinline__ void eq_request(const ExtendQ8Params& p, int b, bool tell, int64_t& q0, int& n, int& before) {
    if (p.groups) {
        const SharedGroup g = p.groups[b];
        q0 = g.first, n = g.count, before = g.len - 1;
        return;
    }
    q0 = p.qo_indptr[b];
    const int64_t m = p.qo_indptr[b + 1] - q0, P = p.prefix_lens[b];
    n = (int)m, before = (int)P;
    if (q0 >= 0 && m >= 0 && m <= p.max_qo_len && P >= 0 && P + m <= p.stride && P + m <= p.max_kv_len) return;
    if (tell && m != 0) report(p.status, RX_DEV_BAD_LENGTH);
    n = 0;
}

// Keys and K/V tiles of the item that starts at packed row `row0`.
__device__ __forceinline__ int eq_keys(const ExtendQ8Params& p, int row0, int rows, int before) {
    return before + (p.groups ? 0 : (min(row0 + EQ_ROWS, rows) - 1) / p.group) + 1;
}

__device__ __forceinline__ int eq_tiles(const ExtendQ8Params& p, int row0, int rows, int before) {
    return (eq_keys(p, row0, rows, before) + EQ_BN - 1) / EQ_BN;
}

// K/V tiles of all of a request's items, for one kv head.
__device__ __forceinline__ int64_t eq_units(const ExtendQ8Params& p, int b, bool tell) {
    int64_t q0, sum = 0;
    int n, before;
    eq_request(p, b, tell, q0, n, before);
    const int rows = n * p.group;
    for (int r = 0; r < rows; r += EQ_ROWS) sum += eq_tiles(p, r, rows, before);
    return sum;
}

// Where unit `at` of request b's (of `units` a kv head) lies: kv head, first row and K/V tile of the item.
__device__ __forceinline__ void eq_locate(const ExtendQ8Params& p, int b, int64_t units, int64_t at, int& g, int& row0, int& j, int& tiles) {
    int64_t q0;
    int n, before;
    eq_request(p, b, false, q0, n, before);
    g = (int)(at / units);
    int64_t left = at - g * units;
    for (row0 = 0;; row0 += EQ_ROWS) {
        tiles = eq_tiles(p, row0, n * p.group, before);
        if (left < tiles) break;
        left -= tiles;
    }
    j = (int)left;
}

// pt_wait for what may take an item's time: a Q buffer, the next item, the scores of a Q tile that the items before did without.
// 2^31 keys, some of every tile at bad slots, take 73 s (4.4 us a tile, 2.3 without), so the bound is 133 s, in the timer's upper
// word (no more code than pt_wait; a bound by the part's tiles cost short prompts 2 %).  The tensor core's warp and the
// converters wait for single tiles, 2 s at most, and would end these waits too.
__device__ __forceinline__ bool eq_wait_item(uint32_t bar, uint32_t parity, volatile int* abort) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        auto now = [] {
            uint32_t t;
            asm volatile("mov.u32 %0, %%globaltimer_hi;" : "=r"(t));
            return t;
        };
        const uint32_t t0 = now();
        do ok = mbar_try_wait(bar, parity);
        while (!ok && !*abort && now() - t0 < 32u);
        if (!ok) *abort = 1;
    }
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Scores and weights of a warp's 32 rows as the tensor core's own fragments have them: lane l holds, of rows l / 4
// (+ 8) of each 16, columns 2 (l % 4), + 1 of every 8 (16x256b), and of the packed weights column l % 4 of
// every 4 (16x128b).  So a lane needs the scales of a quarter of the keys, for four rows.
__device__ __forceinline__ void tmem_ld_scores(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st_weights(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_ld_scores8(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 "
        "{%0,%1,%2,%3}, [%4];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st_scores8(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
        : "memory");
}

__device__ __forceinline__ void tmem_st_weights4(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x1.b32 [%0], {%1,%2};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1])
        : "memory");
}

template <int D, int FMT>
__global__ void __launch_bounds__(EQ_THREADS, 1) extend_q8_kernel(const __grid_constant__ ExtendQ8Params p) {
    using LY = EqLayout<D>;
    constexpr int NK = LY::NK, NV = LY::NV, CPR = LY::CPR, NX = LY::NX;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    const uint32_t bar0 = base + LY::OFF_BAR;
    auto bar = [&](int i) { return bar0 + (uint32_t)(8 * i); };
    volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(gbase + LY::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + LY::OFF_MISC + 4);
    int4* ring = reinterpret_cast<int4*>(gbase + LY::OFF_RING);
    int64_t* scan = reinterpret_cast<int64_t*>(gbase + LY::OFF_SCAN);
    // from a shuffle, so that the compiler knows it the same for the whole warp
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31, tid = threadIdx.x;
    const int G = p.group;

    if (tid == 0) {
        mbar_init(bar(LY::BAR_Q), 32 + 1);   // warp 0's lanes, and lane 0's expect-tx arrival
        for (int i = 0; i < NK; ++i) {
            mbar_init(bar(LY::BAR_KF + i), EQ_CONV / 32);
            mbar_init(bar(LY::BAR_KE + i), 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(bar(LY::BAR_VF + i), EQ_CONV / 32);
            mbar_init(bar(LY::BAR_VE + i), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(LY::BAR_S + t), 1);
            mbar_init(bar(LY::BAR_P + t), 4);          // one arrival per softmax warp, keys 0-63
            mbar_init(bar(LY::BAR_P + 2 + t), 4);      // keys 64-127
            mbar_init(bar(LY::BAR_QE + t), 1);         // Q buffer t read by its item's last S
            mbar_init(bar(LY::BAR_OR + t), 1);         // O_t of an item complete
        }
        for (int i = 0; i < EQ_RING; ++i) {
            mbar_init(bar(LY::BAR_IF + i), 1);
            mbar_init(bar(LY::BAR_IE + i), EQ_CONSUMERS);
        }
        mbar_init(bar(LY::BAR_DONE), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(base + LY::OFF_MISC, LY::TMEM_COLS);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    pdl_wait();                          // what came before has finished; nothing global was touched so far

    // ---------------------------------------------------------------- this CTA's part of the units
    // at least two tiles a CTA; borders close to an item's ends move there
    share_out<EQ_THREADS>(
        p.batch, 2, scan, scan + 16, [&](int b, bool tell) { return eq_units(p, b, tell) * p.hkv; },
        [&](int b, int64_t at, int64_t near) {
            int g, row0, j, tiles;
            eq_locate(p, b, eq_units(p, b, false), at, g, row0, j, tiles);
            return at + (j < near ? -j : tiles - j < near ? tiles - j : 0);
        });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    auto soon = [](uint32_t b, uint32_t parity, volatile int* abort) { return pt_wait(b, parity, abort); };
    auto late = [](uint32_t b, uint32_t parity, volatile int* abort) { return eq_wait_item(b, parity, abort); };
    // The k-th item of this CTA, for a whole warp; false at the end.  The entry is free once every warp has read it.
    auto take = [&](int k, EqItem& it, auto wait) -> bool {
        const int e = k % EQ_RING;
        if (!wait(bar(LY::BAR_IF + e), (k / EQ_RING) & 1, abort_flag)) return false;
        const int4 a = ring[3 * e], c = ring[3 * e + 1], d = ring[3 * e + 2];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(LY::BAR_IE + e));
        auto u = [&](int x) { return __shfl_sync(0xffffffffu, x, 0); };
        it.b = u(a.x), it.g = u(a.y), it.row0 = u(a.z), it.ntiles = u(a.w);
        it.n = u(c.x), it.before = u(c.y), it.j0 = u(c.z), it.j1 = u(c.w);
        it.kv_end = u(d.x), it.q0 = ((int64_t)u(d.w) << 32) | (uint32_t)u(d.z);
        const int f = u(d.y);
        it.whole = f & 1, it.slot = f >> 1;
        return it.b >= 0;
    };

    if (warp < 4 || warp >= 12) {
        regs_decrease<EQ_REGS_OTHER>();
        if (warp == 0) {
            // ------------------------------------------------------------ items and Q
            const uint32_t qs = base + LY::OFF_Q;
            int64_t cur = scan[16];
            const int64_t end = scan[17];
            int b = (int)scan[18], g = 0, row0 = 0, j = 0, tiles = 0, n = 0, before = 0, k = 0;
            int64_t q0 = 0;
            int quse0 = 0, quse1 = 0;    // items so far that used Q buffer 0 / 1
            int4 told[2] = {make_int4(-1, 0, 0, 0), make_int4(-1, 0, 0, 0)};
            bool ok = true;
            if (cur < end) {
                // the border may have moved past the end of its request
                int64_t units = eq_units(p, b, false), at = cur - scan[19];
                while (b + 1 < p.batch && at >= units * p.hkv) {
                    at -= units * p.hkv;
                    units = eq_units(p, ++b, false);
                }
                eq_locate(p, b, units, at, g, row0, j, tiles);
                eq_request(p, b, false, q0, n, before);
            }
            while (ok && cur < end) {
                const int rows = n * G, j1 = (int)min((int64_t)tiles, j + (end - cur));
                const int ntiles = rows - row0 > 128 ? 2 : 1;
                const bool whole = j == 0 && j1 == tiles;
                const int slot = j == 0 ? 1 : 0;
                if (!whole) told[slot] = make_int4(b, g, row0, j1 == tiles ? 1 : 0);
                const int e = k % EQ_RING;
                if (k >= EQ_RING && !(ok = pt_wait(bar(LY::BAR_IE + e), ((k / EQ_RING) - 1) & 1, abort_flag))) break;
                if (lane == 0) {
                    ring[3 * e] = make_int4(b, g, row0, ntiles);
                    ring[3 * e + 1] = make_int4(n, before, j, j1);
                    ring[3 * e + 2] = make_int4(eq_keys(p, row0, rows, before), (whole ? 1 : 0) | (slot << 1),
                                                (int)(uint32_t)q0, (int)(q0 >> 32));
                    mbar_arrive(bar(LY::BAR_IF + e));
                }
                ++k;
                if (quse0 > 0 && !(ok = eq_wait_item(bar(LY::BAR_QE), (quse0 - 1) & 1, abort_flag))) break;
                if (ntiles > 1 && quse1 > 0 && !(ok = eq_wait_item(bar(LY::BAR_QE + 1), (quse1 - 1) & 1, abort_flag))) break;
                quse0 += 1;
                quse1 += ntiles > 1 ? 1 : 0;
                // full 128-row tiles by TMA, one box per 64 columns; a ragged one row by row, two lanes a row, the rows
                // past the end like the last
                const int full = p.q_map_ok && !p.groups && q0 + n <= INT32_MAX ? min(ntiles, (rows - row0) >> 7) : 0;
                if (lane == 0) {
                    fence_proxy_async_smem();
                    mbar_arrive_expect_tx(bar(LY::BAR_Q), (uint32_t)(full * LY::Q_TILE));
                    for (int t = 0; t < full; ++t)
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_3d(qs + (uint32_t)(t * LY::Q_TILE + h * 128 * 128), &p.q_map, h * 64, g * G,
                                        (int)q0 + row0 / G + t * (128 / G), bar(LY::BAR_Q));
                }
                for (int rr = full * 128 + (lane >> 1); rr < ntiles * 128; rr += 16) {
                    const int t = rr >> 7, r = rr & 127, R = min(row0 + rr, rows - 1);
                    const int64_t token = p.groups ? max(p.members[q0 + R / G], 0) : q0 + R / G;
                    const __nv_bfloat16* src = p.q + (token * p.hq + g * G + R % G) * D;
                    const uint32_t to = qs + (uint32_t)(t * LY::Q_TILE + r * 128);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const int c = 2 * i + (lane & 1);
                        cp_async_16(to + (uint32_t)((c >> 3) * 128 * 128 + (((c & 7) ^ (r & 7)) << 4)), src + c * 8, 16);
                    }
                }
                cp_async_arrive_noinc(bar(LY::BAR_Q));
                // on to the next item: row tile, kv head, request
                cur += j1 - j;
                if (cur >= end) break;
                j = 0;
                row0 += EQ_ROWS;
                if (row0 >= rows) {
                    row0 = 0;
                    if (++g == p.hkv) {
                        g = 0;
                        do n = 0;
                        while (++b < p.batch && (eq_request(p, b, false, q0, n, before), n == 0));
                        if (n == 0) break;
                    }
                }
                tiles = eq_tiles(p, row0, n * G, before);
            }
            if (ok) {
                const int e = k % EQ_RING;
                if (k < EQ_RING || pt_wait(bar(LY::BAR_IE + e), ((k / EQ_RING) - 1) & 1, abort_flag)) {
                    if (lane == 0) {
                        ring[3 * e] = make_int4(-1, 0, 0, 0);
                        mbar_arrive(bar(LY::BAR_IF + e));
                    }
                }
            }
            if (lane < 2) p.meta[blockIdx.x * 2 + lane] = lane == 0 ? told[0] : told[1];
            cp_async_wait_all();
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            constexpr uint32_t IDESC_S = idesc_bf16_f32(128, EQ_BN, 0, 0);
            constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, 0, 1);
            const uint32_t qd0 = (uint32_t)sdesc_sw128(base + LY::OFF_Q, 16, 1024);
            const uint32_t kd0 = (uint32_t)sdesc_sw128(base + LY::OFF_K, 16, 1024);
            const uint32_t vd0 = (uint32_t)sdesc_sw128(base + LY::OFF_V, EQ_BN * 128, 1024);
            auto issue_s = [&](int t, int ks) {
                pt_mma_s<D>(tmem + t * EQ_BN, qd0 + (uint32_t)t * (uint32_t)(LY::Q_TILE >> 4), kd0 + (uint32_t)ks * (uint32_t)(LY::KV_TILE >> 4),
                            IDESC_S);
                pt_commit(bar(LY::BAR_S + t));
            };
            auto issue_pv = [&](int t, int vs, int h, bool fresh) {      // keys 64 h .. 64 h + 63
                pt_mma_pv(tmem + LY::COL_O0 + t * D, tmem + t * EQ_BN + h * 32,
                          vd0 + (uint32_t)vs * (uint32_t)(LY::KV_TILE >> 4) + (uint32_t)h * (uint32_t)(64 * 128 >> 4), IDESC_PV, fresh);
            };
            int gt = 0, ic = 0, sc0 = 0, sc1 = 0;    // K/V tiles, items and score steps of Q tile 0 / 1 so far
            bool ok = true;
            EqItem it;
            for (int k = 0; ok && take(k, it, soon); ++k) {
                const int nt = it.ntiles, nkv = it.j1 - it.j0;
                ok = pt_wait(bar(LY::BAR_Q), ic & 1, abort_flag) && pt_wait(bar(LY::BAR_KF + gt % NK), (gt / NK) & 1, abort_flag);
                ic += 1;
                if (!ok) break;
                fence_proxy_async_smem();            // rows and codes that other warps stored, before the tensor core reads them
                tc_fence_after();
                for (int t = 0; t < nt; ++t) {
                    issue_s(t, gt % NK);
                    if (nkv == 1) pt_commit(bar(LY::BAR_QE + t));
                }
                pt_commit(bar(LY::BAR_KE + gt % NK));
                for (int j = 0; ok && j < nkv; ++j) {
                    const int u = gt + j, vs = u % NV, ks = (u + 1) % NK;
                    const bool more = j + 1 < nkv;
                    if (!(ok = pt_wait(bar(LY::BAR_VF + vs), (u / NV) & 1, abort_flag))) break;
                    if (more && !(ok = pt_wait(bar(LY::BAR_KF + ks), ((u + 1) / NK) & 1, abort_flag))) break;
                    fence_proxy_async_smem();
                    for (int t = 0; t < nt; ++t) {
                        const int ph = ((t == 0 ? sc0 : sc1) + j) & 1;
                        for (int h = 0; ok && h < 2; ++h) {
                            ok = pt_wait(bar(LY::BAR_P + 2 * h + t), ph, abort_flag);
                            tc_fence_after();
                            if (ok) issue_pv(t, vs, h, j == 0 && h == 0);
                        }
                        if (!ok) break;
                        if (t == nt - 1) pt_commit(bar(LY::BAR_VE + vs));
                        if (more) {
                            issue_s(t, ks);
                            if (j + 2 == nkv) pt_commit(bar(LY::BAR_QE + t));
                        } else {
                            pt_commit(bar(LY::BAR_OR + t));
                        }
                    }
                    if (ok && more) pt_commit(bar(LY::BAR_KE + ks));
                }
                sc0 += nkv;
                sc1 += nt > 1 ? nkv : 0;
                gt += nkv;
            }
            pt_commit(bar(LY::BAR_DONE));
            __syncwarp();
        } else {
            // ------------------------------------------------------------ K/V tiles
            const int lt = warp < 4 ? tid - 64 : tid - 384 + 64;
            // This thread's 16-byte chunk of every key row it handles: 8 lanes have 4 chunks of a 64-channel half of two
            // neighbouring keys, whose pieces lie in different banks.
            const int c = D == 128 ? (lane & 3) + ((lane >> 1) & 4) : lane & 3;
            const int key0 = (lt >> 5) * (32 / CPR) + (D == 128 ? ((lane >> 3) & 2) + ((lane >> 2) & 1) : lane >> 2);
            constexpr int STEP = EQ_CONV / CPR;              // keys from one of its rows to the next
            static_assert(EQ_CONV % CPR == 0 && STEP % 8 == 0, "one chunk and one swizzle per thread");
            const uint32_t nslots = (uint32_t)p.num_slots;
            const uint32_t pitch = (uint32_t)(p.hkv * D);
            // The tile whose codes are loaded next, and its slots: one tile ahead of the one being stored.
            EqItem it;
            int k = 0, j = 0;
            bool have = take(0, it, soon);
            if (have) j = it.j0;
            const int32_t* slots = nullptr;
            const uint8_t *kb = nullptr, *vb = nullptr;
            const float2* sb = nullptr;
            int32_t sl[NX], ss = -1;
            auto begin = [&]() {
                slots = p.r2t + (int64_t)(p.groups ? p.groups[it.b].src : it.b) * p.stride;
                kb = p.pools.k + (size_t)it.g * D + c * 16;
                vb = p.pools.v + (size_t)it.g * D + c * 16;
                sb = p.pools.scales + it.g;
            };
            auto load_slots = [&]() {
                const int left = it.kv_end - j * EQ_BN;      // keys of this tile and after it
#pragma unroll
                for (int x = 0; x < NX; ++x) {
                    const int key = key0 + x * STEP;
                    sl[x] = key < EQ_BN && key < left ? slots[j * EQ_BN + key] : -1;
                }
                // A place behind the last key has that key's scales, which no row sees: the table may hold any value, so none
                // can say that there is no key.  (With the value changed as it is loaded, or the place kept or worked out again
                // where the scale is, the four long chats took 1710 to 1820 us.)
                ss = lt < EQ_BN ? slots[min(j * EQ_BN + lt, it.kv_end - 1)] : 0;
            };
            auto next = [&]() {
                if (++j == it.j1) {
                    have = take(++k, it, soon);
                    if (!have) return;
                    j = it.j0;
                    begin();
                }
                load_slots();
            };
            // The coming K tile's codes travel to shared memory, to where the thread that widens them reads them; the coming
            // V tile's to registers (both in registers, some were spilled and waited for at once: 720 TFLOP/s).
            // Each chunk's place is filled again as soon as its codes are stored, so a load has a whole tile's time.
            const uint32_t codes = base + LY::OFF_CODES + lt * 16;
            uint4 vr[NX];
            float2 sc = make_float2(0.f, 0.f);
            int32_t kept = 0;                                // ss of the V tile in the registers
            auto fetch_k = [&](int x) {
                const bool in = (uint32_t)sl[x] < nslots;
                cp_async_16(codes + x * EQ_CONV * 16, kb + (size_t)(in ? (uint32_t)sl[x] : 0u) * pitch, in ? 16u : 0u);
            };
            auto fetch_v = [&](int x) {
                vr[x] = make_uint4(0, 0, 0, 0);
                if ((uint32_t)sl[x] < nslots) vr[x] = *reinterpret_cast<const uint4*>(vb + (size_t)(uint32_t)sl[x] * pitch);
            };
            auto load_scale = [&]() {
                kept = ss;
                sc = make_float2(1.f, -1.f);                 // left out
                if ((uint32_t)ss < nslots) sc = sb[(int64_t)(ss >> p.pools.shift) * p.hkv];
                else report(p.status, RX_DEV_BAD_SLOT);
            };
            // channels 16 c .. + 15: two 16-byte pieces of the row's 64-channel half
            const uint32_t piece = (uint32_t)((c >> 2) * EQ_BN * 128 + key0 * 128 + ((2 * c) & 7) * 16) ^ (uint32_t)((key0 & 7) * 16);
            auto store = [&](const uint4& r, int x, uint32_t buf) {
                uint32_t w[8];
                q8_to_bf16<FMT>(r.x, w[0], w[1]);
                q8_to_bf16<FMT>(r.y, w[2], w[3]);
                q8_to_bf16<FMT>(r.z, w[4], w[5]);
                q8_to_bf16<FMT>(r.w, w[6], w[7]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + x * STEP * 128 + (h ? piece ^ 16u : piece)),
                                 "r"(w[4 * h]), "r"(w[4 * h + 1]), "r"(w[4 * h + 2]), "r"(w[4 * h + 3])
                                 : "memory");
            };
            auto publish = [&](uint32_t full) {
                __syncwarp();
                if (lane == 0) mbar_arrive(full);
            };
            bool cur = have;                                 // a tile's codes are on their way
            if (have) {
                begin();
                load_slots();
#pragma unroll
                for (int x = 0; x < NX; ++x) {
                    fetch_k(x);
                    fetch_v(x);
                }
                cp_async_commit();
                load_scale();
                next();
            }
            for (int u = 0; cur; ++u) {
                const int ks = u % NK, vs = u % NV;
                if (u >= NK && !pt_wait(bar(LY::BAR_KE + ks), ((u / NK) - 1) & 1, abort_flag)) break;
                cp_async_wait<0>();
#pragma unroll
                for (int x = 0; x < NX; ++x)
                    if (key0 + x * STEP < EQ_BN) {
                        uint4 r;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                                     : "r"(codes + x * EQ_CONV * 16)
                                     : "memory");
                        store(r, x, base + LY::OFF_K + ks * LY::KV_TILE);
                        if (have) fetch_k(x);
                    }
                cp_async_commit();
                publish(bar(LY::BAR_KF + ks));
                if (u >= NV && !pt_wait(bar(LY::BAR_VE + vs), ((u / NV) - 1) & 1, abort_flag)) break;
                if (lt < EQ_BN) {
                    reinterpret_cast<float*>(gbase + LY::OFF_KS)[vs * EQ_BN + lt] = sc.x * p.scale_log2;
                    reinterpret_cast<float*>(gbase + LY::OFF_VS)[vs * EQ_BN + lt] = sc.y;
                    const bool bad = __any_sync(0xffffffffu, (uint32_t)kept >= nslots || !isfinite(sc.x) || !isfinite(sc.y));
                    if (lane == 0) reinterpret_cast<int*>(gbase + LY::OFF_FLAG)[vs * 4 + lt / 32] = bad ? 1 : 0;
                }
#pragma unroll
                for (int x = 0; x < NX; ++x)
                    if (key0 + x * STEP < EQ_BN) {
                        store(vr[x], x, base + LY::OFF_V + vs * LY::KV_TILE);
                        if (have) fetch_v(x);
                    }
                publish(bar(LY::BAR_VF + vs));
                cur = have;
                if (have) {
                    load_scale();
                    next();
                }
            }
            cp_async_wait_all();
        }
    } else {
        // ------------------------------------------------------------ softmax warpgroups
        regs_increase<EQ_REGS_SOFTMAX>();
        const int t = (warp >> 2) - 1, quarter = warp & 3, r8 = lane >> 2, t4 = lane & 3;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16, half = 16u << 16;
        const uint32_t s_addr = tmem + lane_base + t * EQ_BN;   // scores, then weights over them
        const uint32_t o_addr = tmem + lane_base + LY::COL_O0 + t * D;
        int gt = 0, sc = 0, oc = 0;           // K/V tiles of all items, and score steps and items of this Q tile so far
        bool ok = true;
        EqItem it;
        // of four values, one for each row 8 i + r8 and the same in the row's four lanes: row `lane`'s
        auto of_row = [&](const float* v) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float y = __shfl_sync(0xffffffffu, v[i], 4 * (lane & 7));
                if (lane >> 3 == i) x = y;
            }
            return x;
        };
        for (int k = 0; ok && take(k, it, late); ++k) {
            const int nkv = it.j1 - it.j0;
            if (t >= it.ntiles) {
                gt += nkv;
                continue;
            }
            const int rows = it.n * G, first = it.row0 + t * 128 + quarter * 32;      // the warp's first row
            int lim[4];                          // row 8 i + r8 sees columns 0 .. lim[i] of the coming tile
            float m_ref[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lim[i] = it.before + (p.groups ? 0 : min(first + 8 * i + r8, rows - 1) / G) - it.j0 * EQ_BN;
                m_ref[i] = -INFINITY, l[i] = 0.f;
            }
            for (int j = 0; j < nkv; ++j, ++gt) {
                const int vs = gt % NV;
                if (!(ok = eq_wait_item(bar(LY::BAR_S + t), (sc + j) & 1, abort_flag))) break;
                if (!(ok = pt_wait(bar(LY::BAR_VF + vs), (gt / NV) & 1, abort_flag))) break;     // the scales
                tc_fence_after();
                const float* kscale = reinterpret_cast<const float*>(gbase + LY::OFF_KS) + vs * EQ_BN + 2 * t4;
                const float* vscale = reinterpret_cast<const float*>(gbase + LY::OFF_VS) + vs * EQ_BN + 2 * t4;
                const int4 flag = *reinterpret_cast<const int4*>(gbase + LY::OFF_FLAG + vs * 16);
                float alpha[4], ref[4];
                bool moved = false;
                auto refer = [&](float* mx) {    // the rows' references after scores up to mx in this lane
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
                        float m_new = m_ref[i];
                        if (m_ref[i] == -INFINITY || mx[i] > m_ref[i] + EQ_RESCALE) m_new = fmaxf(m_ref[i], mx[i]);
                        alpha[i] = m_ref[i] == -INFINITY ? 0.f : fast_exp2(m_ref[i] - m_new);
                        moved |= m_new != m_ref[i];
                        l[i] *= alpha[i];
                        m_ref[i] = m_new;
                        ref[i] = m_new == -INFINITY ? 0.f : m_new;
                    }
                    moved = j > 0 && __any_sync(0xffffffffu, moved);
                };
                auto rescale = [&]() {
                    // PV_t(j-1) has completed (S_t(j) was issued after it and is complete), and PV_t(j) waits for
                    // the arrivals below.  Rare: rolled.
                    const float a = of_row(alpha);
#pragma unroll 1
                    for (int cc = 0; cc < D; cc += 32) {
                        float ov[32];
                        tmem_ld32(o_addr + cc, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] *= a;
                        tmem_st32(o_addr + cc, ov);
                    }
                };
                auto publish = [&](int h) {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(LY::BAR_P + 2 * h + t));
                };
                if (flag.x | flag.y | flag.z | flag.w) {
                    // Tiles with a key at a bad slot, or with scales that are not finite, which must not reach rows that do
                    // not see the key: scores and weights are taken out by selection.  Rolled, eight columns a turn.
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c0 = 0; c0 < EQ_BN; c0 += 8) {
                        float v[8];
                        tmem_ld_scores8(s_addr + c0, v);
                        tmem_ld_scores8(s_addr + half + c0, v + 4);
                        tmem_wait_ld();
                        const float2 f = *reinterpret_cast<const float2*>(kscale + c0), w = *reinterpret_cast<const float2*>(vscale + c0);
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            const bool out = c0 + 2 * t4 + (x & 1) > lim[x >> 1] || (x & 1 ? w.y : w.x) == -1.f;
                            v[x] = out ? -INFINITY : v[x] * (x & 1 ? f.y : f.x);
                            mx[x >> 1] = fmaxf(mx[x >> 1], v[x]);
                        }
                        tmem_st_scores8(s_addr + c0, reinterpret_cast<const uint32_t*>(v));
                        tmem_st_scores8(s_addr + half + c0, reinterpret_cast<const uint32_t*>(v + 4));
                    }
                    tmem_wait_st();
                    refer(mx);
#pragma unroll 1
                    for (int c0 = 0; c0 < EQ_BN; c0 += 8) {     // these columns' weights go to columns already read
                        float v[8];
                        uint32_t pk[4];
                        tmem_ld_scores8(s_addr + c0, v);
                        tmem_ld_scores8(s_addr + half + c0, v + 4);
                        tmem_wait_ld();
                        const float2 w = *reinterpret_cast<const float2*>(vscale + c0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float e0 = fast_exp2(v[2 * i] - ref[i]), e1 = fast_exp2(v[2 * i + 1] - ref[i]);
                            l[i] += e0 + e1;
                            pk[i] = pack_bf16x2(v[2 * i] == -INFINITY ? 0.f : e0 * w.x, v[2 * i + 1] == -INFINITY ? 0.f : e1 * w.y);
                        }
                        tmem_st_weights4(s_addr + c0 / 2, pk);
                        tmem_st_weights4(s_addr + half + c0 / 2, pk + 2);
                    }
                    if (moved) rescale();
                    publish(0);
                    publish(1);
                } else {
                    float s[2][64];              // [16 rows][columns 8 i + 2 t4, + 1 of row r8, then of row r8 + 8]
                    tmem_ld_scores(s_addr, s[0]);
                    tmem_ld_scores(s_addr + half, s[1]);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t f = *reinterpret_cast<const uint64_t*>(kscale + 8 * i);
#pragma unroll
                        for (int a = 0; a < 2; ++a)
#pragma unroll
                            for (int x = 0; x < 4; x += 2)
                                f2_unpack(f2_mul(f2_pack(s[a][4 * i + x], s[a][4 * i + x + 1]), f), s[a][4 * i + x], s[a][4 * i + x + 1]);
                    }
                    if (__any_sync(0xffffffffu, lim[0] < EQ_BN - 1)) {       // the causal limit cuts this tile (rows' limits ascend)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                if (8 * i + 2 * t4 + (x & 1) > lim[x >> 1]) s[x >> 2][4 * i + (x & 3)] = -INFINITY;
                    }
                    float mx[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float* v = s[q >> 1] + 2 * (q & 1);
                        float a = v[0], b = v[4], c = v[8], d = v[12];
                        a = fmaxf(a, v[1]), b = fmaxf(b, v[5]), c = fmaxf(c, v[9]), d = fmaxf(d, v[13]);
#pragma unroll
                        for (int i = 4; i < 16; i += 4) {
                            a = fmax3(a, v[4 * i], v[4 * i + 1]);
                            b = fmax3(b, v[4 * i + 4], v[4 * i + 5]);
                            c = fmax3(c, v[4 * i + 8], v[4 * i + 9]);
                            d = fmax3(d, v[4 * i + 12], v[4 * i + 13]);
                        }
                        mx[q] = fmaxf(fmax3(a, b, c), d);
                    }
                    refer(mx);
                    uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
                    // weights in two halves of 64 keys (32 columns), each published as soon as it is stored
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[2][16];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint64_t f = *reinterpret_cast<const uint64_t*>(vscale + 64 * h + 8 * i);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float* v = s[q >> 1] + 32 * h + 4 * i + 2 * (q & 1);
                                float x0, x1;
                                f2_unpack(f2_add(f2_pack(v[0], v[1]), f2_pack(-ref[q], -ref[q])), x0, x1);
                                const uint64_t e2 = f2_pack(fast_exp2(x0), fast_exp2(x1));
                                acc2[q] = f2_add(acc2[q], e2);
                                f2_unpack(f2_mul(e2, f), x0, x1);
                                pk[q >> 1][2 * i + (q & 1)] = pack_bf16x2(x0, x1);
                            }
                        }
                        tmem_st_weights(s_addr + h * 32, pk[0]);
                        tmem_st_weights(s_addr + half + h * 32, pk[1]);
                        if (h == 0 && moved) rescale();
                        publish(h);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float ra, rb;
                        f2_unpack(acc2[q], ra, rb);
                        l[q] += ra + rb;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) lim[i] -= EQ_BN;
            }
            if (!ok) break;
            sc += nkv;
            // O_t is complete once its last PV has been; the next item's first PV, which overwrites it, waits for weights
            // that this warpgroup publishes after these reads
            if (!(ok = pt_wait(bar(LY::BAR_OR + t), oc & 1, abort_flag))) break;
            oc += 1;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            }
            const float sum = of_row(l), top = of_row(m_ref);
            const int R = first + lane;
            const int tok = min(R, rows - 1) / G, h = it.g * G + min(R, rows - 1) % G;
            const int64_t token = p.groups ? p.members[it.q0 + tok] : it.q0 + tok, at = token * p.hq + h;
            const bool valid = R < rows && token >= 0, final = it.whole && !p.groups;
            float* const part_row = it.whole ? p.shared_o + at * D
                                             : p.part_o + (((int64_t)blockIdx.x * 2 + it.slot) * EQ_ROWS + t * 128 + quarter * 32 + lane) * D;
            const float inv = sum == 0.f ? 0.f : 1.f / sum, lse = sum == 0.f ? -INFINITY : top + log2f(sum);      // no key: zeros
#pragma unroll 1
            for (int cc = 0; cc < D; cc += 32) {
                float ov[32];
                tmem_ld32(o_addr + cc, ov);
                tmem_wait_ld();
                if (valid && final) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4*>(p.out + at * D + cc + e) =
                            make_uint4(pack_bf16x2(ov[e] * inv, ov[e + 1] * inv), pack_bf16x2(ov[e + 2] * inv, ov[e + 3] * inv),
                                       pack_bf16x2(ov[e + 4] * inv, ov[e + 5] * inv), pack_bf16x2(ov[e + 6] * inv, ov[e + 7] * inv));
                } else if (valid) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(part_row + cc + e) =
                            make_float4(ov[e] * inv, ov[e + 1] * inv, ov[e + 2] * inv, ov[e + 3] * inv);
                }
                __syncwarp();                    // the whole warp reads the next columns
            }
            if (valid && final && p.lse) p.lse[at] = lse * EQ_LN2;
            if (valid && !final) (it.whole ? p.shared_lse[at] : p.part_lse[(part_row - p.part_o) / D]) = lse;
            __syncwarp();
            tc_fence_before();
        }
    }
    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // copies may still be on their way to shared memory: wait out the time that any of them takes
        if (tid == 0) report(p.status, RX_DEV_TIMEOUT);
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 10000000ull) __nanosleep(1000);
    }
    if (warp == 1) {
        tc_fence_after();
        // every MMA this CTA issued has completed before TMEM is released; this wait does not stop on the abort flag
        volatile int no_abort = 0;
        warp_wait(bar(LY::BAR_DONE), 0, &no_abort, p.status, 500000000ull);
        tmem_dealloc(tmem, LY::TMEM_COLS);
    }
}

// Rows from their parts: blockIdx.x the begun and not ended item, four rows a block, a warp each.
template <int D>
__global__ void __launch_bounds__(128) extend_q8_merge_kernel(const __grid_constant__ ExtendQ8Params p) {
    constexpr int E = D / 32;
    __shared__ int list[EQ_CTAS];
    __shared__ uint32_t room[EQ_CTAS];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int count = parts_of<EQ_CTAS>(p.meta, blockIdx.x, EQ_CTAS, list, room);
    if (count == 0) return;
    const int4 item = p.meta[list[0]];
    int64_t q0;
    int n, before;
    eq_request(p, item.x, false, q0, n, before);
    const int r = blockIdx.y * 4 + warp, R = item.z + r;
    if (R >= n * p.group) return;
    float acc[E];
    const float lse = merge_few<D>(list, count, p.part_o, p.part_lse, EQ_ROWS, r, acc);
    const int64_t token = p.groups ? p.members[q0 + R / p.group] : q0 + R / p.group;
    const int64_t at = token * p.hq + item.y * p.group + R % p.group;
    if (p.groups) {
        if (token < 0) return;
#pragma unroll
        for (int e = 0; e < E; ++e) p.shared_o[at * D + lane * E + e] = acc[e];
        if (lane == 0) p.shared_lse[at] = lse;
        return;
    }
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(p.out + at * D + lane * E + e) = pack_bf16x2(acc[e], acc[e + 1]);
    if (p.lse && lane == 0) p.lse[at] = lse * EQ_LN2;
}

// The current device must be an sm_103: checked once per device.
static int eq_device(const char* fn) {
    static PerDeviceOnce checked;
    return per_device_once(checked, [&] {
        int dev = 0, major = 0, minor = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
            set_error("%s: cannot query the device", fn);
            return (int)RX_ECUDA;
        }
        if (major != 10 || minor != 3) {
            set_error("%s: the tcgen05 kernel needs an sm_103 (GB300) device", fn);
            return (int)RX_EDEVICE;
        }
        return (int)RX_OK;
    });
}

// Tensor map of q as [rows][hq][D] bf16, boxes of a 128-row tile's 64 columns: G heads of 128 / G tokens.  The rows are found through
// qo_indptr, so the host knows no tighter bound than the coordinates'; the kernel addresses only full tiles of a request's rows.
static bool eq_rows_map(CUtensorMap* m, const void* q, int hq, int D, int G) {
    static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    if (!enc || 128 % G != 0) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)hq, (cuuint64_t)INT32_MAX};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)hq * D * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(128 / G)};
    const cuuint32_t elem[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t extend_q8_bytes(const rx_attn_desc* d) {
    const size_t rows = (size_t)EQ_CTAS * 2 * EQ_ROWS;
    return rows * d->head_dim * sizeof(float) + rows * sizeof(float) + (size_t)EQ_CTAS * 2 * sizeof(int4);
}

template <int D, int FMT>
static int launch_extend(const char* fn, const ExtendQ8Params& p, cudaStream_t s) {
    static PerDeviceOnce attr;
    constexpr int smem = EqLayout<D>::ALLOC;
    const int rc = per_device_once(attr, [&] {
        const cudaError_t e = cudaFuncSetAttribute(extend_q8_kernel<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) {
            set_error("%s: cannot set shared memory size: %s", fn, cudaGetErrorString(e));
            return (int)RX_ECUDA;
        }
        // the warpgroups share out the registers the block is launched with: fewer, and they would wait forever
        cudaFuncAttributes fa{};
        if (cudaFuncGetAttributes(&fa, extend_q8_kernel<D, FMT>) != cudaSuccess || fa.numRegs < (int)EQ_REGS_LAUNCH) {
            set_error("%s: kernel built with %d registers per thread; the register split needs %d", fn, fa.numRegs,
                      (int)EQ_REGS_LAUNCH);
            return (int)RX_ECUDA;
        }
        return (int)RX_OK;
    });
    if (rc != RX_OK) return rc;
    cudaError_t e = launch_pdl(extend_q8_kernel<D, FMT>, EQ_CTAS, EQ_THREADS, smem, s, p);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg{};
        const double items = (double)(((int64_t)p.max_qo_len * p.group + EQ_ROWS - 1) / EQ_ROWS) * p.hkv * p.batch;
        cfg.gridDim = dim3((unsigned)std::min<double>(p.groups ? EQ_CTAS : items, EQ_CTAS), EQ_ROWS / 4);
        cfg.blockDim = dim3(128);
        cfg.stream = s;
        cudaLaunchAttribute pdl[1];
        pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        pdl[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = pdl;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, extend_q8_merge_kernel<D>, p);
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("%s: launch failed: %s", fn, cudaGetErrorString(e));
        return RX_ECUDA;
    }
    return RX_OK;
}

static void eq_params(ExtendQ8Params& p, const RowsQ8Args& a, const rx_attn_desc* d, const rx_q8_desc* q8, void* ws) {
    p.q = (const __nv_bfloat16*)a.q;
    p.qo_indptr = a.qo_indptr;
    p.prefix_lens = a.prefix_lens;
    p.r2t = a.r2t;
    p.stride = a.stride;
    p.num_slots = d->num_slots;
    p.pools = {a.k_pool, a.v_pool, a.scales, q8_shift(q8)};
    p.out = (__nv_bfloat16*)a.out;
    p.lse = a.lse;
    p.batch = a.batch;
    p.hq = d->hq;
    p.hkv = d->hkv;
    p.group = d->hq / d->hkv;
    p.max_qo_len = a.max_qo_len;
    p.max_kv_len = a.max_kv_len;
    p.scale_log2 = d->scale * EQ_LOG2E;
    p.status = a.status;
    const size_t rows = (size_t)EQ_CTAS * 2 * EQ_ROWS;
    p.part_o = (float*)ws;
    p.part_lse = p.part_o + rows * d->head_dim;
    p.meta = (int4*)(p.part_lse + rows);
}

static int launch_extend(const char* fn, const ExtendQ8Params& p, const rx_attn_desc* d, const rx_q8_desc* q8, cudaStream_t stream) {
    if (d->head_dim == 128)
        return q8->format == RX_Q8_INT8 ? launch_extend<128, RX_Q8_INT8>(fn, p, stream) : launch_extend<128, RX_Q8_E4M3>(fn, p, stream);
    return q8->format == RX_Q8_INT8 ? launch_extend<64, RX_Q8_INT8>(fn, p, stream) : launch_extend<64, RX_Q8_E4M3>(fn, p, stream);
}

int extend_q8_launch(const char* fn, const RowsQ8Args& a, const rx_attn_desc* d, const rx_q8_desc* q8, void* ws, size_t ws_bytes,
                     cudaStream_t stream) {
    const int dc = eq_device(fn);
    if (dc != RX_OK) return dc;
    const size_t need = extend_q8_bytes(d);
    RX_REQUIRE(ws && ws_bytes >= need && ((uintptr_t)ws & 255) == 0,
               "%s: a 256-byte aligned workspace of %zu bytes is needed (got %zu)", fn, need, ws_bytes);
    RX_REQUIRE((int64_t)a.max_qo_len * (d->hq / d->hkv) < INT32_MAX - EQ_ROWS, "%s: too many rows in a request", fn);
    ExtendQ8Params p{};
    eq_params(p, a, d, q8, ws);
    p.q_map_ok = eq_rows_map(&p.q_map, a.q, d->hq, d->head_dim, p.group) ? 1 : 0;
    return launch_extend(fn, p, d, q8, stream);
}

// A decode batch's groups as the kernels take them: SharedGroup per group, members (-1: not one), and the keys that each
// request takes from its group's shared run.  A group with bad boundaries is left out (its members read their own keys), and so is a member
// that is no request, has fewer keys than the run or is a member already.
__global__ void __launch_bounds__(512) shared_q8_groups_kernel(rx_shared_groups g, int32_t batch, const int32_t* kv_lens, int64_t stride,
                                                               int32_t max_kv_len, SharedGroup* groups, int32_t* members,
                                                               int32_t* shared_of, int32_t* status) {
    pdl_launch_dependents();
    pdl_wait();
    for (int b = threadIdx.x; b < batch; b += blockDim.x) shared_of[b] = 0, members[b] = -1;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = warp; i < g.num_groups; i += blockDim.x / 32) {
        const int32_t first = g.d_group_indptr[i], end = g.d_group_indptr[i + 1], len = g.d_group_len[i];
        const bool good = first >= 0 && end >= first && end <= batch && len >= 1 && len <= stride && len <= max_kv_len;
        if (!good && lane == 0) report(status, RX_DEV_BAD_LENGTH);
        int src = -1;
        for (int m0 = first; good && m0 < end; m0 += 32) {
            const int m = m0 + lane;
            int b = m < end ? g.d_group_members[m] : -1;
            const bool is = b >= 0 && b < batch;
            if (m < end && !is) report(status, RX_DEV_BAD_LENGTH);
            if (!is || kv_lens[b] < len || kv_lens[b] > stride || kv_lens[b] > max_kv_len) b = -1;
            if (b >= 0 && atomicCAS(shared_of + b, 0, len) != 0) {
                report(status, RX_DEV_BAD_LENGTH);
                b = -1;
            }
            if (m < end) members[m] = b;
            const unsigned any = __ballot_sync(0xffffffffu, b >= 0);
            if (src < 0 && any) src = __shfl_sync(0xffffffffu, b, __ffs(any) - 1);
        }
        if (lane == 0) groups[i] = SharedGroup{first, src >= 0 ? end - first : 0, len, src};
    }
}

struct SharedLayout {
    size_t lse, of, members, groups, total;      // shared_o first, the tiles' parts last
};

static SharedLayout shared_layout(const rx_attn_desc* d, int32_t batch, int32_t num_groups) {
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    SharedLayout L{};
    L.lse = up((size_t)batch * d->hq * d->head_dim * sizeof(float));
    L.of = L.lse + up((size_t)batch * d->hq * sizeof(float));
    L.members = L.of + up((size_t)batch * sizeof(int32_t));
    L.groups = L.members + up((size_t)batch * sizeof(int32_t));
    L.total = L.groups + up((size_t)num_groups * sizeof(SharedGroup));
    return L;
}

size_t shared_q8_bytes(const rx_attn_desc* d, int32_t batch, int32_t num_groups) {
    return shared_layout(d, batch, num_groups).total + extend_q8_bytes(d);
}

int shared_q8_launch(const char* fn, RowsQ8Args& a, const rx_attn_desc* d, const rx_q8_desc* q8, const rx_shared_groups* g, void* ws,
                     cudaStream_t stream) {
    const int dc = eq_device(fn);
    if (dc != RX_OK) return dc;
    const SharedLayout L = shared_layout(d, a.batch, g->num_groups);
    unsigned char* w = (unsigned char*)ws;
    ExtendQ8Params p{};
    eq_params(p, a, d, q8, w + L.total);
    p.batch = g->num_groups;
    p.shared_o = (float*)w;
    p.shared_lse = (float*)(w + L.lse);
    p.members = (const int32_t*)(w + L.members);
    p.groups = (const SharedGroup*)(w + L.groups);
    launch_pdl(shared_q8_groups_kernel, 1, 512, 0, stream, *g, a.batch, a.kv_lens, a.stride, a.max_kv_len, (SharedGroup*)(w + L.groups),
               (int32_t*)(w + L.members), (int32_t*)(w + L.of), a.status);
    a.shared_of = (const int32_t*)(w + L.of);
    a.shared_o = p.shared_o;
    a.shared_lse = p.shared_lse;
    return launch_extend(fn, p, d, q8, stream);
}

}  // namespace rx
