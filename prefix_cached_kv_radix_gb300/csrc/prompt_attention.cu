// prompt_attention: causal attention over packed prompts, on tcgen05 tensor cores (bf16).
//
// Row i of a sequence attends rows 0..i of the same sequence; query head h reads kv head
// h / (hq / hkv).  With a running reference m of the row maximum (base 2: s = scale log2(e) q k),
//   P = 2^(s - m),  l += sum P,  O += P V,  o = O / l,  lse = ln 2 (m + log2 l),
// O and l rescaled by 2^(m - m') when the reference moves, which it does only when the row maximum
// has grown by more than 2^8 (P <= 256 stays far from the ends of fp32 and bf16).  S, O, m and l
// are 32-bit; P is rounded to bf16 for the tensor core (unnormalised, at most 2^-8 relative per
// term, which averages out over the keys) while l sums the unrounded values; o is rounded once.
//
// The keys and values lie in rows of the call's own buffers, so every tile is one or two TMA boxes
// (64 columns of 128 rows, 128-byte swizzle, which is the layout tcgen05.mma reads) and no warp
// gathers rows.  A work item is one sequence's kv head and 256 packed rows: the hq / hkv query
// heads of a kv head times as many tokens as fit 128 rows make a Q tile (row = token * heads +
// head), two Q tiles share each K/V tile of 128 keys.  One CTA per SM; the CTAs that run take the
// items of those that have not been launched (clusterlaunchcontrol.try_cancel), so the assignment
// is dynamic without a counter in memory: launches on several streams and replays of captured
// graphs share nothing.  Roles (512 threads):
//   warp 0      decodes the items taken, hands them on through a ring in shared memory, and loads their
//               Q tiles as the buffers come free
//   warp 1      issues the tcgen05.mma: per K/V tile j and Q tile t
//               O_t += P_t(j) V(j) in two halves of 64 keys as P comes in (P from TMEM), then at
//               once S_t(j+1) = Q_t K(j+1)^T over the columns P was read from, or the next item's
//               first scores
//   warp 2      loads K and V tiles into rings of their own, on into the next items, and asks for the next
//               item when it loads an item's last but one tile
//   warp 3      TMEM; clears what must not enter a sum (below)
//   warps 4-7, 8-11   softmax of Q tile 0 and 1, a row per thread
//   warps 12-15 the items' output from TMEM, while the others are on the next item
// While one tile's softmax runs the tensor core works on the other's products.
//
// What bounds it: for long prompts of 128-wide heads the tensor core (32/8 heads, one of 16384 tokens: 1.24
// to 1.37 ms from card to card, 1600 to 1770 TFLOP/s of 1950 measured for a burst and 1706 sustained; of 32768:
// 5.0 to 5.3 ms, 1660 to 1760): a step of 128 keys takes 2700 clocks, of which its products are 2048.  The
// issuing warp decides that: issued by one thread under `if (lane == 0)` the products took 75 clocks each
// instead of 64 (1254 TFLOP/s), and waits where its queue ran dry cost 500 clocks a step.  For 64-wide heads
// the softmax warps' own chain: a step takes about 2450 clocks, of which tensor core and exponentials are
// 1024 each, neither pipe busy for more than 45 % (four prompts of 4096 tokens, 12 heads: 106 us, twice the
// burst rate's time).  For short prompts the passage from one item to the next, 2 to 3 us of which
// instruction fetch is a part (32 prompts of 1024: 234 to 242 us, 1150 to 1180 TFLOP/s; the code was cut from
// 112 to 60 KB, which took that case from 391 to 230 us; 200 prompts of 64 tokens, 12 heads x 64: 51 us), and
// HBM (512 prompts of 64 tokens: 120 us for 670 MB, 82 % of the measured copy rate).
//
// Rows that a row must not see: a masked score is replaced after the product, so nothing of a
// hidden key survives, but P V multiplies hidden values by zero, and zero times an infinity or a
// NaN is not zero.  So in the tiles that the causal mask or the sequence's end cuts, warp 3 clears
// the value rows behind the end (another sequence's, or memory nobody wrote) and takes any
// non-finite elements out; the rows that do attend such a key get them back at the end of the
// item.  A row's result depends on rows 0..i of its own sequence alone.
//
// Every wait is bounded; on time-out the kernel records RX_DEV_TIMEOUT, waits for its copies,
// frees TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "prompt_items.cuh"
#include "prompt_wait.cuh"
#include "radix_attn.h"
#include "rx_common.h"
#include "rx_device.cuh"
#include "rx_kernels.h"
#include "rx_launch.h"

namespace rx {

constexpr int PT_BN = 128;         // keys per K/V tile
constexpr int PT_THREADS = 512;
constexpr int PT_RING = 4;         // items in flight between the roles
constexpr int PT_CONSUMERS = 15;   // MMA warp, K/V warp, clearing warp, eight softmax warps, four output warps
constexpr int PT_LEAD = 2;         // K/V tiles of an item still to be loaded when its successor is asked for
constexpr int PT_CUT = 3;          // K/V tiles of an item that a mask or the sequence's end can cut
// 2 * 128 * 80 + 2 * 128 * 176 = 512 * 128
constexpr uint32_t PT_REGS_SOFTMAX = 176, PT_REGS_OTHER = 80, PT_REGS_LAUNCH = 128;
constexpr float PT_LOG2E = 1.4426950408889634f;
constexpr float PT_LN2 = 0.6931471805599453f;
constexpr float PT_RESCALE = 8.0f;   // log2 units

struct PromptTcParams {
    PromptParams a;
    int32_t group;                 // query heads of a kv head
    int32_t hb, nhb;               // heads of a Q tile (at most 128), head blocks of a kv head
    int32_t tpt;                   // tokens of a Q tile
    PromptDiv by_tokens, by_heads; // tokens of an item, heads of a place
    float scale_log2;
    CUtensorMap q_map, k_map, v_map;
};

template <int D>
struct PtLayout {
    static constexpr int NK = D == 128 ? 3 : 4;    // K ring depth
    static constexpr int NV = D == 128 ? 2 : 4;    // V ring depth
    static constexpr int Q_TILE = 128 * D * 2;
    static constexpr int KV_TILE = PT_BN * D * 2;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + 2 * Q_TILE;
    static constexpr int OFF_V = OFF_K + NK * KV_TILE;
    static constexpr int OFF_BAR = OFF_V + NV * KV_TILE;
    static constexpr int NE = 4;                   // steps whose ends the loads may wait for
    static constexpr int BAR_Q = 0, BAR_KF = 2, BAR_VF = BAR_KF + NK, BAR_E = BAR_VF + NV,
                         BAR_VX = BAR_E + NE,      // a cut V tile is in, but not yet cleared
                         BAR_S = BAR_VX + NV, BAR_P = BAR_S + 2, BAR_QE = BAR_P + 4, BAR_OR = BAR_QE + 2,
                         BAR_OE = BAR_OR + 2, BAR_L = BAR_OE + 2, BAR_IF = BAR_L + 2, BAR_IE = BAR_IF + PT_RING,
                         BAR_IC = BAR_IE + PT_RING,   // every cut tile of an item has been cleared
                         BAR_CLC = BAR_IC + PT_RING, BAR_J = BAR_CLC + 1,   // (SPLIT) the two warpgroups' softmax joined
                         BAR_DONE = BAR_J + 1, NBAR = BAR_DONE + 1;
    static constexpr int OFF_CLC = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;   // answer of try_cancel
    static constexpr int OFF_RING = OFF_CLC + 16;                       // int4 per entry
    static constexpr int OFF_BAD = OFF_RING + 16 * PT_RING;             // non-finite keys: PT_CUT * 4 words per entry
    static constexpr int OFF_INV = OFF_BAD + PT_RING * PT_CUT * 16;     // 1 / l of each row of the Q tiles
    static constexpr int OFF_MISC = OFF_INV + 2 * 128 * 4;              // TMEM address, abort flag
    static constexpr int BYTES = OFF_MISC + 16;
    static constexpr int ALLOC = BYTES + 1024;   // room to align the base to 1024 B
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t COL_O0 = 256;
    static_assert(ALLOC <= 232448, "shared memory budget");
};

// One item as the roles see it: first row, length, first token, head; length < 0 ends the list.
struct PtItem {
    int start, n, t0, head;
    // K/V tiles of Q tile t (none: the tile has no token)
    __device__ __forceinline__ int nkv(int t, int tpt) const {
        const int first = t0 + t * tpt;
        return first < n ? (min(first + tpt, n) - 1) / PT_BN + 1 : 0;
    }
    // first K/V tile that some row of the item does not see whole
    __device__ __forceinline__ int first_cut() const { return (t0 + 1) / PT_BN; }
};

// ---------------------------------------------------------------- work from launches not begun
// Asks for a block of this grid that has not been launched; the 16-byte answer comes with the
// barrier's transaction.
__device__ __forceinline__ void clc_try_cancel(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
                 "r"(bar)
                 : "memory");
}

// The block taken, or -1: none was left (no further request may follow).
__device__ __forceinline__ int clc_answer(uint32_t answer) {
    uint32_t ok, x;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(ok), "=r"(x)
        : "r"(answer)
        : "memory");
    return ok ? (int)x : -1;
}

// ---------------------------------------------------------------- tensor core instructions of a warp
// The whole warp runs the issuing code, so that addresses and descriptors stay warp-uniform, and
// one elected lane issues a group of products.  (Issued under `if (lane == 0)`, one product at a
// time, they took 75 clocks each where the tensor core needs 64.)  Descriptors (sdesc_sw128) come as
// their low word (start address in 16-byte units, leading offset); the high word (stride offset 1024
// bytes, version, 128-byte swizzle) is the same for all.
constexpr uint32_t PT_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);

#define PT_SS(DA, DB, ACC)                                                     \
    "add.u32 a, %1, " #DA ";\n\tadd.u32 b, %2, " #DB ";\n\t"                   \
    "mov.b64 da, {a, %4};\n\tmov.b64 db, {b, %4};\n\t"                         \
    "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, " #ACC ";\n\t"
#define PT_TS(TA, DB, ACC)                                                     \
    "add.u32 a, %1, " #TA ";\n\tadd.u32 b, %2, " #DB ";\n\t"                   \
    "mov.b64 db, {b, %4};\n\t"                                                 \
    "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, " #ACC ";\n\t"
#define PT_GROUP "{\n\t.reg .pred e, t, f;\n\t.reg .b32 a, b;\n\t.reg .b64 da, db;\n\telect.sync _|e, 0xffffffff;\n\t"

// S[128 x 128] = Q K^T over D channels: 16 channels (32 bytes) an instruction, 64 a 16 KB half tile.
template <int D>
__device__ __forceinline__ void pt_mma_s(uint32_t s, uint32_t q, uint32_t k, uint32_t idesc) {
    if constexpr (D == 128)
        asm volatile(PT_GROUP "setp.eq.u32 t, 0, 0;\n\tsetp.ne.u32 f, 0, 0;\n\t" PT_SS(0, 0, f) PT_SS(2, 2, t) PT_SS(4, 4, t)
                         PT_SS(6, 6, t) PT_SS(1024, 1024, t) PT_SS(1026, 1026, t) PT_SS(1028, 1028, t) PT_SS(1030, 1030, t) "}" ::"r"(s),
                     "r"(q), "r"(k), "r"(idesc), "r"(PT_DESC_HI)
                     : "memory");
    else
        asm volatile(PT_GROUP "setp.eq.u32 t, 0, 0;\n\tsetp.ne.u32 f, 0, 0;\n\t" PT_SS(0, 0, f) PT_SS(2, 2, t) PT_SS(4, 4, t)
                         PT_SS(6, 6, t) "}" ::"r"(s),
                     "r"(q), "r"(k), "r"(idesc), "r"(PT_DESC_HI)
                     : "memory");
}

// O[128 x D] += P V over 64 keys: 16 keys (8 TMEM columns of P, 2 KB of V) an instruction; with
// `fresh` the first of them overwrites O.
__device__ __forceinline__ void pt_mma_pv(uint32_t o, uint32_t pt, uint32_t v, uint32_t idesc, bool fresh) {
    asm volatile(PT_GROUP "setp.eq.u32 t, 0, 0;\n\tsetp.eq.u32 f, %5, 0;\n\t" PT_TS(0, 0, f) PT_TS(8, 128, t) PT_TS(16, 256, t)
                     PT_TS(24, 384, t) "}" ::"r"(o),
                 "r"(pt), "r"(v), "r"(idesc), "r"(PT_DESC_HI), "r"(fresh ? 1u : 0u)
                 : "memory");
}
#undef PT_SS
#undef PT_TS
#undef PT_GROUP

__device__ __forceinline__ void pt_commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// SPLIT: an item is one Q tile, and the two softmax warpgroups, S and O take its K/V tiles in turn (even
// and odd ones) and join at the end: half as many steps, one after another, for calls of few items.  (One prompt of 409 tokens, 12 heads x 64: 7.3 us, and 7.9 with one K/V tile after
// another; of 1024 tokens: 10.2 and 11.9.)
template <int D, bool SPLIT>
__global__ void __launch_bounds__(PT_THREADS, 1) prompt_tc_kernel(const __grid_constant__ PromptTcParams p) {
    using LY = PtLayout<D>;
    constexpr int NK = LY::NK, NV = LY::NV;
    constexpr int TILES = SPLIT ? 1 : 2;       // Q tiles of an item
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    const uint32_t bar0 = base + LY::OFF_BAR;
    auto bar = [&](int i) { return bar0 + (uint32_t)(8 * i); };
    volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(gbase + LY::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + LY::OFF_MISC + 4);
    int4* ring = reinterpret_cast<int4*>(gbase + LY::OFF_RING);
    uint32_t* bad = reinterpret_cast<uint32_t*>(gbase + LY::OFF_BAD);
    float* inv_l = reinterpret_cast<float*>(gbase + LY::OFF_INV);
    int32_t* const status = p.a.status;
    // from a shuffle, as the items below: so that the compiler knows them the same for the whole warp
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NK; ++i) mbar_init(bar(LY::BAR_KF + i), 1);
        for (int i = 0; i < LY::NE; ++i) mbar_init(bar(LY::BAR_E + i), 1);
        for (int i = 0; i < NV; ++i) {
            mbar_init(bar(LY::BAR_VF + i), 1);
            mbar_init(bar(LY::BAR_VX + i), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(LY::BAR_Q + t), 1);
            mbar_init(bar(LY::BAR_S + t), 1);
            mbar_init(bar(LY::BAR_P + t), 4);          // one arrival per softmax warp, keys 0-63
            mbar_init(bar(LY::BAR_P + 2 + t), 4);      // keys 64-127
            mbar_init(bar(LY::BAR_QE + t), 1);         // Q buffer t read by its item's last S
            mbar_init(bar(LY::BAR_OR + t), 1);         // O_t of an item complete
            mbar_init(bar(LY::BAR_OE + t), 4);         // and read by the output warps
            mbar_init(bar(LY::BAR_L + t), 4);          // 1 / l of an item's rows written
        }
        for (int i = 0; i < PT_RING; ++i) {
            mbar_init(bar(LY::BAR_IF + i), 1);
            mbar_init(bar(LY::BAR_IE + i), PT_CONSUMERS);
            mbar_init(bar(LY::BAR_IC + i), 1);
        }
        mbar_init(bar(LY::BAR_CLC), 1);
        mbar_init(bar(LY::BAR_J), 8);
        mbar_init(bar(LY::BAR_DONE), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc(base + LY::OFF_MISC, LY::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_launch_dependents();
    pdl_wait();                          // what came before has finished; nothing global was touched so far

    auto ring_item = [&](int k, PtItem& it) {          // item k of this CTA
        const int4 r = ring[k % PT_RING];
        it.start = __shfl_sync(0xffffffffu, r.x, 0), it.n = __shfl_sync(0xffffffffu, r.y, 0);
        it.t0 = __shfl_sync(0xffffffffu, r.z, 0), it.head = __shfl_sync(0xffffffffu, r.w, 0);
    };

    // Asks for a block that has not been launched.  The K/V warp does when it comes to an item's last tiles:
    // asked for as soon as there was room for them, the first few items of each block were shared out at the
    // launch's beginning, whoever was done first (one of 2000 tokens, 32/8 heads x 128: 27 us, and 35; of 4096: 86
    // and 92; 250 prompts of 64 tokens alike).  Warp 0 does where its place has no item.
    auto ask = [&]() {
        if (lane == 0) {
            mbar_arrive_expect_tx(bar(LY::BAR_CLC), 16);
            clc_try_cancel(base + LY::OFF_CLC, bar(LY::BAR_CLC));
        }
    };

    if (warp < 4) {
        regs_decrease<PT_REGS_OTHER>();
        if (warp == 0) {
            // ------------------------------------------------------------ items and Q
            int place = (int)blockIdx.x;
            PromptFinder finder;
            int k = 0, use0 = 0, use1 = 0, asked = 0;
            bool ok = true;
            for (;;) {
                PromptItem w;
                if (finder.find(p.a, place, p.by_tokens, p.by_heads, w)) {
                    PtItem it;
                    it.start = w.start, it.n = w.n, it.t0 = w.tile * p.tpt * TILES, it.head = w.head;
                    const int e = k % PT_RING;
                    ok = k < PT_RING || pt_wait(bar(LY::BAR_IE + e), ((k / PT_RING) - 1) & 1, abort_flag);
                    if (ok && lane == 0) {
                        ring[e] = make_int4(it.start, it.n, it.t0, it.head);
                        mbar_arrive(bar(LY::BAR_IF + e));
                    }
                    ++k;
                    const bool two = TILES > 1 && it.nkv(1, p.tpt) > 0;
                    const int g = it.head / p.nhb, h0 = g * p.group + (it.head - g * p.nhb) * p.hb;
#pragma unroll 1
                    for (int t = 0; ok && t < (two ? 2 : 1); ++t) {
                        const int use = t == 0 ? use0 : use1;
                        ok = use == 0 || pt_wait(bar(LY::BAR_QE + t), (use - 1) & 1, abort_flag);
                        if (!ok) break;
                        use0 += t == 0 ? 1 : 0;
                        use1 += t;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(bar(LY::BAR_Q + t), (uint32_t)(p.hb * p.tpt * D * 2));
#pragma unroll 1
                            for (int c = 0; c < D / 64; ++c)
                                tma_load_3d(base + LY::OFF_Q + t * LY::Q_TILE + c * 128 * 128, &p.q_map, c * 64, h0,
                                            it.start + it.t0 + t * p.tpt, bar(LY::BAR_Q + t));
                        }
                    }
                    if (!ok) break;
                } else {
                    ask();
                }
                if (lane == 0) PromptFinder::check(p.a, place);     // while the answer is on its way
                ok = pt_wait(bar(LY::BAR_CLC), asked & 1, abort_flag);
                if (!ok) break;
                ++asked;
                place = clc_answer(base + LY::OFF_CLC);
                fence_proxy_async_smem();     // the answer is read before the next one is written
                __syncwarp();
                if (place < 0) break;
            }
            if (ok) {
                const int e = k % PT_RING;
                ok = k < PT_RING || pt_wait(bar(LY::BAR_IE + e), ((k / PT_RING) - 1) & 1, abort_flag);
                if (ok && lane == 0) {
                    ring[e] = make_int4(0, -1, 0, 0);
                    mbar_arrive(bar(LY::BAR_IF + e));
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ tcgen05.mma
            constexpr uint32_t IDESC_S = idesc_bf16_f32(128, PT_BN, 0, 0);
            constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, 0, 1);
            const uint32_t qd0 = (uint32_t)sdesc_sw128(base + LY::OFF_Q, 16, 1024);
            const uint32_t kd0 = (uint32_t)sdesc_sw128(base + LY::OFF_K, 16, 1024);
            const uint32_t vd0 = (uint32_t)sdesc_sw128(base + LY::OFF_V, PT_BN * 128, 1024);
            auto issue_s = [&](int t, uint32_t ks, bool last) {     // last: no later S of this item reads Q_t
                pt_mma_s<D>(tmem + t * PT_BN, qd0 + t * (uint32_t)(LY::Q_TILE >> 4), kd0 + ks * (uint32_t)(LY::KV_TILE >> 4), IDESC_S);
                pt_commit(bar(LY::BAR_S + t));
                if (last) pt_commit(bar(LY::BAR_QE + t));
            };
            auto issue_pv = [&](int t, uint32_t vs, int h, bool fresh) {   // keys 64h .. 64h+63 of the tile
                pt_mma_pv(tmem + LY::COL_O0 + t * D, tmem + t * PT_BN + h * 32, vd0 + vs * (uint32_t)(LY::KV_TILE >> 4) + h * 512u,
                          IDESC_PV, fresh);
            };
            auto ready = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test(b, parity)); };
            if constexpr (SPLIT) {
                // K/V tile i of an item goes through S and O of warpgroup i % 2
                int gt = 0;                         // K/V tiles so far
                uint32_t pph = 0, odd = 0, had = 0;   // by bits, as below
                bool ok = true;
                for (int k = 0; ok; ++k) {
                    const int e = k % PT_RING;
                    if (!pt_wait(bar(LY::BAR_IF + e), (k / PT_RING) & 1, abort_flag)) break;
                    PtItem it;
                    ring_item(k, it);
                    if (it.n < 0) break;
                    const int total = it.nkv(0, p.tpt);
                    ok = pt_wait(bar(LY::BAR_Q), k & 1, abort_flag);
#pragma unroll 1
                    for (int i = -2; ok && i < total; ++i) {
                        const uint32_t t = i & 1;
                        if (i >= 0) {
                            const int u = gt + i;
                            ok = pt_wait(bar(LY::BAR_VF + u % NV), (u / NV) & 1, abort_flag) &&
                                 // the previous item's O_t has been read out
                                 (i > 1 || !((had >> t) & 1u) || pt_wait(bar(LY::BAR_OE + t), ((odd >> t) & 1u) ^ 1u, abort_flag));
#pragma unroll 1
                            for (int h = 0; ok && h < 2; ++h) {
                                ok = pt_wait(bar(LY::BAR_P + 2 * h + t), (pph >> t) & 1u, abort_flag);
                                tc_fence_after();
                                if (ok) issue_pv(t, u % NV, h, i < 2 && h == 0);
                            }
                            if (!ok) break;
                            pph ^= 1u << t;
                        }
                        if (i + 2 < total) {
                            const int u = gt + i + 2;
                            ok = pt_wait(bar(LY::BAR_KF + u % NK), (u / NK) & 1, abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            pt_mma_s<D>(tmem + t * PT_BN, qd0, kd0 + (uint32_t)(u % NK) * (uint32_t)(LY::KV_TILE >> 4), IDESC_S);
                            pt_commit(bar(LY::BAR_S + t));
                            if (i + 3 == total) pt_commit(bar(LY::BAR_QE));   // Q read for this item
                        } else if (i >= 0) {
                            pt_commit(bar(LY::BAR_OR + t));                   // O_t of this item complete
                        }
                        if (i >= 0) pt_commit(bar(LY::BAR_E + (gt + i) % LY::NE));
                    }
                    gt += total;
                    odd ^= total > 1 ? 3u : 1u;
                    had |= total > 1 ? 3u : 1u;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(LY::BAR_IE + e));
                }
            } else {
                // ring positions: the next K tile to be multiplied by Q, the V tile of the current step, the step's end
                uint32_t ks = 0, kph = 0, vs = 0, vph = 0, es = 0;
                auto k_next = [&](uint32_t& slot, uint32_t& ph) {
                    if (++slot == NK) slot = 0, ph ^= 1;
                };
                // by bits, one for each Q tile: phase of its P barriers (a step each), parity of its items so
                // far, whether it has had any, and whether S of the coming item's first K tile is on its way
                uint32_t pph = 0, odd = 0, had = 0, issued = 0;
                PtItem nx{};                    // the coming item, where it was there to be read in time
                bool have_nx = false;
                bool ok = true;
                // The tensor core works off what is issued in order and with some 400 clocks of it in its
                // queue; what this warp does between two groups of products has to fit into that.  So the
                // waits for K and V, which are long there, stand where the queue is full, and a step's end is
                // committed once for the K and the V tile that it frees.
                for (int k = 0; ok; ++k) {
                    const int e = k % PT_RING;
                    if (!have_nx) {
                        if (!pt_wait(bar(LY::BAR_IF + e), (k / PT_RING) & 1, abort_flag)) break;
                        ring_item(k, nx);
                    }
                    const PtItem it = nx;
                    if (it.n < 0) break;
                    have_nx = false;
                    const int n0 = it.nkv(0, p.tpt), n1 = TILES > 1 ? it.nkv(1, p.tpt) : 0;
                    const int nkv = max(n0, n1);
#pragma unroll 1
                    for (int t = 0; ok && t < 2; ++t) {
                        const int nt = t == 0 ? n0 : n1;
                        if (nt == 0 || ((issued >> t) & 1u)) continue;
                        ok = pt_wait(bar(LY::BAR_Q + t), (odd >> t) & 1u, abort_flag) && pt_wait(bar(LY::BAR_KF + ks), kph, abort_flag);
                        tc_fence_after();
                        if (ok) issue_s(t, ks, nt == 1);
                    }
                    issued = 0;
                    k_next(ks, kph);
                    bool have_v = false;        // the step's V has been seen to be there
                    for (int j = 0; ok && j < nkv; ++j) {
                        const bool more = j + 1 < nkv;
                        uint32_t vs1 = vs + 1, vph1 = vph;
                        if (vs1 == NV) vs1 = 0, vph1 ^= 1;
                        if (more && !(ok = pt_wait(bar(LY::BAR_KF + ks), kph, abort_flag))) break;
                        if (j + 1 == n0) {                        // the coming item, for its first scores
                            const int e2 = (k + 1) % PT_RING;
                            have_nx = ready(bar(LY::BAR_IF + e2), ((k + 1) / PT_RING) & 1);
                            if (have_nx) ring_item(k + 1, nx);
                        }
                        if (!have_v && !(ok = pt_wait(bar(LY::BAR_VF + vs), vph, abort_flag))) break;
                        have_v = false;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int nt = t == 0 ? n0 : n1;
                            if (j >= nt) continue;
                            // the previous item's O_t has been read out
                            if (j == 0 && ((had >> t) & 1u) && !(ok = pt_wait(bar(LY::BAR_OE + t), ((odd >> t) & 1u) ^ 1u, abort_flag))) break;
#pragma unroll 1
                            for (int h = 0; ok && h < 2; ++h) {
                                ok = pt_wait(bar(LY::BAR_P + 2 * h + t), (pph >> t) & 1u, abort_flag);
                                tc_fence_after();
                                if (ok) issue_pv(t, vs, h, j == 0 && h == 0);
                            }
                            if (!ok) break;
                            pph ^= 1u << t;
                            if (more && (t == 1 || j >= n1)) have_v = ready(bar(LY::BAR_VF + vs1), vph1);
                            // the tile's next scores: of the next step, or of the coming item's first if all they
                            // need is here already; their softmax then runs under this item's last products
                            uint32_t kk = ks, kkph = kph;
                            bool go = j + 1 < nt, last = j + 2 == nt;
                            if (!go) {
                                pt_commit(bar(LY::BAR_OR + t));   // O_t of this item complete
                                if (t == 0 && more) k_next(kk, kkph);
                                if (have_nx && nx.n >= 0) {
                                    const int nn = nx.nkv(t, p.tpt);
                                    last = nn == 1;
                                    go = nn > 0 && ready(bar(LY::BAR_Q + t), ((odd >> t) & 1u) ^ 1u) &&
                                         (t == 0 ? ready(bar(LY::BAR_KF + kk), kkph) : (issued & 1u) != 0);
                                    tc_fence_after();
                                    if (go) issued |= 1u << t;
                                }
                            }
                            if (go) issue_s(t, kk, last);
                        }
                        if (!ok) break;
                        pt_commit(bar(LY::BAR_E + es));       // this step's V and the next one's K are read
                        es = (es + 1) % LY::NE;
                        if (more) k_next(ks, kph);
                        vs = vs1, vph = vph1;
                    }
                    odd ^= n1 > 0 ? 3u : 1u;
                    had |= n1 > 0 ? 3u : 1u;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(LY::BAR_IE + e));
                }
            }
            pt_commit(bar(LY::BAR_DONE));
            __syncwarp();
        } else if (warp == 2) {
            // ------------------------------------------------------------ K and V tiles
            // Step u's end (BAR_E) means that the tensor core is done with V tile u, and with K tile u
            // and, within the item, u + 1.
            int gt = 0, ended = 0;        // tiles loaded, and steps whose end has been waited for, so far
            bool ok = true;
            auto freed = [&](int steps) {
                while (ok && ended < steps) {
                    ok = pt_wait(bar(LY::BAR_E + ended % LY::NE), (ended / LY::NE) & 1, abort_flag);
                    ++ended;
                }
                return ok;
            };
            for (int k = 0; ok; ++k) {
                const int e = k % PT_RING;
                if (!pt_wait(bar(LY::BAR_IF + e), (k / PT_RING) & 1, abort_flag)) break;
                PtItem it;
                ring_item(k, it);
                if (it.n < 0) break;
                const int nkv = max(it.nkv(0, p.tpt), TILES > 1 ? it.nkv(1, p.tpt) : 0);
                const int g = it.head / p.nhb, cut = it.first_cut();
                for (int j = 0; j < nkv; ++j) {
                    const int u = gt + j, ks = u % NK, vs = u % NV;
                    // a cut V tile goes to warp 3 first, which hands it on (at most one per slot is on its way)
                    const uint32_t kf = bar(LY::BAR_KF + ks), vf = bar((j >= cut ? LY::BAR_VX : LY::BAR_VF) + vs);
#pragma unroll 1
                    for (int v = 0; v < 2; ++v) {
                        if (!freed(u + 1 - (v ? NV : NK))) break;
                        const uint32_t full = v ? vf : kf, to = base + (v ? LY::OFF_V + vs * LY::KV_TILE : LY::OFF_K + ks * LY::KV_TILE);
                        if (lane == 0) {
                            mbar_arrive_expect_tx(full, LY::KV_TILE);
#pragma unroll 1
                            for (int c = 0; c < D / 64; ++c)
                                tma_load_3d(to + c * PT_BN * 128, v ? &p.v_map : &p.k_map, c * 64, g, it.start + j * PT_BN, full);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (j == max(nkv - PT_LEAD, 0)) ask();
                }
                gt += nkv;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(LY::BAR_IE + e));
            }
        } else {
            // ------------------------------------------------------------ cut V tiles
            int gt = 0;
            uint32_t ph = 0;                                // phase of each slot's BAR_VX
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int e = k % PT_RING;
                if (!pt_wait(bar(LY::BAR_IF + e), (k / PT_RING) & 1, abort_flag)) break;
                PtItem it;
                ring_item(k, it);
                if (it.n < 0) break;
                const int nkv = max(it.nkv(0, p.tpt), TILES > 1 ? it.nkv(1, p.tpt) : 0), cut = it.first_cut();
                uint32_t* mask = bad + e * PT_CUT * 4;      // read by the softmax warps before the entry is used again
                if (lane < PT_CUT * 4) mask[lane] = 0;
                __syncwarp();
                for (int j = cut; j < nkv; ++j) {
                    const int vs = (gt + j) % NV;
                    ok = pt_wait(bar(LY::BAR_VX + vs), (ph >> vs) & 1, abort_flag);
                    ph ^= 1u << vs;
                    if (!ok) break;
                    uint4* tile = reinterpret_cast<uint4*>(gbase + LY::OFF_V + vs * LY::KV_TILE);   // [D / 64][128 rows][8]
                    const int rows = it.n - j * PT_BN;      // rows of the sequence in this tile
                    if (rows < PT_BN) {
#pragma unroll 1
                        for (int i = rows * 8 + lane; i < PT_BN * 8; i += 32)
#pragma unroll
                            for (int c = 0; c < D / 64; ++c) tile[c * PT_BN * 8 + i] = make_uint4(0, 0, 0, 0);
                        __syncwarp();
                    }
                    // 0 * x summed over the tile: NaN if and only if some x is not finite
                    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
                    __nv_bfloat162 acc[4] = {zero, zero, zero, zero};
#pragma unroll 4
                    for (int i = lane; i < PT_BN * D / 8; i += 32) {
                        const uint4 x = tile[i];
                        acc[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.x), zero, acc[0]);
                        acc[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.y), zero, acc[1]);
                        acc[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.z), zero, acc[2]);
                        acc[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.w), zero, acc[3]);
                    }
                    const float2 f0 = __bfloat1622float2(__hadd2(acc[0], acc[1])), f1 = __bfloat1622float2(__hadd2(acc[2], acc[3]));
                    const float sum = f0.x + f0.y + f1.x + f1.y;
                    if (__any_sync(0xffffffffu, sum != sum)) {
#pragma unroll 1
                        for (int i = lane; i < PT_BN * D / 8; i += 32) {
                            uint4 x = tile[i];
                            uint32_t* w = reinterpret_cast<uint32_t*>(&x);
                            bool any = false;
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                if ((w[c] & 0x7f80u) == 0x7f80u) w[c] &= 0xffff0000u, any = true;
                                if ((w[c] & 0x7f800000u) == 0x7f800000u) w[c] &= 0x0000ffffu, any = true;
                            }
                            if (any) {
                                tile[i] = x;
                                const int row = (i >> 3) & (PT_BN - 1);
                                atomicOr(mask + (j - cut) * 4 + (row >> 5), 1u << (row & 31));
                            }
                        }
                    }
                    fence_proxy_async_smem();               // cleared before the tensor core reads
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(LY::BAR_VF + vs));
                }
                if (!ok) break;
                gt += nkv;
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(LY::BAR_IC + e));
                    mbar_arrive(bar(LY::BAR_IE + e));
                }
            }
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------ softmax warpgroups
        regs_increase<PT_REGS_SOFTMAX>();
        const int t = (warp >> 2) - 1;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + t * PT_BN;   // scores, then P over them
        const uint32_t o_addr = tmem + lane_base + LY::COL_O0 + t * D;   // rescaled here, read out by the output warps
        const float sl = p.scale_log2;
        const int row_tok = r / p.hb, row_head = r - row_tok * p.hb;
        int sc = 0, oc = 0;                   // score steps, and items (SPLIT: joins), of this Q tile so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int e = k % PT_RING;
            if (!pt_wait(bar(LY::BAR_IF + e), (k / PT_RING) & 1, abort_flag)) break;
            PtItem it;
            ring_item(k, it);
            if (it.n < 0) break;
            const int total = it.nkv(0, p.tpt);            // (SPLIT) K/V tiles of both warpgroups
            const int nkv = SPLIT ? (total + 1 - t) / 2 : it.nkv(t, p.tpt);
            const int tok = it.t0 + (SPLIT ? 0 : t * p.tpt) + row_tok;
            const int pos = min(tok, it.n - 1);          // attends keys 0..pos
            float m_ref = -INFINITY, l = 0.f;
            for (int j = 0; j < nkv; ++j) {
                if (!pt_wait(bar(LY::BAR_S + t), (sc + j) & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                float s[PT_BN];
#pragma unroll
                for (int c = 0; c < PT_BN; c += 32) tmem_ld32(s_addr + c, s + c);
                tmem_wait_ld();
                const int lim = pos - (SPLIT ? 2 * j + t : j) * PT_BN;   // columns past lim are masked
                if (lim < PT_BN - 1) {
#pragma unroll
                    for (int c = 0; c < PT_BN; c += 32) {
                        const int left = lim - c;      // of these 32 columns, 0 .. left are seen
                        const uint32_t see = left >= 31 ? 0xffffffffu : left < 0 ? 0u : (2u << left) - 1u;
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (!((see >> x) & 1u)) s[c + x] = -INFINITY;
                    }
                }
                float mx8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mx8[i] = s[i];
#pragma unroll
                for (int c = 8; c + 16 <= PT_BN; c += 16)
#pragma unroll
                    for (int i = 0; i < 8; ++i) mx8[i] = fmax3(mx8[i], s[c + i], s[c + 8 + i]);
#pragma unroll
                for (int i = 0; i < 8; ++i) mx8[i] = fmaxf(mx8[i], s[PT_BN - 8 + i]);
                float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
                mx *= sl;
                float m_new = m_ref;
                if (m_ref == -INFINITY || mx > m_ref + PT_RESCALE) m_new = fmaxf(m_ref, mx);
                const float alpha = (m_ref == -INFINITY) ? 0.f : fast_exp2(m_ref - m_new);
                const bool rescale = j > 0 && __any_sync(0xffffffffu, m_new != m_ref);
                l *= alpha;
                m_ref = m_new;
                const float sub = m_new == -INFINITY ? 0.f : m_new;   // nothing but -inf so far
                const uint64_t sl2 = f2_pack(sl, sl), nm2 = f2_pack(-sub, -sub);
                uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
                // P in two halves of 64 keys (32 columns), each published as soon as it is stored
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[PT_BN / 4];
#pragma unroll
                    for (int cc = 0; cc < PT_BN / 2; cc += 2) {
                        const int c = h * (PT_BN / 2) + cc;
                        const uint64_t x2 = f2_fma(f2_pack(s[c], s[c + 1]), sl2, nm2);
                        float x0, x1;
                        f2_unpack(x2, x0, x1);
                        const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
                        acc2[(c >> 1) & 3] = f2_add(acc2[(c >> 1) & 3], f2_pack(e0, e1));
                        pk[cc >> 1] = pack_bf16x2(e0, e1);
                    }
                    tmem_st32u(s_addr + h * 32, pk);
                    if (h == 0 && rescale) {
                        // PV_t(j-1) has completed (S_t(j) was issued after it and is complete),
                        // and PV_t(j) waits for the arrival below.  Rare: rolled.
#pragma unroll 1
                        for (int cc = 0; cc < D; cc += 32) {
                            float ov[32];
                            tmem_ld32(o_addr + cc, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 32; ++x) ov[x] *= alpha;
                            tmem_st32(o_addr + cc, ov);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(LY::BAR_P + 2 * h + t));
                }
                const uint64_t a01 = f2_add(f2_add(acc2[0], acc2[1]), f2_add(acc2[2], acc2[3]));
                float ra, rb;
                f2_unpack(a01, ra, rb);
                l += ra + rb;
            }
            if (!ok) break;
            sc += nkv;
            if constexpr (SPLIT) {
                // Both warpgroups' maximum and sum of each row through the output's factors: first m, then
                // l 2^(m - M), then the factor 2^(m - M) / L of each one's O.
                float* const mine = inv_l + t * 128 + r;
                const float* const other = inv_l + (1 - t) * 128 + r;
                auto joined = [&]() {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(LY::BAR_J));
                    const bool got = pt_wait(bar(LY::BAR_J), oc & 1, abort_flag);
                    ++oc;
                    return got;
                };
                if (k > 0 && !pt_wait(bar(LY::BAR_OE), (k - 1) & 1, abort_flag)) break;   // the last item's have been read
                *mine = m_ref;
                if (!joined()) break;
                const float m = fmaxf(m_ref, *other);
                const float a = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - m);
                if (!joined()) break;
                *mine = l * a;
                if (!joined()) break;
                const float sum = l * a + *other;
                if (!joined()) break;
                *mine = a / sum;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(LY::BAR_L + t));
                const int g = it.head / p.nhb, hh = (it.head - g * p.nhb) * p.hb + row_head;
                if (t == 0 && p.a.lse && row_tok < p.tpt && tok < it.n && hh < p.group)
                    p.a.lse[((int64_t)it.start + tok) * p.a.hq + g * p.group + hh] = (m + log2f(sum)) * PT_LN2;
            } else if (nkv > 0) {
                // 1 / l for the output warps, once they have read the last item's
                if (oc > 0 && !pt_wait(bar(LY::BAR_OE + t), (oc - 1) & 1, abort_flag)) break;
                oc += 1;
                inv_l[t * 128 + r] = 1.f / l;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(LY::BAR_L + t));
                const int g = it.head / p.nhb, hh = (it.head - g * p.nhb) * p.hb + row_head;
                if (p.a.lse && row_tok < p.tpt && tok < it.n && hh < p.group)
                    p.a.lse[((int64_t)it.start + tok) * p.a.hq + g * p.group + hh] = (m_ref + log2f(l)) * PT_LN2;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(LY::BAR_IE + e));
        }
    } else {
        // ------------------------------------------------------------ output
        regs_decrease<PT_REGS_OTHER>();
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const int row_tok = r / p.hb, row_head = r - row_tok * p.hb;
        uint32_t ph = 0;                         // phases of the tiles' barriers (bit t), an item each
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int e = k % PT_RING;
            if (!pt_wait(bar(LY::BAR_IF + e), (k / PT_RING) & 1, abort_flag)) break;
            PtItem it;
            ring_item(k, it);
            if (it.n < 0) break;
            const int g = it.head / p.nhb, hh = (it.head - g * p.nhb) * p.hb + row_head;
            const uint32_t* mask = bad + e * PT_CUT * 4;
            const int nt = TILES > 1 && it.nkv(1, p.tpt) > 0 ? 2 : 1;
            const bool both = SPLIT && it.nkv(0, p.tpt) > 1;      // O_1 holds the odd K/V tiles' part
#pragma unroll 1
            for (int t = 0; t < nt; ++t) {
                ok = pt_wait(bar(LY::BAR_L + t), SPLIT ? k & 1 : (ph >> t) & 1, abort_flag) &&
                     pt_wait(bar(LY::BAR_OR + t), (ph >> t) & 1, abort_flag) && pt_wait(bar(LY::BAR_IC + e), (k / PT_RING) & 1, abort_flag);
                if constexpr (SPLIT)
                    ok = ok && pt_wait(bar(LY::BAR_L + 1), k & 1, abort_flag) &&
                         (!both || pt_wait(bar(LY::BAR_OR + 1), (ph >> 1) & 1, abort_flag));
                if (!ok) break;
                ph ^= both ? 3u : 1u << t;
                tc_fence_after();
                const bool any = __any_sync(0xffffffffu, lane < PT_CUT * 4 && mask[lane] != 0);
                const float inv = inv_l[t * 128 + r], inv1 = SPLIT ? inv_l[128 + r] : 0.f;
                const int tok = it.t0 + t * p.tpt + row_tok;
                const bool valid = row_tok < p.tpt && tok < it.n && hh < p.group;
                const uint32_t o_addr = tmem + ((uint32_t)(quarter * 32) << 16) + LY::COL_O0 + t * D;
                __nv_bfloat16* orow =
                    (__nv_bfloat16*)p.a.out + ((int64_t)it.start + tok) * p.a.out_stride + (int64_t)(g * p.group + hh) * D;
                // Four neighbouring lanes trade 16-byte pieces so that together they write 64 bytes of one row
                // at a time: whole sectors, and a quarter of the lines an instruction touches.
                uint64_t to[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    to[i] = __shfl_sync(0xffffffffu, (unsigned long long)(uintptr_t)(valid ? orow : nullptr), (lane & ~3) + i);
#pragma unroll 1
                for (int cc = 0; cc < D; cc += 32) {
                    float ov[32];
                    tmem_ld32(o_addr + cc, ov);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 32; ++x) ov[x] *= inv;
                    if constexpr (SPLIT) {
                        if (both) {
                            float o1[32];
                            tmem_ld32(o_addr + D + cc, o1);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 32; ++x) ov[x] = fmaf(o1[x], inv1, ov[x]);
                        }
                    }
                    if (cc + 32 == D) {          // read: the next item's first product may overwrite it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (both) mbar_arrive(bar(LY::BAR_OE + 1));
                            mbar_arrive(bar(LY::BAR_OE + t));
                        }
                    }
                    uint32_t w[16];                  // four pieces of 8 columns
#pragma unroll
                    for (int x = 0; x < 16; ++x) w[x] = pack_bf16x2(ov[2 * x], ov[2 * x + 1]);
#pragma unroll
                    for (int b = 1; b < 4; b <<= 1)  // piece c of lane l changes places with piece l of lane c
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (!(c & b))
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    const bool up = lane & b;
                                    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[4 * c + x] : w[4 * (c ^ b) + x], b);
                                    if (up) w[4 * c + x] = got;
                                    else w[4 * (c ^ b) + x] = got;
                                }
#pragma unroll
                    for (int i = 0; i < 4; ++i)      // piece lane % 4 of row i of the four
                        if (to[i])
                            reinterpret_cast<uint4*>((uintptr_t)to[i] + cc * 2)[lane & 3] =
                                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    __syncwarp();                    // the whole warp reads the next columns
                }
                // the non-finite values of the keys this row attends, added to what was just stored (by other
                // lanes: seen after the warp's barrier above)
                if (any && valid) {
#pragma unroll 1
                    for (int w = 0; w < PT_CUT * 4; ++w)
#pragma unroll 1
                        for (uint32_t b = mask[w]; b; b &= b - 1) {
                            const int key = it.first_cut() * PT_BN + w * 32 + __ffs(b) - 1;
                            if (key > tok) break;
                            const __nv_bfloat16* vr =
                                (const __nv_bfloat16*)p.a.v + ((int64_t)it.start + key) * p.a.v_stride + (int64_t)g * D;
#pragma unroll 1
                            for (int x = 0; x < D; ++x) {
                                const float f = __bfloat162float(vr[x]);
                                if (!isfinite(f)) orow[x] = __float2bfloat16_rn(__bfloat162float(orow[x]) + f);
                            }
                        }
                }
                __syncwarp();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(LY::BAR_IE + e));
        }
    }
    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // Copies and an answer may still be on their way to shared memory.  What phase of which barrier
        // each went to is not worth keeping for this case: wait out the time that any of them takes.
        if (threadIdx.x == 0) report(status, RX_DEV_TIMEOUT);
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 10000000ull) __nanosleep(1000);
    }
    if (warp == 3) {
        tc_fence_after();
        // every MMA this CTA issued has completed before TMEM is released; this wait does not stop
        // on the abort flag (only on its own time bound)
        volatile int no_abort = 0;
        warp_wait(bar(LY::BAR_DONE), 0, &no_abort, status, 500000000ull);
        tmem_dealloc(tmem, LY::TMEM_COLS);
    }
}

// cuTensorMapEncodeTiled from the driver, resolved once through the runtime (no -lcuda).
static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// Tensor map of bf16 rows [rows][heads][D], `stride` elements between rows: boxes of 64 columns x
// `heads_box` heads x `rows_box` rows, 128-byte swizzle.  Rows past the end read as zeros.
static bool rows_map(CUtensorMap* m, const void* ptr, int64_t rows, int heads, int D, int64_t stride, int heads_box, int rows_box) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)heads_box, (cuuint32_t)rows_box};
    const cuuint32_t elem[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, elem,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The device's SM count; 0 with a message where the current device is not an sm_103.
static int device_sms() {
    static PerDeviceOnce once;
    static int counts[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        set_error("prompt_attention: cannot query the device");
        return 0;
    }
    per_device_once(once, [&] {
        int major = 0, minor = 0, n = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            set_error("prompt_attention: cannot query the device");
            return (int)RX_ECUDA;
        }
        if (major != 10 || minor != 3) {
            set_error("prompt_attention: the tcgen05 kernel needs an sm_103 (GB300) device");
            return (int)RX_EDEVICE;
        }
        counts[dev] = n;
        return (int)RX_OK;
    });
    return counts[dev];
}

template <int D, bool SPLIT>
static int launch_pt(const PromptTcParams& p, unsigned grid, cudaStream_t stream) {
    static PerDeviceOnce attr;
    const int rc = per_device_once(attr, [] {
        const cudaError_t e =
            cudaFuncSetAttribute(prompt_tc_kernel<D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, PtLayout<D>::ALLOC);
        if (e != cudaSuccess) {
            set_error("prompt_attention: cannot set shared memory size: %s", cudaGetErrorString(e));
            return (int)RX_ECUDA;
        }
        // the warpgroups re-split the registers the block is launched with (setmaxnreg); the shares
        // must add up to no more than that, or the increasing warps would wait forever
        static_assert(256 * PT_REGS_OTHER + 256 * PT_REGS_SOFTMAX <= PT_THREADS * PT_REGS_LAUNCH, "register split");
        cudaFuncAttributes fa{};
        if (cudaFuncGetAttributes(&fa, prompt_tc_kernel<D, SPLIT>) != cudaSuccess || fa.numRegs < (int)PT_REGS_LAUNCH) {
            set_error("prompt_attention: kernel built with %d registers per thread; the register split needs %d", fa.numRegs,
                      (int)PT_REGS_LAUNCH);
            return (int)RX_ECUDA;
        }
        return (int)RX_OK;
    });
    if (rc != RX_OK) return rc;
    launch_pdl(prompt_tc_kernel<D, SPLIT>, grid, PT_THREADS, PtLayout<D>::ALLOC, stream, p);   // an error shows in cudaGetLastError
    return RX_OK;
}

static int launch_prompt_tc(const PromptParams& a, int head_dim, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms <= 0) return RX_EDEVICE;
    PromptTcParams p{};
    p.a = a;
    p.group = a.hq / a.hkv;
    p.hb = std::min(p.group, 128);
    p.nhb = (p.group + p.hb - 1) / p.hb;
    p.tpt = 128 / p.hb;
    // A scale of zero as the least number above it: masked scores are -inf, and -inf times it has to stay so.
    // Scores are below 2^128: it moves none by more than 2^-21.  By its bits, as the calling thread may have
    // the processor take numbers this small for zero.
    const float sl = a.scale * PT_LOG2E;
    int32_t bits;
    std::memcpy(&bits, &sl, sizeof bits);
    bits = std::max(bits, 1);            // -0 has the sign bit
    std::memcpy(&p.scale_log2, &bits, sizeof bits);
    const int64_t heads = (int64_t)a.hkv * p.nhb;
    // Two Q tiles an item share its K/V tiles and keep the tensor core busy in turn (1.4 us a step of
    // 128 keys); one, its K/V tiles split between two softmax warpgroups, while even those items are no
    // more than the SMs, or two an SM if the sequences are long.  (12 heads x 64, one Q tile and two: 2000 tokens
    // 15.2 and 22.4 us, 3000 22.6 and 31.2; 12 of 128 6.7 and 6.2; at four an SM 5000 tokens 49.7 and 48.4.
    // 32/8 heads x 128: 700 tokens 12.4 and 14.0, 1100 16.7 and 18.2; 6 of 100 9.4 and 7.9.)
    const int64_t one = prompt_items(a.total, a.batch, p.tpt) * heads;
    const bool split = one <= sms || (one <= 2 * sms && a.total >= 512ll * a.batch);
    const int tokens = split ? p.tpt : 2 * p.tpt;
    const int64_t items = prompt_items(a.total, a.batch, tokens) * heads;
    RX_REQUIRE(items < (1ll << 31), "prompt_attention: too many rows");
    p.a.by_level = prompt_by_level(items, sms, a.batch, 2 * a.total * a.hkv * head_dim * 2);
    p.by_tokens = PromptDiv(tokens);
    p.by_heads = PromptDiv((int)heads);
    RX_REQUIRE(rows_map(&p.q_map, a.q, a.total, a.hq, head_dim, a.q_stride, p.hb, p.tpt) &&
                   rows_map(&p.k_map, a.k, a.total, a.hkv, head_dim, a.k_stride, 1, PT_BN) &&
                   rows_map(&p.v_map, a.v, a.total, a.hkv, head_dim, a.v_stride, 1, PT_BN),
               "prompt_attention: the driver made no tensor map of these rows");
    if (split) return head_dim == 128 ? launch_pt<128, true>(p, (unsigned)items, stream) : launch_pt<64, true>(p, (unsigned)items, stream);
    return head_dim == 128 ? launch_pt<128, false>(p, (unsigned)items, stream) : launch_pt<64, false>(p, (unsigned)items, stream);
}

}  // namespace rx

using namespace rx;

extern "C" int prompt_attention(const rx_attn_desc* desc, int32_t batch, const void* d_q, int64_t q_stride, const void* d_k,
                                int64_t k_stride, const void* d_v, int64_t v_stride, const int64_t* d_indptr, void* d_out,
                                int64_t out_stride, float* d_lse, int64_t total, int32_t* d_status, void* stream) {
    RX_TRACE("prompt_attention");
    RX_REQUIRE(desc && batch >= 0 && total >= 0 && total <= INT32_MAX, "prompt_attention: bad arguments");
    RX_REQUIRE(desc->dtype == RX_F32 || desc->dtype == RX_BF16, "prompt_attention: unknown dtype %d", desc->dtype);
    RX_REQUIRE(desc->hq > 0 && desc->hkv > 0 && desc->hq <= 65536 && desc->hq % desc->hkv == 0, "prompt_attention: bad head counts");
    RX_REQUIRE(desc->head_dim == 64 || desc->head_dim == 128, "prompt_attention: head_dim must be 64 or 128");
    RX_REQUIRE(std::isfinite(desc->scale * PT_LOG2E) && desc->scale >= 0.f, "prompt_attention: scale must be finite and not negative");
    if (batch == 0 || total == 0) return RX_OK;
    RX_REQUIRE(d_q && d_k && d_v && d_indptr && d_out, "prompt_attention: null device pointer");
    const int64_t elt = desc->dtype == RX_F32 ? 4 : 2, D = desc->head_dim;
    const struct {
        const void* p;
        int64_t stride, row;
    } rows[] = {{d_q, q_stride, desc->hq * D}, {d_k, k_stride, desc->hkv * D}, {d_v, v_stride, desc->hkv * D},
                {d_out, out_stride, desc->hq * D}};
    for (const auto& r : rows)
        RX_REQUIRE(((uintptr_t)r.p & 15) == 0 && r.stride * elt % 16 == 0 && r.stride >= r.row && r.stride < (1ll << 34),
                   "prompt_attention: rows must be 16-byte aligned and at least a row apart");
    PromptParams p{};
    p.batch = batch;
    p.hq = desc->hq;
    p.hkv = desc->hkv;
    p.total = total;
    p.q = d_q;
    p.k = d_k;
    p.v = d_v;
    p.out = d_out;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.out_stride = out_stride;
    p.indptr = d_indptr;
    p.lse = d_lse;
    p.scale = desc->scale;
    p.status = d_status;
    const int rc = desc->dtype == RX_F32 ? launch_prompt_simt(p, desc->head_dim, (cudaStream_t)stream)
                                         : launch_prompt_tc(p, desc->head_dim, (cudaStream_t)stream);
    if (rc != RX_OK) return rc;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("prompt_attention: launch failed: %s", cudaGetErrorString(e));
        return RX_ECUDA;
    }
    return RX_OK;
}
