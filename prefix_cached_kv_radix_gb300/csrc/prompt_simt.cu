// prompt_attention in 32 bits on CUDA cores: causal attention over packed prompts.
//
// Row i of a sequence attends rows 0..i of the same sequence:  o = softmax(scale q K^T) V, one
// pass over the keys with a running maximum m and sum l, the accumulator rescaled by 2^(m - m')
// when the maximum moves.  Bound by the fused multiply-adds (4 head_dim flops per query head, row
// and key); tensor cores would round the products' inputs, so they are not used for 32-bit rows.
//
// One block per (sequence, query head, 64 rows), keys in tiles of 64.  A thread owns 8 rows x 64 / TX keys of
// the scores and 8 rows x head_dim / TX columns of the output, both in registers and as pairs of rows: the
// packed (two-wide) multiply-add takes two rows of Q, or of P, which lie side by side in shared memory (Q
// is stored by channel, P by key), and one value of K, or V, twice.  What limits it beside the multiply-adds is
// the shared loads that feed them: with TX = 16 (128 threads, two blocks an SM) 12 of 16 bytes for 64 of
// them, with TX = 8 (64 threads, four blocks an SM, 254 registers) 16 for 128.  The few blocks of an SM run
// beside one another, one's softmax under another's products.  P takes the place of the K tile it came from;
// where there is room (head_dim 64, TX 16) the next K tile has a buffer of its own and comes in meanwhile.
// Rows of Q, K and P are padded by 16 bytes so that eight threads reading eight rows hit all banks.
//
// Probabilities are 2^(s sl - m), sl = scale log2(e): one multiply-add, rounded once where the result
// is small, and the special-function unit (2^-22 relative).  l is summed per thread and joined at the
// end; the accumulator is rescaled only in tiles where a row's maximum moved.
//
// Measured, against 79 TFLOP/s of the multiply-add pipe: 8 ragged prompts of up to 2001 tokens, 16/4 heads x
// 64, 0.43 ms (49; with pairs of channels instead of rows 0.48), four of 4096 tokens 54, one of 8192 tokens, 16/4
// heads x 128, 58.  Small calls are one block's chain of tiles: one of 300 tokens, 12 heads x 64, 23 us.
//
// A value row that a row may not see enters none of its sums, so an infinity or a NaN there (a later
// token, the next sequence's row) stays where it is.
#include <cuda_runtime.h>

#include <algorithm>

#include "prompt_items.cuh"
#include "radix_attn.h"
#include "rx_common.h"
#include "rx_device.cuh"
#include "rx_kernels.h"
#include "rx_launch.h"

namespace rx {

constexpr int PS_BM = 64, PS_BN = 64;
constexpr float PS_LOG2E = 1.4426950408889634f;
constexpr float PS_LN2 = 0.6931471805599453f;
constexpr int PS_ALONE = 120000;   // bytes of shared memory with which a block has an SM to itself

template <int D, int TX_>
struct PsLayout {
    static constexpr int TX = TX_;                         // threads across the keys (and the columns)
    static constexpr int THREADS = PS_BM / 8 * TX;
    static constexpr int NC = PS_BN / TX;                  // keys of a thread
    static constexpr int LDQ = PS_BM + 4;                  // floats between channels of Q (stored by channel)
    static constexpr int LD = D + 4;                       // floats between rows of K
    static constexpr int NK = D == 64 && TX == 16 ? 2 : 1; // K buffers
    static constexpr int LDP = PS_BM + 4;                  // floats between keys of P (stored by key)
    static constexpr int K_SIZE = PS_BN * LD;
    static constexpr int OFF_K = D * LDQ;
    static constexpr int OFF_V = OFF_K + NK * K_SIZE;
    static constexpr int BYTES = (OFF_V + PS_BN * D) * 4;
    static constexpr int BLOCKS = TX == 8 ? 4 : 2;         // per SM
    static_assert(PS_BN * LDP <= K_SIZE, "P takes the place of K");
    static_assert(BLOCKS * (BYTES + 1024) <= 233472, "shared memory of the blocks of an SM");
};

// `rows` rows of D floats, `stride` apart, to shared rows LD apart; rows from `have` on are zeros.
template <int D, int LD, int THREADS>
__device__ __forceinline__ void ps_load(uint32_t dst, const float* src, int64_t stride, int rows, int have) {
    constexpr int V = D / 4;
    for (int i = threadIdx.x; i < rows * V; i += THREADS) {
        const int r = i / V, c = i % V;
        cp_async_16(dst + (uint32_t)(r * LD + c * 4) * 4, src + (int64_t)min(r, max(have - 1, 0)) * stride + c * 4,
                    r < have ? 16u : 0u);
    }
    cp_async_commit();
}

template <int D, int TX>
__global__ void __launch_bounds__(PsLayout<D, TX>::THREADS, PsLayout<D, TX>::BLOCKS)
    prompt_simt_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ PromptDiv by_rows,
                       const __grid_constant__ PromptDiv by_heads) {
    using LY = PsLayout<D, TX>;
    constexpr int LD = LY::LD, LDP = LY::LDP, LDQ = LY::LDQ, NC = LY::NC, THREADS = LY::THREADS;
    constexpr int OC = D / TX / 4;                           // 4-column groups of a thread
    extern __shared__ __align__(16) float sm[];
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t sb = smem_u32(sm);
    PromptItem it;
    PromptFinder finder;
    if (!finder.find(p, (int)blockIdx.x, by_rows, by_heads, it)) {
        if (threadIdx.x == 0) PromptFinder::check(p, (int)blockIdx.x);
        return;
    }
    const int h = it.head, g = h / (p.hq / p.hkv);
    const int row0 = it.tile * PS_BM, rows = min(PS_BM, it.n - row0);
    const float* q = (const float*)p.q + (int64_t)(it.start + row0) * p.q_stride + (int64_t)h * D;
    const float* k = (const float*)p.k + (int64_t)it.start * p.k_stride + (int64_t)g * D;
    const float* v = (const float*)p.v + (int64_t)it.start * p.v_stride + (int64_t)g * D;
    const int keys = row0 + rows;                            // keys the block needs
    const int nkv = (keys + PS_BN - 1) / PS_BN;
    const int ty = threadIdx.x / TX, tx = threadIdx.x % TX;  // rows ty*8.., keys tx + TX c, columns (tx + TX c)*4
    // A scale of zero as the least number above it: masked scores are -inf, and -inf times it has to stay so.
    // Scores are below 2^128: it moves none by more than 2^-21.
    const float sl = fmaxf(p.scale * PS_LOG2E, 0x1p-149f);
    auto load_k = [&](int j) {
        ps_load<D, LD, THREADS>(sb + (LY::OFF_K + j % LY::NK * LY::K_SIZE) * 4, k + (int64_t)(j * PS_BN) * p.k_stride, p.k_stride,
                                PS_BN, keys - j * PS_BN);
    };
    auto load_v = [&](int j) {
        ps_load<D, D, THREADS>(sb + LY::OFF_V * 4, v + (int64_t)(j * PS_BN) * p.v_stride, p.v_stride, PS_BN, keys - j * PS_BN);
    };
    load_k(0);
    load_v(0);
    {   // Q, stored by channel: a warp takes 32 bytes of 16 rows at a time, whole sectors and all banks
        constexpr int N = PS_BM * D / 4 / THREADS;
        const int row = threadIdx.x % 16 + threadIdx.x / 32 % (PS_BM / 16) * 16;
        const int c0 = threadIdx.x / 16 % 2 + threadIdx.x / (2 * PS_BM) * 2;
        float4 x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int w = i * THREADS / 32;                  // warps' worths before this one
            const int r = row + w % (PS_BM / 16) * 16, c = (c0 + w / (PS_BM / 16) * 2) * 4;
            x[i] = r < rows ? *reinterpret_cast<const float4*>(q + (int64_t)r * p.q_stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int w = i * THREADS / 32;
            float* to = sm + (c0 + w / (PS_BM / 16) * 2) * 4 * LDQ + row + w % (PS_BM / 16) * 16;
            to[0] = x[i].x, to[LDQ] = x[i].y, to[2 * LDQ] = x[i].z, to[3 * LDQ] = x[i].w;
        }
    }
    if (threadIdx.x == 0) PromptFinder::check(p, (int)blockIdx.x);    // under the first loads
    float m[8], l[8];                                        // row maximum times sl; this thread's part of the sum
    uint64_t o[4][OC * 4];                                   // rows 2i and 2i + 1 of a column
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < OC * 4; ++c) o[i][c] = 0ull;
    for (int j = 0; j < nkv; ++j) {
        const int k0 = j * PS_BN;
        float* const kt = sm + LY::OFF_K + j % LY::NK * LY::K_SIZE;
        if constexpr (LY::NK == 2) {
            if (j + 1 < nkv) load_k(j + 1);
            else cp_async_commit();
            cp_async_wait<2>();                              // all but this tile's V and the next K
        } else {
            cp_async_wait<1>();
        }
        __syncthreads();
        // scores of two rows at a time
        uint64_t s2[4][NC];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c) s2[i][c] = 0ull;
#pragma unroll 8
        for (int d = 0; d < D; d += 4) {
            float b[NC][4];
#pragma unroll
            for (int c = 0; c < NC; ++c) *reinterpret_cast<float4*>(b[c]) = *reinterpret_cast<const float4*>(kt + (tx + TX * c) * LD + d);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const ulonglong2 a0 = *reinterpret_cast<const ulonglong2*>(sm + (d + x) * LDQ + ty * 8);
                const ulonglong2 a1 = *reinterpret_cast<const ulonglong2*>(sm + (d + x) * LDQ + ty * 8 + 4);
                const uint64_t a[4] = {a0.x, a0.y, a1.x, a1.y};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const uint64_t w = f2_pack(b[c][x], b[c][x]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s2[i][c] = f2_fma(a[i], w, s2[i][c]);
                }
            }
        }
        const bool cut = k0 + PS_BN - 1 > row0;              // a mask or the end of the sequence cuts this tile
        float pr[NC][8];
        bool moved = false;
        float corr[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = row0 + ty * 8 + i;
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                float x, y;
                f2_unpack(s2[i / 2][c], x, y);
                pr[c][i] = i % 2 ? y : x;
                if (cut && k0 + tx + TX * c > r) pr[c][i] = -INFINITY;
                mx = fmaxf(mx, pr[c][i]);
            }
#pragma unroll
            for (int w = TX / 2; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float mn = fmaxf(m[i], mx * sl);
            const float sub = mn == -INFINITY ? 0.f : mn;    // nothing but -inf so far
            corr[i] = fast_exp2(m[i] - sub);
            moved |= mn != m[i];
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                pr[c][i] = fast_exp2(fmaf(pr[c][i], sl, -sub));
                sum += pr[c][i];
            }
            l[i] = fmaf(l[i], corr[i], sum);
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t c2 = f2_pack(corr[2 * i], corr[2 * i + 1]);
#pragma unroll
                for (int c = 0; c < OC * 4; ++c) o[i][c] = f2_fma(o[i][c], c2, 0ull);
            }
        }
        __syncthreads();                                     // K is read: P takes its place
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; i += 4)
                *reinterpret_cast<float4*>(kt + (tx + TX * c) * LDP + ty * 8 + i) =
                    make_float4(pr[c][i], pr[c][i + 1], pr[c][i + 2], pr[c][i + 3]);
        cp_async_wait<LY::NK == 2 ? 1 : 0>();                // V is in
        __syncthreads();
        // A hidden key has P = 0, and 0 times its value is 0 unless that is not finite: only a cut tile that
        // has such a value (their sum with factors of 0 is NaN) adds key by key for the rows that attend it.
        bool apart = false;
        if (cut) {
            float z = 0.f;
            for (int i = threadIdx.x; i < PS_BN * D / 4; i += THREADS) {
                const float4 x = *reinterpret_cast<const float4*>(sm + LY::OFF_V + i * 4);
                z = fmaf(x.x, 0.f, z), z = fmaf(x.y, 0.f, z), z = fmaf(x.z, 0.f, z), z = fmaf(x.w, 0.f, z);
            }
            apart = __syncthreads_or(z != z);
        }
        auto pv = [&](int kk, bool guarded) {
            const ulonglong2 pa = *reinterpret_cast<const ulonglong2*>(kt + kk * LDP + ty * 8);
            const ulonglong2 pb = *reinterpret_cast<const ulonglong2*>(kt + kk * LDP + ty * 8 + 4);
            const uint64_t pp[4] = {pa.x, pa.y, pb.x, pb.y};
#pragma unroll
            for (int c = 0; c < OC; ++c) {
                const float4 w = *reinterpret_cast<const float4*>(sm + LY::OFF_V + kk * D + (tx + TX * c) * 4);
                const uint64_t w2[4] = {f2_pack(w.x, w.x), f2_pack(w.y, w.y), f2_pack(w.z, w.z), f2_pack(w.w, w.w)};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint64_t r = f2_fma(pp[i], w2[x], o[i][c * 4 + x]);
                        if (!guarded) {
                            o[i][c * 4 + x] = r;
                        } else {
                            float lo, hi, lo0, hi0;
                            f2_unpack(r, lo, hi);
                            f2_unpack(o[i][c * 4 + x], lo0, hi0);
                            const int row = row0 + ty * 8 + 2 * i;
                            o[i][c * 4 + x] = f2_pack(k0 + kk <= row ? lo : lo0, k0 + kk <= row + 1 ? hi : hi0);
                        }
                    }
            }
        };
        if (apart) {
#pragma unroll 1
            for (int kk = 0; kk < PS_BN; ++kk) pv(kk, true);
        } else {
#pragma unroll 8
            for (int kk = 0; kk < PS_BN; ++kk) pv(kk, false);
        }
        __syncthreads();                                     // P and V are read
        if (j + 1 < nkv) {
            if constexpr (LY::NK == 1) load_k(j + 1);
            load_v(j + 1);
        }
    }
    cp_async_wait_all();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = ty * 8 + i;
        float sum = l[i];
#pragma unroll
        for (int w = TX / 2; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        if (r >= rows) continue;
        const float inv = 1.f / sum;
        float* orow = (float*)p.out + (int64_t)(it.start + row0 + r) * p.out_stride + (int64_t)h * D;
#pragma unroll
        for (int c = 0; c < OC; ++c) {
            float w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float lo, hi;
                f2_unpack(o[i / 2][c * 4 + x], lo, hi);
                w[x] = (i % 2 ? hi : lo) * inv;
            }
            *reinterpret_cast<float4*>(orow + (tx + TX * c) * 4) = make_float4(w[0], w[1], w[2], w[3]);
        }
        if (p.lse && tx == 0) p.lse[(int64_t)(it.start + row0 + r) * p.hq + h] = (m[i] + log2f(sum)) * PS_LN2;
    }
}

template <int D, int TX>
static int launch_ps(const PromptParams& p, unsigned grid, bool alone, cudaStream_t stream) {
    using LY = PsLayout<D, TX>;
    constexpr int MORE = std::max(LY::BYTES, PS_ALONE);
    static PerDeviceOnce attr;
    const int rc = per_device_once(attr, [] {
        const cudaError_t e = cudaFuncSetAttribute(prompt_simt_kernel<D, TX>, cudaFuncAttributeMaxDynamicSharedMemorySize, MORE);
        if (e != cudaSuccess) {
            set_error("prompt_attention: cannot set shared memory size: %s", cudaGetErrorString(e));
            return (int)RX_ECUDA;
        }
        return (int)RX_OK;
    });
    if (rc != RX_OK) return rc;
    launch_pdl(prompt_simt_kernel<D, TX>, grid, LY::THREADS, alone ? MORE : LY::BYTES, stream, p, PromptDiv(PS_BM), PromptDiv(p.hq));
    return RX_OK;
}

int launch_prompt_simt(PromptParams p, int head_dim, cudaStream_t stream) {
    const int64_t items = prompt_items(p.total, p.batch, PS_BM) * p.hq;
    if (items >= (1ll << 31)) {
        set_error("prompt_attention: too many rows");
        return RX_EINVAL;
    }
    // TX = 8 has half the threads of an item, so that it takes longer: for calls of many items, where the
    // items beside it fill the SM, and of sequences long enough that the products are most of it.  (12
    // heads x 64, TX 8 and 16: one of 7680 tokens 1653 and 1717 us, of 5120 875 and 786, of 300 40 and 23; 20 of
    // 500 187 and 198, 100 of 200 325 and 311.  With head_dim 128 its output would not fit the registers.)
    const bool wide = head_dim == 64 && items > 2 * 152 * PsLayout<64, 8>::BLOCKS && p.total >= 256ll * p.batch;
    // One block an SM, the longest first, for calls of up to a few items an SM: two on one SM would each take
    // nearly twice as long beside SMs that are idle (or soon are).  Not for short sequences, whose items are
    // alike.  (12 heads x 64, one block and two: 640 tokens 41 and 53 us, 1280 76 and 124, 1920 155 and 183,
    // 2560 261 and 240; 10 of 64 9.1 and 12.0, 18 of 64 16 and 12.  16 heads x 128: 300 37 and 41, 1280 158 and
    // 224, 1920 346 and 327.)
    const bool alone = items <= 152 || (items <= 152 * 5 / 2 && p.total >= 256ll * p.batch);
    p.by_level = prompt_by_level(items, 152 * (alone ? 1 : wide ? PsLayout<64, 8>::BLOCKS : PsLayout<64, 16>::BLOCKS), p.batch,
                                 2 * p.total * p.hkv * head_dim * 4);
    const unsigned grid = (unsigned)items;
    if (head_dim == 128) return launch_ps<128, 16>(p, grid, alone, stream);
    return wide ? launch_ps<64, 8>(p, grid, alone, stream) : launch_ps<64, 16>(p, grid, alone, stream);
}

}  // namespace rx
