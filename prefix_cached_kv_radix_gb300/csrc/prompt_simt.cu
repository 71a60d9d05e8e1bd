// prompt_attention in 32 bits on CUDA cores: causal attention over packed prompts.
//
// Row i of a sequence attends rows 0..i of the same sequence:  o = softmax(scale q K^T) V, one
// pass over the keys with a running maximum m and sum l, the accumulator rescaled by e^(m - m')
// when the maximum moves.  Bound by the fused multiply-adds (4 head_dim flops per query head, row
// and key); tensor cores would round the products' inputs, so they are not used for 32-bit rows.
//
// One block of 256 threads per (sequence, query head, 128 rows), keys in tiles of 64.  A thread
// owns 8 rows x 4 keys of the scores and 8 rows x head_dim / 16 columns of the output, both in
// registers: per 16 bytes it reads from shared memory it does 5 packed (two-wide) multiply-adds in
// the first product and 8 in the second, so the arithmetic, not shared memory, sets the pace.  K is
// fetched while the block works on P V and V while it works on Q K^T (cp.async).  Rows of Q and K
// are padded by 16 bytes so that eight threads reading eight rows hit all banks.
//
// A value row that a row may not see enters none of its sums: in the tiles a mask cuts, a key's
// product is added only for the rows that attend it, so an infinity or a NaN there (a later token,
// the next sequence's row) stays where it is.
#include <cuda_runtime.h>

#include <algorithm>

#include "prompt_items.cuh"
#include "radix_attn.h"
#include "rx_common.h"
#include "rx_device.cuh"
#include "rx_kernels.h"

namespace rx {

constexpr int PS_BM = 128, PS_BN = 64, PS_THREADS = 256;

template <int D>
struct PsLayout {
    static constexpr int LD = D + 4;                       // floats between rows of Q and K
    static constexpr int OFF_K = PS_BM * LD;
    static constexpr int OFF_V = OFF_K + PS_BN * LD;
    static constexpr int LDP = PS_BM + 4;                  // floats between keys of P (stored by key)
    static constexpr int OFF_P = OFF_V + PS_BN * D;
    static constexpr int BYTES = (OFF_P + PS_BN * LDP) * 4;
};

// `rows` rows of D floats, `stride` apart, to shared rows LD apart; rows from `have` on are zeros.
template <int D, int LD>
__device__ __forceinline__ void ps_load(uint32_t dst, const float* src, int64_t stride, int rows, int have) {
    constexpr int V = D / 4;
    for (int i = threadIdx.x; i < rows * V; i += PS_THREADS) {
        const int r = i / V, c = i % V;
        cp_async_16(dst + (uint32_t)(r * LD + c * 4) * 4, src + (int64_t)min(r, max(have - 1, 0)) * stride + c * 4,
                    r < have ? 16u : 0u);
    }
    cp_async_commit();
}

template <int D>
__global__ void __launch_bounds__(PS_THREADS) prompt_simt_kernel(const __grid_constant__ PromptParams p,
                                                                  const __grid_constant__ PromptDiv by_rows,
                                                                  const __grid_constant__ PromptDiv by_heads) {
    using LY = PsLayout<D>;
    constexpr int LD = LY::LD, LDP = LY::LDP, OC = D / 64;   // OC: 4-column groups of a thread
    extern __shared__ __align__(16) float sm[];
    const uint32_t sb = smem_u32(sm);
    PromptItem it;
    PromptFinder finder;
    if (!finder.find(p, (int)blockIdx.x, by_rows, by_heads, it)) return;
    const int h = it.head, g = h / (p.hq / p.hkv);
    const int row0 = it.tile * PS_BM, rows = min(PS_BM, it.n - row0);
    const float* q = (const float*)p.q + (int64_t)(it.start + row0) * p.q_stride + (int64_t)h * D;
    const float* k = (const float*)p.k + (int64_t)it.start * p.k_stride + (int64_t)g * D;
    const float* v = (const float*)p.v + (int64_t)it.start * p.v_stride + (int64_t)g * D;
    const int keys = row0 + rows;                            // keys the block needs
    const int nkv = (keys + PS_BN - 1) / PS_BN;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;  // rows ty*8.., keys tx + 16 j, columns tx*4 + 64 c

    ps_load<D, LD>(sb, q, p.q_stride, PS_BM, rows);
    ps_load<D, LD>(sb + LY::OFF_K * 4, k, p.k_stride, PS_BN, keys);
    float m[8], l[8];
    uint64_t o[8][OC * 2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < OC * 2; ++c) o[i][c] = 0ull;
    }
    for (int j = 0; j < nkv; ++j) {
        const int k0 = j * PS_BN;
        ps_load<D, D>(sb + LY::OFF_V * 4, v + (int64_t)k0 * p.v_stride, p.v_stride, PS_BN, keys - k0);
        cp_async_wait<1>();                                  // Q and this tile of K are in
        __syncthreads();
        // scores: two channels at a time, the even and the odd ones summed apart
        uint64_t s2[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) s2[i][c] = 0ull;
#pragma unroll 2
        for (int d = 0; d < D; d += 4) {
            ulonglong2 a[8], b[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = *reinterpret_cast<const ulonglong2*>(sm + (ty * 8 + i) * LD + d);
#pragma unroll
            for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const ulonglong2*>(sm + LY::OFF_K + (tx + 16 * c) * LD + d);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    s2[i][c] = f2_fma(a[i].x, b[c].x, s2[i][c]);
                    s2[i][c] = f2_fma(a[i].y, b[c].y, s2[i][c]);
                }
        }
        const bool cut = k0 + PS_BN - 1 > row0;              // a mask or the end of the sequence cuts this tile
        float pr[4][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = row0 + ty * 8 + i;
            float sc[4], mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float x, y;
                f2_unpack(s2[i][c], x, y);
                sc[c] = (x + y) * p.scale;
                if (cut && k0 + tx + 16 * c > r) sc[c] = -INFINITY;
                mx = fmaxf(mx, sc[c]);
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float mn = fmaxf(m[i], mx);
            const float sub = mn == -INFINITY ? 0.f : mn;    // nothing but -inf so far
            const float corr = expf(m[i] - sub);
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                pr[c][i] = expf(sc[c] - sub);
                sum += pr[c][i];
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            l[i] = l[i] * corr + sum;
            m[i] = mn;
            const uint64_t c2 = f2_pack(corr, corr);
#pragma unroll
            for (int c = 0; c < OC * 2; ++c) o[i][c] = f2_fma(o[i][c], c2, 0ull);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 8; i += 4)
                *reinterpret_cast<float4*>(sm + LY::OFF_P + (tx + 16 * c) * LDP + ty * 8 + i) =
                    make_float4(pr[c][i], pr[c][i + 1], pr[c][i + 2], pr[c][i + 3]);
        cp_async_wait<0>();                                  // V is in
        __syncthreads();                                     // P is written, K is read
        if (j + 1 < nkv)
            ps_load<D, LD>(sb + LY::OFF_K * 4, k + (int64_t)(k0 + PS_BN) * p.k_stride, p.k_stride, PS_BN, keys - k0 - PS_BN);
        const int nk = min(PS_BN, keys - k0);
        auto pv = [&](int kk, bool guarded) {
            const float4 pa = *reinterpret_cast<const float4*>(sm + LY::OFF_P + kk * LDP + ty * 8);
            const float4 pb = *reinterpret_cast<const float4*>(sm + LY::OFF_P + kk * LDP + ty * 8 + 4);
            const float pp[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
            ulonglong2 w[OC];
#pragma unroll
            for (int c = 0; c < OC; ++c) w[c] = *reinterpret_cast<const ulonglong2*>(sm + LY::OFF_V + kk * D + tx * 4 + 64 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (guarded && k0 + kk > row0 + ty * 8 + i) continue;
                const uint64_t p2 = f2_pack(pp[i], pp[i]);
#pragma unroll
                for (int c = 0; c < OC; ++c) {
                    o[i][2 * c] = f2_fma(p2, w[c].x, o[i][2 * c]);
                    o[i][2 * c + 1] = f2_fma(p2, w[c].y, o[i][2 * c + 1]);
                }
            }
        };
        if (cut) {
#pragma unroll 1
            for (int kk = 0; kk < nk; ++kk) pv(kk, true);
        } else {
#pragma unroll 4
            for (int kk = 0; kk < PS_BN; ++kk) pv(kk, false);
        }
        __syncthreads();                                     // P and V are read
    }
    cp_async_wait_all();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = ty * 8 + i;
        if (r >= rows) continue;
        const float inv = 1.f / l[i];
        float* orow = (float*)p.out + (int64_t)(it.start + row0 + r) * p.out_stride + (int64_t)h * D;
#pragma unroll
        for (int c = 0; c < OC; ++c) {
            float4 w;
            f2_unpack(o[i][2 * c], w.x, w.y);
            f2_unpack(o[i][2 * c + 1], w.z, w.w);
            w.x *= inv, w.y *= inv, w.z *= inv, w.w *= inv;
            *reinterpret_cast<float4*>(orow + tx * 4 + 64 * c) = w;
        }
        if (p.lse && tx == 0) p.lse[(int64_t)(it.start + row0 + r) * p.hq + h] = m[i] + logf(l[i]);
    }
}

template <int D>
static int launch_ps(const PromptParams& p, unsigned grid, cudaStream_t stream) {
    static PerDeviceOnce attr;
    const int rc = per_device_once(attr, [] {
        const cudaError_t e =
            cudaFuncSetAttribute(prompt_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, PsLayout<D>::BYTES);
        if (e != cudaSuccess) {
            set_error("prompt_attention: cannot set shared memory size: %s", cudaGetErrorString(e));
            return (int)RX_ECUDA;
        }
        return (int)RX_OK;
    });
    if (rc != RX_OK) return rc;
    prompt_simt_kernel<D><<<grid, PS_THREADS, PsLayout<D>::BYTES, stream>>>(p, PromptDiv(PS_BM), PromptDiv(p.hq));
    return RX_OK;
}

int launch_prompt_simt(const PromptParams& p, int head_dim, cudaStream_t stream) {
    const int64_t items = prompt_items(p.total, p.batch, PS_BM) * p.hq;
    if (items >= (1ll << 31)) {
        set_error("prompt_attention: too many rows");
        return RX_EINVAL;
    }
    return head_dim == 128 ? launch_ps<128>(p, (unsigned)items, stream) : launch_ps<64>(p, (unsigned)items, stream);
}

}  // namespace rx
