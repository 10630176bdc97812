// Dense attention over the paged latent-KV cache for a batch whose sequences share a prefix.
//
// For query token t of sequence b at position p and head h: z_s = scale * q[t,h,:] . kv[s,:] for s = 0..p,
// out[t,h,:] = softmax(z) . kv[:, :512], lse[t,h] = logsumexp(z) ("Optimizing Inference for Hybrid Attention
// Architectures: From Operator Fusion to Sequence Sharding", section "Breaking Down the Computational Path of
// Hybrid Attention", step 2, without the selection).  Positions below prefix_len are read through sequence 0.
//
// One warp per (token, head) and a running maximum and sum over its keys.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kWarps = 4;

// Values 2*lane + 64*i, +1 (i = 0..8) of a cache row.
template <bool KVFP8>
__device__ __forceinline__ void load_row(const uint8_t* cache, int64_t row, int lane, float (&x)[18]) {
    if constexpr (KVFP8) {
        const uint8_t* src = cache + row * kKvFp8RowBytes;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t c = __ldg(reinterpret_cast<const uint16_t*>(src + 64 * i) + lane);
            const float s = __ldg(reinterpret_cast<const float*>(src + kKvFp8ScaleOff) + i / 2);
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
            float lo, hi;
            asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
                : "=f"(lo), "=f"(hi)
                : "r"(h2));
            x[2 * i] = lo * s;
            x[2 * i + 1] = hi * s;
        }
        const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(src + kKvFp8RopeOff) + lane);
        x[16] = __uint_as_float(v << 16);
        x[17] = __uint_as_float(v & 0xFFFF0000u);
    } else {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(cache + row * 1152);
#pragma unroll
        for (int i = 0; i < 9; ++i) {
            const uint32_t v = __ldg(src + 32 * i + lane);
            x[2 * i] = __uint_as_float(v << 16);
            x[2 * i + 1] = __uint_as_float(v & 0xFFFF0000u);
        }
    }
}

template <bool KVFP8>
__global__ void __launch_bounds__(32 * kWarps) prefix_simple_kernel(const PrefixParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (r >= (int64_t)p.total_q * p.heads) return;
    const int t = (int)(r / p.heads);
    int b = -1, c0 = 0, c1 = 0;
    for (int j = 0; j < p.batch; ++j) {
        c0 = __ldg(p.cu_q_lens + j);
        c1 = __ldg(p.cu_q_lens + j + 1);
        if (c0 <= t && t < c1) {
            b = j;
            break;
        }
    }
    const int L = b < 0 ? 0 : __ldg(p.seq_lens + b);
    if (b < 0 || (int64_t)c1 - c0 > (int64_t)L - p.prefix_len || (int64_t)L > (int64_t)p.max_pages * 64) {
        if (lane == 0) raise_error(p.err, DSA_DEVERR_SEQ);
        return;
    }
    const int pos = L - (c1 - t);
    float q[18];
#pragma unroll
    for (int i = 0; i < 9; ++i) {
        const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(p.q + r * 576) + 32 * i + lane);
        q[2 * i] = __uint_as_float(v << 16);
        q[2 * i + 1] = __uint_as_float(v & 0xFFFF0000u);
    }
    float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    for (int s = 0; s <= pos; ++s) {
        const int32_t pg = __ldg(p.page_table + (int64_t)(s < p.prefix_len ? 0 : b) * p.max_pages + s / 64);
        if (pg < 0 || pg >= p.num_pages) {
            if (lane == 0) raise_error(p.err, DSA_DEVERR_PAGE);
            continue;
        }
        float x[18], z = 0.f;
        load_row<KVFP8>(p.kv_cache, (int64_t)pg * 64 + (s & 63), lane, x);
#pragma unroll
        for (int i = 0; i < 18; ++i) z = fmaf(q[i], x[i], z);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, off);
        z *= p.scale_log2;
        if (z == -INFINITY) continue;  // weight 0
        const float mn = fmaxf(m, z), a = exp2f(m - mn), e = exp2f(z - mn);
        l = l * a + e;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = acc[i] * a + e * x[i];
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        reinterpret_cast<uint32_t*>(p.out + r * 512)[32 * i + lane] = f2_to_bf2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if (lane == 0 && p.lse) p.lse[r] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_prefix(const PrefixLaunch& L, cudaStream_t stream) {
    const PrefixParams& p = L.params;
    const int64_t rows = (int64_t)p.total_q * p.heads;
    const unsigned blocks = (unsigned)((rows + kWarps - 1) / kWarps);
    if (p.kv_fp8)
        prefix_simple_kernel<true><<<blocks, 32 * kWarps, 0, stream>>>(p);
    else
        prefix_simple_kernel<false><<<blocks, 32 * kWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dsa
