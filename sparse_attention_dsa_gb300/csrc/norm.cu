// Root-mean-square norm with the residual's addition, to bf16 and to E4M3 codes with scales: what stands in front of a
// projection ("Day0 Inference Support and Performance Optimization for New LLM Architectures", section 3.3: input
// preparation ahead of the indexer; sections 4 and 4.1 for the FP8 and MXFP8 forms).
//
// Mathematics, per row: h = x + residual, s = bf16(h), y = h / sqrt(mean(h^2) + eps) * weight, in fp32 from the unrounded h
// (one rounding less than from the stored sum).  Codes are made of the fp32 y: per row or tile of 128, scale = absmax / 448
// (1 for a group of zeros) and E4M3(y / scale); per 32, scale = 2^(floor(log2(absmax)) - 8).
//
// What bounds it: HBM for long steps (every element is read and written once), launch and one round of loads and
// reductions for short ones.  So a row is held in registers between its only load and its stores, as 16-byte pieces: a row
// of up to 1024 values by a warp (no block barrier), a longer one by a block.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace dsa {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kRowsPerBlock = 4;  // rows of a warp each
constexpr int kMaxWarps = 32;

// Of all threads that share a row.  The block's result is in every thread; `slots` is used once a call.
template <bool kWarpRow, typename F>
__device__ __forceinline__ float reduce_row(float v, float* slots, F op) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = op(v, __shfl_xor_sync(kAll, v, off));
    if (kWarpRow) return v;
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    v = slots[lane < warps ? lane : 0];
    if (lane >= warps) v = 0.f;  // (neutral: sums of squares and absolute maxima)
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = op(v, __shfl_xor_sync(kAll, v, off));
    return v;
}

// Piece i of thread t is piece t + i * width of the row, so that a warp's loads are whole lines and a group of 32 or 128
// values lies in neighbouring lanes.
template <int P, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kRowsPerBlock : 1024) norm_kernel(const NormParams p) {
    __shared__ float sums[kMaxWarps], maxima[kMaxWarps];
    const int t = kWarpRow ? threadIdx.x & 31 : threadIdx.x, width = kWarpRow ? 32 : blockDim.x;
    const int64_t row = kWarpRow ? (int64_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5) : blockIdx.x;
    if (kWarpRow && row >= p.rows) return;
    const int pieces = p.dim >> 3;
    const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.x_stride);
    const uint4* res = reinterpret_cast<const uint4*>(p.residual + row * p.dim);
    const uint4* weight = reinterpret_cast<const uint4*>(p.weight);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 xv[P], rv[P], wv[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int at = t + i * width;
        xv[i] = at < pieces ? x[at] : zero;
        rv[i] = p.residual != nullptr && at < pieces ? res[at] : zero;
        wv[i] = at < pieces ? __ldg(weight + at) : zero;
    }
    float h[P][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        unpack8(xv[i], h[i]);
        if (p.residual != nullptr) {
            float r[8];
            unpack8(rv[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] += r[j];
        }
        float part[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) part[j] = fmaf(h[i][j], h[i][j], h[i][j + 4] * h[i][j + 4]);
        ss += (part[0] + part[1]) + (part[2] + part[3]);
    }
    ss = reduce_row<kWarpRow>(ss, sums, [](float a, float b) { return a + b; });
    const float r = __frsqrt_rn(__fdiv_rn(ss, (float)p.dim) + p.eps);
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int at = t + i * width;
        if (p.sum != nullptr && at < pieces) reinterpret_cast<uint4*>(p.sum + row * p.dim)[at] = pack8(h[i]);
        float w[8];
        unpack8(wv[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = at < pieces ? h[i][j] * r * w[j] : 0.f;
        if (p.out != nullptr && at < pieces) reinterpret_cast<uint4*>(p.out + row * p.out_stride)[at] = pack8(h[i]);
        most = fmaxf(most, absmax8(h[i]));
    }
    if (p.codes == nullptr) return;
    uint2* codes = reinterpret_cast<uint2*>(p.codes + row * p.dim);
    if (p.group == 0) {
        most = reduce_row<kWarpRow>(most, maxima, [](float a, float b) { return fmaxf(a, b); });
        const float scale = group_scale(most);
        if (t == 0) static_cast<float*>(p.scale)[row] = scale;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (t + i * width < pieces) codes[t + i * width] = codes8(h[i], scale);
        return;
    }
    const int lanes = p.group >> 3;  // 16 of a tile, 4 of an MX group
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int at = t + i * width;
        float m = absmax8(h[i]);
        m = fmaxf(m, __shfl_xor_sync(kAll, m, 1));
        m = fmaxf(m, __shfl_xor_sync(kAll, m, 2));
        if (lanes == 16) {
            m = fmaxf(m, __shfl_xor_sync(kAll, m, 4));
            m = fmaxf(m, __shfl_xor_sync(kAll, m, 8));
        }
        if (at >= pieces) continue;
        const int64_t group = row * (pieces / lanes) + at / lanes;
        if (p.mx) {
            const int e = mx_exponent(m);
            if (at % lanes == 0) static_cast<uint8_t*>(p.scale)[group] = (uint8_t)(e + 127);
            codes[at] = codes8_exp(h[i], e);
        } else {
            const float scale = group_scale(m);
            if (at % lanes == 0) static_cast<float*>(p.scale)[group] = scale;
            codes[at] = codes8(h[i], scale);
        }
    }
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t stream) {
    if (p.rows <= 0) return cudaSuccess;
    const int pieces = p.dim / 8;
    if (pieces <= 128) {
        const dim3 grid((unsigned)((p.rows + kRowsPerBlock - 1) / kRowsPerBlock)), block(32 * kRowsPerBlock);
        auto kernel = pieces <= 32 ? norm_kernel<1, true> : pieces <= 64 ? norm_kernel<2, true> : norm_kernel<4, true>;
        kernel<<<grid, block, 0, stream>>>(p);
    } else {
        const int threads = ((pieces + 1) / 2 + 31) / 32 * 32;
        norm_kernel<2, false><<<dim3((unsigned)p.rows), dim3((unsigned)threads), 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace dsa
