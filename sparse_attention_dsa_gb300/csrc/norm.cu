// Root-mean-square norm with the residual's addition, to bf16 and to E4M3 codes with scales: what stands in front of a
// projection ("Day0 Inference Support and Performance Optimization for New LLM Architectures", section 3.3: input
// preparation ahead of the indexer; sections 4 and 4.1 for the FP8 and MXFP8 forms).
//
// Mathematics, per row: h = x + residual, s = bf16(h), y = h / sqrt(mean(h^2) + eps) * weight, in fp32 from the unrounded h
// (one rounding less than from the stored sum).  Codes are made of the fp32 y: per row or tile of 128, scale = absmax / 448
// (1 for a group of zeros) and E4M3(y / scale); per 32, scale = 2^(floor(log2(absmax)) - 8).
//
// What bounds it: HBM for long steps (every element is read and written once), launch and one round of loads and
// reductions for short ones.  So a row is held between its only load and its stores, as 16-byte pieces: a row of up to 1024
// values by a warp (no block barrier), a longer one by a block.  It is in registers but for some values of a thread with four
// pieces, whose 64 registers do not suffice (up to 72 bytes a thread are kept in local memory): with more registers fewer rows
// are in flight (8192 rows of 8192 to FP8 tiles 135 us, for 72), and with the weights, which make the difference, loaded only behind the
// reduction their latency stands in each row's way (96).
//
// Measured (one GB300; 20 calls in a graph; in brackets with L2 flushed before each): 32 rows of 4096 with the residual
// 2.0 us (7.3), 1171 of 1536 to MXFP8 3.1 (9.3), latency; 4096 of 512 2.5 (9.3); 8192 rows of 8192 with the residual 78.5 us to
// bf16 (85; 537 MB, 6.8 TB/s, 1.01 of the copy bandwidth), 72 to FP8 in tiles (79; 472 MB, 6.5 TB/s, 0.97), 69.5 to MXFP8 (77; 472 MB,
// 6.8 TB/s); 16384 of 4096 with the residual to FP8 rows 75 (81; 470 MB, 0.93).
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
constexpr int kFewRows = 1216;    // eight blocks for each SM
constexpr float kSmallMean = 0x1p-100f;  // of squares: below, some of a row's may be subnormal

// Of all threads that share a row.  The block's result is in every thread; `slots` are its own until all have read it.
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
// (An instance for each kind of codes: with the choice inside, all paid for the registers of the largest, 101 us for 79.)
enum Codes { kNone, kRow, kTile, kMx };
template <int P, bool kWarpRow, Codes kCodes>
__global__ void __launch_bounds__(kWarpRow ? 32 * kRowsPerBlock : 1024, kWarpRow ? 8 : 1) norm_kernel(const NormParams p) {
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
    const float mean = __fdiv_rn(ss, (float)p.dim) + p.eps;
    float r = __frsqrt_rn(mean);
    // Squares beyond fp32's range, or so small that they lose bits: the row times a power of two (its sum is stored before).  (In
    // place and with the same slots: with others 8192 rows of 8192 took 78 us to FP8 tiles, not 72; as a function of its own 84.)
    const bool scaled = ss == INFINITY || mean < kSmallMean;
    if (__builtin_expect(scaled, 0)) {
        const float f = ss == INFINITY ? 0x1p-72f : 0x1p80f;  // largest squares below 2^128 / 16384; the smallest numbers' normal
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int at = t + i * width;
            if (p.sum != nullptr && at < pieces) reinterpret_cast<uint4*>(p.sum + row * p.dim)[at] = pack8(h[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[i][j] *= f;
                ss = fmaf(h[i][j], h[i][j], ss);
            }
        }
        if (!kWarpRow) __syncthreads();  // everyone has read the slots
        ss = reduce_row<kWarpRow>(ss, sums, [](float a, float b) { return a + b; });
        r = __frsqrt_rn(__fdiv_rn(ss, (float)p.dim) + p.eps * f * f);
    }
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int at = t + i * width;
        if (p.sum != nullptr && !scaled && at < pieces) reinterpret_cast<uint4*>(p.sum + row * p.dim)[at] = pack8(h[i]);
        float w[8];
        unpack8(wv[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = at < pieces ? h[i][j] * r * w[j] : 0.f;
        if (p.out != nullptr && at < pieces) reinterpret_cast<uint4*>(p.out + row * p.out_stride)[at] = pack8(h[i]);
        if (kCodes == kRow) most = fmaxf(most, absmax8(h[i]));
    }
    if (kCodes == kNone) return;
    uint2* codes = reinterpret_cast<uint2*>(p.codes + row * p.dim);
    if (kCodes == kRow) {
        most = reduce_row<kWarpRow>(most, maxima, [](float a, float b) { return fmaxf(a, b); });
        const float scale = group_scale(most);
        if (t == 0) static_cast<float*>(p.scale)[row] = scale;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (t + i * width < pieces) codes[t + i * width] = codes8(h[i], scale);
        return;
    }
    // groups of 16 lanes (a tile) or 4 (MX)
    constexpr int lanes = kCodes == kTile ? 16 : 4;
    float m[P];
#pragma unroll
    for (int i = 0; i < P; ++i) m[i] = absmax8(h[i]);
#pragma unroll
    for (int off = 1; off < 4; off <<= 1)
#pragma unroll
        for (int i = 0; i < P; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(kAll, m[i], off));
    const int64_t first = row * (pieces / lanes);
    if (kCodes == kMx) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int at = t + i * width, e = mx_exponent(m[i]);
            const uint2 c = codes8_exp(h[i], e);
            if (at < pieces) {
                codes[at] = c;
                if (at % 4 == 0) static_cast<uint8_t*>(p.scale)[first + at / 4] = (uint8_t)(e + 127);
            }
        }
        return;
    }
#pragma unroll
    for (int off = 4; off < 16; off <<= 1)
#pragma unroll
        for (int i = 0; i < P; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(kAll, m[i], off));
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int at = t + i * width;
        const float scale = group_scale(m[i]);
        if (at < pieces) {
            codes[at] = codes8(h[i], scale);
            if (at % 16 == 0) static_cast<float*>(p.scale)[first + at / 16] = scale;
        }
    }
}

template <Codes kCodes>
void launch(const NormParams& p, cudaStream_t stream) {
    const int pieces = p.dim / 8;
    if (pieces <= 128) {
        const dim3 grid((unsigned)((p.rows + kRowsPerBlock - 1) / kRowsPerBlock)), block(32 * kRowsPerBlock);
        auto kernel = pieces <= 32 ? norm_kernel<1, true, kCodes> : pieces <= 64 ? norm_kernel<2, true, kCodes> : norm_kernel<4, true, kCodes>;
        kernel<<<grid, block, 0, stream>>>(p);
        return;
    }
    // A piece a thread for few rows (32 rows of 4096: 2.0 us, with four 2.3; 1171 of 1536 3.5 and 3.9), four for many, whose
    // loads are in flight together and meet at a quarter of the barriers (8192 rows of 8192, bf16: 79 us, with one 92, with
    // two 108; 16384 of 4096, row codes: 69, 89, 99), and for rows that are longer than a block's threads.
    const int each = p.rows <= kFewRows && pieces <= 1024 ? 1 : 4;
    auto kernel = each == 1 ? norm_kernel<1, false, kCodes> : norm_kernel<4, false, kCodes>;
    const int threads = ((pieces + each - 1) / each + 31) / 32 * 32;
    kernel<<<dim3((unsigned)p.rows), dim3((unsigned)threads), 0, stream>>>(p);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t stream) {
    if (p.rows <= 0) return cudaSuccess;
    if (p.codes == nullptr)
        launch<kNone>(p, stream);
    else if (p.mx)
        launch<kMx>(p, stream);
    else if (p.group == 0)
        launch<kRow>(p, stream);
    else
        launch<kTile>(p, stream);
    return cudaGetLastError();
}

}  // namespace dsa
