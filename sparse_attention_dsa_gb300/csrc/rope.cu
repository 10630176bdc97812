// Position rotation on the way into the caches and of a step's queries ("Day0 Inference Support and
// Performance Optimization for New LLM Architectures", section 3.3: the indexer's inputs are prepared ahead
// of the indexer; sections 4 and 4.1 for the FP8 and MXFP8 forms they are stored in).
//
// Mathematics: pair (x1, x2) of a row at position p becomes (x1 cos - x2 sin, x1 sin + x2 cos) with the 32
// angles of table row p.  The products are rounded before the sum (no fused multiply-add), so the result is
// the one that elementary fp32 operations give, and is rounded once more, to the stored type.
// Quantisation: scale = absmax / 448 per group (1 for an all-zero group) and E4M3(x / scale), correctly
// rounded divisions; MXFP8 groups of 32 take 2^(floor(log2(absmax)) - 8).
//
// What bounds it: HBM for long steps (every byte is read and written once), launch and a chain of four
// dependent loads (query offsets -> length -> page and table row) for short ones.  So a row is held as
// 16-byte pieces, one to three a lane, whose loads are issued before that chain starts, and a 64-dim rotary
// block is 8 neighbouring lanes: interleaved pairs lie inside a piece, the halves' partner is the piece four
// further, fetched by a shuffle.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;

// Two E4M3 codes (a in the low byte), nearest-even, saturating at +-448.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Eight bf16 values of a 16-byte piece.
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(f2_to_bf2(x[0], x[1]), f2_to_bf2(x[2], x[3]), f2_to_bf2(x[4], x[5]), f2_to_bf2(x[6], x[7]));
}
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], scale);
    return make_uint2(codes2(y[0], y[1]) | (codes2(y[2], y[3]) << 16), codes2(y[4], y[5]) | (codes2(y[6], y[7]) << 16));
}
__device__ __forceinline__ float absmax8(const float (&x)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    return m;
}
// absmax / 448 in fp32 (1 for an all-zero group)
__device__ __forceinline__ float group_scale(float amax) { return amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f; }

// Shared exponent of an MX group: floor(log2(absmax)) - 8 within the E8M0 range, 0 for an all-zero group.
// (Subnormal maxima lie below the clamp either way; infinities and NaN take the top exponent.)
__device__ __forceinline__ int mx_exponent(float amax) {
    if (!(amax > 0.f)) return 0;
    const int e = (int)(__float_as_uint(amax) >> 23) - 127 - 8;
    return max(-127, min(127, e));
}
// 2^e for e in [-127, 127] (2^-127 is subnormal)
__device__ __forceinline__ float exp2_int(int e) {
    return e > -127 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(0x00400000u);
}

// Rotates piece j (0..7) of a 64-dim rotary block in place.  Every lane of the warp calls it; `partner` is
// the lane that holds piece j ^ 4 of the same block (any lane when !on).
__device__ __forceinline__ void rotate_piece(float (&x)[8], const uint4& own, int j, bool on, int partner,
                                             bool interleaved, const float* row) {
    uint4 o;
    o.x = __shfl_sync(kAll, own.x, partner);
    o.y = __shfl_sync(kAll, own.y, partner);
    o.z = __shfl_sync(kAll, own.z, partner);
    o.w = __shfl_sync(kAll, own.w, partner);
    if (!on) return;
    const float4* t4 = reinterpret_cast<const float4*>(row);
    if (interleaved) {
        const float4 c = __ldg(t4 + j), s = __ldg(t4 + 8 + j);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(a, cc[i]), __fmul_rn(b, ss[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(a, ss[i]), __fmul_rn(b, cc[i]));
        }
    } else {
        float y[8];
        unpack8(o, y);
        const int q = 2 * (j & 3);
        const float4 c0 = __ldg(t4 + q), c1 = __ldg(t4 + q + 1), s0 = __ldg(t4 + 8 + q), s1 = __ldg(t4 + 9 + q);
        const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // first half: x1 cos - x2 sin; second half: x1 sin + x2 cos
            if (j < 4)
                x[i] = __fsub_rn(__fmul_rn(x[i], cc[i]), __fmul_rn(y[i], ss[i]));
            else
                x[i] = __fadd_rn(__fmul_rn(y[i], ss[i]), __fmul_rn(x[i], cc[i]));
        }
    }
}

// Sequence b, length L and position of token t, found by one warp (every lane returns the same).  False,
// with the error bit raised, when no sequence owns t or its position is inconsistent.
__device__ __forceinline__ bool locate(const RopeParams& r, int t, int lane, int* b_out, int* pos_out) {
    int b = -1, pos = 0;
    for (int j0 = 0; j0 < r.batch; j0 += 32) {
        const int j = j0 + lane;
        int c0 = 0, c1 = 0, L = 0;
        if (j < r.batch) {
            c0 = __ldg(r.cu_q_lens + j);
            c1 = __ldg(r.cu_q_lens + j + 1);
            L = __ldg(r.seq_lens + j);  // beside the offsets: one link less in the chain of loads
        }
        const uint32_t hit = __ballot_sync(kAll, c0 <= t && t < c1);
        if (hit) {
            const int src = __ffs(hit) - 1;
            c0 = __shfl_sync(kAll, c0, src);
            c1 = __shfl_sync(kAll, c1, src);
            L = __shfl_sync(kAll, L, src);
            const int64_t p = (int64_t)L - c1 + t;
            if (c1 - c0 <= L && (int64_t)L <= (int64_t)r.max_pages * 64) {
                b = j0 + src;
                pos = (int)p;
            }
            break;
        }
    }
    if (b < 0 || pos >= r.table_len) {
        if (lane == 0) raise_error(r.err, b < 0 ? DSA_DEVERR_SEQ : DSA_DEVERR_ROPE);
        return false;
    }
    *b_out = b;
    *pos_out = pos;
    return true;
}

constexpr int kAppendWarps = 8;

// One warp per token.  Lane pieces: kv pieces lane and lane + 32 (the latent part, 16 lanes a 128-dim tile);
// a third piece is the rotary part in lanes 0-7 and the indexer key in lanes 16-31.
__global__ void __launch_bounds__(32 * kAppendWarps) rope_append_kernel(const RopeAppendParams p) {
    const RopeParams& r = p.r;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kAppendWarps + warp;
    if (t >= r.total_q) return;
    const bool has_kv = p.kv_new != nullptr, has_k = p.k_new != nullptr;
    const int Di = r.idx_dim;
    const int kp = lane - 16;  // indexer key piece
    const bool k_on = has_k && kp >= 0 && 8 * kp < Di;
    const bool rot_on = has_kv && lane < 8;
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0, v2 = v0;
    if (has_kv) {
        const uint4* src = reinterpret_cast<const uint4*>(p.kv_new + t * p.kv_stride);
        v0 = __ldg(src + lane);
        v1 = __ldg(src + 32 + lane);
        if (lane < 8) v2 = __ldg(src + 64 + lane);
    }
    if (k_on) v2 = __ldg(reinterpret_cast<const uint4*>(p.k_new + t * p.k_stride) + kp);
    int b, pos;
    if (!locate(r, (int)t, lane, &b, &pos)) return;  // uniform over the warp
    const int32_t pg = __ldg(r.page_table + (int64_t)b * r.max_pages + pos / 64);
    if (pg < 0 || pg >= r.num_pages) {
        if (lane == 0) raise_error(r.err, DSA_DEVERR_PAGE);
        return;
    }
    const int64_t row = (int64_t)pg * 64 + (pos & 63);
    // the rotary piece and the key's rotated pieces
    float x[8];
    unpack8(v2, x);
    {
        const int b8 = r.idx_begin >> 3;  // -1 >> 3 = -1: no piece qualifies below
        const int j = lane < 8 ? lane : kp - b8;
        const bool on = rot_on || (k_on && r.idx_begin >= 0 && j >= 0 && j < 8);
        const int partner = on ? (lane < 8 ? lane ^ 4 : 16 + b8 + (j ^ 4)) : lane;
        rotate_piece(x, v2, j, on, partner, lane < 8 ? r.kv_interleaved != 0 : r.idx_interleaved != 0,
                     r.table + (int64_t)pos * 64);
    }
    if (has_kv && !p.kv_fp8) {
        uint4* dst = reinterpret_cast<uint4*>(p.kv_cache + row * 1152);
        dst[lane] = v0;
        dst[32 + lane] = v1;
        if (lane < 8) dst[64 + lane] = pack8(x);
    } else if (has_kv) {
        uint8_t* dst = p.kv_cache + row * kKvFp8RowBytes;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float y[8];
            unpack8(k == 0 ? v0 : v1, y);
            float m = absmax8(y);
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
            const float scale = group_scale(m);
            reinterpret_cast<uint2*>(dst)[32 * k + lane] = codes8(y, scale);
            if ((lane & 15) == 0) *reinterpret_cast<float*>(dst + kKvFp8ScaleOff + 4 * (2 * k + (lane >> 4))) = scale;
        }
        if (lane < 8) reinterpret_cast<uint4*>(dst + kKvFp8RopeOff)[lane] = pack8(x);
    }
    if (has_k && r.idx_dtype == DSA_BF16) {
        if (k_on) reinterpret_cast<uint4*>(p.k_cache + row * Di * 2)[kp] = pack8(x);
    } else if (has_k) {
        float m = k_on ? absmax8(x) : 0.f;
        m = fmaxf(m, __shfl_xor_sync(kAll, m, 1));
        m = fmaxf(m, __shfl_xor_sync(kAll, m, 2));
        if (r.idx_dtype == DSA_MXFP8_E4M3) {
            const int e = mx_exponent(m);
            if (k_on) {
                reinterpret_cast<uint2*>(p.k_cache + row * Di)[kp] = codes8(x, exp2_int(e));
                if ((kp & 3) == 0) static_cast<uint8_t*>(p.k_scale)[row * (Di / 32) + (kp >> 2)] = (uint8_t)(e + 127);
            }
        } else {
            m = fmaxf(m, __shfl_xor_sync(kAll, m, 4));
            m = fmaxf(m, __shfl_xor_sync(kAll, m, 8));
            const float scale = group_scale(m);
            if (k_on) {
                reinterpret_cast<uint2*>(p.k_cache + row * Di)[kp] = codes8(x, scale);
                if (kp == 0) static_cast<float*>(p.k_scale)[row] = scale;
            }
        }
    }
}

constexpr int kQueryWarps = 8;
constexpr int kSteps = 4;  // pieces a lane has in flight

// A token's work is a list of warp steps: step i < pe_steps rotates heads 4i..4i+3 (8 lanes a head), later
// ones hold two indexer rows (16 lanes a row).  gridDim.y CTAs share a token's steps.
__global__ void __launch_bounds__(32 * kQueryWarps) rope_queries_kernel(const RopeQueriesParams p) {
    const RopeParams& r = p.r;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x;
    const int Di = r.idx_dim;
    const int pe_steps = p.q_pe ? (p.heads + 3) / 4 : 0;
    const int steps = pe_steps + (p.q_idx_in ? (p.idx_heads + 1) / 2 : 0);
    const int stride = (int)gridDim.y * kQueryWarps;
    int b = 0, pos = 0;
    bool located = false;
    for (int s0 = (int)blockIdx.y * kQueryWarps + warp; s0 < steps; s0 += stride * kSteps) {
        uint4 v[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int s = s0 + k * stride;
            v[k] = make_uint4(0, 0, 0, 0);
            if (s < pe_steps) {
                const int h = 4 * s + (lane >> 3);
                if (h < p.heads)
                    v[k] = *reinterpret_cast<const uint4*>(p.q_pe + t * p.q_pe_token_stride + h * p.q_pe_head_stride +
                                                           8 * (lane & 7));
            } else if (s < steps) {
                const int h = 2 * (s - pe_steps) + (lane >> 4);
                if (h < p.idx_heads && 8 * (lane & 15) < Di)
                    v[k] = *reinterpret_cast<const uint4*>(p.q_idx_in + t * p.q_idx_stride + (int64_t)h * Di +
                                                           8 * (lane & 15));
            }
        }
        if (!located) {
            if (!locate(r, (int)t, lane, &b, &pos)) return;  // uniform over the warp
            located = true;
        }
        const float* row = r.table + (int64_t)pos * 64;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int s = s0 + k * stride;
            if (s >= steps) break;  // uniform over the warp
            float x[8];
            unpack8(v[k], x);
            if (s < pe_steps) {
                const int h = 4 * s + (lane >> 3);
                rotate_piece(x, v[k], lane & 7, true, lane ^ 4, r.kv_interleaved != 0, row);
                if (h < p.heads)
                    reinterpret_cast<uint4*>(p.q + (t * p.heads + h) * 576 + 512)[lane & 7] = pack8(x);
                continue;
            }
            const int h = 2 * (s - pe_steps) + (lane >> 4), kp = lane & 15;
            const bool on = h < p.idx_heads && 8 * kp < Di;
            const int b8 = r.idx_begin >> 3, j = kp - b8;
            const bool rot = on && r.idx_begin >= 0 && j >= 0 && j < 8;
            rotate_piece(x, v[k], j, rot, rot ? (lane & 16) + b8 + (j ^ 4) : lane, r.idx_interleaved != 0, row);
            const int64_t out = t * p.idx_heads + h;
            if (r.idx_dtype == DSA_BF16) {
                if (on) reinterpret_cast<uint4*>(p.q_idx + out * Di * 2)[kp] = pack8(x);
                continue;
            }
            float m = on ? absmax8(x) : 0.f;
            m = fmaxf(m, __shfl_xor_sync(kAll, m, 1));
            m = fmaxf(m, __shfl_xor_sync(kAll, m, 2));
            if (r.idx_dtype == DSA_MXFP8_E4M3) {
                const int e = mx_exponent(m);
                if (on) {
                    reinterpret_cast<uint2*>(p.q_idx + out * Di)[kp] = codes8(x, exp2_int(e));
                    if ((kp & 3) == 0) static_cast<uint8_t*>(p.q_scale)[out * (Di / 32) + (kp >> 2)] = (uint8_t)(e + 127);
                }
            } else {
                m = fmaxf(m, __shfl_xor_sync(kAll, m, 4));
                m = fmaxf(m, __shfl_xor_sync(kAll, m, 8));
                const float scale = group_scale(m);
                if (on) {
                    reinterpret_cast<uint2*>(p.q_idx + out * Di)[kp] = codes8(x, scale);
                    if (kp == 0) static_cast<float*>(p.q_scale)[out] = scale;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams& p, cudaStream_t stream) {
    const unsigned blocks = (unsigned)(((int64_t)p.r.total_q + kAppendWarps - 1) / kAppendWarps);
    rope_append_kernel<<<blocks, 32 * kAppendWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_rope_queries(const RopeQueriesParams& p, cudaStream_t stream) {
    // few tokens: each one's steps are spread over several CTAs, until the SMs have one each
    const int steps = (p.q_pe ? (p.heads + 3) / 4 : 0) + (p.q_idx_in ? (p.idx_heads + 1) / 2 : 0);
    int parts = 1;
    while (parts * kQueryWarps < steps && (int64_t)p.r.total_q * parts < 2 * p.num_sms) ++parts;
    rope_queries_kernel<<<dim3((unsigned)p.r.total_q, (unsigned)parts), 32 * kQueryWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dsa
