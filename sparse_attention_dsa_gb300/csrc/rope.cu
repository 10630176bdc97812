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
// What bounds it: HBM for long steps (every byte is read and written once), launch and a chain of three
// dependent loads (query offsets and length -> page and table row -> stores) for short ones.  So a row is held
// as 16-byte pieces, one to three a lane, whose loads are issued before that chain starts, and a 64-dim rotary
// block is 8 neighbouring lanes: interleaved pairs lie inside a piece, the halves' partner is the piece four
// further, fetched by a shuffle.
//
// Measured (one GB300; 20 calls in a graph, so that up to some 100 MB stay in L2; in brackets with L2 flushed before each).
// rope_append: 4 tokens 2.5 us (3.3), latency; 380 tokens to FP8 4.7 us (7.4): every warp looks through the sequences, 32 a
// round trip (one token of each of 32, 256, 1024 sequences: 3.4, 4.8, 10.2 us); 24693 tokens to FP8 15.1 us (20.5); eight
// ragged chunks of up to 4096 tokens, bf16, 10.6 us (17.9: 75.8 MB in and out, 4.2 TB/s, 0.63 of the copy bandwidth: each
// warp has three loads a lane on their way and then its own chain).  Two tokens a warp were no faster.
// rope_queries: 32 tokens 2.5 us (3.7), 4096 tokens of 128 + 64 heads to MXFP8 46.2 us (50.1; 237 MB, 5.1 TB/s, 0.75),
// to bf16 50.0 (49.3; 269 MB, 0.79), to FP8 52 to 59 (56.1: the quotients' reciprocals and corrections).
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;

// Two fp32 products, or products and sums, in one instruction (rounded like the single ones).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

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
__device__ __forceinline__ uint2 pack_codes(const float (&y)[8]) {
    return make_uint2(codes2(y[0], y[1]) | (codes2(y[2], y[3]) << 16), codes2(y[4], y[5]) | (codes2(y[6], y[7]) << 16));
}
// E4M3 codes of x / scale, the quotient rounded to fp32 first (so that both appends make the same codes).  With the
// correctly rounded reciprocal, y = x inv is within two units in the last place, y s - x is exact, and
// y - (y s - x) inv differs from the quotient by 2^-23 units before its rounding (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990): three packed operations a pair where a division
// takes ten a value.  (The signs are such that -0 stays -0.)  Scales whose products could leave fp32's range divide.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
    const float inv = __frcp_rn(scale);
    float y[8];
    if (scale > 0x1p-80f && scale < 0x1p80f) {
        const float2 inv2 = make_float2(inv, inv), minus2 = make_float2(-inv, -inv), scale2 = make_float2(scale, scale);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 v = mul2(make_float2(x[i], x[i + 1]), inv2);
            const float2 q = fma2(fma2(v, scale2, make_float2(-x[i], -x[i + 1])), minus2, v);
            y[i] = q.x;
            y[i + 1] = q.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], scale);
    }
    return pack_codes(y);
}
// The same for a scale of 2^e, -127 <= e <= 120: the product with 2^-e, a normal number, is the quotient.
__device__ __forceinline__ uint2 codes8_exp(const float (&x)[8], int e) {
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 v = mul2(make_float2(x[i], x[i + 1]), make_float2(inv, inv));
        y[i] = v.x;
        y[i + 1] = v.y;
    }
    return pack_codes(y);
}
__device__ __forceinline__ float absmax8(const float (&x)[8]) {
    const float a = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fabsf(x[2]));
    const float b = fmaxf(fmaxf(fabsf(x[3]), fabsf(x[4])), fabsf(x[5]));
    return fmaxf(fmaxf(fmaxf(a, b), fmaxf(fabsf(x[6]), fabsf(x[7]))), 0.f);  // (the 0: a group of NaN alone)
}
// absmax / 448 in fp32 (1 for an all-zero group); the product with 1/448 and one correction, as above (no quotient by 448
// comes closer to halfway between two fp32 numbers than a 14th of their distance)
__device__ __forceinline__ float group_scale(float amax) {
    if (!(amax > 0x1p-80f && amax < 0x1p120f)) return amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    const float c = 1.f / 448.f, y = amax * c;
    return __fmaf_rn(__fmaf_rn(-448.f, y, amax), c, y);
}

// Shared exponent of an MX group: floor(log2(absmax)) - 8 within the E8M0 range, 0 for an all-zero group.  (Subnormal
// maxima lie below the range either way; an infinity gives 120.)
__device__ __forceinline__ int mx_exponent(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    return bits == 0u ? 0 : max(-127, (int)(bits >> 23) - 127 - 8);
}

// A 64-dim rotary block is 8 pieces of 8 values.  Value i of piece j becomes x_i c_i + o_i s_i, o_i its partner in the
// pair and s_i the sine with the sign of its side.
// The cosines and signed sines of values 4 h .. 4 h + 3 of a piece, from the position's table row.
struct TableTurn {
    const float* row;
    int j;
    __device__ __forceinline__ void get(int h, bool interleaved, float (&c)[4], float (&s)[4]) const {
        if (interleaved) {  // pairs (2i, 2i + 1) of the piece, angles 4j ..
            const float2 a = __ldg(reinterpret_cast<const float2*>(row) + 2 * j + h);
            const float2 b = __ldg(reinterpret_cast<const float2*>(row) + 16 + 2 * j + h);
            c[0] = c[1] = a.x;
            c[2] = c[3] = a.y;
            s[0] = -b.x;
            s[1] = b.x;
            s[2] = -b.y;
            s[3] = b.y;
        } else {  // partner in piece j ^ 4, angles 8 (j & 3) ..
            const float4 a = __ldg(reinterpret_cast<const float4*>(row) + 2 * (j & 3) + h);
            const float4 b = __ldg(reinterpret_cast<const float4*>(row) + 8 + 2 * (j & 3) + h);
            const bool first = j < 4;
            c[0] = a.x;
            c[1] = a.y;
            c[2] = a.z;
            c[3] = a.w;
            s[0] = first ? -b.x : b.x;
            s[1] = first ? -b.y : b.y;
            s[2] = first ? -b.z : b.z;
            s[3] = first ? -b.w : b.w;
        }
    }
};
// The same held in registers, for all the rows of a token.
struct Turn {
    float c[2][4], s[2][4];
    __device__ __forceinline__ void load(const TableTurn& t, bool interleaved) {
        t.get(0, interleaved, c[0], s[0]);
        t.get(1, interleaved, c[1], s[1]);
    }
    __device__ __forceinline__ void get(int h, bool, float (&cc)[4], float (&ss)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            cc[i] = c[h][i];
            ss[i] = s[h][i];
        }
    }
};
// x: piece `own`, rotated in place where `on`.  `partner`: the lane that holds piece j ^ 4 (any lane where there is none);
// `halves`: some lane of the warp pairs by halves (the same in every lane; every lane calls).  The sums are single
// operations: a packed product and a packed sum were compiled to one fused operation, which does not round the product.
template <typename T>
__device__ __forceinline__ void rotate_piece(float (&x)[8], const uint4& own, bool on, int partner, bool interleaved,
                                             bool halves, const T& turn) {
    uint32_t w[4] = {own.x, own.y, own.z, own.w};
    if (halves) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __shfl_sync(kAll, w[i], partner);
    }
    if (!on) return;
    auto half = [&](int h, const float2& o0, const float2& o1) {
        float c[4], s[4];
        turn.get(h, interleaved, c, s);
        const float2 a0 = mul2(make_float2(x[4 * h], x[4 * h + 1]), make_float2(c[0], c[1]));
        const float2 a1 = mul2(make_float2(x[4 * h + 2], x[4 * h + 3]), make_float2(c[2], c[3]));
        const float2 b0 = mul2(o0, make_float2(s[0], s[1])), b1 = mul2(o1, make_float2(s[2], s[3]));
        x[4 * h] = __fadd_rn(a0.x, b0.x);
        x[4 * h + 1] = __fadd_rn(a0.y, b0.y);
        x[4 * h + 2] = __fadd_rn(a1.x, b1.x);
        x[4 * h + 3] = __fadd_rn(a1.y, b1.y);
    };
    auto pair = [](uint32_t v) { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u)); };
    if (interleaved) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            half(h, make_float2(x[4 * h + 1], x[4 * h]), make_float2(x[4 * h + 3], x[4 * h + 2]));
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) half(h, pair(w[2 * h]), pair(w[2 * h + 1]));
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
            if (c0 >= 0 && c1 - c0 <= L && (int64_t)L <= (int64_t)r.max_pages * 64) {
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
__global__ void __launch_bounds__(32 * kAppendWarps, 6) rope_append_kernel(const RopeAppendParams p) {
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
        const bool inter = lane < 8 ? r.kv_interleaved != 0 : r.idx_interleaved != 0;
        rotate_piece(x, v2, on, partner, inter, !r.kv_interleaved || !r.idx_interleaved,
                     TableTurn{r.table + (int64_t)pos * 64, j});
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
                reinterpret_cast<uint2*>(p.k_cache + row * Di)[kp] = codes8_exp(x, e);
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

// Warps of a CTA and warp steps in flight (4096 tokens to MXFP8: 47.0 us; with two steps 58.7, with six 53.6, with eight
// 49.2; with two warps 46.7, with eight 51.1; 6 or 10 CTAs an SM instead of 8: 48.6, 52.8).
constexpr int kQueryWarps = 4;
constexpr int kSteps = 4;

// Position of token t, found by warp 0 for the CTA; -1 where it has none.
__device__ __forceinline__ int cta_position(const RopeParams& r, int t, int warp, int lane) {
    __shared__ int found;
    if (warp == 0) {
        int b, pos;
        const bool ok = locate(r, t, lane, &b, &pos);
        if (lane == 0) found = ok ? pos : -1;
    }
    __syncthreads();
    return found;
}

// A token's work is two lists of warp steps, each shared by the warps of its CTAs (blockIdx.y): heads 4s .. 4s + 3 of
// the attention's queries (8 lanes a head, `pe_parts` CTAs), and two indexer rows (16 lanes a row, the other CTAs); a
// warp takes at most kSteps steps, all in flight at once.  IDX: dsa_dtype_t of the indexer's output.
template <int IDX>
__global__ void __launch_bounds__(32 * kQueryWarps, 8) rope_queries_kernel(const RopeQueriesParams p, int pe_parts) {
    const RopeParams& r = p.r;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x;
    if ((int)blockIdx.y < pe_parts) {
        const int stride = pe_parts * kQueryWarps, s0 = (int)blockIdx.y * kQueryWarps + warp;
        const int j = lane & 7, h0 = lane >> 3;  // piece, head of the step
        const uint16_t* src = p.q_pe + t * p.q_pe_token_stride + h0 * p.q_pe_head_stride + 8 * j;
        uint4 v[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int h = 4 * (s0 + k * stride);
            v[k] = h + h0 < p.heads ? *reinterpret_cast<const uint4*>(src + h * p.q_pe_head_stride) : make_uint4(0, 0, 0, 0);
        }
        const int pos = cta_position(r, (int)t, warp, lane);
        if (pos < 0) return;
        const bool inter = r.kv_interleaved != 0;
        Turn turn;
        turn.load({r.table + (int64_t)pos * 64, j}, inter);
        uint16_t* dst = p.q + (t * p.heads + h0) * 576 + 512 + 8 * j;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int h = 4 * (s0 + k * stride);
            if (h >= p.heads) break;  // uniform over the warp
            float x[8];
            unpack8(v[k], x);
            rotate_piece(x, v[k], true, lane ^ 4, inter, !inter, turn);
            if (h + h0 < p.heads) *reinterpret_cast<uint4*>(dst + h * 576) = pack8(x);
        }
        return;
    }
    const int Di = r.idx_dim, stride = ((int)gridDim.y - pe_parts) * kQueryWarps;
    const int s0 = ((int)blockIdx.y - pe_parts) * kQueryWarps + warp;
    const int kp = lane & 15, h0 = lane >> 4;  // piece, row of the step
    const bool in = 8 * kp < Di;
    const uint16_t* src = p.q_idx_in + t * p.q_idx_stride + h0 * Di + 8 * kp;
    uint4 w[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const int h = 2 * (s0 + k * stride);
        w[k] = h + h0 < p.idx_heads && in ? *reinterpret_cast<const uint4*>(src + h * Di) : make_uint4(0, 0, 0, 0);
    }
    const int pos = cta_position(r, (int)t, warp, lane);
    if (pos < 0) return;
    const int b8 = r.idx_begin >> 3, j = kp - b8;
    const bool inter = r.idx_interleaved != 0;
    const bool turns = in && r.idx_begin >= 0 && j >= 0 && j < 8;
    const int partner = turns ? (lane & 16) + b8 + (j ^ 4) : lane;
    Turn turn;
    if (turns) turn.load({r.table + (int64_t)pos * 64, j}, inter);
    const int64_t row0 = t * p.idx_heads + h0;
    uint8_t* dst = p.q_idx + row0 * Di * (IDX == DSA_BF16 ? 2 : 1) + kp * (IDX == DSA_BF16 ? 16 : 8);
    const int row_bytes = IDX == DSA_BF16 ? 2 * Di : Di;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const int h = 2 * (s0 + k * stride);
        if (h >= p.idx_heads) break;  // uniform over the warp
        const bool on = h + h0 < p.idx_heads && in;
        float x[8];
        unpack8(w[k], x);
        if (r.idx_begin >= 0) rotate_piece(x, w[k], turns, partner, inter, !inter, turn);
        if constexpr (IDX == DSA_BF16) {
            if (on) *reinterpret_cast<uint4*>(dst + h * row_bytes) = pack8(x);
        } else {
            float m = absmax8(x);  // 0 where there is no piece
            m = fmaxf(m, __shfl_xor_sync(kAll, m, 1));
            m = fmaxf(m, __shfl_xor_sync(kAll, m, 2));
            if constexpr (IDX == DSA_MXFP8_E4M3) {
                const int e = mx_exponent(m);
                if (on) {
                    *reinterpret_cast<uint2*>(dst + h * row_bytes) = codes8_exp(x, e);
                    if ((kp & 3) == 0)
                        static_cast<uint8_t*>(p.q_scale)[(row0 + h) * (Di / 32) + (kp >> 2)] = (uint8_t)(e + 127);
                }
            } else {
                m = fmaxf(m, __shfl_xor_sync(kAll, m, 4));
                m = fmaxf(m, __shfl_xor_sync(kAll, m, 8));
                const float scale = group_scale(m);
                if (on) {
                    *reinterpret_cast<uint2*>(dst + h * row_bytes) = codes8(x, scale);
                    if (kp == 0) static_cast<float*>(p.q_scale)[row0 + h] = scale;
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
    // CTAs of each kind a token: enough for kSteps steps a warp; with few tokens more, until the SMs have two each
    const int pe = p.q_pe ? (p.heads + 3) / 4 : 0, idx = p.q_idx_in ? (p.idx_heads + 1) / 2 : 0;
    auto parts = [&](int steps) {
        int n = steps > 0 ? 1 : 0;
        while (n * kQueryWarps < steps && (n * kQueryWarps * kSteps < steps || (int64_t)p.r.total_q * n < p.num_sms)) ++n;
        return n;
    };
    const int pe_parts = parts(pe);
    const dim3 grid((unsigned)p.r.total_q, (unsigned)(pe_parts + parts(idx))), block(32 * kQueryWarps);
    if (p.r.idx_dtype == DSA_MXFP8_E4M3)
        rope_queries_kernel<DSA_MXFP8_E4M3><<<grid, block, 0, stream>>>(p, pe_parts);
    else if (p.r.idx_dtype == DSA_FP8_E4M3)
        rope_queries_kernel<DSA_FP8_E4M3><<<grid, block, 0, stream>>>(p, pe_parts);
    else
        rope_queries_kernel<DSA_BF16><<<grid, block, 0, stream>>>(p, pe_parts);
    return cudaGetLastError();
}

}  // namespace dsa
