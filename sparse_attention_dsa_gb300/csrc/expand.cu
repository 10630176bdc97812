// Causal attention of prompts with keys and values of every head, made of the paged latent rows (latent attention in its
// expanded form; the absorbed form is prefix.cu's and sfa_impl.cuh's: "Optimizing Inference for Hybrid Attention
// Architectures: From Operator Fusion to Sequence Sharding", section "Breaking Down the Computational Path of Hybrid
// Attention", step 2, without the selection).
//
// With c_s the latent part and r_s the rotary part of position s, and head h's weights wk, wv (128 x 512 each):
//   k[s, h] = [wk c_s | r_s] (192 dims),  v[s, h] = wv c_s (128 dims),
//   z_s = scale * q[t, h] . k[s, h] for s = 0..p_t,  out[t, h] = softmax(z) . v,  lse[t, h] = logsumexp(z).
// A (query, position, head) takes 2 (192 + 128) operations where the absorbed form takes 2 (576 + 512), and a (position,
// head) 2 x 256 x 512 for its keys and values, so this is the form for many queries a sequence.  Keys are rounded to
// bf16, as a projection would leave them (the queries they meet are bf16), values and weights to f16, small ones to bf16.
//
// Four kernels, chained by programmatic launches:
//   gather:  the pages' rows as tiles (of 128 positions, a sequence's own) of nine 16 KB pieces (64 dims of 128 positions;
//            zeros behind the last position; FP8 rows as f16, and then the weights, too), the layout that the tensor cores
//            read (128-byte swizzle); and the plan: where each sequence's tiles and blocks of 256 queries are;
//   keys:    K and V = W c: a matrix product of all tiles and heads, CTA pairs (256 positions x a head's 256 rows);
//   attend:  a CTA takes 256 queries of a head as two tiles of 128 that share K and V; all such items, each as long as its
//            tiles of keys, are cut into equal parts, one for each CTA (long ones behind a whole item each), or (where that does not
//            pay) they are taken whole in turn;
//   combine: the results of items that were cut.
//
// What bounds it, and measured (one GB300; calls in a graph, in brackets with L2 flushed before).  The tensor pipe: a tile of
// 128 x 128 is 1280 cycles of products, in which its softmax (about 1150) and its group's wait for the other tile's products pass.
// An 8192-token prompt of 128 heads 1775 to 1960 us (1910 to 1970), by the card and its power limit, 3.02 TFLOP, up to 1.70 PFLOP/s,
// 0.9 of the measured cuBLAS rate, of which gathering 8, keys 170 (275 GFLOP; their 537 MB are written at HBM's pace for
// writes).  4096 queries behind 12288 of 16 heads 402 to 411 us (405 to 430), 0.88 of it: the parts' results and their combination
// 15.  Eight ragged prompts of up to 1171 queries, 32 heads, FP8 rows 173 to 175 us (181 to 184): a quarter of the pairs in
// its tiles are masked, an item of some six tiles costs about two more, keys 48.  Three prompts of up to 200 queries, 16 heads
// 24 us (34): three kernels' latency, one after another.  With small values (kSmall) everywhere: 503 for the chunk, 217, 27 for the
// short ones, 2295 for the long one.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace dsa {
namespace {

constexpr uint32_t kAllLanes = 0xFFFFFFFFu;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kUnit = 128 * 128;               // 16 KB: 128 positions x 64 dims, or 64 positions x 128 dims
constexpr int kTileBytes = kExpandTileBytes;   // latent and rotary parts of 128 positions: nine units
constexpr int kHeadTile = kExpandHeadTileBytes;  // keys (two units) and values (two) of 128 positions of a head
constexpr int kBlockRows = kExpandBlockRows;

// What the gathering kernel leaves of its plan (int32): a PlanHead, then for each sequence its first tile, its first block
// of queries and its first place on the line (one more of each than sequences), and first_bad.  Between the head and these,
// with parts: the parts' first places on the line of all heads (int64).
struct PlanHead {
    int32_t tiles;    // in use
    int32_t blocks;   // of queries, of a head
    int32_t counter;  // whole items handed out
    int32_t parts;    // the line of items is cut in so many parts; 0: whole items
    int32_t group;    // whole items: heads that are worked on together
    int32_t whole;    // with parts: the last so many blocks of each head are whole items in front of them
    int32_t head_line;  // with parts: places of a head's other blocks
    int32_t sorted;   // whole items: block_order() holds
    int32_t wide;     // some values are kept as bf16 (see kSmall)
    int32_t pad;
};
__device__ __forceinline__ PlanHead* plan_head(const ExpandParams& p) { return reinterpret_cast<PlanHead*>(p.plan); }
__device__ __forceinline__ long long* part_begins(const ExpandParams& p) { return reinterpret_cast<long long*>(plan_head(p) + 1); }
// (whole items: in the same place) a head's blocks, those with the most tiles first
__device__ __forceinline__ int32_t* block_order(const ExpandParams& p) { return reinterpret_cast<int32_t*>(part_begins(p)); }
constexpr int kSortBlocks = 256;
static_assert(kSortBlocks <= 2 * (kExpandCtas + 1), "block_order()");
__device__ __forceinline__ int32_t* tile_begin(const ExpandParams& p) { return p.plan + kExpandPlanHead; }
__device__ __forceinline__ int32_t* block_begin(const ExpandParams& p) { return tile_begin(p) + p.batch + 1; }
__device__ __forceinline__ int32_t* place_begin(const ExpandParams& p) { return block_begin(p) + p.batch + 1; }
// First position of a sequence that has no finite values or no page (INT32_MAX: none): rows that see it are NaN.  -1: the
// sequence is left out, as its tiles do not fit.
__device__ __forceinline__ int32_t* first_bad(const ExpandParams& p) { return place_begin(p) + p.batch + 1; }
static_assert(kExpandPlanHead == sizeof(PlanHead) / 4 + 2 * (kExpandCtas + 1), "expand_plan_bytes()");

// The line: the blocks of head 0, of head 1, ..., each kItemCost places for what it costs beside its tiles (its queries' load,
// its first scores' latency, its result) and one for each tile of keys.  It is cut into equal parts, of kMinPlaces at least
// on average, or its items are taken whole in turn:
//   * whole, where the estimate of the last CTA's time is no longer than with parts (three short prompts 24.0 us, cut 31.4;
//     eight ragged ones 174, cut 187; but 256 items of 112 tiles, for 152 CTAs, 465, cut 404);
//     With parts, each CTA takes first one whole item (the last blocks of the heads, as many as all heads have CTAs for), where
//     those leave every CTA a part: CTAs at the same head then meet its keys at about the same time, from L2
//     instead of HBM, where parts alone begin anywhere (4096 queries behind 12288 of 16 heads 401 us for 417, the last
//     1569 and 2048 of 27359 and 28000 positions 803 for 863).
//   * whole, where the longest item is no more than 1 / kWholeItems of a CTA's share: heads go in groups whose keys and
//     values (kGroupBytes) stay in L2 while all their blocks meet them (the 8192-token prompt of 128 heads 1912 us, at the power
//     limit; head by head 1935, all heads together 2099, cut 2139).
constexpr int kItemCost = 2;  // (1 and 3: no difference beyond the runs')
constexpr int kMinPlaces = 4;
constexpr int kWholeItems = 8;
constexpr int kCutCost = 8;  // what cutting costs a CTA: writing parts, combining
constexpr int64_t kGroupBytes = 48 << 20;
__device__ __forceinline__ int tiles_before(int place, int n) { return min(n, max(0, place - kItemCost)); }
// Tiles of keys that n queries from position pos0 see.
__device__ __forceinline__ int tiles_seen(int pos0, int n) { return (pos0 + n + 127) / 128; }
// Places of a sequence's first i blocks, all of them whole, its first query at position pos0: block j takes kItemCost +
// tiles_seen(pos0 + 256 j, 256) = kItemCost + tiles_seen(pos0, 0) + 2 (j + 1).
static_assert(kBlockRows == 256, "two tiles more for each block");
__device__ __forceinline__ int64_t places_before(int pos0, int64_t i) { return i * (kItemCost + tiles_seen(pos0, 0)) + i * (i + 1); }
__device__ __forceinline__ int64_t places_of(int pos0, int n) {
    const int64_t whole = places_before(pos0, n / kBlockRows);
    return n % kBlockRows ? whole + kItemCost + tiles_seen(pos0, n) : whole;
}
// The plan and the lengths are read from L2: the combining kernel looks at them before it has waited for the kernel in front.
__device__ __forceinline__ int ld_plan(const int32_t* a) { return __ldcg(a); }
// The last of a[0 .. n - 1] (ascending) that is not above x; a[0] is not.  Called by a whole warp.
__device__ __forceinline__ int last_not_above(const int32_t* a, int n, int x, int lane) {
    int lo = 0;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const uint32_t le = __ballot_sync(kAllLanes, step * lane < n && ld_plan(a + lo + step * lane) <= x);  // (lane 0's always)
        const int k = 31 - __clz(le);
        lo += step * k;
        n = min(step, n - step * k);
    }
    return lo;
}

__device__ __forceinline__ float exp2_fast(float x) {  // relative error about 2^-22; exp2(-inf) = +0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Queries and positions of sequence b; false when they are inconsistent.
__device__ __forceinline__ bool sequence(const ExpandParams& p, int b, int* c0, int* n, int* L) {
    const int a = p.cu_q_lens[b], e = p.cu_q_lens[b + 1];
    *c0 = a;
    *n = 0;
    *L = p.seq_lens[b];
    if (a < 0 || e < a || e > p.total_q) return false;
    *n = e - a;
    if (*n == 0) return true;
    return *n <= *L && (int64_t)*L <= (int64_t)p.max_pages * 64 && *L <= INT32_MAX - 255;
}

// The sequence that a tile belongs to: the last one that begins no later and has tiles.
__device__ __forceinline__ int sequence_of_tile(const ExpandParams& p, int tile) {
    const int32_t* begin = tile_begin(p);
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (begin[mid] <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Values and weights are multiplied as f16 (11 bits, for bf16's 8: the output's error, 2 bf16 roundings less, fell from
// 0.0030 to 0.0022 of its norm, of which 0.0017 are its own rounding).  Values are kept times kValueGain, which is taken out of
// the result: exact down to 2^-16 and up to 65504 / kValueGain.
constexpr float kValueGain = 4.f;
constexpr float kValueLimit = 16380.f;  // times kValueGain it is 65520, which rounds to f16's infinity
// Smaller ones lose bits (f16's steps end at 2^-24, that is 2^-26 of a value), so that a vector of small values alone would be
// coarse or 0.  Where a position's largest value of a head, not 0, is below 2^-13 (as f16, times kValueGain: kSmall), the 32
// positions that a warp of the keys kernel writes are kept, with their weights, as bf16: any magnitude, 8 bits.  Elsewhere a
// value is off by 2^-27 at most, 2^-14 of its vector's largest.  The choice is a byte for each 32 positions of a head (`forms`),
// which says how the weights are rounded and how the products of those positions are issued.
constexpr uint32_t kSmall = 0x1000;  // 2^-11
__device__ __forceinline__ uint32_t f2_to_h2(float a, float b) {  // a in the low half
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// FP8 rows are multiplied as f16, too (a code's four bits times a scale lose 2^-11 of it, for bf16's 2^-8: error 0.0022 instead of
// 0.0031), and the weights with them.  A position's row, and kGainRows rows of the weights together, are kept times a power of
// two that brings their largest magnitude to 2^14 or more, at least kRowGain or kWeightGain: down to 2^-28 of the largest no bit
// is lost.  The keys kernel takes both out of its sums.
constexpr float kRowGain = 4.f;
constexpr int kRowGainLog2 = 2, kWeightGainLog2 = 4, kMostGainLog2 = 62;  // (the products of two stay within fp32)
constexpr float kWeightGain = 16.f;
constexpr int kGainRows = 16;  // (a factor for each column of a result instead: eight ragged prompts 193 us for 174)
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// The gain's exponent for a largest magnitude with this exponent of its own (128: not finite).
__device__ __forceinline__ int gain_log2(int largest, int least) { return max(least, min(kMostGainLog2, 14 - largest)); }
// Eight E4M3 codes times a scale (in fp32), rounded to f16.
__device__ __forceinline__ uint4 codes_to_h8(uint32_t lo, uint32_t hi, float scale) {
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint16_t pair = (uint16_t)((j < 2 ? lo : hi) >> (16 * (j & 1)));
        float a, b;
        asm("{\n\t.reg .b32 h2;\n\t.reg .f16 l, h;\n\tcvt.rn.f16x2.e4m3x2 h2, %2;\n\tmov.b32 {l, h}, h2;\n\t"
            "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
            : "=f"(a), "=f"(b)
            : "h"(pair));
        out[j] = f2_to_h2(a * scale, b * scale);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}
// The magnitude of a code without its sign (0x7F: NaN, as 480).
__device__ __forceinline__ float code_value(uint32_t c) {
    return (c >> 3) ? (float)(8 + (c & 7)) * power_of_two((int)(c >> 3) - 10) : (float)(c & 7) * 0x1p-9f;
}
// Whether one of sixteen codes, none a NaN, times a finite scale is beyond f16's range (a rare path).
__device__ __forceinline__ bool codes_beyond(const uint4& code, float scale) {
    if (!(fabsf(scale) < INFINITY)) return false;
    const uint32_t w[4] = {code.x, code.y, code.z, code.w};
    bool found = false;
#pragma unroll 1
    for (int j = 0; j < 16; ++j) {
        const uint32_t c = (w[j >> 2] >> (8 * (j & 3))) & 0x7Fu;
        found |= c != 0x7Fu && code_value(c) * fabsf(scale) * kRowGain >= 65520.f;
    }
    return found;
}
// Nonzero in the sign bits' places where one of two f16 values has an exponent of all ones (it carries into them).
__device__ __forceinline__ uint32_t not_finite2(uint32_t h) { return ((h & 0x7C007C00u) + 0x04000400u) & 0x80008000u; }

// ---------------------------------------------------------------------------------------------------------
// gather: a block takes 16 positions at a time, a warp two of them (with 64 a block, 4096 positions took 11.7 us).  Every block numbers the sequences' tiles for
// itself (each thread a run of sequences, then a scan of the threads' sums), which costs less than a kernel in front; the
// first one leaves the plan.  Rows of a page that is out of range become NaN, and so the scores of whoever sees them.
// Bound by HBM and L2: 1152 or 656 bytes read, 1152 written a position.
// ---------------------------------------------------------------------------------------------------------
constexpr int kGatherWarps = 8;
constexpr int kGatherThreads = 32 * kGatherWarps;
constexpr int kGatherRows = 2 * kGatherWarps;
constexpr int kGatherUnits = 128 / kGatherRows;  // of a tile

__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const ExpandParams p) {
    __shared__ long long scan[3][kGatherWarps];
    __shared__ int longest[kGatherWarps];
    __shared__ __align__(16) int block_tiles[kSortBlocks];
    __shared__ int2 found[2];  // (sequence, first tile), one for each parity of the loop
    __shared__ uint32_t largest_weight[2][kGatherWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool plans = blockIdx.x == 0;
    grid_dependency_wait();
    allow_dependent_launch();
    const int run = (p.batch + kGatherThreads - 1) / kGatherThreads;
    const int b0 = min(p.batch, tid * run), b1 = min(p.batch, b0 + run);
    long long sum[3] = {0, 0, 0};  // tiles, blocks, places
    int most = 0;
    for (int b = b0; b < b1; ++b) {
        int c0, n, L;
        if (!sequence(p, b, &c0, &n, &L)) {
            if (plans) raise_error(p.err, DSA_DEVERR_SEQ);
            continue;
        }
        if (n == 0) continue;
        sum[0] += (L + 127) / 128;
        sum[1] += (n + kBlockRows - 1) / kBlockRows;
        sum[2] += places_of(L - n, n);
        most = max(most, kItemCost + (L + 127) / 128);
    }
    long long incl[3] = {sum[0], sum[1], sum[2]};
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const long long o = __shfl_up_sync(kAllLanes, incl[i], off);
            if (lane >= off) incl[i] += o;
        }
        most = max(most, __shfl_xor_sync(kAllLanes, most, off));
    }
    if (lane == 31) {
        for (int i = 0; i < 3; ++i) scan[i][warp] = incl[i];
        longest[warp] = most;
    }
    __syncthreads();
    long long before[3], all[3] = {0, 0, 0};
    for (int i = 0; i < 3; ++i) {
        before[i] = incl[i] - sum[i];
        for (int w = 0; w < kGatherWarps; ++w) {
            if (w < warp) before[i] += scan[i][w];
            all[i] += scan[i][w];
        }
    }
    const int tiles = (int)(all[0] < p.cap_tiles ? all[0] : p.cap_tiles);
    if (plans) {
        for (int w = 0; w < kGatherWarps; ++w) most = max(most, longest[w]);
        long long at[3] = {before[0], before[1], before[2]};
        for (int b = b0; b < b1; ++b) {
            int c0, n, L;
            const bool ok = sequence(p, b, &c0, &n, &L) && n > 0;
            const int mine = ok ? (L + 127) / 128 : 0, parts = ok ? (n + kBlockRows - 1) / kBlockRows : 0;
            // (more pages than were announced, or offsets that run backwards: left out)
            const bool fits = at[0] + mine <= p.cap_tiles && at[1] + parts <= p.cap_blocks;
            if (ok && !fits) raise_error(p.err, DSA_DEVERR_SEQ);
            tile_begin(p)[b] = (int32_t)(at[0] < p.cap_tiles ? at[0] : p.cap_tiles);
            block_begin(p)[b] = (int32_t)(at[1] < p.cap_blocks ? at[1] : p.cap_blocks);
            place_begin(p)[b] = (int32_t)at[2];  // (looked at where all of it is within 32 bits)
            first_bad(p)[b] = ok && !fits ? -1 : INT32_MAX;
            at[0] += mine;
            at[1] += parts;
            if (ok) at[2] += places_of(L - n, n);
        }
        // (what does not fit leaves places that nobody works on)
        const int blocks = (int)(all[1] < p.cap_blocks ? all[1] : p.cap_blocks);
        const long long line = all[2] * p.heads;
        int parts = (int)(line / kMinPlaces < p.ctas ? max(1LL, line / kMinPlaces) : p.ctas);
        // how long the last CTA takes with whole items (its share and half an item; no more than one item each), and with parts
        const long long alone = all[1] * p.heads <= p.ctas ? most : line / p.ctas + most / 2, cut = line / parts + kCutCost;
        if (all[1] > p.cap_blocks || all[2] > INT32_MAX || alone <= cut || line >= (long long)kWholeItems * p.ctas * most) parts = 0;
        const int whole = parts == p.ctas && (long long)(most + kMinPlaces) * p.ctas <= line ? min(p.ctas / p.heads, blocks - 1) : 0;
        // Items of several sequences are taken in the order of their lengths, so that the CTAs end together (eight ragged prompts of
        // 32 heads, FP8 rows: 175 us, sequence by sequence 180); of one they
        // are in that order, and so many blocks that they are not sorted end together anyway.
        const bool sorted = parts == 0 && p.batch > 1 && blocks <= kSortBlocks && all[1] == blocks && blocks * p.heads > p.ctas;
        if (tid == 0) {
            PlanHead h = {};
            h.sorted = sorted;
            h.tiles = tiles;
            h.blocks = blocks;
            h.parts = parts;
            h.whole = whole;
            h.counter = p.ctas;  // every CTA takes the item of its own number first
            h.group = max(1, min(p.heads, (int)(kGroupBytes / kHeadTile) / max(1, tiles)));
            *plan_head(p) = h;
            tile_begin(p)[p.batch] = tiles;
            block_begin(p)[p.batch] = blocks;
            place_begin(p)[p.batch] = (int32_t)all[2];
            if (p.cu_q_lens[0] != 0 || p.cu_q_lens[p.batch] != p.total_q) raise_error(p.err, DSA_DEVERR_SEQ);
        }
        if (sorted) {
            static_assert(kGatherThreads == kSortBlocks, "a block a thread");
            block_tiles[tid] = -1;
            __syncthreads();
            int at = (int)before[1];
            for (int b = b0; b < b1; ++b) {
                int c0, n, L;
                if (!sequence(p, b, &c0, &n, &L)) continue;
                for (int q = 0; q < n; q += kBlockRows) block_tiles[at++] = tiles_seen(L - n + q, min(kBlockRows, n - q));
            }
            __syncthreads();
            const int mine = block_tiles[tid];
            int rank = 0;
#pragma unroll 4
            for (int i = 0; i < kSortBlocks; i += 4) {
                const int4 v = *reinterpret_cast<const int4*>(block_tiles + i);
                rank += v.x > mine || (v.x == mine && i < tid);
                rank += v.y > mine || (v.y == mine && i + 1 < tid);
                rank += v.z > mine || (v.z == mine && i + 2 < tid);
                rank += v.w > mine || (v.w == mine && i + 3 < tid);
            }
            if (tid < blocks) block_order(p)[rank] = tid;
        }
        if (parts > 0) {
            __syncthreads();  // the arrays are there
            // Position of a block's first query, its sequence's first place, and its number in it.
            auto look_up = [&](int block, int* n, int* pos0, int* first) {
                int lo = 0, hi = p.batch;  // the last sequence that begins no later
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (ld_plan(block_begin(p) + mid) <= block) lo = mid;
                    else hi = mid;
                }
                *n = p.cu_q_lens[lo + 1] - p.cu_q_lens[lo];
                *pos0 = p.seq_lens[lo] - *n;
                *first = ld_plan(place_begin(p) + lo);
                return block - ld_plan(block_begin(p) + lo);
            };
            int n, pos0, first;
            if (tid == 0) {
                int32_t head_line = (int32_t)all[2];
                if (whole > 0) {
                    const int i = look_up(blocks - whole, &n, &pos0, &first);
                    head_line = first + (int32_t)places_before(pos0, i);
                }
                plan_head(p)->head_line = head_line;
                part_begins(p)[0] = 0;
            }
            // CTA c's part is its share of all places without its whole item (in 1 / parts of a place)
            long long share = tid < parts ? line : 0;
            if (tid < whole * p.heads) {
                const int i = look_up(blocks - 1 - tid / p.heads, &n, &pos0, &first), q = i * kBlockRows;
                share -= (long long)parts * (kItemCost + tiles_seen(pos0 + q, min(kBlockRows, n - q)));
            }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long o = __shfl_up_sync(kAllLanes, share, off);
                if (lane >= off) share += o;
            }
            if (lane == 31) scan[0][warp] = share;
            __syncthreads();
            for (int w = 0; w < warp; ++w) share += scan[0][w];
            if (tid < p.ctas) part_begins(p)[tid + 1] = share / parts;
        }
    }
    if (p.kv_fp8) {  // the heads' weights as f16 (by the last blocks first: the first ones have the plan and the first rows)
        static_assert(kGainRows * 512 / 8 == 4 * kGatherThreads, "four pieces a thread");
        bool beyond = false;
        uint32_t turn = 0;
        for (int i = (int)gridDim.x - 1 - (int)blockIdx.x; i < p.heads * (256 / kGainRows); i += (int)gridDim.x, turn ^= 1u) {
            const uint4* src = reinterpret_cast<const uint4*>(p.w_kv) + (int64_t)i * 4 * kGatherThreads + tid;
            uint4* dst = reinterpret_cast<uint4*>(p.weights16) + (int64_t)i * 4 * kGatherThreads + tid;
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = src[k * kGatherThreads];
            uint32_t most = 0;  // as bf16 bits, in either half
#pragma unroll
            for (int k = 0; k < 4; ++k)
                most = __vmaxu2(__vmaxu2(most, __vmaxu2(v[k].x & 0x7FFF7FFFu, v[k].y & 0x7FFF7FFFu)),
                                __vmaxu2(v[k].z & 0x7FFF7FFFu, v[k].w & 0x7FFF7FFFu));
            most = __reduce_max_sync(kAllLanes, max(most & 0xFFFFu, most >> 16));
            if (lane == 0) largest_weight[turn][warp] = most;
            __syncthreads();
            most = __reduce_max_sync(kAllLanes, largest_weight[turn][lane % kGatherWarps]);
            const int log2 = gain_log2((int)(most >> 7) - 127, kWeightGainLog2);
            const float gain = power_of_two(log2);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = __uint_as_float(w[j] << 16), b = __uint_as_float(w[j] & 0xFFFF0000u);
                    h[j] = f2_to_h2(a * gain, b * gain);
                    if (not_finite2(h[j]) != 0)
                        beyond |= (fabsf(a) < INFINITY && fabsf(a) * kWeightGain >= 65520.f) ||
                                  (fabsf(b) < INFINITY && fabsf(b) * kWeightGain >= 65520.f);
                }
                dst[k * kGatherThreads] = make_uint4(h[0], h[1], h[2], h[3]);
            }
            if (tid == 0) p.weight_scale[i] = power_of_two(-log2);
        }
        if (beyond) raise_error(p.err, DSA_DEVERR_RANGE);
    }
    const int64_t units = (int64_t)kGatherUnits * tiles;
    uint32_t turn = 0;
    for (int64_t i = blockIdx.x; i < units; i += gridDim.x, turn ^= 1u) {
        const int tile = (int)(i / kGatherUnits), row0 = kGatherRows * (int)(i % kGatherUnits);
        if (tile >= before[0] && tile < before[0] + sum[0]) {  // a sequence of this thread's run
            long long at = before[0];
            for (int b = b0; b < b1; ++b) {
                int c0, n, L;
                if (!sequence(p, b, &c0, &n, &L) || n == 0) continue;
                if (tile < at + (L + 127) / 128) {
                    found[turn] = make_int2(b, (int)at);
                    break;
                }
                at += (L + 127) / 128;
            }
        }
        __syncthreads();
        const int b = found[turn].x, base = 128 * (tile - found[turn].y) + row0;
        const int L = p.seq_lens[b];
        const int pg = base < L ? p.page_table[(int64_t)b * p.max_pages + (base >> 6)] : 0;
        const bool in = pg >= 0 && pg < p.num_pages;
        if (!in && tid == 0) raise_error(p.err, DSA_DEVERR_PAGE);
        uint8_t* dst = p.latents + (int64_t)tile * kTileBytes;
        const uint4 zero = make_uint4(0, 0, 0, 0), nan = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);  // (as f16, too)
#pragma unroll
        for (int j = warp; j < kGatherRows; j += kGatherWarps) {
            const int row = row0 + j, of_page = (base & 63) + j;
            const bool have = in && base + j < L;
            const uint4 none = in || base + j >= L ? zero : nan;
            auto put = [&](int chunk, uint4 v) {  // 16-byte chunk of the row's 72
                *reinterpret_cast<uint4*>(dst + (chunk >> 3) * kUnit + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)) = v;
            };
            if (!p.kv_fp8 || !have) {
                if (p.kv_fp8 && lane == 0) p.row_scale[(int64_t)tile * 128 + row] = 1.f;
                const uint4* src = reinterpret_cast<const uint4*>(p.kv_cache + ((int64_t)pg * 64 + of_page) * 1152);
                uint4 v[3];
#pragma unroll
                for (int k = 0; k < 3; ++k) v[k] = have && lane + 32 * k < 72 ? src[lane + 32 * k] : none;
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (lane + 32 * k < 72) put(lane + 32 * k, v[k]);
            } else {
                const uint8_t* src = p.kv_cache + ((int64_t)pg * 64 + of_page) * kKvFp8RowBytes;
                const uint4 code = reinterpret_cast<const uint4*>(src)[lane];
                const float scale = reinterpret_cast<const float*>(src + kKvFp8ScaleOff)[lane >> 3];
                const uint4 rot = lane < 8 ? reinterpret_cast<const uint4*>(src + kKvFp8RopeOff)[lane] : zero;
                uint32_t most = __vmaxu4(__vmaxu4(code.x & 0x7F7F7F7Fu, code.y & 0x7F7F7F7Fu),
                                         __vmaxu4(code.z & 0x7F7F7F7Fu, code.w & 0x7F7F7F7Fu));
                most = __vmaxu2(most & 0x00FF00FFu, (most >> 8) & 0x00FF00FFu);
                const float largest = fabsf(code_value(max(most & 0xFFFFu, most >> 16)) * scale);
                const int log2 = gain_log2((int)(__reduce_max_sync(kAllLanes, __float_as_uint(largest)) >> 23) - 127, kRowGainLog2);
                if (lane == 0) p.row_scale[(int64_t)tile * 128 + row] = power_of_two(-log2);
                float gained = scale * power_of_two(log2);
                // (codes of 0 beside a scale that the gain takes beyond fp32 are 0; others with such a scale are beyond range)
                if (fabsf(gained) == INFINITY && fabsf(scale) < INFINITY) gained = copysignf(FLT_MAX, scale);
                const uint4 lo = codes_to_h8(code.x, code.y, gained), hi = codes_to_h8(code.z, code.w, gained);
                put(2 * lane, lo);
                put(2 * lane + 1, hi);
                if (lane < 8) put(64 + lane, rot);
                // (an infinity makes what the keys kernel finds; here is known whether it was one before)
                const uint32_t odd = not_finite2(lo.x) | not_finite2(lo.y) | not_finite2(lo.z) | not_finite2(lo.w) |
                                     not_finite2(hi.x) | not_finite2(hi.y) | not_finite2(hi.z) | not_finite2(hi.w);
                if (odd != 0 && codes_beyond(code, scale)) raise_error(p.err, DSA_DEVERR_RANGE);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------------------
// keys: D (256 positions x 256) = c W[h]^T for each pair of tiles and each head, cta_group::2: CTA c of the pair holds
// tile 2 i + c and rows 128 c .. of the head's weights (c = 0: keys, 1: values), both in chunks of 64 inner dims; its
// tensor memory receives its tile's keys and values.  A pair's tile takes half of what two single ones would from L2 (64 bytes
// a cycle and SM), which would bound it otherwise.  8192 positions of 128 heads: 170 us, 1.6 PFLOP/s (head after head; tile
// after tile 180; without its stores 137: 537 MB, which writes alone take 134 us for).
// ---------------------------------------------------------------------------------------------------------
constexpr int kKeysThreads = 256;  // warp 0: TMA, 1: products, 2: tensor memory, 4-7: results
constexpr int kKeysResultWarp = 4;
constexpr int kKeysStages = 6;
constexpr int kPiece = 32 * 128;  // 32 positions x 64 dims
template <bool F16>  // FP8 rows
constexpr uint32_t kIdescKeys = make_idesc(256, 256, F16 ? 0 : 1, F16 ? 0 : 1, 0, 0);

struct KeysCtrl {
    uint64_t full[kKeysStages], empty[kKeysStages];
    uint64_t d_full[2], d_empty[2];
    uint64_t drained;
    uint32_t tmem_base;
    int32_t failed;
};
constexpr int kKeysSmem = 1024 + kKeysStages * 2 * kUnit + 4 * 2 * kPiece + (int)sizeof(KeysCtrl);
static_assert(kKeysSmem <= 232448, "shared memory of one CTA");

template <bool F16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kKeysThreads, 1)
    keys_kernel(const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CUtensorMap wmap, const ExpandParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* o_s = smem + kKeysStages * 2 * kUnit;
    KeysCtrl* ctl = reinterpret_cast<KeysCtrl*>(o_s + 4 * 2 * kPiece);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_ctarank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (tid == 0) {
        prefetch_tensormap(&cmap);
        prefetch_tensormap(&wmap);
        for (int i = 0; i < kKeysStages; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->d_full[i], 1);
            mbar_init(&ctl->d_empty[i], 8);  // the result warps of both CTAs
        }
        mbar_init(&ctl->drained, 1);
        ctl->failed = 0;
        fence_mbar_init();
    }
    __syncwarp();
    cluster_arrive();
    if (warp == 2) {
        tmem_pair_alloc(&ctl->tmem_base, 512);
        tmem_pair_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    cluster_wait();  // the peer's barriers exist before anything arrives on them
    tc_fence_after();
    grid_dependency_wait();
    allow_dependent_launch();
    const uint32_t tmem = ctl->tmem_base;
    const int tiles = plan_head(p)->tiles;
    // unit u: tile pair u % tile_pairs of head u / tile_pairs, so that all pairs of CTAs are at the same few heads' weights
    const int tile_pairs = (tiles + 1) / 2;
    const int64_t units = (int64_t)tile_pairs * p.heads;
    auto leader = [&](uint64_t* bar) { return mapa_shared(smem_u32(bar), 0); };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(kAllLanes, mbar_wait(bar, parity, p.err, p.wait_ns)) != 0;
    };
    bool ok = true;

    // (loads and products by one thread each: see the attention's products)
    auto wait_one = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, p.err, p.wait_ns); };
    if (warp == 0) {
        if (elect_one_sync()) {
            const uint32_t full = leader(&ctl->full[0]);
            uint32_t n = 0;
            for (int64_t u = pair; ok && u < units; u += pairs) {
                const int tile = 2 * (int)(u % tile_pairs) + rank, head = (int)(u / tile_pairs);
#pragma unroll 1
                for (int k = 0; k < 8; ++k, ++n) {
                    const uint32_t slot = n % kKeysStages;
                    if (!(ok = wait_one(&ctl->empty[slot], ((n / kKeysStages) & 1u) ^ 1u))) break;
                    uint8_t* dst = smem + slot * 2 * kUnit;
                    if (rank == 0) mbar_arrive_expect_tx(&ctl->full[slot], 4 * kUnit);
                    // (the tile behind the last one, where their number is odd, has its place but no rows of its own)
                    tma_pair_load_3d(dst, &cmap, full + 8 * slot, 0, 0, 9 * tile + k);
                    tma_pair_load_3d(dst + kUnit, &wmap, full + 8 * slot, 64 * k, 128 * rank, head);
                }
            }
        }
        ok = __all_sync(kAllLanes, ok);
    } else if (warp == 1 && rank == 0) {
        if (elect_one_sync()) {
            const uint64_t ad = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
            uint32_t n = 0, t = 0;
            for (int64_t u = pair; ok && u < units; u += pairs, ++t) {
                const uint32_t buf = t & 1u;
                if (!(ok = wait_one(&ctl->d_empty[buf], ((t >> 1) & 1u) ^ 1u))) break;
                tc_fence_after();
#pragma unroll 1
                for (int k = 0; k < 8; ++k, ++n) {
                    const uint32_t slot = n % kKeysStages;
                    if (!(ok = wait_one(&ctl->full[slot], (n / kKeysStages) & 1u))) break;
                    const uint64_t a = ad + (uint64_t)(slot * (2 * kUnit / 16));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma_pair_f16_ss(tmem + 256 * buf, a + (uint64_t)(2 * j), a + (uint64_t)(kUnit / 16 + 2 * j),
                                         kIdescKeys<F16>, k == 0 && j == 0 ? 0u : 1u);
                    umma_pair_commit(&ctl->empty[slot], 3);
                }
                if (ok) umma_pair_commit(&ctl->d_full[buf], 3);
            }
            // drain (default limit): every product of the pair is done before its memory is given back
            umma_pair_commit(&ctl->drained, 1);
            mbar_wait(&ctl->drained, 0, p.err);
        }
        ok = __all_sync(kAllLanes, ok);
    } else if (warp >= kKeysResultWarp) {
        // warp w has positions 32 w .. of its CTA's tile, a lane each: keys in columns 0-127, values behind them
        const int ew = warp - kKeysResultWarp;
        const uint32_t trow = tmem + ((uint32_t)(32 * ew) << 16);
        const uint32_t d_empty = leader(&ctl->d_empty[0]);
        uint8_t* stage = o_s + ew * 2 * kPiece;
        uint32_t t = 0;
        for (int64_t u = pair; ok && u < units; u += pairs, ++t) {
            const int tile = 2 * (int)(u % tile_pairs) + rank, head = (int)(u / tile_pairs);
            const uint32_t buf = t & 1u;
            // (FP8 rows: what the position and the weights' rows were multiplied by, taken out)
            const float row_scale = F16 ? p.row_scale[(int64_t)tile * 128 + 32 * ew + lane] : 1.f;
            const float4* weight_scale = reinterpret_cast<const float4*>(p.weight_scale + head * (256 / kGainRows));
            if (!(ok = wait(&ctl->d_full[buf], (t >> 1) & 1u))) break;
            tc_fence_after();
            uint8_t* dst = p.kv + ((int64_t)tile * p.heads + head) * kHeadTile;
            // dims 64 c .. of the values: unit 2 + position / 64
            auto values_at = [&](int c) { return dst + (2 + (ew >> 1)) * kUnit + c * (kUnit / 2) + (ew & 1) * kPiece; };
            auto give_back = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(d_empty + 8 * buf);
            };
            bool bad = false, beyond = false;  // a value is not finite as f16; and is finite itself
            uint32_t most = 0, any = 0;        // the position's largest value as f16, in either half; all values' bits
            bool wide = false;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {  // 64 columns each
                float v[4][16];
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld16(trow + 256 * buf + 64 * c + 16 * k, v[k]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_regs_ready(v[k]);
                if (F16) {
                    static_assert(kGainRows == 16, "of a load of 16 columns");
                    const float4 of = weight_scale[c];
                    const float f[4] = {row_scale * of.x, row_scale * of.y, row_scale * of.z, row_scale * of.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[k][i] *= f[k];
                }
                uint4 w[8];
                if (c < 2) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float* f = &v[k >> 1][8 * (k & 1)];
                        w[k] = make_uint4(f2_to_bf2(f[0], f[1]), f2_to_bf2(f[2], f[3]), f2_to_bf2(f[4], f[5]), f2_to_bf2(f[6], f[7]));
                    }
                } else {
                    uint32_t here = 0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float* f = &v[k >> 1][8 * (k & 1)];
                        uint32_t* h = reinterpret_cast<uint32_t*>(&w[k]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            h[i] = f2_to_h2(f[2 * i] * kValueGain, f[2 * i + 1] * kValueGain);
                            here = __vmaxu2(here, h[i] & 0x7FFF7FFFu);
                            any |= __float_as_uint(f[2 * i]) | __float_as_uint(f[2 * i + 1]);
                        }
                    }
                    most = __vmaxu2(most, here);
                    // A weight of 0 times a value that is not finite is NaN, for rows that do not see the position too: its
                    // values become 0, and the rows that do see it NaN at the end.
                    if (max(here & 0xFFFFu, here >> 16) >= 0x7C00u) {
                        bad = true;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int i = 0; i < 16; ++i) beyond |= fabsf(v[k][i]) < INFINITY && fabsf(v[k][i]) >= kValueLimit;
#pragma unroll
                        for (int k = 0; k < 8; ++k) w[k] = make_uint4(0, 0, 0, 0);
                    }
                    if (c == 3) {
                        wide = __any_sync(kAllLanes, max(most & 0xFFFFu, most >> 16) < kSmall && (any << 1) != 0);
                        if (!wide) give_back();
                    }
                }
                uint8_t* at = stage + (c & 1) * kPiece;
                if (lane == 0) bulk_wait_read<1>();
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) st_shared_v4(smem_u32(at) + lane * 128 + ((k ^ (lane & 7)) << 4), w[k]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    // keys: unit c, positions in rows of 128 bytes
                    if (tile < tiles) bulk_copy_s2g(c < 2 ? dst + c * kUnit + ew * kPiece : values_at(c - 2), at, kPiece);
                    bulk_commit();
                }
            }
            if (__builtin_expect(wide, 0)) {
                if (lane == 0) bulk_wait_all();  // the same places are written once more
                __syncwarp();
#pragma unroll 1
                for (int c = 128; c < 256; c += 16) {
                    float v[16];
                    tmem_ld16(trow + 256 * buf + c, v);
                    tmem_ld_wait();
                    tmem_regs_ready(v);
                    const float f = F16 ? row_scale * p.weight_scale[head * (256 / kGainRows) + c / kGainRows] : 1.f;
                    uint32_t h[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[i] = bad ? 0u : f2_to_bf2(v[2 * i] * f * kValueGain, v[2 * i + 1] * f * kValueGain);
                    uint8_t* at = stage + ((c >> 6) & 1) * kPiece + lane * 128;
                    const int chunk = (c >> 3) & 7;
                    st_shared_v4(smem_u32(at) + ((chunk ^ (lane & 7)) << 4), make_uint4(h[0], h[1], h[2], h[3]));
                    st_shared_v4(smem_u32(at) + (((chunk + 1) ^ (lane & 7)) << 4), make_uint4(h[4], h[5], h[6], h[7]));
                }
                give_back();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    for (int c = 0; c < 2; ++c) {  // (a group for each piece, as above)
                        if (tile < tiles) bulk_copy_s2g(values_at(c), stage + c * kPiece, kPiece);
                        bulk_commit();
                    }
                }
            }
            if (lane == 0 && tile < tiles) {
                p.forms[((int64_t)tile * p.heads + head) * 4 + ew] = wide;
                if (wide) plan_head(p)->wide = 1;
            }
            if (bad && tile < tiles) {
                const int b = sequence_of_tile(p, tile);
                if (beyond) raise_error(p.err, DSA_DEVERR_RANGE);
                atomicMin(first_bad(p) + b, 128 * (tile - tile_begin(p)[b]) + 32 * ew + lane);
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    if (!ok && lane == 0) ctl->failed = 1;
    tc_fence_before();
    __syncthreads();
    if (ctl->failed && tid == 0) {
        // a wait gave up: nobody consumed the copies still in flight, so leave them time to land (they take
        // microseconds) before this shared memory is given back
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
    }
    cluster_sync();  // neither CTA leaves before the other's products, copies and arrivals are done
    tc_fence_after();
    if (warp == 2) tmem_pair_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------------------------------------
// attend: S_w = Q_w K^T and O_w += P_w V for the two query tiles w = 0, 1 in turn, all in tensor memory (P over its own S as
// 16-bit pairs), so that the softmax of one tile runs under the products of the other.  K and V come in 16 KB units (bulk
// copies of what the keys kernel left in the tensor cores' layout) through a ring, each unit freed by the products that read it
// last.  The running maximum is raised only when it grows by more than 2^kRaise.
// Tried and not kept: results by warps of their own (the softmax's registers), one barrier for all units of a tile's keys or
// values (the ring refills later: 440 us for 420 where keys come from HBM), both groups at the same queries' tiles of
// keys in turn where there are no more than 128 (as long: it reads twice the keys a step), cut items joined by the last CTA
// with a part (its code took registers from the softmax's loop: 1.3 times the time of all).
// ---------------------------------------------------------------------------------------------------------
constexpr int kAttendThreads = 352;  // warps 0-3 and 4-7: softmax of the two query tiles, 8: loads, 9: products, 10: segments
constexpr int kLoadWarp = 8;
constexpr int kProductWarp = 9;
// (With segments looked up by the loads' warp, between its loads, three short prompts took 23.3 us, for 22.4; but an 8192-token
// prompt of 128 heads in a long loop, at the power limit, 1.3% less than with this warp.)
constexpr int kPlanWarp = 10;
constexpr int kRing = 8;             // units of K and V, in turn K K K V V
constexpr int kQTile = 3 * kUnit;    // 128 queries x 192 dims
constexpr int kTileUnits = 5;
constexpr int kOCol = 256;           // tensor memory: S (and P in its first half) at 0 and 128, O at 256 and 384
constexpr uint32_t kIdescQK = make_idesc(128, 128, 1, 1, 0, 0);
constexpr uint32_t kIdescPV = make_idesc(128, 128, 0, 0, 0, 1);
constexpr uint32_t kIdescWide = make_idesc(128, 128, 1, 1, 0, 1) - kIdescPV;  // what bf16 operands add to it
constexpr float kRaise = 4.f;  // the running maximum (log2) is raised only when it grows by more than this
// Weights are taken relative to 2^-kLift of the running maximum: as f16, up to 2^(kRaise + kLift) = 2^15, they keep their
// precision down to 2^-25 of the largest one's, so that a long context's many small weights beside a large one are not lost.
constexpr float kLift = 11.f;

// What a CTA works on at a time: a block of queries of a head, with the tiles of keys from j0 to j1 (all of them, or a part)
struct Segment {
    int32_t row0, nrows;  // query tokens (none: no more segments)
    int32_t head, seq;
    int32_t pos0;         // position of the first
    int32_t tile0;        // first tile of the sequence's keys
    int32_t n0, n1;       // tiles that queries 0-127, 128-255 see
    int32_t j0, j1;
    int32_t bad;          // first position without finite values (see first_bad())
    int32_t wide;         // some values of the call are bf16 (see kSmall)
};
// In flight between the roles of a CTA (with 3 it keeps items that another could begin: eight ragged prompts 178 us for 174).
constexpr int kSegments = 2;
// 32 bytes: one whole sector where `whole` says that dst is 32-byte aligned, as 16-byte pieces otherwise (arrays may begin at
// any multiple of 16).
__device__ __forceinline__ void st_global_32(void* dst, const uint32_t* v, bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

struct AttendCtrl {
    uint64_t q_full[2], q_empty[2];
    uint64_t full[kRing], empty[kRing];
    uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
    uint64_t seg_full[kSegments], seg_empty[kSegments];
    uint64_t drained;
    uint32_t tmem_base;
    int32_t failed;
    Segment segments[kSegments];
};
__device__ __forceinline__ bool is_whole(const Segment& s) { return s.j0 == 0 && s.j1 == max(s.n0, s.n1); }
// Query tile w's tiles of a segment: from j0 to here.
__device__ __forceinline__ int seg_end(const Segment& s, int w) { return min(s.j1, w == 0 ? s.n0 : s.n1); }

// Rows and keys of block i of sequence b; false where the sequence is left out.
__device__ __forceinline__ bool block_rows(const ExpandParams& p, int b, int i, Segment* s) {
    const int c0 = ld_plan(p.cu_q_lens + b), n = ld_plan(p.cu_q_lens + b + 1) - c0, q = i * kBlockRows;
    s->seq = b;
    s->row0 = c0 + q;
    s->nrows = min(kBlockRows, n - q);
    s->pos0 = ld_plan(p.seq_lens + b) - n + q;
    s->tile0 = ld_plan(tile_begin(p) + b);
    s->n0 = tiles_seen(s->pos0, min(s->nrows, 128));
    s->n1 = s->nrows > 128 ? tiles_seen(s->pos0, s->nrows) : 0;
    s->bad = ld_plan(first_bad(p) + b);
    return s->bad >= 0;
}
// The block at place x of a head's line: its sequence and number there, its first place, and that of the next block.
// Called by a whole warp.
struct Place {
    int b, i, begin, end;
};
__device__ __forceinline__ Place block_at(const ExpandParams& p, int x, int lane) {
    Place w;
    w.b = last_not_above(place_begin(p), p.batch, x, lane);
    const int n = ld_plan(p.cu_q_lens + w.b + 1) - ld_plan(p.cu_q_lens + w.b), pos0 = ld_plan(p.seq_lens + w.b) - n;
    const int first = ld_plan(place_begin(p) + w.b);
    int lo = 0, hi = (n + kBlockRows - 1) / kBlockRows;  // the last block that begins no later
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (places_before(pos0, mid) <= x - first) lo = mid;
        else hi = mid;
    }
    w.i = lo;
    w.begin = first + (int)places_before(pos0, lo);
    w.end = first + (int)((lo + 1) * kBlockRows <= n ? places_before(pos0, lo + 1) : places_of(pos0, n));
    return w;
}
// Part k of the line starts here.
__device__ __forceinline__ int64_t part_begin(const ExpandParams& p, int k) { return __ldcg(part_begins(p) + k); }
// How the values of a tile and head are kept: a byte for each 32 positions, 1 for bf16.
__device__ __forceinline__ uint32_t forms_of(const ExpandParams& p, int tile, int head) {
    return reinterpret_cast<const uint32_t*>(p.forms)[(int64_t)tile * p.heads + head];
}
// Weights of a tile's positions that are kept as bf16, from f16 in place.  (Rolled up: with a second conversion beside the first, in
// the softmax's loop or in a loop of its own, calls without such values took 2 to 3% longer instead of 1.)
__device__ __forceinline__ void widen(uint32_t scol, uint32_t forms) {
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
        if (!((forms >> (8 * g)) & 1u)) continue;
        float h[16];  // pairs
        tmem_ld16(scol + 16 * g, h);
        tmem_ld_wait();
        tmem_regs_ready(h);
        uint32_t packed[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
            packed[i] = f2_to_bf2(e.x, e.y);
        }
        tmem_st16_u32(scol + 16 * g, packed);
    }
    tmem_st_wait();
}
// Where CTA c leaves a part of an item: at most the first and the last segment of its part of the line are parts of items, and
// the last begins its item.
__device__ __forceinline__ float* part_slot(const ExpandParams& p, int c, bool first_tile) {
    return p.partial + (int64_t)(2 * c + (first_tile ? 1 : 0)) * kExpandPartFloats;
}
// The result of a query tile, or of its part of an item: behind the tile's last products, by the warps of its softmax.  (Parts
// are combined by a kernel of their own: done here by an item's last part, the code for it cost the softmax's loop its
// registers, called or not: 2250 us for an 8192-token prompt of 128 heads that takes 1735.)
__device__ __forceinline__ void write_result(const ExpandParams& p, AttendCtrl* ctl, uint32_t seg, uint32_t ocol, bool have, float m_used,
                                          float l_sum) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, w = warp >> 2, row = 128 * w + (tid & 127);
    const Segment& it = ctl->segments[seg];
    const int nrows = it.nrows;
    const bool whole = is_whole(it), first_tile = it.j0 == 0;
    const int64_t at = (int64_t)(it.row0 + row) * p.heads + it.head;
    const bool poisoned = it.bad <= it.pos0 + row;
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->seg_empty[seg]);
    auto free_o = [&] {  // in registers: the next products may have it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->o_free[w]);
    };
    auto read_o = [&](int c, float (&o)[2][16]) {
        tmem_ld16(ocol + c, o[0]);
        tmem_ld16(ocol + c + 16, o[1]);
        tmem_ld_wait();
        tmem_regs_ready(o[0]);
        tmem_regs_ready(o[1]);
    };
    uint16_t* dst = p.out + at * 128;
    if (whole) {
        if (poisoned) l_sum = NAN;
        const float inv = l_sum == 0.f ? 0.f : 1.f / (kValueGain * l_sum);
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
            float o[2][16];
            read_o(c, o);
            if (row < nrows) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = f2_to_bf2(o[k][2 * i] * inv, o[k][2 * i + 1] * inv);
                    st_global_32(dst + c + 16 * k, v, p.sectors);
                }
            }
        }
        free_o();
        if (row < nrows && p.lse) p.lse[at] = l_sum == 0.f ? -INFINITY : (m_used + log2f(l_sum)) * kLn2;
        return;
    }
    float* slot = part_slot(p, blockIdx.x, first_tile);
    if (have) {
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
            float o[2][16];
            read_o(c, o);
            if (row < nrows) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(o[k >> 1][8 * (k & 1) + i] * (1.f / kValueGain));
                    st_global_32(slot + row * 128 + c + 8 * k, v, p.sectors);
                }
            }
        }
        free_o();
    }
    if (row < nrows) reinterpret_cast<float2*>(slot + kBlockRows * 128)[row] = make_float2(m_used, l_sum);
}

constexpr int kAttendSmem = 1024 + 2 * kQTile + kRing * kUnit + (int)sizeof(AttendCtrl);
static_assert(kAttendSmem <= 232448, "shared memory of one CTA");

__global__ void __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap nopemap, const __grid_constant__ CUtensorMap pemap, const ExpandParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* ring = smem + 2 * kQTile;
    AttendCtrl* ctl = reinterpret_cast<AttendCtrl*>(ring + kRing * kUnit);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        prefetch_tensormap(&nopemap);
        prefetch_tensormap(&pemap);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->q_full[i], 1);
            mbar_init(&ctl->q_empty[i], 1);
            mbar_init(&ctl->s_full[i], 1);
            mbar_init(&ctl->p_full[i], 4);
            mbar_init(&ctl->o_full[i], 1);
            mbar_init(&ctl->o_free[i], 4);
        }
        for (int i = 0; i < kSegments; ++i) {
            mbar_init(&ctl->seg_full[i], 1);
            mbar_init(&ctl->seg_empty[i], 10);  // the softmax warps, loads, products
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
        }
        mbar_init(&ctl->drained, 1);
        ctl->failed = 0;
        fence_mbar_init();
    }
    if (warp == kProductWarp) {
        tmem_alloc(&ctl->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dependency_wait();
    allow_dependent_launch();
    const uint32_t tmem = ctl->tmem_base;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(kAllLanes, mbar_wait(bar, parity, p.err, p.wait_ns)) != 0;
    };
    bool ok = true;

    if (warp == kLoadWarp) {
        // ---------------- what the segments need in the order of its use ----------------
        if (elect_one_sync()) {
            auto wait_one = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, p.err, p.wait_ns); };
            uint32_t u = 0, used[2] = {0, 0};  // units, segments that used each query tile
            for (uint32_t n = 0; ok; ++n) {
                if (!(ok = wait_one(&ctl->seg_full[n % kSegments], (n / kSegments) & 1u))) break;
                const Segment s = ctl->segments[n % kSegments];
                mbar_arrive(&ctl->seg_empty[n % kSegments]);
                if (s.nrows == 0) break;
                const uint8_t* kv = p.kv + ((int64_t)s.tile0 * p.heads + s.head) * kHeadTile;
                const uint8_t* rotary = p.latents + (int64_t)s.tile0 * kTileBytes + 8 * kUnit;
                auto load_q = [&](int w) {
                    if (!wait_one(&ctl->q_empty[w], (used[w] & 1u) ^ 1u)) return false;
                    ++used[w];
                    mbar_arrive_expect_tx(&ctl->q_full[w], kQTile);
                    uint8_t* dst = smem + w * kQTile;
                    tma_load_3d(dst, &nopemap, &ctl->q_full[w], 0, s.head, s.row0 + 128 * w);
                    tma_load_3d(dst + kUnit, &nopemap, &ctl->q_full[w], 64, s.head, s.row0 + 128 * w);
                    tma_load_3d(dst + 2 * kUnit, &pemap, &ctl->q_full[w], 0, s.head, s.row0 + 128 * w);
                    return true;
                };
                if (s.j0 < s.n0) ok = load_q(0);
                for (int j = s.j0; ok && j < s.j1; ++j) {
                    const uint8_t* tile = kv + (int64_t)j * p.heads * kHeadTile;
#pragma unroll 1
                    for (int k = 0; ok && k < kTileUnits; ++k, ++u) {
                        const uint32_t slot = u % kRing;
                        if (!(ok = wait_one(&ctl->empty[slot], ((u / kRing) & 1u) ^ 1u))) break;
                        const uint8_t* src = k == 2 ? rotary + (int64_t)j * kTileBytes : tile + (k < 2 ? k : k - 1) * kUnit;
                        mbar_arrive_expect_tx(&ctl->full[slot], kUnit);
                        bulk_copy_g2s(ring + slot * kUnit, src, kUnit, &ctl->full[slot]);
                        if (j == s.j0 && k == 2 && s.j0 < s.n1) ok = load_q(1);
                    }
                }
            }
        }
        ok = __all_sync(kAllLanes, ok);
    } else if (warp == kPlanWarp) {
        // ---------------- segments, looked up ahead of their use ----------------
        const PlanHead plan = *plan_head(p);
        uint32_t n = 0;
        Segment s;
        s.wide = plan.wide;
        auto publish = [&] {
            if (!wait(&ctl->seg_empty[n % kSegments], ((n / kSegments) & 1u) ^ 1u)) return false;
            if (lane == 0) {
                ctl->segments[n % kSegments] = s;
                mbar_arrive(&ctl->seg_full[n % kSegments]);
            }
            __syncwarp();
            ++n;
            return true;
        };
        if (plan.parts > 0) {
            // this CTA's whole item, if it has one, and its part of the line: the other blocks of head 0, of head 1, ...
            if ((int)blockIdx.x < plan.whole * p.heads) {
                const int block = plan.blocks - 1 - (int)blockIdx.x / p.heads;
                const int b = last_not_above(block_begin(p), p.batch, block, lane);
                s.head = (int)blockIdx.x % p.heads;
                if (block_rows(p, b, block - block_begin(p)[b], &s)) {
                    s.j0 = 0;
                    s.j1 = max(s.n0, s.n1);
                    ok = publish();
                }
            }
            const int64_t head_line = plan.head_line, x1 = part_begin(p, blockIdx.x + 1);
            int64_t x = part_begin(p, blockIdx.x);
            while (ok && x < x1) {
                s.head = (int)(x / head_line);
                const int at = (int)(x - s.head * head_line);
                const Place w = block_at(p, at, lane);
                const int n_tiles = w.end - w.begin - kItemCost;
                const int64_t left = x1 - s.head * head_line;  // the part's end on this head's line
                s.j0 = tiles_before(at - w.begin, n_tiles);
                s.j1 = left >= w.end ? n_tiles : tiles_before((int)left - w.begin, n_tiles);
                if (s.j1 > s.j0 && block_rows(p, w.b, w.i, &s)) ok = publish();
                x = s.head * head_line + w.end;
            }
        } else {
            // Whole items, as CTAs become free.  Heads in groups whose keys fit L2, the last ones, whose keys were made last,
            // first; in a group the longest items first (or the last blocks, of a sequence the ones with the most keys).
            const int64_t n_items = (int64_t)plan.blocks * p.heads, group_items = (int64_t)plan.blocks * plan.group;
            int64_t index = blockIdx.x;
            while (ok && index < n_items) {
                const int group = (int)(index / group_items), rest = (int)(index - group * group_items);
                const int heads = min(plan.group, p.heads - group * plan.group), turn = rest / heads;
                const int block = plan.sorted ? ld_plan(block_order(p) + turn) : plan.blocks - 1 - turn;
                s.head = p.heads - 1 - (group * plan.group + rest % heads);
                const int b = last_not_above(block_begin(p), p.batch, block, lane);
                if (block_rows(p, b, block - block_begin(p)[b], &s)) {
                    s.j0 = 0;
                    s.j1 = max(s.n0, s.n1);
                    ok = publish();
                }
                int next = 0;
                if (lane == 0) next = atomicAdd(&plan_head(p)->counter, 1);
                index = __shfl_sync(kAllLanes, next, 0);
            }
        }
        s.nrows = 0;
        if (ok) ok = publish();
    } else if (warp == kProductWarp) {
        // ---------------- S_w(j) = Q_w K(j)^T and O_w += P_w(j) V(j), the two query tiles in turn ----------------
        // The steps of all segments form one row: a step's scores are asked for between the products of the weights of the
        // step before it, also where that is the last of another segment.  One thread does it all: with waits and elections
        // of the whole warp a unit's four products took 440 cycles to issue, and to be done 256.
        if (elect_one_sync()) {
            auto wait_one = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, p.err, p.wait_ns); };
            const uint64_t qd = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
            const uint64_t kd = smem_desc(smem_u32(ring), 16, 1024, kSwizzle128B);
            const uint64_t vd = smem_desc(smem_u32(ring), kUnit / 2, 1024, kSwizzle128B);  // MN-major, dims 64.. half a unit on
            uint32_t segs[2] = {0, 0}, tiles_done[2] = {0, 0};
            struct Step {
                uint32_t u;              // its first unit
                uint32_t forms;          // of its values, a byte for each 32 positions
                bool have[2];            // which query tiles have it
                bool first[2], last[2];  // of its segment
            };
            auto qk = [&](int w, const Step& t) {
                if (!t.have[w]) return true;
                if (t.first[w] && !wait_one(&ctl->q_full[w], segs[w] & 1u)) return false;
                const bool shared = t.have[w ^ 1];  // the other query tile reads these keys, too: the first waits, the second frees
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const uint32_t at = t.u + k, slot = at % kRing;
                    if ((w == 0 || !shared) && !wait_one(&ctl->full[slot], (at / kRing) & 1u)) return false;
                    if (k == 0) tc_fence_after();
                    const uint64_t a = qd + (uint64_t)((w * kQTile + k * kUnit) / 16), b = kd + (uint64_t)(slot * (kUnit / 16));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16_ss(tmem + 128 * w, a + (uint64_t)(2 * kk), b + (uint64_t)(2 * kk), kIdescQK,
                                    k == 0 && kk == 0 ? 0u : 1u);
                    if (k == 2) umma_commit(&ctl->s_full[w]);
                    if (w == 1 || !shared) umma_commit(&ctl->empty[slot]);
                }
                if (t.last[w]) umma_commit(&ctl->q_empty[w]);
                return true;
            };
            auto pv = [&](int w, const Step& t) {
                if (!t.have[w]) return true;
                uint32_t idesc[4];  // of 32 positions each
#pragma unroll
                for (int i = 0; i < 4; ++i) idesc[i] = kIdescPV + ((t.forms >> (8 * i)) & 1u) * kIdescWide;
                if (!wait_one(&ctl->p_full[w], tiles_done[w] & 1u)) return false;
                ++tiles_done[w];
                if (t.first[w] && !wait_one(&ctl->o_free[w], (segs[w] & 1u) ^ 1u)) return false;
                const bool shared = t.have[w ^ 1];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t at = t.u + 3 + k, slot = at % kRing;
                    if ((w == 0 || !shared) && !wait_one(&ctl->full[slot], (at / kRing) & 1u)) return false;
                    if (k == 0) tc_fence_after();
                    const uint64_t b = vd + (uint64_t)(slot * (kUnit / 16));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16_ts(tmem + kOCol + 128 * w, tmem + 128 * w + 32 * k + 8 * kk, b + (uint64_t)(128 * kk),
                                    idesc[2 * k + (kk >> 1)], t.first[w] && k == 0 && kk == 0 ? 0u : 1u);
                    if (w == 1 || !shared) umma_commit(&ctl->empty[slot]);
                }
                if (t.last[w]) {
                    umma_commit(&ctl->o_full[w]);
                    ++segs[w];
                }
                return true;
            };
            uint32_t u = 0;
            Step before = {};
            for (uint32_t n = 0; ok; ++n) {
                if (!(ok = wait_one(&ctl->seg_full[n % kSegments], (n / kSegments) & 1u))) break;
                const Segment s = ctl->segments[n % kSegments];
                mbar_arrive(&ctl->seg_empty[n % kSegments]);
                if (s.nrows == 0) break;
                for (int j = s.j0; ok && j < s.j1; ++j, u += kTileUnits) {
                    Step now;
                    now.u = u;
                    now.forms = s.wide ? forms_of(p, s.tile0 + j, s.head) : 0;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        now.have[w] = j < seg_end(s, w);
                        now.first[w] = j == s.j0;
                        now.last[w] = j == seg_end(s, w) - 1;
                    }
                    ok = pv(0, before) && qk(0, now) && pv(1, before) && qk(1, now);
                    before = now;
                }
            }
            ok = ok && pv(0, before) && pv(1, before);
            // drain (default limit): every product is done before its memory is given back
            umma_commit(&ctl->drained);
            mbar_wait(&ctl->drained, 0, p.err);
        }
        ok = __all_sync(kAllLanes, ok);
    } else {
        // ---------------- softmax: a thread has a query of its warp group's tile ----------------
        const int w = warp >> 2, r = tid & 127;
        const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t scol = trow + 128 * w, ocol = trow + kOCol + 128 * w;
        uint32_t tile = 0, used = 0;
        for (uint32_t n = 0; ok; ++n) {
            if (!(ok = wait(&ctl->seg_full[n % kSegments], (n / kSegments) & 1u))) break;
            const Segment& it = ctl->segments[n % kSegments];  // read again behind the loop, to spare its registers
            if (it.nrows == 0) break;
            const int end = seg_end(it, w), begin = it.j0, first = it.pos0 + 128 * w;
            auto give_back = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->seg_empty[n % kSegments]);
            };
            if (end <= begin && (is_whole(it) || 128 * w >= it.nrows)) {  // nothing for this query tile
                give_back();
                continue;
            }
            float m_used = -INFINITY, l_sum = 0.f;  // what weights are relative to (log2): the maximum - kLift; their sum
#pragma unroll 1
            for (int j = begin; j < end; ++j, ++tile) {
                const bool wide = it.wide != 0;
                if (!(ok = wait(&ctl->s_full[w], tile & 1u))) break;
                tc_fence_after();
                float s[8][16];
#pragma unroll
                for (int k = 0; k < 8; ++k) tmem_ld16(scol + 16 * k, s[k]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 8; ++k) tmem_regs_ready(s[k]);
                if (128 * j + 128 > first + 1) {  // some query does not see all of it
                    const int seen = first + r + 1 - 128 * j;
#pragma unroll
                    for (int k = 0; k < 128; ++k)
                        if (k >= seen) s[k >> 4][k & 15] = -INFINITY;
                }
                float mx[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) mx[i] = s[0][i];
#pragma unroll
                for (int k = 1; k < 8; ++k)
#pragma unroll
                    for (int i = 0; i < 16; ++i) mx[i] = fmaxf(mx[i], s[k][i]);
#pragma unroll
                for (int h = 8; h > 0; h >>= 1)
#pragma unroll
                    for (int i = 0; i < h; ++i) mx[i] = fmaxf(mx[i], mx[i + h]);
                const float mt = mx[0] * p.scale_log2;
                const bool raise = mt > m_used + (kRaise + kLift);
                const float m_new = raise ? mt - kLift : m_used;
                const float alpha = raise && m_used != -INFINITY ? exp2f(m_used - m_new) : 1.f;
                const float mu = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet: exp2(-inf) = 0
                if (__any_sync(kAllLanes, alpha != 1.f)) {  // (the products before this tile's scores are done)
#pragma unroll 1
                    for (int c = 0; c < 128; c += 16) {
                        float o[16];
                        tmem_ld16(ocol + c, o);
                        tmem_ld_wait();
                        tmem_regs_ready(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= alpha;
                        tmem_st16(ocol + c, o);
                    }
                }
                // weights: the sum takes the fp32 values, the products their rounding to f16 (at most 2^-11 of each, unbiased), and those
                // once more to bf16 where the values are (see kSmall)
                float2 sum[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
                const float2 scale2 = make_float2(p.scale_log2, p.scale_log2), mu2 = make_float2(-mu, -mu);
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    uint32_t packed[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float* x = &s[k + (i >> 4)][i & 15];
                        float2 e = fma2(make_float2(x[0], x[1]), scale2, mu2);
                        e.x = exp2_fast(e.x);
                        e.y = exp2_fast(e.y);
                        packed[i / 2] = f2_to_h2(e.x, e.y);
                        sum[(i / 2) & 3] = add2(sum[(i / 2) & 3], e);
                    }
                    tmem_st16_u32(scol + 8 * k, packed);
                }
                const float2 half = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                l_sum = l_sum * alpha + (half.x + half.y);
                m_used = m_new;
                tmem_st_wait();
                if (__builtin_expect(wide, 0)) widen(scol, forms_of(p, it.tile0 + j, it.head));
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->p_full[w]);
            }
            if (!ok) break;
            // ---- the result, or a part's ----
            const bool have = end > begin;
            if (have) {
                if (!(ok = wait(&ctl->o_full[w], used & 1u))) break;
                ++used;
                tc_fence_after();
            }
            write_result(p, ctl, n % kSegments, ocol, have, m_used, l_sum);
        }
    }
    if (!ok && lane == 0) ctl->failed = 1;
    tc_fence_before();
    __syncthreads();
    if (ctl->failed && tid == 0) {
        // a wait gave up: nobody consumed the copies still in flight, so leave them time to land (they take
        // microseconds) before this shared memory is given back
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == kProductWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------------------------------------
// combine: items that were cut, 32 rows a block, four a warp; of a row's parts (m_k in log2 units, l_k, O_k)
//   M = max m_k, L = sum_k l_k 2^(m_k - M), out = sum_k 2^(m_k - M) O_k / L, lse = (M + log2 L) ln 2
// ---------------------------------------------------------------------------------------------------------
constexpr int kCombineWarps = 8;
constexpr int kRowsPerWarp = 4;
constexpr int kCombineRows = kRowsPerWarp * kCombineWarps;
constexpr int kBatches = 2;  // of rows, one after another (all blocks are resident at once)

__global__ void __launch_bounds__(32 * kCombineWarps) combine_kernel(const ExpandParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = blockIdx.x + 1;
    // The plan is older than the attention: its blocks, when they let this kernel start, had waited for the end of what
    // made it.  So the item is looked up while the attention still runs.  (No block returns before its end, though: what is
    // launched behind this kernel takes the end of all blocks for the end of the attention.)
    const bool begins = k < ld_plan(&plan_head(p)->parts);
    int64_t begin = 0;
    int n_tiles = 0, last = k;
    auto cut = [&](int part) {  // the item's tiles in front of a part
        const int64_t at = part_begin(p, part) - begin;
        return at >= kItemCost + n_tiles ? n_tiles : at <= 0 ? 0 : tiles_before((int)at, n_tiles);
    };
    Segment s;
    s.nrows = 0;
    if (begins) {
        // the item in which part k begins; the first part that begins inside it takes care of it
        const int64_t head_line = ld_plan(&plan_head(p)->head_line), x = part_begin(p, k);
        s.head = (int)(x / head_line);
        const Place w = block_at(p, (int)(x - s.head * head_line), lane);
        begin = s.head * head_line + w.begin;
        n_tiles = w.end - w.begin - kItemCost;
        const int here = cut(k);
        if (here <= 0 || here >= n_tiles || cut(k - 1) > 0 || !block_rows(p, w.b, w.i, &s)) s.nrows = 0;
        while (last + 1 < p.ctas && cut(last + 1) < n_tiles) ++last;
    }
    grid_dependency_wait();
    allow_dependent_launch();
    if (s.nrows == 0) return;
    const int bad = first_bad(p)[s.seq];
#pragma unroll 1
    for (int batch = 0; batch < kBatches; ++batch) {
        const int row0 = kCombineRows * (kBatches * blockIdx.y + batch) + kRowsPerWarp * warp;
        if (row0 >= s.nrows) return;
        // all rows' loads of a part are in flight together (rows behind the last are within the slot)
        auto part = [&](int c) { return part_slot(p, c, c == k - 1); };
        auto stats = [&](int c, int i) { return reinterpret_cast<const float2*>(part(c) + kBlockRows * 128)[row0 + i]; };
        float M[kRowsPerWarp], L[kRowsPerWarp];
        float4 sum[kRowsPerWarp];
#pragma unroll
        for (int i = 0; i < kRowsPerWarp; ++i) {
            M[i] = -INFINITY;
            L[i] = 0.f;
            sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 2
        for (int c = k - 1; c <= last; ++c)
#pragma unroll
            for (int i = 0; i < kRowsPerWarp; ++i) M[i] = fmaxf(M[i], stats(c, i).x);
#pragma unroll 2
        for (int c = k - 1; c <= last; ++c) {
#pragma unroll
            for (int i = 0; i < kRowsPerWarp; ++i) {
                const float2 ml = stats(c, i);
                const float4 o = reinterpret_cast<const float4*>(part(c) + (row0 + i) * 128)[lane];
                // (no score above -inf: no weight, unless a NaN is among them; its O may never have been written)
                const float w = ml.x > -INFINITY ? exp2f(ml.x - M[i]) : ml.y == 0.f ? 0.f : NAN;
                L[i] += ml.y * w;
                sum[i].x += w == 0.f ? 0.f : w * o.x;
                sum[i].y += w == 0.f ? 0.f : w * o.y;
                sum[i].z += w == 0.f ? 0.f : w * o.z;
                sum[i].w += w == 0.f ? 0.f : w * o.w;
            }
        }
#pragma unroll
        for (int i = 0; i < kRowsPerWarp; ++i) {
            if (row0 + i >= s.nrows) break;
            if (bad <= s.pos0 + row0 + i) L[i] = NAN;
            const float inv = L[i] == 0.f ? 0.f : 1.f / L[i];
            const int64_t at = (int64_t)(s.row0 + row0 + i) * p.heads + s.head;
            reinterpret_cast<uint2*>(p.out + at * 128)[lane] =
                make_uint2(f2_to_bf2(sum[i].x * inv, sum[i].y * inv), f2_to_bf2(sum[i].z * inv, sum[i].w * inv));
            if (lane == 0 && p.lse) p.lse[at] = L[i] == 0.f ? -INFINITY : (M[i] + log2f(L[i])) * kLn2;
        }
    }
}

}  // namespace

cudaError_t launch_expand(const ExpandLaunch& L, cudaStream_t stream) {
    const ExpandParams& p = L.params;
    if (p.total_q <= 0) return cudaSuccess;
    auto keys = p.kv_fp8 ? keys_kernel<true> : keys_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(keys, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttendSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // (FP8 rows: the weights are converted by the same blocks, many heads' also where there are few rows: 100 tokens of 128
    // heads took 172 us with a block for each 16 rows alone)
    const int64_t weights = p.kv_fp8 ? (int64_t)p.heads * (256 / kGainRows) : 0, blocks = 8 * L.num_sms;
    const int64_t gathered = std::max(weights, (int64_t)kGatherUnits * p.cap_tiles);
    cfg.gridDim = dim3((unsigned)std::min(gathered, blocks));
    cfg.blockDim = dim3(kGatherThreads);
    if ((e = cudaLaunchKernelEx(&cfg, gather_kernel, p)) != cudaSuccess) return e;
    const int64_t units = (int64_t)((p.cap_tiles + 1) / 2) * p.heads;
    const int pairs = L.num_sms / 2;
    cfg.gridDim = dim3((unsigned)(2 * (units < pairs ? units : pairs)));
    cfg.blockDim = dim3(kKeysThreads);
    cfg.dynamicSmemBytes = kKeysSmem;
    if ((e = cudaLaunchKernelEx(&cfg, keys, L.cmap, L.wmap, p)) != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)p.ctas);
    cfg.blockDim = dim3(kAttendThreads);
    cfg.dynamicSmemBytes = kAttendSmem;
    if ((e = cudaLaunchKernelEx(&cfg, attend_kernel, L.nopemap, L.pemap, p)) != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)p.ctas, kBlockRows / (kBatches * kCombineRows));
    cfg.blockDim = dim3(32 * kCombineWarps);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, combine_kernel, p);
}

}  // namespace dsa
