// Causal attention of prompts with keys and values of every head, made of the paged latent rows (latent attention in its
// expanded form; the absorbed form is prefix.cu's and sfa_impl.cuh's: "Optimizing Inference for Hybrid Attention
// Architectures: From Operator Fusion to Sequence Sharding", section "Breaking Down the Computational Path of Hybrid
// Attention", step 2, without the selection).
//
// With c_s the latent part and r_s the rotary part of position s, and head h's weights wk, wv (128 x 512 each):
//   k[s, h] = [wk c_s | r_s] (192 dims),  v[s, h] = wv c_s (128 dims),
//   z_s = scale * q[t, h] . k[s, h] for s = 0..p_t,  out[t, h] = softmax(z) . v,  lse[t, h] = logsumexp(z).
// A (query, position, head) takes 2 (192 + 128) operations where the absorbed form takes 2 (576 + 512), and a (position,
// head) 2 x 256 x 512 for its keys and values, so this is the form for many queries a sequence.  Keys and values are
// rounded to bf16, as a projection would leave them.
//
// Four kernels, chained by programmatic launches:
//   plan:    where each sequence's positions lie (tiles of 128, a sequence's own) and the list of blocks of 256 queries;
//   gather:  the pages' rows as tiles of nine 16 KB pieces (64 dims of 128 positions, FP8 rows as bf16; zeros behind the
//            last position), the layout that the tensor cores read (128-byte swizzle);
//   keys:    K and V = W c: a matrix product of all tiles and heads, CTA pairs (256 positions x a head's 256 rows);
//   attend:  a CTA takes 256 queries of a head as two tiles of 128 that share K and V.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

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

// What the plan kernel leaves, at the start of the plan area (int32), tile_begin [batch + 1], first_bad [batch], then
// blocks, an int2 each.
struct PlanHead {
    int32_t tiles;    // in use
    int32_t blocks;   // in the list
    int32_t counter;  // work items handed out
    int32_t unused;
};
__device__ __forceinline__ PlanHead* plan_head(const ExpandParams& p) { return reinterpret_cast<PlanHead*>(p.plan); }
__device__ __forceinline__ int32_t* tile_begin(const ExpandParams& p) { return p.plan + 4; }
// First position of a sequence that has no finite values or no page (INT32_MAX: none): rows that see it are NaN.
__device__ __forceinline__ int32_t* first_bad(const ExpandParams& p) { return p.plan + 4 + p.batch + 1; }
__device__ __forceinline__ int2* blocks(const ExpandParams& p) { return reinterpret_cast<int2*>(p.plan + expand_plan_ints(p.batch)); }

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

// ---------------------------------------------------------------------------------------------------------
// plan: one block.  Every thread counts a run of sequences; a scan of the threads' sums numbers tiles and blocks.
// ---------------------------------------------------------------------------------------------------------
constexpr int kPlanThreads = 512;

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

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const ExpandParams p) {
    __shared__ long long scan[2][kPlanThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dependency_wait();
    allow_dependent_launch();
    const int run = (p.batch + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(p.batch, tid * run), b1 = min(p.batch, b0 + run);
    long long tiles = 0, count = 0;
    for (int b = b0; b < b1; ++b) {
        int c0, n, L;
        if (!sequence(p, b, &c0, &n, &L)) {
            raise_error(p.err, DSA_DEVERR_SEQ);
            continue;
        }
        if (n > 0) {
            tiles += (L + 127) / 128;
            count += (n + kBlockRows - 1) / kBlockRows;
        }
    }
    long long ti = tiles, ci = count;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long to = __shfl_up_sync(kAllLanes, ti, off), co = __shfl_up_sync(kAllLanes, ci, off);
        if (lane >= off) {
            ti += to;
            ci += co;
        }
    }
    if (lane == 31) {
        scan[0][warp] = ti;
        scan[1][warp] = ci;
    }
    __syncthreads();
    long long at = ti - tiles, block = ci - count, all_tiles = 0, all_blocks = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) {
            at += scan[0][w];
            block += scan[1][w];
        }
        all_tiles += scan[0][w];
        all_blocks += scan[1][w];
    }
    for (int b = b0; b < b1; ++b) {
        int c0, n, L;
        const bool ok = sequence(p, b, &c0, &n, &L) && n > 0;
        const int mine = ok ? (L + 127) / 128 : 0, parts = ok ? (n + kBlockRows - 1) / kBlockRows : 0;
        // (more pages than were announced, or offsets that run backwards: left out)
        const bool fits = at + mine <= p.cap_tiles && block + parts <= p.cap_blocks;
        if (ok && !fits) raise_error(p.err, DSA_DEVERR_SEQ);
        tile_begin(p)[b] = (int32_t)(at < p.cap_tiles ? at : p.cap_tiles);
        first_bad(p)[b] = INT32_MAX;
        for (int i = 0; i < parts && block + i < p.cap_blocks; ++i)
            blocks(p)[block + i] = make_int2(fits ? b : -1, i * kBlockRows);
        at += mine;
        block += parts;
    }
    if (tid == 0) {
        PlanHead h;
        h.tiles = (int32_t)(all_tiles < p.cap_tiles ? all_tiles : p.cap_tiles);
        h.blocks = (int32_t)(all_blocks < p.cap_blocks ? all_blocks : p.cap_blocks);
        h.counter = 0;
        h.unused = 0;
        *plan_head(p) = h;
        tile_begin(p)[p.batch] = h.tiles;
        if (p.cu_q_lens[0] != 0 || p.cu_q_lens[p.batch] != p.total_q) raise_error(p.err, DSA_DEVERR_SEQ);
    }
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

// ---------------------------------------------------------------------------------------------------------
// gather: a block per half tile (64 positions, one page), a warp per position.  Bound by HBM and L2: 1152 or 656 bytes
// read, 1152 written a position.
// ---------------------------------------------------------------------------------------------------------
constexpr int kGatherWarps = 8;

__global__ void __launch_bounds__(32 * kGatherWarps) gather_kernel(const ExpandParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    allow_dependent_launch();
    const int halves = 2 * plan_head(p)->tiles;
    for (int i = blockIdx.x; i < halves; i += gridDim.x) {
        const int tile = i >> 1, b = sequence_of_tile(p, tile), base = 128 * (tile - tile_begin(p)[b]) + 64 * (i & 1);
        const int L = p.seq_lens[b];
        const int pg = base < L ? p.page_table[(int64_t)b * p.max_pages + (base >> 6)] : 0;
        const bool in = pg >= 0 && pg < p.num_pages;
        if (!in && threadIdx.x == 0) {
            raise_error(p.err, DSA_DEVERR_PAGE);
            atomicMin(first_bad(p) + b, base);
        }
        uint8_t* dst = p.latents + (int64_t)tile * kTileBytes;
#pragma unroll 2
        for (int j = warp; j < 64; j += kGatherWarps) {
            const int row = 64 * (i & 1) + j;
            const bool have = in && base + j < L;
            auto put = [&](int chunk, uint4 v) {  // 16-byte chunk of the row's 72
                *reinterpret_cast<uint4*>(dst + (chunk >> 3) * kUnit + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)) = v;
            };
            const uint4 zero = make_uint4(0, 0, 0, 0);
            if (!p.kv_fp8) {
                const uint4* src = reinterpret_cast<const uint4*>(p.kv_cache + ((int64_t)pg * 64 + j) * 1152);
                uint4 v[3];
#pragma unroll
                for (int k = 0; k < 3; ++k) v[k] = have && lane + 32 * k < 72 ? src[lane + 32 * k] : zero;
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (lane + 32 * k < 72) put(lane + 32 * k, v[k]);
            } else {
                const uint8_t* src = p.kv_cache + ((int64_t)pg * 64 + j) * kKvFp8RowBytes;
                const uint4 code = have ? reinterpret_cast<const uint4*>(src)[lane] : zero;
                const float scale = have ? reinterpret_cast<const float*>(src + kKvFp8ScaleOff)[lane >> 3] : 0.f;
                const uint4 rot = have && lane < 8 ? reinterpret_cast<const uint4*>(src + kKvFp8RopeOff)[lane] : zero;
                put(2 * lane, e4m3x8_to_bf16x8(make_uint2(code.x, code.y), scale));
                put(2 * lane + 1, e4m3x8_to_bf16x8(make_uint2(code.z, code.w), scale));
                if (lane < 8) put(64 + lane, rot);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------------------
// keys: D (256 positions x 256) = c W[h]^T for each pair of tiles and each head, cta_group::2: CTA c of the pair holds
// tile 2 i + c and rows 128 c .. of the head's weights (c = 0: keys, 1: values), both in chunks of 64 inner dims; its
// tensor memory receives its tile's keys and values.
// ---------------------------------------------------------------------------------------------------------
constexpr int kKeysThreads = 256;  // warp 0: TMA, 1: products, 2: tensor memory, 4-7: results
constexpr int kKeysResultWarp = 4;
constexpr int kKeysStages = 6;
constexpr int kPiece = 32 * 128;  // 32 positions x 64 dims
constexpr uint32_t kIdescKeys = make_idesc(256, 256, 1, 1, 0, 0);

struct KeysCtrl {
    uint64_t full[kKeysStages], empty[kKeysStages];
    uint64_t d_full[2], d_empty[2];
    uint64_t drained;
    uint32_t tmem_base;
    int32_t failed;
};
constexpr int kKeysSmem = 1024 + kKeysStages * 2 * kUnit + 4 * 2 * kPiece + (int)sizeof(KeysCtrl);
static_assert(kKeysSmem <= 232448, "shared memory of one CTA");

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
    const int64_t units = (int64_t)((tiles + 1) / 2) * p.heads;
    const int64_t u0 = units * pair / pairs, u1 = units * (pair + 1) / pairs;  // unit: tiles u / heads, head u % heads
    auto leader = [&](uint64_t* bar) { return mapa_shared(smem_u32(bar), 0); };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(kAllLanes, mbar_wait(bar, parity, p.err, p.wait_ns)) != 0;
    };
    bool ok = true;

    if (warp == 0) {
        const uint32_t full = leader(&ctl->full[0]);
        uint32_t n = 0;
        for (int64_t u = u0; ok && u < u1; ++u) {
            const int tile = 2 * (int)(u / p.heads) + rank, head = (int)(u % p.heads);
#pragma unroll 1
            for (int k = 0; k < 8; ++k, ++n) {
                const uint32_t slot = n % kKeysStages;
                if (!(ok = wait(&ctl->empty[slot], ((n / kKeysStages) & 1u) ^ 1u))) break;
                if (elect_one_sync()) {
                    uint8_t* dst = smem + slot * 2 * kUnit;
                    if (rank == 0) mbar_arrive_expect_tx(&ctl->full[slot], 4 * kUnit);
                    // (the tile behind the last one, where their number is odd, has its place but no rows of its own)
                    tma_pair_load_3d(dst, &cmap, full + 8 * slot, 0, 0, 9 * tile + k);
                    tma_pair_load_3d(dst + kUnit, &wmap, full + 8 * slot, 64 * k, 128 * rank, head);
                }
            }
        }
    } else if (warp == 1 && rank == 0) {
        const uint64_t ad = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
        uint32_t n = 0, t = 0;
        for (int64_t u = u0; ok && u < u1; ++u, ++t) {
            const uint32_t buf = t & 1u;
            if (!(ok = wait(&ctl->d_empty[buf], ((t >> 1) & 1u) ^ 1u))) break;
#pragma unroll 1
            for (int k = 0; k < 8; ++k, ++n) {
                const uint32_t slot = n % kKeysStages;
                if (!(ok = wait(&ctl->full[slot], (n / kKeysStages) & 1u))) break;
                tc_fence_after();
                if (elect_one_sync()) {
                    const uint64_t a = ad + (uint64_t)(slot * (2 * kUnit / 16));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma_pair_f16_ss(tmem + 256 * buf, a + (uint64_t)(2 * j), a + (uint64_t)(kUnit / 16 + 2 * j),
                                         kIdescKeys, k == 0 && j == 0 ? 0u : 1u);
                    umma_pair_commit(&ctl->empty[slot], 3);
                    if (k == 7) umma_pair_commit(&ctl->d_full[buf], 3);
                }
            }
        }
        // drain (default limit): every product of the pair is done before its memory is given back
        if (elect_one_sync()) {
            umma_pair_commit(&ctl->drained, 1);
            mbar_wait(&ctl->drained, 0, p.err);
        }
        __syncwarp();
    } else if (warp >= kKeysResultWarp) {
        // warp w has positions 32 w .. of its CTA's tile, a lane each: keys in columns 0-127, values behind them
        const int ew = warp - kKeysResultWarp;
        const uint32_t trow = tmem + ((uint32_t)(32 * ew) << 16);
        const uint32_t d_empty = leader(&ctl->d_empty[0]);
        uint8_t* stage = o_s + ew * 2 * kPiece;
        uint32_t t = 0;
        for (int64_t u = u0; ok && u < u1; ++u, ++t) {
            const int tile = 2 * (int)(u / p.heads) + rank, head = (int)(u % p.heads);
            const uint32_t buf = t & 1u;
            if (!(ok = wait(&ctl->d_full[buf], (t >> 1) & 1u))) break;
            tc_fence_after();
            uint8_t* dst = p.kv + ((int64_t)tile * p.heads + head) * kHeadTile;
            bool finite = true;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {  // 64 columns each
                float v[4][16];
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld16(trow + 256 * buf + 64 * c + 16 * k, v[k]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_regs_ready(v[k]);
                if (c == 3) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(d_empty + 8 * buf);
                }
                uint4 w[8];
                uint32_t odd = 0;  // an exponent of all ones carries into the sign bit's place
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float* f = &v[k >> 1][8 * (k & 1)];
                    w[k] = make_uint4(f2_to_bf2(f[0], f[1]), f2_to_bf2(f[2], f[3]), f2_to_bf2(f[4], f[5]), f2_to_bf2(f[6], f[7]));
                    const uint32_t e = 0x7F807F80u, one = 0x00800080u;
                    odd |= ((w[k].x & e) + one) | ((w[k].y & e) + one) | ((w[k].z & e) + one) | ((w[k].w & e) + one);
                }
                // a weight of 0 times a value that is not finite is NaN, for rows that do not see the position too: its
                // values become 0, and the rows that do see it NaN at the end
                if (c >= 2 && (odd & 0x80008000u) != 0) {
                    finite = false;
#pragma unroll
                    for (int k = 0; k < 8; ++k) w[k] = make_uint4(0, 0, 0, 0);
                }
                uint8_t* at = stage + (c & 1) * kPiece;
                if (lane == 0) bulk_wait_read<1>();
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) st_shared_v4(smem_u32(at) + lane * 128 + ((k ^ (lane & 7)) << 4), w[k]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    // keys: unit c, positions in rows of 128 bytes; values: unit 2 + position / 64, of it dims 64 (c - 2) ..
                    uint8_t* to = c < 2 ? dst + c * kUnit + ew * kPiece
                                        : dst + (2 + (ew >> 1)) * kUnit + (c - 2) * (kUnit / 2) + (ew & 1) * kPiece;
                    if (tile < tiles) bulk_copy_s2g(to, at, kPiece);
                    bulk_commit();
                }
            }
            if (!finite && tile < tiles) {
                const int b = sequence_of_tile(p, tile);
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
// attend
// ---------------------------------------------------------------------------------------------------------
constexpr int kAttendThreads = 320;  // warps 0-3 and 4-7: softmax of the two query tiles, 8: loads, 9: products
constexpr int kLoadWarp = 8;
constexpr int kProductWarp = 9;
constexpr int kRing = 8;             // units of K and V, in turn K K K V V
constexpr int kQTile = 3 * kUnit;    // 128 queries x 192 dims
constexpr int kTileUnits = 5;
constexpr int kOCol = 256;           // tensor memory: S (and P in its first half) at 0 and 128, O at 256 and 384
constexpr uint32_t kIdescQK = make_idesc(128, 128, 1, 1, 0, 0);
constexpr uint32_t kIdescPV = make_idesc(128, 128, 1, 1, 0, 1);
constexpr float kRaise = 8.f;  // the running maximum (log2) is raised only when it grows by more than this

struct AttendItem {
    int32_t row0, nrows;  // query tokens (none: no more items)
    int32_t head, seq;
    int32_t pos0;         // position of the first
    int32_t tile0;        // first tile of the sequence's keys
    int32_t n0, n1;       // tiles that queries 0-127, 128-255 see
};
struct AttendCtrl {
    uint64_t q_full[2], q_empty[2];
    uint64_t full[kRing], empty[kRing];
    uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
    uint64_t item_full[2], item_empty[2];
    uint64_t drained;
    uint32_t tmem_base;
    int32_t failed;
    AttendItem items[2];
};
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
            mbar_init(&ctl->item_full[i], 1);
            mbar_init(&ctl->item_empty[i], 9);  // the softmax warps and the products'
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
    // item number n of this CTA, once it is there; false: gave up
    auto next_item = [&](uint32_t n, AttendItem* it) {
        if (!wait(&ctl->item_full[n & 1u], (n >> 1) & 1u)) return false;
        *it = ctl->items[n & 1u];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->item_empty[n & 1u]);
        return true;
    };
    bool ok = true;

    if (warp == kLoadWarp) {
        // ---------------- items, and what each needs in the order of its use ----------------
        const int n_blocks = plan_head(p)->blocks;
        const int64_t n_items = (int64_t)n_blocks * p.heads;
        uint32_t n = 0, u = 0, used[2] = {0, 0};  // items, units, items that used each query tile
        while (ok) {
            // heads one after another, so that a head's keys stay in L2 for its blocks; the last blocks (the most keys) first
            AttendItem it;
            it.nrows = 0;
            int index = 0;
            if (lane == 0) index = atomicAdd(&plan_head(p)->counter, 1);
            index = __shfl_sync(kAllLanes, index, 0);
            if (index < n_items) {
                const int2 blk = blocks(p)[n_blocks - 1 - index % n_blocks];
                if (blk.x < 0) continue;
                const int c0 = p.cu_q_lens[blk.x], nq = p.cu_q_lens[blk.x + 1] - c0;
                it.head = index / n_blocks;
                it.seq = blk.x;
                it.row0 = c0 + blk.y;
                it.nrows = min(kBlockRows, nq - blk.y);
                it.pos0 = p.seq_lens[blk.x] - nq + blk.y;
                it.tile0 = tile_begin(p)[blk.x];
                it.n0 = (it.pos0 + min(it.nrows, 128) + 127) / 128;
                it.n1 = it.nrows > 128 ? (it.pos0 + it.nrows + 127) / 128 : 0;
            }
            if (!(ok = wait(&ctl->item_empty[n & 1u], ((n >> 1) & 1u) ^ 1u))) break;
            if (lane == 0) {
                ctl->items[n & 1u] = it;
                mbar_arrive(&ctl->item_full[n & 1u]);
            }
            __syncwarp();
            ++n;
            if (it.nrows == 0) break;
            const uint8_t* kv = p.kv + ((int64_t)it.tile0 * p.heads + it.head) * kHeadTile;
            const uint8_t* rotary = p.latents + (int64_t)it.tile0 * kTileBytes + 8 * kUnit;
            const int tiles = max(it.n0, it.n1);
            auto load_q = [&](int w) {
                if (!wait(&ctl->q_empty[w], (used[w] & 1u) ^ 1u)) return false;
                ++used[w];
                if (elect_one_sync()) {
                    mbar_arrive_expect_tx(&ctl->q_full[w], kQTile);
                    uint8_t* dst = smem + w * kQTile;
                    tma_load_3d(dst, &nopemap, &ctl->q_full[w], 0, it.head, it.row0 + 128 * w);
                    tma_load_3d(dst + kUnit, &nopemap, &ctl->q_full[w], 64, it.head, it.row0 + 128 * w);
                    tma_load_3d(dst + 2 * kUnit, &pemap, &ctl->q_full[w], 0, it.head, it.row0 + 128 * w);
                }
                return true;
            };
            if (!(ok = load_q(0))) break;
            for (int j = 0; ok && j < tiles; ++j) {
                const uint8_t* tile = kv + (int64_t)j * p.heads * kHeadTile;
#pragma unroll 1
                for (int k = 0; k < kTileUnits; ++k, ++u) {
                    const uint32_t slot = u % kRing;
                    if (!(ok = wait(&ctl->empty[slot], ((u / kRing) & 1u) ^ 1u))) break;
                    if (elect_one_sync()) {
                        const uint8_t* src = k == 2 ? rotary + (int64_t)j * kTileBytes : tile + (k < 2 ? k : k - 1) * kUnit;
                        mbar_arrive_expect_tx(&ctl->full[slot], kUnit);
                        bulk_copy_g2s(ring + slot * kUnit, src, kUnit, &ctl->full[slot]);
                    }
                    if (j == 0 && k == 2 && it.n1 > 0 && !(ok = load_q(1))) break;
                }
            }
        }
    } else if (warp == kProductWarp) {
        // ---------------- S_w(j) = Q_w K(j)^T and O_w += P_w(j) V(j), the two query tiles in turn ----------------
        const uint64_t qd = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
        const uint64_t kd = smem_desc(smem_u32(ring), 16, 1024, kSwizzle128B);
        const uint64_t vd = smem_desc(smem_u32(ring), kUnit / 2, 1024, kSwizzle128B);  // MN-major, dims 64.. half a unit on
        uint32_t u = 0, used[2] = {0, 0}, tiles_done[2] = {0, 0};
        for (uint32_t n = 0; ok; ++n) {
            AttendItem it;
            if (!(ok = next_item(n, &it)) || it.nrows == 0) break;
            const int tiles = max(it.n0, it.n1);
            auto count = [&](int w) { return w == 0 ? it.n0 : it.n1; };
            // the ring's unit k of tile j (K: 0-2, V: 3, 4)
            auto qk = [&](int w, int j) {
                if (j >= count(w)) return true;
                if (j == 0 && !wait(&ctl->q_full[w], used[w] & 1u)) return false;
                const bool other = w == 0 && j < it.n1;  // the other query tile reads these keys, too
#pragma unroll 1
                for (int k = 0; k < 3; ++k) {
                    const uint32_t at = u + kTileUnits * j + k, slot = at % kRing;
                    if (!wait(&ctl->full[slot], (at / kRing) & 1u)) return false;
                    tc_fence_after();
                    if (elect_one_sync()) {
                        const uint64_t a = qd + (uint64_t)((w * kQTile + k * kUnit) / 16), b = kd + (uint64_t)(slot * (kUnit / 16));
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16_ss(tmem + 128 * w, a + (uint64_t)(2 * kk), b + (uint64_t)(2 * kk), kIdescQK,
                                        k == 0 && kk == 0 ? 0u : 1u);
                        if (!other) umma_commit(&ctl->empty[slot]);
                        if (k == 2) {
                            umma_commit(&ctl->s_full[w]);
                            if (j == count(w) - 1) umma_commit(&ctl->q_empty[w]);
                        }
                    }
                }
                return true;
            };
            auto pv = [&](int w, int j) {
                if (j >= count(w)) return true;
                if (!wait(&ctl->p_full[w], tiles_done[w] & 1u)) return false;
                ++tiles_done[w];
                if (j == 0 && !wait(&ctl->o_free[w], (used[w] & 1u) ^ 1u)) return false;
                const bool other = w == 0 && j < it.n1, last = j == count(w) - 1;
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    const uint32_t at = u + kTileUnits * j + 3 + k, slot = at % kRing;
                    if (!wait(&ctl->full[slot], (at / kRing) & 1u)) return false;
                    tc_fence_after();
                    if (elect_one_sync()) {
                        const uint64_t b = vd + (uint64_t)(slot * (kUnit / 16));
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16_ts(tmem + kOCol + 128 * w, tmem + 128 * w + 32 * k + 8 * kk, b + (uint64_t)(128 * kk),
                                        kIdescPV, j == 0 && k == 0 && kk == 0 ? 0u : 1u);
                        if (!other) umma_commit(&ctl->empty[slot]);
                        if (k == 1 && last) umma_commit(&ctl->o_full[w]);
                    }
                }
                return true;
            };
            ok = qk(0, 0) && qk(1, 0);
            for (int j = 0; ok && j < tiles; ++j) ok = pv(0, j) && qk(0, j + 1) && pv(1, j) && qk(1, j + 1);
            u += kTileUnits * tiles;
            ++used[0];
            if (it.n1 > 0) ++used[1];
        }
        // drain (default limit): every product is done before its memory is given back
        if (elect_one_sync()) {
            umma_commit(&ctl->drained);
            mbar_wait(&ctl->drained, 0, p.err);
        }
        __syncwarp();
    } else {
        // ---------------- softmax: a thread has a query of its warp group's tile ----------------
        const int w = warp >> 2, r = tid & 127;
        const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t scol = trow + 128 * w, ocol = trow + kOCol + 128 * w;
        uint32_t tile = 0, used = 0;
        for (uint32_t n = 0; ok; ++n) {
            AttendItem it;
            if (!(ok = next_item(n, &it)) || it.nrows == 0) break;
            const int tiles = w == 0 ? it.n0 : it.n1;
            if (tiles == 0) continue;
            const int first = it.pos0 + 128 * w, limit = first + r + 1;  // positions this query sees: below `limit`
            float m_used = -INFINITY, l_sum = 0.f;
#pragma unroll 1
            for (int j = 0; j < tiles; ++j, ++tile) {
                if (!(ok = wait(&ctl->s_full[w], tile & 1u))) break;
                tc_fence_after();
                float s[8][16];
#pragma unroll
                for (int k = 0; k < 8; ++k) tmem_ld16(scol + 16 * k, s[k]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 8; ++k) tmem_regs_ready(s[k]);
                if (128 * j + 128 > first + 1) {  // some query does not see all of it
                    const int seen = limit - 128 * j;
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
                const bool raise = mt > m_used + kRaise;
                const float m_new = raise ? mt : m_used;
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
                // weights: the sum takes the fp32 values, the products their rounding to bf16 (at most 2^-8 of each, unbiased)
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
                        packed[i / 2] = f2_to_bf2(e.x, e.y);
                        sum[(i / 2) & 3] = add2(sum[(i / 2) & 3], e);
                    }
                    tmem_st16_u32(scol + 8 * k, packed);
                }
                const float2 half = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                l_sum = l_sum * alpha + (half.x + half.y);
                m_used = m_new;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->p_full[w]);
            }
            if (!ok) break;
            // ---- the result ----
            if (!(ok = wait(&ctl->o_full[w], used & 1u))) break;
            ++used;
            tc_fence_after();
            if (*const_cast<volatile int32_t*>(first_bad(p) + it.seq) < limit) l_sum = NAN;
            const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
            const int row = 128 * w + r;
            const int64_t at = (int64_t)(it.row0 + row) * p.heads + it.head;
            uint4* dst = reinterpret_cast<uint4*>(p.out + at * 128);
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                float o[2][16];
                tmem_ld16(ocol + c, o[0]);
                tmem_ld16(ocol + c + 16, o[1]);
                tmem_ld_wait();
                tmem_regs_ready(o[0]);
                tmem_regs_ready(o[1]);
                if (row < it.nrows) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float* f = &o[k >> 1][8 * (k & 1)];
                        dst[c / 8 + k] = make_uint4(f2_to_bf2(f[0] * inv, f[1] * inv), f2_to_bf2(f[2] * inv, f[3] * inv),
                                                    f2_to_bf2(f[4] * inv, f[5] * inv), f2_to_bf2(f[6] * inv, f[7] * inv));
                    }
                }
            }
            if (row < it.nrows && p.lse) p.lse[at] = l_sum == 0.f ? -INFINITY : (m_used + log2f(l_sum)) * kLn2;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->o_free[w]);
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

}  // namespace

cudaError_t launch_expand(const ExpandLaunch& L, cudaStream_t stream) {
    const ExpandParams& p = L.params;
    if (p.total_q <= 0) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(keys_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttendSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    if ((e = cudaLaunchKernelEx(&cfg, plan_kernel, p)) != cudaSuccess) return e;
    const int64_t halves = 2 * (int64_t)p.cap_tiles;
    cfg.gridDim = dim3((unsigned)(halves < 8 * L.num_sms ? halves : 8 * L.num_sms));
    cfg.blockDim = dim3(32 * kGatherWarps);
    if ((e = cudaLaunchKernelEx(&cfg, gather_kernel, p)) != cudaSuccess) return e;
    const int64_t units = (int64_t)((p.cap_tiles + 1) / 2) * p.heads;
    const int pairs = L.num_sms / 2;
    cfg.gridDim = dim3((unsigned)(2 * (units < pairs ? units : pairs)));
    cfg.blockDim = dim3(kKeysThreads);
    cfg.dynamicSmemBytes = kKeysSmem;
    if ((e = cudaLaunchKernelEx(&cfg, keys_kernel, L.cmap, L.wmap, p)) != cudaSuccess) return e;
    const int64_t items = (int64_t)p.cap_blocks * p.heads;
    cfg.gridDim = dim3((unsigned)(items < L.num_sms ? items : L.num_sms));
    cfg.blockDim = dim3(kAttendThreads);
    cfg.dynamicSmemBytes = kAttendSmem;
    return cudaLaunchKernelEx(&cfg, attend_kernel, L.nopemap, L.pemap, p);
}

}  // namespace dsa
