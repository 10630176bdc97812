// Products of every head with its own weights, around attention over latent rows (latent attention in its absorbed form:
// "Optimizing Inference for Hybrid Attention Architectures: From Operator Fusion to Sequence Sharding", section "Breaking
// Down the Computational Path of Hybrid Attention"; the queries and outputs of its step 2 live in the latent space):
//   absorb:  q[t, h, 0:512] = sum_d q_nope[t, h, d] wk[h, d, :]     (a head's key weights, 128 x 512)
//   values:  out[t, h, :]   = sum_c o[t, h, c] wv[h, :, c]          (a head's value weights, 128 x 512)
// Products of bf16 are exact in fp32 and summed in fp32; the sum is rounded once, to the bf16 that attention and the next
// projection take.
//
// Work.  A unit is 128 tokens by one slab of weights: absorb 128 x 256 (half of a head's latent dims), values 512 x 128.
// Units are numbered tokens by tokens, all slabs of 128 tokens and then the next, and CTAs take every grid-th, so that at any
// time all of them are at the same rows: their reads and writes are whole rows of all heads (slab by slab, with the slab
// kept in shared memory, 4096 tokens of 128 heads took 156 us and 139 so; 2111 tokens' values 63 and 58).
// A unit's inner dims go in chunks of 64, token rows (by TMA from the caller's strides; rows behind the last token are
// zeros) and weights together, through a ring of stages; one thread fills it, one issues the products.  The accumulator
// in tensor memory is double: four warps round a unit to bf16 and store it by TMA (32 tokens x 64 dims at a time, clipped at
// the last token) while the next one is multiplied.
//
// What bounds it: HBM.  Absorb writes 1024 bytes for 256 read, and writes alone run at 4.0 TB/s here (filling memory), 134 us for
// the 537 MB of 4096 tokens of 128 heads.  These take 141 us, and read 248 MB where 151 are needed: 211 with dense rows (some
// of a head's token rows come again for its second slab), 37 more where rows are 384 bytes apart (probably what fetches of 256 bytes
// take along of their neighbours).  Values reads four times what it writes: 2111 tokens of 128 heads 58 us for 363 MB, 6.3 TB/s, 0.92 of
// the copy bandwidth.  Few tokens: each head's weights once, and latency; 32 tokens of 128 heads 6.2 us (L2 flushed
// before each call 13.5 to 15.5), 130 tokens of 16 heads 4.8 (11.4).
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr uint32_t kAllLanes = 0xFFFFFFFFu;
constexpr int kTokens = 128;           // of a unit
constexpr int kChunk = kTokens * 128;  // 64 dims of its tokens
constexpr int kPiece = 32 * 128;       // what a warp stores at a time
constexpr int kPieces = 2;             // of them in flight
constexpr int kThreads = 256;          // warp 0: TMA, 1: products, 2: tensor memory, 4-7: results
constexpr int kResultWarp = 4;

template <bool VALUES>
struct Form {
    static constexpr int kN = VALUES ? 128 : 256;   // output dims of a unit
    static constexpr int kChunks = VALUES ? 8 : 2;  // of 64 inner dims
    static constexpr int kStage = kChunk + kN * 128;
    static constexpr int kStages = VALUES ? 6 : 4;
    static constexpr int kSlabs = VALUES ? 1 : 2;   // of a head
    // weights as [inner][n] (absorb: MN-major) or [n][inner] (values)
    static constexpr uint32_t kIdesc = make_idesc(kTokens, kN, 1, 1, 0, VALUES ? 0 : 1);
};

struct Ctrl {
    uint64_t full[6], empty[6];
    uint64_t d_full[2], d_empty[2];
    uint64_t drained;
    uint32_t tmem_base;
    int32_t failed;
};
template <bool VALUES>
constexpr int kSmem = 1024 + Form<VALUES>::kStages * Form<VALUES>::kStage + 4 * kPieces * kPiece + (int)sizeof(Ctrl);
static_assert(kSmem<true> <= 232448 && kSmem<false> <= 232448, "shared memory of one CTA");

// Unit u: its first token, head and first output dim.
struct Unit {
    int token, head, col;
};
template <bool VALUES>
__device__ __forceinline__ Unit unit_of(const HeadsParams& p, int64_t u) {
    const int slabs = p.heads * Form<VALUES>::kSlabs, tile = (int)(u / slabs), slab = (int)(u - (int64_t)tile * slabs);
    return {kTokens * tile, slab / Form<VALUES>::kSlabs, Form<VALUES>::kN * (slab % Form<VALUES>::kSlabs)};
}

template <bool VALUES>
__global__ void __launch_bounds__(kThreads, 1)
    heads_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
                 const __grid_constant__ CUtensorMap omap, const HeadsParams p) {
    using F = Form<VALUES>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* o_s = smem + F::kStages * F::kStage;
    Ctrl* ctl = reinterpret_cast<Ctrl*>(o_s + 4 * kPieces * kPiece);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        prefetch_tensormap(&amap);
        prefetch_tensormap(&wmap);
        prefetch_tensormap(&omap);
        for (int i = 0; i < F::kStages; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->d_full[i], 1);
            mbar_init(&ctl->d_empty[i], 4);
        }
        mbar_init(&ctl->drained, 1);
        ctl->failed = 0;
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_alloc(&ctl->tmem_base, 2 * F::kN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    auto wait_one = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, p.err, p.wait_ns); };
    bool ok = true;

    if (warp == 0) {
        // ---------------- loads ----------------
        if (elect_one_sync()) {
            uint32_t n = 0;
            for (int64_t u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
                const Unit it = unit_of<VALUES>(p, u);
#pragma unroll 1
                for (int k = 0; k < F::kChunks; ++k, ++n) {
                    const uint32_t slot = n % F::kStages;
                    if (!(ok = wait_one(&ctl->empty[slot], ((n / F::kStages) & 1u) ^ 1u))) break;
                    uint8_t* dst = smem + slot * F::kStage;
                    mbar_arrive_expect_tx(&ctl->full[slot], F::kStage);
                    tma_load_3d(dst, &amap, &ctl->full[slot], 64 * k, it.head, it.token);
                    if (VALUES) {
                        tma_load_3d(dst + kChunk, &wmap, &ctl->full[slot], 64 * k, 128, it.head);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            tma_load_3d(dst + kChunk + 64 * 128 * j, &wmap, &ctl->full[slot], it.col + 64 * j, 64 * k, it.head);
                    }
                }
            }
        }
        ok = __all_sync(kAllLanes, ok);
    } else if (warp == 1) {
        // ---------------- products ----------------
        if (elect_one_sync()) {
            const uint64_t ad = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
            const uint64_t wd = smem_desc(smem_u32(smem + kChunk), VALUES ? 16 : 64 * 128, 1024, kSwizzle128B);
            uint32_t n = 0, t = 0;
            for (int64_t u = blockIdx.x; ok && u < p.units; u += gridDim.x, ++t) {
                const uint32_t buf = t & 1u, d = tmem + F::kN * buf;
                if (!(ok = wait_one(&ctl->d_empty[buf], ((t >> 1) & 1u) ^ 1u))) break;
                tc_fence_after();
#pragma unroll 1
                for (int k = 0; k < F::kChunks; ++k, ++n) {
                    const uint32_t slot = n % F::kStages;
                    if (!(ok = wait_one(&ctl->full[slot], (n / F::kStages) & 1u))) break;
                    const uint64_t at = (uint64_t)(slot * (F::kStage / 16));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma_f16_ss(d, ad + at + (uint64_t)(2 * j), wd + at + (uint64_t)((VALUES ? 2 : 128) * j), F::kIdesc,
                                    k == 0 && j == 0 ? 0u : 1u);
                    umma_commit(&ctl->empty[slot]);
                }
                if (ok) umma_commit(&ctl->d_full[buf]);
            }
            // drain (default limit): every product is done before its memory is given back
            umma_commit(&ctl->drained);
            mbar_wait(&ctl->drained, 0, p.err);
        }
        ok = __all_sync(kAllLanes, ok);
    } else if (warp >= kResultWarp) {
        // ---------------- results: warp w has tokens 32 w .. 32 w + 31 of a unit ----------------
        const int ew = warp - kResultWarp;
        const uint32_t trow = tmem + ((uint32_t)(32 * ew) << 16);
        uint8_t* stage = o_s + ew * kPieces * kPiece;
        uint32_t t = 0, piece = 0;
        for (int64_t u = blockIdx.x; ok && u < p.units; u += gridDim.x, ++t) {
            const Unit it = unit_of<VALUES>(p, u);
            const int token = it.token + 32 * ew;
            const uint32_t buf = t & 1u;
            if (!(ok = __all_sync(kAllLanes, wait_one(&ctl->d_full[buf], (t >> 1) & 1u)))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < F::kN; c += 64, ++piece) {
                float v[4][16];
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld16(trow + F::kN * buf + c + 16 * k, v[k]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_regs_ready(v[k]);
                if (c + 64 == F::kN) {  // the last of it is in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->d_empty[buf]);
                }
                uint8_t* at = stage + (piece % kPieces) * kPiece;
                if (lane == 0) bulk_wait_read<kPieces - 1>();  // the store that had this place has read it
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float* f = &v[k >> 1][8 * (k & 1)];
                    st_shared_v4(smem_u32(at) + lane * 128 + ((k ^ (lane & 7)) << 4),
                                 make_uint4(f2_to_bf2(f[0], f[1]), f2_to_bf2(f[2], f[3]), f2_to_bf2(f[4], f[5]),
                                            f2_to_bf2(f[6], f[7])));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (token < p.total_q) tma_store_3d(&omap, at, it.col + c, it.head, token);
                    bulk_commit();
                }
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
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, 2 * F::kN);
}

}  // namespace

cudaError_t launch_heads(const HeadsLaunch& L, cudaStream_t stream) {
    HeadsParams p = L.params;
    if (p.total_q <= 0) return cudaSuccess;
    p.units = ((int64_t)p.total_q + kTokens - 1) / kTokens * p.heads * (p.values ? Form<true>::kSlabs : Form<false>::kSlabs);
    auto kernel = p.values ? heads_kernel<true> : heads_kernel<false>;
    const int smem = p.values ? kSmem<true> : kSmem<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = p.units < L.num_sms ? p.units : L.num_sms;
    kernel<<<dim3((unsigned)grid), dim3(kThreads), smem, stream>>>(L.amap, L.wmap, L.omap, p);
    return cudaGetLastError();
}

}  // namespace dsa
