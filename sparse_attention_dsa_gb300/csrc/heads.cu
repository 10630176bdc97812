// Products of every head with its own weights, around attention over latent rows (latent attention in its absorbed form:
// "Optimizing Inference for Hybrid Attention Architectures: From Operator Fusion to Sequence Sharding", section "Breaking
// Down the Computational Path of Hybrid Attention"; the queries and outputs of its step 2 live in the latent space):
//   absorb:  q[t, h, 0:512] = sum_d q_nope[t, h, d] wk[h, d, :]     (a head's key weights, 128 x 512)
//   values:  out[t, h, :]   = sum_c o[t, h, c] wv[h, :, c]          (a head's value weights, 128 x 512)
// Products of bf16 are exact in fp32 and summed in fp32; the sum is rounded once, to the bf16 that attention and the next
// projection take.
//
// Work.  A unit is 128 tokens by one slab of weights: absorb 128 x 256 (half of a head's latent dims), values 512 x 128.
// Units are numbered slab by slab, and each CTA takes an equal run of them, so that a slab stays in shared memory for all
// the tokens that meet it there.  Both products go over their inner dims in chunks of 64:
//   weights: a ring of 128 KB, a slab's chunks in turn (absorb: two slabs; values: one), each freed by the last product that
//   reads it, so that the next slab's chunks come in under the last products of this one;
//   tokens: a ring of 16 KB chunks by TMA from the caller's strides (rows behind the last token are zeros);
//   the accumulator in tensor memory is double: four warps round a unit to bf16 and store it by TMA (32 tokens x 64 dims at a
//   time, clipped at the last token) while the next one is multiplied.
// What bounds it: HBM (absorb writes 1024 bytes for 256 read, values the other way around).
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr uint32_t kAllLanes = 0xFFFFFFFFu;
constexpr int kTokens = 128;         // of a unit
constexpr int kChunk = kTokens * 128;  // 64 dims of its tokens
constexpr int kWeights = 128 * 1024;
constexpr int kPiece = 32 * 128;     // what a warp stores at a time
constexpr int kThreads = 256;        // warp 0: TMA, 1: products, 2: tensor memory, 4-7: results
constexpr int kResultWarp = 4;

template <bool VALUES>
struct Form {
    static constexpr int kN = VALUES ? 128 : 256;         // output dims of a unit
    static constexpr int kChunks = VALUES ? 8 : 2;        // of 64 inner dims
    static constexpr int kWSlot = kN * 128;               // a chunk of a slab
    static constexpr int kWSlots = kWeights / kWSlot;
    static constexpr int kASlots = VALUES ? 5 : 4;        // values reads most of its bytes, absorb writes them
    static constexpr int kPieces = VALUES ? 1 : 2;        // a warp's stores in flight
    // weights as [inner][n] (absorb: MN-major) or [n][inner] (values)
    static constexpr uint32_t kIdesc = make_idesc(kTokens, kN, 1, 1, 0, VALUES ? 0 : 1);
};

struct Ctrl {
    uint64_t w_full[8], w_empty[8];
    uint64_t a_full[5], a_empty[5];
    uint64_t d_full[2], d_empty[2];
    uint64_t drained;
    uint32_t tmem_base;
    int32_t failed;
};
template <bool VALUES>
constexpr int kSmem = 1024 + kWeights + Form<VALUES>::kASlots * kChunk + 4 * Form<VALUES>::kPieces * kPiece + (int)sizeof(Ctrl);
static_assert(kSmem<true> <= 232448 && kSmem<false> <= 232448, "shared memory of one CTA");

template <bool VALUES>
__global__ void __launch_bounds__(kThreads, 1)
    heads_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
                 const __grid_constant__ CUtensorMap omap, const HeadsParams p) {
    using F = Form<VALUES>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* w_s = smem;
    uint8_t* a_s = w_s + kWeights;
    uint8_t* o_s = a_s + F::kASlots * kChunk;
    Ctrl* ctl = reinterpret_cast<Ctrl*>(o_s + 4 * F::kPieces * kPiece);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        prefetch_tensormap(&amap);
        prefetch_tensormap(&wmap);
        prefetch_tensormap(&omap);
        for (int i = 0; i < F::kWSlots; ++i) {
            mbar_init(&ctl->w_full[i], 1);
            mbar_init(&ctl->w_empty[i], 1);
        }
        for (int i = 0; i < F::kASlots; ++i) {
            mbar_init(&ctl->a_full[i], 1);
            mbar_init(&ctl->a_empty[i], 1);
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
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(kAllLanes, mbar_wait(bar, parity, p.err, p.wait_ns)) != 0;
    };
    const int u0 = (int)(p.units * blockIdx.x / gridDim.x), u1 = (int)(p.units * (blockIdx.x + 1) / gridDim.x);
    // unit u: slab u / tiles, tokens from kTokens * (u % tiles); a slab's first unit here loads it, its last frees it
    auto first_of_slab = [&](int u) { return u == u0 || u % p.tiles == 0; };
    auto last_of_slab = [&](int u) { return u == u1 - 1 || (u + 1) % p.tiles == 0; };
    bool ok = true;

    if (warp == 0) {
        // ---------------- loads, in the order of their use ----------------
        uint32_t w = 0, a = 0;  // chunks so far
        for (int u = u0; ok && u < u1; ++u) {
            const int slab = u / p.tiles, token = kTokens * (u % p.tiles);
            const int head = VALUES ? slab : slab >> 1, col = VALUES ? 0 : 256 * (slab & 1);
            const bool fresh = first_of_slab(u);
#pragma unroll 1
            for (int k = 0; k < F::kChunks; ++k, ++a) {
                if (fresh) {
                    const uint32_t slot = w % F::kWSlots;
                    if (!(ok = wait(&ctl->w_empty[slot], ((w / F::kWSlots) & 1u) ^ 1u))) break;
                    if (elect_one_sync()) {
                        mbar_arrive_expect_tx(&ctl->w_full[slot], F::kWSlot);
                        uint8_t* dst = w_s + slot * F::kWSlot;
                        if (VALUES) {
                            tma_load_3d(dst, &wmap, &ctl->w_full[slot], 64 * k, 128, head);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                tma_load_3d(dst + 64 * 128 * j, &wmap, &ctl->w_full[slot], col + 64 * j, 64 * k, head);
                        }
                    }
                    ++w;
                }
                const uint32_t slot = a % F::kASlots;
                if (!(ok = wait(&ctl->a_empty[slot], ((a / F::kASlots) & 1u) ^ 1u))) break;
                if (elect_one_sync()) {
                    mbar_arrive_expect_tx(&ctl->a_full[slot], kChunk);
                    tma_load_3d(a_s + slot * kChunk, &amap, &ctl->a_full[slot], 64 * k, head, token);
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- products ----------------
        uint32_t w = 0, a = 0, n = 0;  // w: first chunk of the slab
        const uint64_t ad = smem_desc(smem_u32(a_s), 16, 1024, kSwizzle128B);
        const uint64_t wd = smem_desc(smem_u32(w_s), VALUES ? 16 : 64 * 128, 1024, kSwizzle128B);
        for (int u = u0; ok && u < u1; ++u, ++n) {
            const bool fresh = first_of_slab(u), last = last_of_slab(u);
            const uint32_t buf = n & 1u, d = tmem + F::kN * buf;
            if (!(ok = wait(&ctl->d_empty[buf], ((n >> 1) & 1u) ^ 1u))) break;
#pragma unroll 1
            for (int k = 0; k < F::kChunks; ++k, ++a) {
                const uint32_t ws = (w + k) % F::kWSlots, as = a % F::kASlots;
                if (fresh && !(ok = wait(&ctl->w_full[ws], ((w + k) / F::kWSlots) & 1u))) break;
                if (!(ok = wait(&ctl->a_full[as], (a / F::kASlots) & 1u))) break;
                tc_fence_after();
                if (elect_one_sync()) {
                    const uint64_t x = ad + (uint64_t)(as * (kChunk / 16)), y = wd + (uint64_t)(ws * (F::kWSlot / 16));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma_f16_ss(d, x + (uint64_t)(2 * j), y + (uint64_t)((VALUES ? 2 : 128) * j), F::kIdesc,
                                    k == 0 && j == 0 ? 0u : 1u);
                    umma_commit(&ctl->a_empty[as]);
                    if (last) umma_commit(&ctl->w_empty[ws]);
                    if (k == F::kChunks - 1) umma_commit(&ctl->d_full[buf]);
                }
            }
            if (last) w += F::kChunks;
        }
        // drain (default limit): every product is done before its memory is given back
        if (elect_one_sync()) {
            umma_commit(&ctl->drained);
            mbar_wait(&ctl->drained, 0, p.err);
        }
        __syncwarp();
    } else if (warp >= kResultWarp) {
        // ---------------- results: warp w has tokens 32 w .. 32 w + 31 of a unit ----------------
        const int ew = warp - kResultWarp;
        const uint32_t trow = tmem + ((uint32_t)(32 * ew) << 16);
        uint8_t* stage = o_s + ew * F::kPieces * kPiece;
        uint32_t n = 0, piece = 0;
        for (int u = u0; ok && u < u1; ++u, ++n) {
            const int slab = u / p.tiles, token = kTokens * (u % p.tiles) + 32 * ew;
            const int head = VALUES ? slab : slab >> 1, col = VALUES ? 0 : 256 * (slab & 1);
            const uint32_t buf = n & 1u;
            if (!(ok = wait(&ctl->d_full[buf], (n >> 1) & 1u))) break;
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
                uint8_t* at = stage + (piece % F::kPieces) * kPiece;
                if (lane == 0) bulk_wait_read<F::kPieces - 1>();  // the store that had this place has read it
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
                    if (token < p.total_q) tma_store_3d(&omap, at, col + c, head, token);
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
    p.tiles = (p.total_q + kTokens - 1) / kTokens;
    p.units = (int64_t)p.tiles * p.heads * (p.values ? 1 : 2);
    auto kernel = p.values ? heads_kernel<true> : heads_kernel<false>;
    const int smem = p.values ? kSmem<true> : kSmem<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = p.units < L.num_sms ? p.units : L.num_sms;
    kernel<<<dim3((unsigned)grid), dim3(kThreads), smem, stream>>>(L.amap, L.wmap, L.omap, p);
    return cudaGetLastError();
}

}  // namespace dsa
