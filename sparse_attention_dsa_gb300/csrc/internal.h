// Launch descriptions shared between the C-ABI layer (api.cu) and the kernel translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa.h"

namespace dsa {

constexpr int kMaxStages = 8;

// ---- lightning indexer + Top-K -----------------------------------------------------------------------
struct IndexerParams {
    const float* q_scale;  // [T, Hi] (FP8 only)
    const float* w;        // [T, Hi]
    const float* k_scale;  // [num_pages, 64] (FP8 only)
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* cu_q_lens;
    int32_t* topk;  // [T, K]
    int32_t* err;   // device error word
    int32_t batch;
    int32_t total_q;
    int32_t num_pages;
    int32_t max_pages;
    int32_t top_k;
    int32_t qb;              // query tokens per cluster work item
    int32_t blocks_per_seq;  // ceil(max_q_len / qb)
    int32_t chunk;           // positions per CTA (multiple of 128)
    int32_t stages;          // filled in by the launcher
    int32_t* rows_out;       // [T, K] physical cache row of every selected position (-1 for padding), or null
    const void* q_idx_codes;  // MXFP8: the q_idx codes [T, Hi, Di] (dequantised at set-up instead of loaded by TMA)
    float* topk_score;        // [T, K] fp32 score of every selected position (-inf for padding), or null
    int32_t pos_begin;        // only positions in [pos_begin, pos_end) are candidates (pos_begin % 64 == 0)
    int32_t pos_end;
    uint64_t wait_ns;         // limit of every pipeline wait (drains keep the default limit)
};

struct IndexerLaunch {
    CUtensorMap kmap;  // 3-D view [num_pages][64][Di] of the indexer K cache
    CUtensorMap qmap;  // 2-D view [T*Hi][Di] of q_idx
    IndexerParams params;
    int items;    // work items (clusters)
    int cluster;  // CTAs per cluster
    int idx_heads;
    int idx_dim;
    bool fp8;
    bool mx;         // FP8 with one E8M0 scale per 32 elements (q_scale / k_scale hold scale bytes)
    int smem_limit;  // opt-in dynamic shared memory per block
    bool check_occupancy;
};

// UMMA N of the kernel variant serving (Hi, Di, dtype, qb), 0 when no variant exists.
int indexer_variant_n(int idx_heads, int idx_dim, int fp8, int qb);  // fp8: 0 bf16, 1 row scales, 2 MXFP8
// Dynamic shared memory of that variant for the given pipeline depth, positions per CTA and cluster size.
size_t indexer_smem_estimate(int idx_heads, int idx_dim, int fp8, int qb, int stages, int chunk, int cluster);  // fp8 as above
cudaError_t launch_indexer(const IndexerLaunch& launch, cudaStream_t stream);

// ---- sparse flash attention --------------------------------------------------------------------------
struct SfaParams {
    const uint16_t* q;         // [T, Hq, D] bf16 bits
    const uint16_t* kv_cache;  // [num_pages, 64, D] bf16 bits, or FP8 rows of kKvFp8RowBytes (kv_fp8)
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* cu_q_lens;
    const int32_t* topk;  // [T, K]
    uint16_t* out;        // [T, Hq, Dv] bf16 bits
    float* lse;           // [T, Hq] or null
    int32_t* err;
    int32_t batch;
    int32_t total_q;
    int32_t num_pages;
    int32_t max_pages;
    int32_t top_k;
    int32_t heads;
    int32_t kv_dim;
    int32_t v_dim;
    float scale_log2;  // softmax_scale * log2(e)
    int32_t splits;    // position splits per query (filled in by the launcher)
    int32_t early_setup;  // launched right behind this library's indexer: only topk comes from it
    float* merge;         // split-merge scratch: sfa_merge_floats_per_cta() floats per CTA of the grid
    int32_t kv_fp8;       // kv_cache rows are in the FP8 row layout
    const int32_t* rows_in;  // [T, K] physical rows of topk written by the indexer phase in the same launch, or null
    int32_t one_query_per_seq;  // every sequence has exactly one query token: token t belongs to sequence t
    int32_t pos_begin;          // Top-K entries outside [pos_begin, pos_end) are skipped (a context shard)
    int32_t pos_end;
    uint64_t wait_ns;           // limit of every pipeline wait (drains keep the default limit)
};

struct SfaLaunch {
    CUtensorMap qmap;  // 2-D view [T*Hq][576] of q, 128-row boxes
    SfaParams params;
    int smem_limit;
    int num_sms;
    bool after_indexer;  // the previous kernel in the stream is this library's indexer (programmatic launch)
};

cudaError_t launch_sfa(const SfaLaunch& launch, cudaStream_t stream);

// Position splits the attention launcher starts from for these sizes on `num_sms` SMs (before its
// co-residency check), and the most entries one split may hold.
int sfa_splits(int64_t total_q, int32_t top_k, int num_sms);
constexpr int kSfaMaxEntries = 2048;
// FP8 latent-KV row: 512 E4M3 codes (4 tiles of 128), 4 fp32 tile scales, 64 bf16 rotary values
constexpr int kKvFp8RowBytes = 656;
constexpr int kKvFp8ScaleOff = 512;
constexpr int kKvFp8RopeOff = 528;

// ---- appending a step's rows to the paged caches ------------------------------------------------------
struct AppendParams {
    const uint16_t* k_new;   // [T, Di] bf16 bits or null
    const uint16_t* kv_new;  // [T, 576] bf16 bits or null
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* cu_q_lens;
    uint8_t* k_cache;   // bf16 rows of Di, or E4M3 rows of Di bytes (idx_fp8)
    float* k_scale;     // [num_pages * 64] (idx_fp8)
    uint8_t* kv_cache;  // bf16 rows of 576, or FP8 rows of kKvFp8RowBytes (kv_fp8)
    int32_t* err;
    int32_t batch;
    int32_t total_q;
    int32_t num_pages;
    int32_t max_pages;
    int32_t idx_dim;
    int32_t idx_fp8;
    int32_t kv_fp8;
};
cudaError_t launch_append(const AppendParams& p, cudaStream_t stream);

// Single-launch decode (indexer + Top-K + attention of each token in one cluster, one kernel).  Returns
// cudaErrorNotSupported, without launching anything, when the sizes do not map one query token to one
// cluster (the caller then launches the two kernels).
cudaError_t launch_decode(const IndexerLaunch& indexer, const SfaLaunch& attention, cudaStream_t stream);
// Whether launch_decode would launch for these plans (no launch).
bool decode_single_launch(const IndexerLaunch& indexer, const SfaLaunch& attention);

// Split-merge scratch of the attention kernel: each CTA of a grid with position splits owns one region
// of kSfaMergeRows partial O rows (256 fp32 each; P * ceil(128 / P) of them are used) and 128
// (max, sum) pairs.
constexpr int kSfaMergeRows = 136;
constexpr size_t kSfaMergeFloatsPerCta = (size_t)kSfaMergeRows * 256 + 2 * 128;
// The largest grid (in CTAs) the attention launcher can choose with position splits for these sizes
// (0 when it never splits): at most 256 SMs' worth, or more when top_k forces splits.
size_t sfa_merge_ctas(int64_t total_q, int32_t top_k);
// Bytes of workspace the library uses: the 256-byte error word area, plus the attention merge scratch.
constexpr size_t kErrorWordArea = 256;

// ---- context-parallel decode: merge of shard Top-K lists, combine of shard attention outputs -----------
struct MergeParams {
    const int32_t* idx;   // [shards, T, K] shard-local selections (positions, -1 padded)
    const float* score;   // [shards, T, K] their scores
    int32_t* out_idx;     // [T, K]
    float* out_score;     // [T, K] or null
    int32_t shards;
    int32_t total_q;
    int32_t top_k;
};
size_t merge_smem_bytes(int shards, int top_k);
cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream);

struct CombineParams {
    const uint16_t* out_in;  // [shards, T, Hq, Dv] bf16 bits
    const float* lse_in;     // [shards, T, Hq]
    uint16_t* out;           // [T, Hq, Dv] bf16 bits
    float* lse;              // [T, Hq] or null
    int32_t shards;
    int32_t total_q;
    int32_t heads;
    int32_t v_dim;
};
cudaError_t launch_combine(const CombineParams& p, cudaStream_t stream);

// ---- position rotation: appending rotated rows, rotating a step's queries -------------------------------
struct RopeParams {
    const float* table;  // [table_len, 64] fp32: 32 cosines, 32 sines
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* cu_q_lens;
    int32_t* err;
    int32_t table_len;
    int32_t kv_interleaved;
    int32_t idx_interleaved;
    int32_t idx_begin;  // first rotated dim of an indexer row, or -1
    int32_t batch;
    int32_t total_q;
    int32_t num_pages;
    int32_t max_pages;
    int32_t idx_dim;
    int32_t idx_dtype;  // dsa_dtype_t
};
struct RopeAppendParams {
    RopeParams r;
    const uint16_t* k_new;   // bf16 bits, rows k_stride elements apart, or null
    const uint16_t* kv_new;  // bf16 bits, rows kv_stride elements apart, or null
    int64_t k_stride;
    int64_t kv_stride;
    uint8_t* k_cache;
    void* k_scale;  // fp32 [num_pages * 64], or E8M0 bytes [num_pages * 64, Di / 32]
    uint8_t* kv_cache;
    int32_t kv_fp8;
};
struct RopeQueriesParams {
    RopeParams r;
    const uint16_t* q_pe;  // bf16 bits or null; may alias q
    int64_t q_pe_token_stride;
    int64_t q_pe_head_stride;
    uint16_t* q;               // [T, Hq, 576] bf16 bits
    const uint16_t* q_idx_in;  // bf16 bits or null; may be q_idx (bf16)
    int64_t q_idx_stride;
    uint8_t* q_idx;  // [T, Hi, Di]
    void* q_scale;   // fp32 [T, Hi], or E8M0 bytes [T, Hi, Di / 32]
    int32_t heads;
    int32_t idx_heads;
    int32_t num_sms;
};
cudaError_t launch_rope_append(const RopeAppendParams& p, cudaStream_t stream);
cudaError_t launch_rope_queries(const RopeQueriesParams& p, cudaStream_t stream);

// ---- dense attention over the latent-KV cache with a shared prefix --------------------------------------
struct PrefixParams {
    const uint16_t* q;        // [T, Hq, 576] bf16 bits
    const uint8_t* kv_cache;  // bf16 rows, or FP8 rows of kKvFp8RowBytes
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* cu_q_lens;
    uint16_t* out;  // [T, Hq, 512] bf16 bits
    float* lse;     // [T, Hq] or null
    int32_t* err;
    int32_t batch;
    int32_t total_q;
    int32_t num_pages;
    int32_t max_pages;
    int32_t heads;
    int32_t prefix_len;
    int32_t kv_fp8;
    float scale_log2;  // softmax_scale * log2(e)
    uint64_t wait_ns;
    int32_t max_q_len;
    // filled in by plan_prefix()
    int32_t packed;         // rows of different sequences share tiles over the prefix
    int32_t packed_tiles;   // 128-row tiles of all the batch's rows
    int32_t tiles_per_seq;  // 128-row tiles of the longest sequence's rows, 0 where items are numbered by the rows in front
    int32_t prefix_tiles;   // 128-position tiles of the prefix
    int32_t row_tiles;      // 128-row tiles that attend to the prefix
    int32_t n_items;
    int32_t slot_by_item;   // where partial results lie (partial_slot)
    int32_t planned;  // the items' tiles are divided evenly among the CTA pairs (else: whole items in turn)
    // workspace (planned)
    int32_t* plan;  // merged: an int4 for each part; packed: behind those, an int2 for each item (see the kernels)
    float* partial;  // slots of kPartialFloats
    int32_t convert_ahead;  // plan_prefix(): the prefix's FP8 rows are converted to f16 first
    uint8_t* ahead;         // those rows [ceil(prefix_len / 64) * 64][576] f16, or null
};
constexpr int kLongestContext = INT32_MAX - 255;  // the end of a context's last tile is a position, too
constexpr int kPrefixPairs = 76;     // CTA pairs of the largest grid: one CTA on each of 152 SMs
constexpr int kPlanItems = 2048;     // most items that are divided evenly
constexpr int kPackItems = 4096;     // the same where rows are packed
constexpr int kDivideCost = 11;      // what dividing costs each pair, in tiles
constexpr int kPartCost = 1;         // what a partial result costs, in tiles
constexpr int kWholeTiles = 16;      // longer own contexts are always divided
constexpr int kAheadGain = 100;      // tiles that converting ahead must save
// A partial result: O [128][512] fp32 (unnormalised), then (maximum in log2 units, sum) per row.
constexpr int kPartialFloats = 128 * 512 + 2 * 128;
void plan_prefix(PrefixParams* p, int max_pages);  // from the sizes alone
size_t prefix_plan_bytes(const PrefixParams& p);
size_t prefix_partial_bytes(const PrefixParams& p);
size_t prefix_ahead_bytes(const PrefixParams& p);
size_t prefix_workspace_bound(const PrefixParams& p, int max_pages);  // the three, of any call that is no larger
struct PrefixLaunch {
    CUtensorMap qmap;  // 3-D view [9][T*Hq][64] of q: 64-dim atoms of 64 rows, nine at a time
    // 4-D views [pages][9][64][64] of 16-bit rows (the bf16 cache, or the prefix's FP8 rows converted ahead)
    CUtensorMap kmap;  // atoms of a page three at a time (converted rows: one)
    CUtensorMap vmap;  // four atoms (256 dims) at a time
    CUtensorMap codemap;  // FP8 rows, 4-D view [num_pages][4][64][128] of their codes: two scale tiles at a time
    CUtensorMap rotmap;   // FP8 rows, 3-D view [num_pages][64][656] bytes: the rotary part of a page
    PrefixParams params;
};
cudaError_t launch_prefix(const PrefixLaunch& launch, cudaStream_t stream);

// Sets the message returned by dsa_last_error_message() on this host thread.
void set_last_error(const char* message);

// Limit of the kernels' pipeline waits for launches made from now on (dsa_set_wait_limit_ns).
uint64_t wait_limit_ns();

// The host half of dsa_indexer_topk: every argument check and the launch plan, nothing enqueued (*launch
// is false when there is nothing to launch); then the launch itself.
dsa_status_t prepare_indexer_call(const dsa_dims_t* dims, const void* q_idx, const void* q_scale, const float* w,
                                  const void* k_cache, const void* k_scale, const int32_t* page_table,
                                  const int32_t* seq_lens, const int32_t* cu_q_lens, int32_t* topk_idx,
                                  float* topk_score, void* workspace, IndexerLaunch* launch_out, bool* launch);
dsa_status_t launch_indexer_call(const IndexerLaunch& launch, void* stream);

// Candidates one dsa_topk_merge call may hold per query token (shards * top_k): its shared-memory keys.
constexpr int kMaxMergeCandidates = 16384;

}  // namespace dsa
