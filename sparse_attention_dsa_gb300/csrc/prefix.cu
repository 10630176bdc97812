// Dense attention over the paged latent-KV cache for a batch whose sequences share a prefix, for sm_103a.
//
// For query token t of sequence b at position p and head h: z_s = scale * q[t,h,:] . kv[s,:] for s = 0..p,
// out[t,h,:] = softmax(z) . kv[:, :512], lse[t,h] = logsumexp(z) ("Optimizing Inference for Hybrid Attention
// Architectures: From Operator Fusion to Sequence Sharding", section "Breaking Down the Computational Path of
// Hybrid Attention", step 2, without the selection).  Positions below prefix_len are read through sequence 0.
//
// Rows.  A query row is one (token, head); the latent rows are the keys and values of every head, so a
// product tile takes 128 rows whatever tokens and heads they are.  An item is such a tile with the positions
// it attends to, in tiles of 128:
//   * merged: the tile's rows belong to one sequence and its positions are the prefix and then the sequence's
//     own; with all its tiles in one place the result is written directly;
//   * packed: an item of 128 rows of any sequences over the prefix, and for each sequence items over its own
//     positions; the partial results of a row are combined by a second kernel.  Fewer tiles pass over the prefix
//     where a sequence's rows do not fill one.
// The tiles of all items form one line (each item with a few places for what it costs beside its tiles) that is
// cut into equal parts, one for each CTA pair, so that the work is even whatever the lengths are; an item cut in
// two or more is combined from its parts.  Short merged items are taken whole instead, in turn.  plan_prefix()
// chooses, with the times of each way.
//
// One CTA pair (a cluster of two, cta_group::2) works on 128 rows, 64 in each CTA, because a 128 x 512 fp32
// accumulator would fill the tensor memory of one: the pair's products of 128 rows put the first half of the
// columns into lanes 0-63 and the second half into lanes 64-127, so O takes 256 columns, two S tiles 64 each.
//   S (128 x 128) = Q K^T: CTA c holds Q of its rows and K of page c of the tile (64 rows x 576 dims);
//   O (128 x 512) += P V: CTA c holds P of its rows and V of both pages for dims 256c .. 256c + 255.
// K and V are rings of shared-memory slots filled by TMA straight from the pages, K 192 dims and V 64 positions
// x 256 dims at a time (a copy takes some 270 cycles to issue, whatever its size), each freed by the commit of
// the products that read it.  A tile's P V is
// issued behind the next tile's Q K^T, so the softmax of one tile runs under the products of the other.
//   softmax: thread (row, column half), 64 scores each; the two halves of a row exchange their maxima through
// shared memory.  The running maximum is raised only when it grows by more than 2^8.
//   Tiles that some row does not see whole (the prefix's or a context's end, the causal edge) take their V
// through registers, where infinities and NaN become 0: 0 x inf would reach rows that do not see them.
//   FP8 rows become f16 in the rings (eight warps), or, a prefix's that several tiles of rows attend to, once ahead.
//
// What bounds it, and measured (one GB300, warm).  A 128 x 128 tile costs 2 x 128 x 128 x (576 + 512) operations, 1.42 us on
// a pair at the measured cuBLAS rate: prefix tiles, whose rows are in L2, take 1.30 us, bound by the tensor pipe and by
// the shared-memory reads of Q K^T, which fill it.  Own bf16 rows are read once by one pair: 1.8 us a tile with all
// pairs at it, 0.92 of the copy bandwidth.  Own FP8 rows: 3.1 us, bound by shared memory (245 KB of
// operands, 280 KB for codes arriving, read and written back, a CTA and tile).  32 sequences of 1024 positions behind 16384, 128 heads:
// 91 to 93 us, 1.6 PFLOP/s; 64 x 16 heads, 500 behind 32741: 58 us; 8 prompts of up to 257 queries x 32 heads behind 4096: 277
// to 304 us (the power limit), 1.6 to 1.7 PFLOP/s; one short item: 12 us, all latency.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr uint32_t kAllLanes = 0xFFFFFFFFu;
constexpr float kLn2 = 0.69314718055994531f;

// An ordinary load of an input.  These kernels may be resident before the kernel that writes their inputs has ended
// (they wait for its end before they load): not a case for loads that take memory as constant for a kernel's duration.
template <typename T>
__device__ __forceinline__ T ld_input(const T* p) {
    return *p;
}

// ---------------------------------------------------------------------------------------------------------
// Items and their division among the CTA pairs (used by both kernels)
// ---------------------------------------------------------------------------------------------------------
struct Item {
    int row0, nrows;    // rows of [T * Hq]
    int b;              // sequence, or -1: packed rows over the prefix
    int tiles_a;        // tiles of the prefix, then
    int tiles_b;        // tiles of the sequence's own positions, from position base_b
    int base_b;
    int hi_all, hi_max;  // positions below hi_all are seen by every row, those from hi_max on by none
    int pos0, lrow0;    // position of the sequence's first query; first row within the sequence's rows
};

// Offsets and length of sequence b; false when they are inconsistent.
__device__ __forceinline__ bool sequence(const PrefixParams& p, int b, int* c0, int* n, int* L) {
    const int a = ld_input(p.cu_q_lens + b), e = ld_input(p.cu_q_lens + b + 1);
    *L = ld_input(p.seq_lens + b);
    *c0 = a;
    *n = e - a;
    if (a < 0 || e < a || e > p.total_q || *n > p.max_q_len) return false;
    if (*n == 0) return true;
    if (*L > kLongestContext) return false;
    return (int64_t)*n <= (int64_t)*L - p.prefix_len && (int64_t)*L <= (int64_t)p.max_pages * 64;
}

// The sequence through whose page table the prefix is read: the first whose context covers it (0 if there is none: no
// sequence has a query behind the prefix then).  Called by a whole warp; mine: seq_lens[lane], -1 where there is none.
__device__ __forceinline__ int prefix_source(const PrefixParams& p, int mine, int lane) {
    for (int j0 = 0;;) {
        const uint32_t hit = __ballot_sync(kAllLanes, mine >= p.prefix_len && (int64_t)mine <= (int64_t)p.max_pages * 64);
        if (hit) return j0 + __ffs(hit) - 1;
        j0 += 32;
        if (j0 >= p.batch) return 0;
        mine = j0 + lane < p.batch ? ld_input(p.seq_lens + j0 + lane) : -1;
    }
}
__device__ __forceinline__ int first_length(const PrefixParams& p, int lane) {
    return lane < p.batch ? ld_input(p.seq_lens + lane) : -1;
}

// Number of sequence b's first item among the sequences' items, c0 its first query.  Where one sequence has many queries
// and most have few, tiles_per_seq numbers a sequence would be empty ones nearly all (tiles_per_seq is 0 then): b +
// floor(c0 * heads / 128) is never less than the number of tiles in front of it.
__device__ __forceinline__ int64_t first_item(const PrefixParams& p, int b, int c0) {
    return p.tiles_per_seq > 0 ? (int64_t)b * p.tiles_per_seq : b + (int64_t)c0 * p.heads / 128;
}
// The sequence of item j then: the last one whose first item is not behind it.
__device__ __forceinline__ int search_item(const PrefixParams& p, int j) {
    int b = 0, hi = min(p.batch, j + 1);
    while (hi - b > 1) {
        const int mid = (b + hi) / 2;
        if (first_item(p, mid, ld_input(p.cu_q_lens + mid)) <= j) b = mid;
        else hi = mid;
    }
    return b;
}

// SEARCH: items are numbered by the rows in front of them (an instance of its own: with the choice in the code of every role
// 32 x 64 heads of FP8 rows behind 16000 took 74.3 us instead of 71.2).
template <bool SEARCH>
__device__ __forceinline__ Item decode_item(const PrefixParams& p, int i) {
    Item it;
    it.b = -1;
    it.tiles_a = p.prefix_tiles;
    it.tiles_b = it.base_b = it.pos0 = it.lrow0 = 0;
    it.hi_all = it.hi_max = p.prefix_len;
    const int nt = p.packed ? p.packed_tiles : 0;
    if (i < nt) {
        it.row0 = 128 * i;
        it.nrows = min(128, p.total_q * p.heads - it.row0);
        return it;
    }
    const int j = i - nt;
    it.b = SEARCH ? search_item(p, j) : j / p.tiles_per_seq;
    int c0, n, L;
    bool ok = sequence(p, it.b, &c0, &n, &L);
    if (SEARCH) {
        const int64_t lrow0 = 128 * (j - first_item(p, it.b, c0));  // (a row that no sequence has: inconsistent offsets)
        ok = ok && lrow0 >= 0 && lrow0 < (int64_t)n * p.heads;
        it.lrow0 = ok ? (int)lrow0 : 0;
    } else {
        it.lrow0 = 128 * (j - it.b * p.tiles_per_seq);
    }
    it.row0 = ok ? c0 * p.heads + it.lrow0 : 0;
    it.nrows = ok ? min(128, n * p.heads - it.lrow0) : 0;
    if (it.nrows <= 0) {
        it.nrows = it.tiles_a = 0;
        return it;
    }
    if (p.packed) it.tiles_a = 0;
    it.pos0 = L - n;
    it.hi_all = it.pos0 + it.lrow0 / p.heads + 1;
    it.hi_max = it.pos0 + (it.lrow0 + it.nrows - 1) / p.heads + 1;
    it.base_b = p.prefix_len & ~63;
    it.tiles_b = (it.hi_max - it.base_b + 127) / 128;
    return it;
}

// Part k of a line of W tiles cut in G parts starts at floor(k W / G); the part that holds tile w.
__device__ __forceinline__ int part_begin(int k, int W, int G) { return (int)((int64_t)k * W / G); }
__device__ __forceinline__ int part_of(int w, int W, int G) { return (int)((((int64_t)w + 1) * G - 1) / W); }

// Where pair k leaves its partial result of an item.  By item: there are at most item + pair of them before this one (packed:
// every segment has a result to combine).  By pair: of merged items only a pair's first and last segment can be cut, and a
// segment with the item's first tile is the last one.
__device__ __forceinline__ int64_t partial_slot(const PrefixParams& p, int item, int k, bool has_first_tile) {
    return p.slot_by_item ? item + k : 2 * k + (has_first_tile ? 1 : 0);
}

// On the line an item is kItemCost places longer than its tiles, in front of them: what its queries' load, its
// first tile's latency and its result cost in tiles.  Parts are no shorter than kMinPlaces on average.
// (20 sequences of 4096 positions, 128 heads: 28.1, 26.7, 25.9, 26.6, 27.5 us with 1, 2, 3, 4, 6 places.)
// A tile of FP8 rows that are converted in passing takes three places.  A cut gives the tiles that begin before it to
// the part before it.
constexpr int kItemCost = 3;
constexpr int kMinPlaces = 2 + kItemCost;
__device__ __forceinline__ int parts_for(int W, int pairs) { return max(1, min(pairs, W / kMinPlaces)); }
__device__ __forceinline__ int cost_a(const PrefixParams& p) { return p.kv_fp8 && p.ahead == nullptr ? 3 : 1; }
__device__ __forceinline__ int cost_b(const PrefixParams& p) { return p.kv_fp8 ? 3 : 1; }
__device__ __forceinline__ int places(const PrefixParams& p, const Item& it) {
    return it.tiles_a + it.tiles_b > 0 ? kItemCost + it.tiles_a * cost_a(p) + it.tiles_b * cost_b(p) : 0;
}
// Tiles of an item that begin before its place o.
__device__ __forceinline__ int tiles_before(const PrefixParams& p, const Item& it, int o) {
    const int ca = cost_a(p), cb = cost_b(p), x = max(0, o - kItemCost), a = it.tiles_a * ca;
    return x <= a ? (x + ca - 1) / ca : min(it.tiles_a + it.tiles_b, it.tiles_a + (x - a + cb - 1) / cb);
}
// First and last part of an item of `n` places from place `before` of the line.
__device__ __forceinline__ void parts_of_item(const PrefixParams& p, const Item& it, int before, int n, int W, int G, int* k0,
                                              int* k1) {
    *k0 = part_of(before + kItemCost, W, G);  // the part of its first tile's first place, and of its last tile's
    *k1 = part_of(before + n - (it.tiles_b > 0 ? cost_b(p) : cost_a(p)), W, G);
}

// ---------------------------------------------------------------------------------------------------------
// The attention kernel
// ---------------------------------------------------------------------------------------------------------
// warp 0: TMA, 1: products, 4-7: softmax; bf16: 8-11 V of edge tiles; FP8: 2, 3, 8, 9 convert K, 10-13 V
constexpr int kSoftmaxWarp = 4;
constexpr int kFillWarp = 8;
constexpr int kFillWarps = 4;  // of each kind
constexpr int kMaxWarps = 14;
template <bool KVFP8>
constexpr int kThreads = 32 * (KVFP8 ? kMaxWarps : kFillWarp + kFillWarps);
constexpr int kQAtoms = 9;                  // 64-dim pieces of a row
constexpr int kAtom = 64 * 128;             // 64 rows x 128 bytes, 128-byte swizzle
// K ring: the nine atoms of a tile, handed over in three units: bf16 three atoms each (one copy each), FP8 four, four
// and the rotary atom
constexpr int kKUnits = 3;
template <bool KVFP8>
__host__ __device__ constexpr int unit_atom(int j) { return (KVFP8 ? 4 : 3) * j; }
template <bool KVFP8>
__host__ __device__ constexpr int unit_atoms(int j) { return KVFP8 ? (j < 2 ? 4 : 1) : 3; }
constexpr int kVSlots = 2;                  // V ring: slots of 64 positions x 256 dims
constexpr int kVSlot = 4 * kAtom;
constexpr int kPBytes = 2 * kAtom;          // 64 rows x 128 positions
constexpr int kSCol = 256;                  // tensor memory: O in columns 0-255, S tiles at 256 and 320
template <bool KVFP8>
constexpr uint32_t kIdescQK = make_idesc(128, 128, KVFP8 ? 0 : 1, KVFP8 ? 0 : 1, 0, 0);
template <bool KVFP8>
constexpr uint32_t kIdescPV = make_idesc(128, 256, KVFP8 ? 0 : 1, KVFP8 ? 0 : 1, 0, 1);
// Raise the running maximum (log2) only when it grows by more than this.
template <bool KVFP8>
constexpr float kRaise = KVFP8 ? 4.f : 8.f;
// Weights are taken relative to 2^-kLift of the running maximum: f16 weights of up to 2^(kRaise + kLift) = 2^15 keep
// their precision down to 2^-25 of the largest one's, so that a long context's many small weights beside a large
// one are not lost (bf16 has fp32's range).
template <bool KVFP8>
constexpr float kLift = KVFP8 ? 11.f : 0.f;

struct Segment {
    Item it;
    int index;   // item number
    int u0, u1;  // tiles of the item
};

struct Ctrl {
    uint64_t q_full, q_empty;
    uint64_t k_full[kKUnits], k_empty[kKUnits];
    uint64_t v_full[kVSlots], v_empty[kVSlots];
    uint64_t v_turn[kVSlots];  // bf16: the slot is free for an edge tile's V (once for each edge tile)
    uint64_t s_full[2], s_empty[2];
    uint64_t p_full, pv_done, o_free, edge_full, drained, exchanged;
    // FP8: bf16 queries, codes and rotary parts are here; are converted
    uint64_t q_raw, q_conv, k_raw[3], k_conv[3], v_raw[2], v_conv[2];
    uint32_t tmem_base;
    int32_t failed;
    int32_t prefix_source;
    int32_t first_place;  // this pair's first item (in `first`) and its place in it
    Segment first;
    int32_t scan[kMaxWarps];
    float exchange[2][128];
    // bf16: the first position whose V was cleaned in an edge tile of a segment (numbered from 1, one slot for each parity):
    // segment << 32 | INT32_MAX - position
    unsigned long long cleaned[2];
};
constexpr int kSmem = 1024 + 2 * kQAtoms * kAtom + kVSlots * kVSlot + kPBytes + (int)sizeof(Ctrl);
static_assert(kSmem <= 232448, "shared memory of one CTA");
static_assert(kPackItems >= kPlanItems && kPackItems * 4 <= kQAtoms * kAtom, "the plan's scan is done in the K ring's memory");

// Where a role stands in its pair's list of segments.
struct Walk {
    int item, tile, left;  // next item, place in it, places left (planned) or the stride (whole items)
    bool decoded;          // the segment passed in holds the next item already
};

template <bool SEARCH>
__device__ __forceinline__ bool next_segment(const PrefixParams& p, Walk& w, Segment& s) {
    if (p.planned) {
        while (w.left > 0 && w.item < p.n_items) {
            if (!w.decoded) s.it = decode_item<SEARCH>(p, w.item);
            w.decoded = false;
            const int tiles = s.it.tiles_a + s.it.tiles_b;
            if (tiles > 0) {  // w.tile counts places
                s.index = w.item;
                const int n = places(p, s.it);
                s.u0 = tiles_before(p, s.it, w.tile);
                s.u1 = w.tile + w.left >= n ? tiles : tiles_before(p, s.it, w.tile + w.left);
                w.left -= n - w.tile;
            }
            ++w.item;
            w.tile = 0;
            if (tiles > 0 && s.u1 > s.u0) return true;
        }
        return false;
    }
    while (w.item >= 0) {  // whole items, the ones with the most positions (the last of each sequence) first
        if (!w.decoded) s.it = decode_item<SEARCH>(p, w.item);
        w.decoded = false;
        s.index = w.item;
        s.u0 = 0;
        s.u1 = s.it.tiles_a + s.it.tiles_b;
        w.item -= w.left;
        if (s.u1 > 0) return true;
    }
    return false;
}

// Tile u of an item: its first position, the range that exists, its page-table row, whether every row sees it whole.
struct Tile {
    int base, lo, hi;
    const int32_t* pages;
    bool edge;
    bool copied;  // FP8: its rows have been converted ahead
};
// shared: the page-table row of the prefix.
__device__ __forceinline__ Tile tile_of(const PrefixParams& p, const int32_t* shared, const Item& it, int u) {
    Tile t;
    if (u < it.tiles_a) {
        t.base = 128 * u;
        t.lo = 0;
        t.hi = p.prefix_len;
        t.pages = shared;
        t.edge = t.base + 128 > t.hi;
        t.copied = p.ahead != nullptr;
    } else {
        t.base = it.base_b + 128 * (u - it.tiles_a);
        t.lo = p.prefix_len;
        t.hi = it.hi_max;
        t.pages = p.page_table + (int64_t)it.b * p.max_pages;
        t.edge = t.base < t.lo || t.base + 128 > it.hi_all;
        t.copied = false;
    }
    return t;
}
// Table entry of half h (64 positions) of a tile; kNoPage where it has no position that exists.  The entry is
// checked where it is used, a tile later, so that nothing waits for its load here.
constexpr int kNoPage = INT32_MIN;
__device__ __forceinline__ int page_of(const Tile& t, int h) {
    const int first = t.base + 64 * h;
    return first < t.hi ? ld_input(t.pages + (first >> 6)) : kNoPage;
}

// Infinities and NaN of a pair (bf16, or f16) become 0.
template <uint32_t kExponent = 0x7F80u>
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
    if ((v & kExponent) == kExponent) v &= 0xFFFF0000u;
    if ((v & (kExponent << 16)) == kExponent << 16) v &= 0x0000FFFFu;
    return v;
}

// FP8 rows are multiplied as f16, q and the weights with them: a code's four significant bits times a scale of eleven
// lose three bits less than in bf16 (errors of 2^-11 against 2^-8), and a pair of codes takes two instructions rather
// than six.  Rows are kept times kF16Gain, which cancels in the scores (q is divided by it) and is taken out of the
// result; the largest values are 65504 / kF16Gain.  A row's scale is some 450 times smaller than its largest value: it is
// kept 2^8 times larger, and the codes (whose range is small) as much smaller, so that both are exact down to
// values of 2^-16.
constexpr float kF16Gain = 4.f;
constexpr float kScaleGain = 256.f * kF16Gain;
constexpr uint32_t kCodeGain = 0x1C001C00u;  // 2^-8 twice
__device__ __forceinline__ uint32_t f2_to_h2(float a, float b) {  // a in the low half
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// Eight E4M3 codes times a scale, given as a f16 pair of scale * kScaleGain.
__device__ __forceinline__ uint4 codes_to_h8(uint32_t lo, uint32_t hi, uint32_t scale2) {
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint16_t pair = (uint16_t)((j < 2 ? lo : hi) >> (16 * (j & 1)));
        asm("{\n\t.reg .b32 h;\n\tcvt.rn.f16x2.e4m3x2 h, %1;\n\tmul.rn.f16x2 h, h, %3;\n\tmul.rn.f16x2 %0, h, %2;\n\t}"
            : "=r"(out[j])
            : "h"(pair), "r"(scale2), "r"(kCodeGain));
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}
// Eight bf16 values times a power of two.
__device__ __forceinline__ uint4 bf8_to_h8(uint4 v, float gain) {
    auto pair = [&](uint32_t w) { return f2_to_h2(__uint_as_float(w << 16) * gain, __uint_as_float(w & 0xFFFF0000u) * gain); };
    return make_uint4(pair(v.x), pair(v.y), pair(v.z), pair(v.w));
}
// What lies beyond f16's range must not pass for an infinity: q of the other sign would make a score of -inf of it, and the
// position would drop out of the result.  A row of K or q with such an element gets a NaN, so that every row of the result
// that sees it does, and is reported.
// Nonzero in the sign bits' places where a f16 value of the eight has an exponent of all ones (it carries into them).
__device__ __forceinline__ uint32_t not_finite(const uint4& h) {
    const uint32_t c = 0x7C007C00u, one = 0x04000400u;
    return (((h.x & c) + one) | ((h.y & c) + one) | ((h.z & c) + one) | ((h.w & c) + one)) & 0x80008000u;
}
// Whether one of eight bf16 values is finite, and infinite as f16 times gain.
__device__ __forceinline__ bool values_over(const uint4& v, float gain) {
    const uint4 h = bf8_to_h8(v, gain);
    if (not_finite(h) == 0) return false;
    const uint32_t from[4] = {v.x, v.y, v.z, v.w}, to[4] = {h.x, h.y, h.z, h.w};
    bool found = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int at = 16 * (j & 1);
        found |= ((to[j >> 1] >> at) & 0x7FFFu) == 0x7C00u && ((from[j >> 1] >> at) & 0x7F80u) != 0x7F80u;
    }
    return found;
}
// Whether one of sixteen codes times their scale is infinite as f16, or the scale itself (64 and more); neither is a NaN.
// No element of a smaller scale than kLargestScale is: 65520 / (448 * kF16Gain) = 36.56.
constexpr float kLargestScale = 36.5f;
__device__ __forceinline__ bool codes_over(const uint4& code, float scale) {
    if (!(fabsf(scale) > kLargestScale)) return false;
    const uint32_t scale2 = f2_to_h2(scale * kScaleGain, scale * kScaleGain);
    if ((scale2 & 0x7FFFu) == 0x7C00u) return true;
    const uint4 lo = codes_to_h8(code.x, code.y, scale2), hi = codes_to_h8(code.z, code.w, scale2);
    const uint32_t to[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    bool found = false;
#pragma unroll
    for (int j = 0; j < 16; ++j) found |= ((to[j >> 1] >> (16 * (j & 1))) & 0x7FFFu) == 0x7C00u;
    return found;
}
constexpr uint32_t kNaN2 = 0x7E007E00u;  // f16 twice
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float exp2_fast(float x) {  // relative error about 2^-22; exp2(-inf) = +0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool KVFP8, bool SEARCH>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads<KVFP8>, 1)
    prefix_pair_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap codemap,
                       const __grid_constant__ CUtensorMap rotmap, const PrefixParams p) {
    constexpr int kThreads = dsa::kThreads<KVFP8>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* q_s = smem;
    uint8_t* k_s = q_s + kQAtoms * kAtom;
    uint8_t* v_s = k_s + kQAtoms * kAtom;
    uint8_t* p_s = v_s + kVSlots * kVSlot;
    Ctrl* ctl = reinterpret_cast<Ctrl*>(p_s + kPBytes);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_ctarank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    // ---- set-up (before the division of the work: its loads hide it) ----
    if (tid == 0) {
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
        if (KVFP8) {
            prefetch_tensormap(&codemap);
            prefetch_tensormap(&rotmap);
        }
        mbar_init(&ctl->q_full, 1);
        mbar_init(&ctl->q_empty, 1);
        for (int i = 0; i < kKUnits; ++i) {
            mbar_init(&ctl->k_full[i], 1);
            mbar_init(&ctl->k_empty[i], 1);
        }
        for (int i = 0; i < kVSlots; ++i) {
            mbar_init(&ctl->v_full[i], 1);
            mbar_init(&ctl->v_empty[i], 1);
            mbar_init(&ctl->v_turn[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->s_full[i], 1);
            mbar_init(&ctl->s_empty[i], 8);  // the softmax warps of both CTAs
        }
        mbar_init(&ctl->p_full, 8);
        mbar_init(&ctl->pv_done, 1);
        mbar_init(&ctl->o_free, 8);
        mbar_init(&ctl->edge_full, 2 * kFillWarps);
        mbar_init(&ctl->drained, 1);
        if (KVFP8) {
            mbar_init(&ctl->q_raw, 1);
            mbar_init(&ctl->q_conv, 4 * kFillWarps);
            for (int i = 0; i < 3; ++i) {
                mbar_init(&ctl->k_raw[i], 1);
                mbar_init(&ctl->k_conv[i], 2 * kFillWarps);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&ctl->v_raw[i], 1);
                mbar_init(&ctl->v_conv[i], 2 * kFillWarps);
            }
        }
        mbar_init(&ctl->exchanged, 4);
        ctl->failed = 0;
        ctl->cleaned[0] = ctl->cleaned[1] = 0;
        fence_mbar_init();
    }
    __syncwarp();
    cluster_arrive();
    if (warp == 2) {
        tmem_pair_alloc(&ctl->tmem_base, 512);
        tmem_pair_relinquish();
    }
    // everything above may run before the previous kernel of the stream has ended, nothing below may; the
    // combining kernel, launched behind this one in the same way, does likewise
    grid_dependency_wait();
    allow_dependent_launch();

    // ---- the division of the work ----
    if (pair == 0 && rank == 0) {  // inconsistent sequences and tokens of no sequence are reported once
        for (int b = tid; b < p.batch; b += kThreads) {
            int c0, n, L;
            if (!sequence(p, b, &c0, &n, &L)) raise_error(p.err, DSA_DEVERR_SEQ);
        }
        if (tid == 0 && (ld_input(p.cu_q_lens) != 0 || ld_input(p.cu_q_lens + p.batch) != p.total_q))
            raise_error(p.err, DSA_DEVERR_SEQ);
    }
    constexpr int kSourceWarp = 3;
    const int first_L = warp == kSourceWarp ? first_length(p, lane) : 0;  // looked at behind the plan's own loads
    Walk start;
    bool idle = false;
    if (p.planned) {
        // places before each item: every thread a run of items, then a scan of the threads' sums
        int32_t* cum = reinterpret_cast<int32_t*>(k_s);
        const int run = (p.n_items + kThreads - 1) / kThreads;
        const int i0 = min(p.n_items, tid * run), i1 = min(p.n_items, i0 + run);
        int sum = 0;
        Item mine;  // the last of the run, the only one as a rule
        for (int i = i0; i < i1; ++i) {
            mine = decode_item<SEARCH>(p, i);
            cum[i] = places(p, mine);
            sum += cum[i];
        }
        int incl = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(kAllLanes, incl, off);
            if (lane >= off) incl += o;
        }
        if (lane == 31) ctl->scan[warp] = incl;
        __syncthreads();
        int before = incl - sum, W = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += ctl->scan[w];
            W += ctl->scan[w];
        }
        const int G = parts_for(W, pairs);
        idle = pair >= G || W == 0;
        const int w0 = idle ? 0 : part_begin(pair, W, G);
        if (idle && rank == 0 && tid == 0) reinterpret_cast<int4*>(p.plan)[pair] = make_int4(0, 0, 0, 0);
        for (int i = i0; i < i1; ++i) {
            const int tiles = cum[i];
            if (run > 1) mine = decode_item<SEARCH>(p, i);
            // for the combining kernel: packed, the parts of every item; merged, for each part that begins inside an
            // item, as the second of that item's parts, the item's rows, parts (first, and count << 8) and number
            const bool here = w0 >= before && w0 < before + tiles;
            if (rank == 0 && (p.packed ? pair == 0 : here && !idle)) {
                int k0 = 0, count = 0;
                if (tiles > 0) {
                    int k1;
                    parts_of_item(p, mine, before, tiles, W, G, &k0, &k1);
                    count = k1 - k0 + 1;
                }
                if (p.packed)
                    reinterpret_cast<int2*>(p.plan + 4 * kPrefixPairs)[i] = make_int2(k0, count);
                else
                    reinterpret_cast<int4*>(p.plan)[pair] =
                        make_int4(mine.row0, count > 1 && k0 == pair - 1 ? mine.nrows : 0, k0 | (count << 8), i);
            }
            if (here) {
                ctl->first.index = i;
                ctl->first.it = mine;
                ctl->first_place = w0 - before;
            }
            before += tiles;
        }
        fence_proxy_async_smem();  // the scan's memory is the K ring's, which the async proxy writes next
        start.left = idle ? 0 : part_begin(pair + 1, W, G) - w0;
    } else {
        if (tid == 0) {
            ctl->first.index = p.n_items - 1 - pair;
            ctl->first.it = decode_item<SEARCH>(p, p.n_items - 1 - pair);  // no more pairs than items
            ctl->first_place = 0;
        }
        start.left = pairs;
    }
    if (warp == kSourceWarp) {
        const int b = prefix_source(p, first_L, lane);
        if (lane == 0) ctl->prefix_source = b;
    }
    tc_fence_before();
    __syncthreads();
    start.item = ctl->first.index;
    start.tile = ctl->first_place;
    start.decoded = true;
    cluster_wait();  // the peer's barriers exist before anything arrives on them
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const int32_t* shared = p.page_table + (int64_t)ctl->prefix_source * p.max_pages;
    auto leader = [&](uint64_t* bar) { return mapa_shared(smem_u32(bar), 0); };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(kAllLanes, mbar_wait(bar, parity, p.err, p.wait_ns)) != 0;
    };
    const bool softmax_warp = warp >= kSoftmaxWarp && warp < kSoftmaxWarp + 4;
    bool ok = true;

    if (warp == 0) {
        // ---------------- loads: Q of a segment, then K(u) and V(u - 1) in the order of their use ----------------
        Walk w = start;
        Segment s = ctl->first;
        uint32_t seg = 0, kphase = 1, vphase = 1;  // a tile takes every slot of both rings once
        const uint32_t q_full = leader(&ctl->q_full), k_full = leader(&ctl->k_full[0]), v_full = leader(&ctl->v_full[0]);
        while (ok && next_segment<SEARCH>(p, w, s)) {
            Tile t = tile_of(p, shared, s.it, s.u0), tv = t;
            int page0 = page_of(t, 0), page1 = page_of(t, 1), vpage0 = 0, vpage1 = 0;
            if (seg > 0 && !(ok = wait(&ctl->q_empty, (seg - 1) & 1u))) break;
            if (elect_one_sync()) {
                if (KVFP8) {
                    mbar_arrive_expect_tx(&ctl->q_raw, kQAtoms * kAtom);
                    tma_load_3d(q_s, &qmap, &ctl->q_raw, 0, s.it.row0 + 64 * rank, 0);
                } else {
                    if (rank == 0) mbar_arrive_expect_tx(&ctl->q_full, 2 * kQAtoms * kAtom);
                    tma_pair_load_3d(q_s, &qmap, q_full, 0, s.it.row0 + 64 * rank, 0);
                }
            }
            ++seg;
            for (int u = s.u0; ok && u <= s.u1; ++u) {
                Tile tn = t;
                int next0 = kNoPage, next1 = kNoPage, later = kNoPage;
                if (u + 1 < s.u1) {
                    tn = tile_of(p, shared, s.it, u + 1);
                    next0 = page_of(tn, 0);
                    next1 = page_of(tn, 1);
                }
                if (u + 2 < s.u1 && (u + 2 >= s.it.tiles_a || p.row_tiles <= 2)) {
                    const Tile t2 = tile_of(p, shared, s.it, u + 2);
                    if (!t2.copied) later = page_of(t2, rank);
                }
                if (u < s.u1) {
                    // entries out of range are reported; behind the last page the copy writes zeros
                    const bool in0 = page0 >= 0 && page0 < p.num_pages, in1 = page1 >= 0 && page1 < p.num_pages;
                    if (((!in0 && page0 != kNoPage) || (!in1 && page1 != kNoPage)) && rank == 0 && lane == 0)
                        raise_error(p.err, DSA_DEVERR_PAGE);
                    if (!in0) page0 = p.num_pages;
                    if (!in1) page1 = p.num_pages;
                    if (KVFP8 && t.copied) {  // rows converted ahead lie in the order of their positions
                        page0 = t.base >> 6;
                        page1 = page0 + 1;
                    }
                    const int page = rank == 0 ? page0 : page1;
#pragma unroll
                    for (int j = 0; j < kKUnits; ++j) {
                        if (!(ok = wait(&ctl->k_empty[j], kphase))) break;
                        if (elect_one_sync()) {
                            constexpr int kBytes = unit_atoms<KVFP8>(0) * kAtom;
                            uint8_t* dst = k_s + j * kBytes;
                            const uint32_t bar = k_full + 8 * j;
                            if (KVFP8 && !t.copied) {
                                // the codes of four atoms into the middle two, or the rotary part (see the conversion)
                                if (rank == 0) mbar_arrive(&ctl->k_full[j]);
                                mbar_arrive_expect_tx(&ctl->k_raw[j], (j < 2 ? 2 : 1) * kAtom);
                                if (j < 2)
                                    tma_load_4d(dst + kAtom, &codemap, &ctl->k_raw[j], 0, 0, 2 * j, page);
                                else
                                    tma_load_3d(dst, &rotmap, &ctl->k_raw[j], kKvFp8RopeOff, 0, page);
                            } else {
                                if (rank == 0) mbar_arrive_expect_tx(&ctl->k_full[j], 2 * unit_atoms<KVFP8>(j) * kAtom);
                                tma_pair_load_4d(dst, KVFP8 && j < 2 ? &vmap : &kmap, bar, 0, 0, unit_atom<KVFP8>(j), page);
                            }
                        }
                    }
                    kphase ^= 1u;
                }
                if (ok && u > s.u0) {
#pragma unroll 1
                    for (int h = 0; h < kVSlots; ++h) {
                        if (!(ok = wait(&ctl->v_empty[h], vphase))) break;
                        if (elect_one_sync()) {
                            const int page = h == 0 ? vpage0 : vpage1;
                            uint8_t* dst = v_s + h * kVSlot;
                            if (KVFP8 && !tv.copied) {
                                if (rank == 0) mbar_arrive(&ctl->v_full[h]);
                                mbar_arrive_expect_tx(&ctl->v_raw[h], 2 * kAtom);
                                tma_load_4d(dst + kAtom, &codemap, &ctl->v_raw[h], 0, 0, 2 * rank, page);
                            } else if (!KVFP8 && tv.edge) {
                                // filled by the warps below, which have a barrier of their own
                                if (rank == 0) mbar_arrive(&ctl->v_full[h]);
                                mbar_arrive(&ctl->v_turn[h]);
                            } else {
                                if (rank == 0) mbar_arrive_expect_tx(&ctl->v_full[h], 2 * kVSlot);
                                tma_pair_load_4d(dst, &vmap, v_full + 8 * h, 0, 0, 4 * rank, page);
                            }
                        }
                    }
                    vphase ^= 1u;
                }
                // A ring holds one tile, so a copy is asked for about one tile before its use: less than HBM's latency.
                // The tile after the next is brought to L2, unless it is the prefix's and so in L2 for the other pairs.
                if (later >= 0 && later < p.num_pages && elect_one_sync()) {
                    const uint32_t bytes = 64 * (KVFP8 ? kKvFp8RowBytes : 1152);
                    l2_prefetch(p.kv_cache + (int64_t)later * bytes, bytes);
                }
                vpage0 = page0;
                vpage1 = page1;
                tv = t;
                page0 = next0;
                page1 = next1;
                t = tn;
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------- products: S(u) = Q K(u)^T, then O += P(u - 1) V(u - 1) ----------------
        Walk w = start;
        Segment s = ctl->first;
        uint32_t seg = 0, tile = 0, edges = 0, k_raws = 0, v_raws = 0;
        const uint64_t qd = smem_desc(smem_u32(q_s), 16, 1024, kSwizzle128B);
        const uint64_t kd = smem_desc(smem_u32(k_s), 16, 1024, kSwizzle128B);
        const uint64_t pd = smem_desc(smem_u32(p_s), 16, 1024, kSwizzle128B);
        const uint64_t vd = smem_desc(smem_u32(v_s), kAtom, 1024, kSwizzle128B);  // MN-major, atoms kAtom apart
        auto pv = [&](uint32_t n, bool first, bool edge, bool raw) {  // n: the tile's number among all of this pair's
            if (!wait(&ctl->p_full, n & 1u)) return false;
            if (!KVFP8 && edge && !wait(&ctl->edge_full, edges++ & 1u)) return false;
            if (first && seg > 1 && !wait(&ctl->o_free, seg & 1u)) return false;
#pragma unroll
            for (int h = 0; h < kVSlots; ++h) {
                if (!wait(&ctl->v_full[h], n & 1u)) return false;
                if (KVFP8 && raw && !wait(&ctl->v_conv[h], v_raws & 1u)) return false;
                tc_fence_after();
                if (elect_one_sync()) {
                    const uint64_t pa = pd + (uint64_t)(h * (kAtom / 16)), b = vd + (uint64_t)(h * (kVSlot / 16));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            umma_pair_f16_ss(tmem + 128 * j, pa + (uint64_t)(2 * kk),
                                             b + (uint64_t)(j * (2 * kAtom / 16) + 128 * kk), kIdescPV<KVFP8>,
                                             first && h == 0 && kk == 0 ? 0u : 1u);
                    umma_pair_commit(&ctl->v_empty[h], 3);
                    if (h == 1) umma_pair_commit(&ctl->pv_done, 3);
                }
            }
            if (raw) ++v_raws;
            return true;
        };
        while (ok && next_segment<SEARCH>(p, w, s)) {
            if (!(ok = wait(KVFP8 ? &ctl->q_conv : &ctl->q_full, seg & 1u))) break;
            ++seg;
            bool edge = false, raw = false;
            for (int u = s.u0; ok && u < s.u1; ++u, ++tile) {
                const uint32_t buf = tile & 1u;
                const bool last = u == s.u1 - 1;
                const Tile cur = tile_of(p, shared, s.it, u);
                const bool cur_raw = KVFP8 && !cur.copied;
                if (!(ok = wait(&ctl->s_empty[buf], ((tile >> 1) & 1u) ^ 1u))) break;
#pragma unroll
                for (int j = 0; j < kKUnits; ++j) {
                    if (!(ok = wait(&ctl->k_full[j], tile & 1u))) break;
                    if (KVFP8 && cur_raw && !(ok = wait(&ctl->k_conv[j], k_raws & 1u))) break;
                    tc_fence_after();
                    if (elect_one_sync()) {
                        constexpr uint32_t kStep = kAtom / 16;
                        const uint32_t d = tmem + kSCol + 64 * buf;
#pragma unroll
                        for (int kk = 0; kk < 4 * unit_atoms<KVFP8>(j); ++kk) {
                            const uint32_t at = (unit_atom<KVFP8>(j) + kk / 4) * kStep + 2 * (kk & 3);
                            umma_pair_f16_ss(d, qd + at, kd + at, kIdescQK<KVFP8>, j == 0 && kk == 0 ? 0u : 1u);
                        }
                        umma_pair_commit(&ctl->k_empty[j], 3);
                        if (j == kKUnits - 1) {
                            umma_pair_commit(&ctl->s_full[buf], 3);
                            if (last) umma_pair_commit(&ctl->q_empty, 3);
                        }
                    }
                }
                if (cur_raw) ++k_raws;
                if (ok && u > s.u0) ok = pv(tile - 1, u == s.u0 + 1, edge, raw);
                edge = cur.edge;
                raw = cur_raw;
            }
            if (ok) ok = pv(tile - 1, s.u1 == s.u0 + 1, edge, raw);
        }
        // drain (default limit): every product of the pair is done before its memory is given back
        if (elect_one_sync()) {
            umma_pair_commit(&ctl->drained, 1);
            mbar_wait(&ctl->drained, 0, p.err);
        }
        __syncwarp();
    } else if (softmax_warp) {
        // ---------------- softmax: thread (row, half of the positions) ----------------
        Walk w = start;
        Segment s = ctl->first;
        const int st = tid - 32 * kSoftmaxWarp;  // lane of tensor memory
        const int half = st >> 6, r = st & 63;
        const uint32_t trow = tmem + ((uint32_t)(st & ~31) << 16);
        const uint32_t s_empty = leader(&ctl->s_empty[0]), p_full = leader(&ctl->p_full), o_free = leader(&ctl->o_free);
        const uint32_t p_row = smem_u32(p_s) + half * kAtom + r * 128;
        uint32_t tile = 0, swaps = 0, seg = 0;
        // A value of the row's other half (tensor-memory lane st ^ 64).  Two buffers, and a bounded wait instead
        // of a block barrier, so that a warp that has given up stops no other.
        auto swap = [&](float mine, float* other) {
            ctl->exchange[swaps & 1u][st] = mine;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->exchanged);
            if (!wait(&ctl->exchanged, swaps & 1u)) return false;
            *other = ctl->exchange[swaps & 1u][st ^ 64];
            ++swaps;
            return true;
        };
        bool have = next_segment<SEARCH>(p, w, s);
        int first_pg = have ? page_of(tile_of(p, shared, s.it, s.u0), half) : kNoPage;
        while (have) {
            const int tr = 64 * rank + r;  // row of the tile
            // positions this row sees: below `limit`
            const int limit = s.it.b < 0 ? p.prefix_len : s.it.pos0 + (s.it.lrow0 + tr) / p.heads + 1;
            float m_used = -INFINITY, l_sum = 0.f;
            Tile t = tile_of(p, shared, s.it, s.u0);
            int pg = first_pg;
#pragma unroll 1
            for (int u = s.u0; u < s.u1; ++u, ++tile) {
                const uint32_t buf = tile & 1u;
                const Tile cur = t;
                const bool bad_page = pg < 0 || pg >= p.num_pages;
                if (u + 1 < s.u1) {
                    t = tile_of(p, shared, s.it, u + 1);
                    pg = page_of(t, half);
                }
                if (!(ok = wait(&ctl->s_full[buf], (tile >> 1) & 1u))) break;
                tc_fence_after();
                float sv[64];
                {
                    float a0[16], a1[16], a2[16], a3[16];
                    const uint32_t col = trow + kSCol + 64 * buf;
                    tmem_ld16(col, a0);
                    tmem_ld16(col + 16, a1);
                    tmem_ld16(col + 32, a2);
                    tmem_ld16(col + 48, a3);
                    tmem_ld_wait();
                    tmem_regs_ready(a0);
                    tmem_regs_ready(a1);
                    tmem_regs_ready(a2);
                    tmem_regs_ready(a3);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        sv[j] = a0[j];
                        sv[16 + j] = a1[j];
                        sv[32 + j] = a2[j];
                        sv[48 + j] = a3[j];
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(s_empty + 8 * buf);
                if (cur.edge || bad_page) {
                    const int first = cur.base + 64 * half;
                    const int lo = bad_page ? 64 : cur.lo - first, hi = min(cur.hi, limit) - first;
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (j < lo || j >= hi) sv[j] = -INFINITY;
                }
                float mx[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) mx[k] = fmaxf(fmaxf(sv[k], sv[k + 16]), fmaxf(sv[k + 32], sv[k + 48]));
#pragma unroll
                for (int n = 8; n > 0; n >>= 1)
#pragma unroll
                    for (int k = 0; k < n; ++k) mx[k] = fmaxf(mx[k], mx[k + n]);
                float other;
                if (!(ok = swap(mx[0], &other))) break;
                const float mt = fmaxf(mx[0], other) * p.scale_log2;
                const bool raise = mt > m_used + kRaise<KVFP8>;
                const float m_new = raise ? mt : m_used;
                const float alpha = (raise && m_used != -INFINITY) ? exp2f(m_used - m_new) : 1.f;
                const float mu = m_new == -INFINITY ? 0.f : m_new - kLift<KVFP8>;  // nothing seen yet: exp2(-inf) = 0
                // weights: the sum takes the fp32 values, the products their rounding to bf16 or f16 (at most
                // 2^-8 or 2^-11 of each, unbiased), so that lse keeps fp32 accuracy
                uint32_t packed[32];
                float ps[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    const float e0 = exp2_fast(fmaf(sv[j], p.scale_log2, -mu));
                    const float e1 = exp2_fast(fmaf(sv[j + 1], p.scale_log2, -mu));
                    packed[j / 2] = KVFP8 ? f2_to_h2(e0, e1) : f2_to_bf2(e0, e1);
                    ps[(j / 2) & 7] += e0 + e1;
                }
                const float rs = ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
                // the previous tile's P V is done: P may be overwritten, O is still
                if (tile > 0 && !(ok = wait(&ctl->pv_done, (tile - 1) & 1u))) break;
                tc_fence_after();
                if (u > s.u0 && __any_sync(kAllLanes, alpha != 1.f)) {
#pragma unroll 1
                    for (int c = 0; c < 256; c += 16) {
                        float o[16];
                        tmem_ld16(trow + c, o);
                        tmem_ld_wait();
                        tmem_regs_ready(o);
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] *= alpha;
                        tmem_st16(trow + c, o);
                    }
                    tmem_st_wait();
                }
                l_sum = l_sum * alpha + rs;
                m_used = m_new;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    st_shared_v4(p_row + ((c ^ (r & 7)) << 4),
                                 make_uint4(packed[4 * c], packed[4 * c + 1], packed[4 * c + 2], packed[4 * c + 3]));
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(p_full);
            }
            if (!ok) break;
            // the next segment, looked up while this one's last products run
            Segment ahead = s;
            have = next_segment<SEARCH>(p, w, ahead);
            if (have) first_pg = page_of(tile_of(p, shared, ahead.it, ahead.u0), half);
            // ---- the segment's result: O / l and lse, or O, m and l for the combining kernel ----
            if (!(ok = wait(&ctl->pv_done, (tile - 1) & 1u))) break;
            tc_fence_after();
            float other;
            if (!(ok = swap(l_sum, &other))) break;
            float l = half == 0 ? l_sum + other : other + l_sum;  // the same sum in both halves
            if (!KVFP8) {
                // An infinite value of weight 0 is NaN where V comes as it is; V of edge tiles had it cleaned, so that the rows
                // that do not see it are not, and those that do become NaN here.
                const unsigned long long bad = *const_cast<volatile unsigned long long*>(&ctl->cleaned[++seg & 1u]);
                if ((uint32_t)(bad >> 32) == seg && limit > INT32_MAX - (int)(uint32_t)bad) l = NAN;
            }
            const float m = m_used - kLift<KVFP8>;  // what O and l are relative to
            const bool whole = s.u0 == 0 && s.u1 == s.it.tiles_a + s.it.tiles_b && !p.packed;
            float* slot = p.partial + partial_slot(p, s.index, pair, s.u0 == 0) * kPartialFloats;
            constexpr float kTakeOut = KVFP8 ? 1.f / kF16Gain : 1.f;
            const float inv = l == 0.f ? 0.f : kTakeOut / l;
            // A thread holds 256 values of its row.  They pass through this warp's part of the P memory, 128 bytes
            // a row at a time, so that a store instruction writes four whole 128-byte lines (row by row it touched
            // 32, and took 6400 cycles a segment).
            const uint32_t stage = smem_u32(p_s) + half * kAtom + (r & 32) * 128;
            const int sub = lane >> 3, piece = lane & 7, row_first = 64 * rank + (r & 32);
            auto write_lines = [&](uint8_t* dst, int64_t pitch) {  // dst: this warp's first row, its 128 bytes
                __syncwarp();
                uint4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int lr = 4 * k + sub;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v[k].x), "=r"(v[k].y), "=r"(v[k].z), "=r"(v[k].w)
                                 : "r"(stage + lr * 128 + ((piece ^ (lr & 7)) << 4))
                                 : "memory");
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (row_first + 4 * k + sub < s.it.nrows)
                        *reinterpret_cast<uint4*>(dst + (4 * k + sub) * pitch + 16 * piece) = v[k];
                __syncwarp();
            };
            if (row_first >= s.it.nrows) {
                // none of this warp's rows exists
            } else if (whole) {
                uint8_t* dst = reinterpret_cast<uint8_t*>(p.out + ((int64_t)s.it.row0 + row_first) * 512 + 256 * half);
#pragma unroll 1
                for (int c = 0; c < 256; c += 64) {
                    float o[4][16];
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_ld16(trow + c + 16 * k, o[k]);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_regs_ready(o[k]);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float* v = &o[k >> 1][8 * (k & 1)];
                        st_shared_v4(p_row + ((k ^ (r & 7)) << 4),
                                     make_uint4(f2_to_bf2(v[0] * inv, v[1] * inv), f2_to_bf2(v[2] * inv, v[3] * inv),
                                                f2_to_bf2(v[4] * inv, v[5] * inv), f2_to_bf2(v[6] * inv, v[7] * inv)));
                    }
                    write_lines(dst + 2 * c, 1024);
                }
                if (tr < s.it.nrows && half == 0 && p.lse)
                    p.lse[(int64_t)s.it.row0 + tr] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            } else {
                uint8_t* dst = reinterpret_cast<uint8_t*>(slot + row_first * 512 + 256 * half);
                float o[2][16];
                tmem_ld16(trow, o[0]);
                tmem_ld16(trow + 16, o[1]);
#pragma unroll 1
                for (int c = 0; c < 256; c += 32) {
                    tmem_ld_wait();
                    tmem_regs_ready(o[0]);
                    tmem_regs_ready(o[1]);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float* v = &o[k >> 2][4 * (k & 3)];
                        st_shared_v4(p_row + ((k ^ (r & 7)) << 4),
                                     make_uint4(__float_as_uint(v[0] * kTakeOut), __float_as_uint(v[1] * kTakeOut),
                                                __float_as_uint(v[2] * kTakeOut), __float_as_uint(v[3] * kTakeOut)));
                    }
                    if (c + 32 < 256) {  // the next ones come while these are written
                        tmem_ld16(trow + c + 32, o[0]);
                        tmem_ld16(trow + c + 48, o[1]);
                    }
                    write_lines(dst + 4 * c, 2048);
                }
                if (tr < s.it.nrows && half == 0) reinterpret_cast<float2*>(slot + 128 * 512)[tr] = make_float2(m, l);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(o_free);
            s = ahead;
        }
    } else if (!KVFP8 && warp >= kFillWarp) {
        // ---------------- V of edge tiles, through registers ----------------
        Walk w = start;
        Segment s = ctl->first;
        const int fw = warp - kFillWarp;
        static_assert(kFillWarps == 4, "16 rows of a page each");
        const uint32_t edge_full = leader(&ctl->edge_full);
        // The ring does not wait for these warps at other tiles, so its own phases may pass them by (a parity names one
        // of two phases).  v_turn has one phase for each edge tile, and the ring stays there until the tile is filled.
        uint32_t turn = 0, seg = 0;
        static_assert(kVSlots == 2, "one slot for each page of a tile");
        while (ok && next_segment<SEARCH>(p, w, s)) {
            ++seg;
            for (int u = s.u0; ok && u < s.u1; ++u) {
                const Tile t = tile_of(p, shared, s.it, u);
                if (!t.edge) continue;
                int bad = INT32_MAX;  // first position that this lane has to clean
                // A row of 32 chunks (8 dims) at a time; rows 16 fw .. 16 fw + 15 of both pages are this warp's.  All is
                // loaded and looked at before the slots are waited for: only the stores are on the way to the products.
                const int row0 = 16 * fw;
                uint4 v[2][16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int pg = page_of(t, h), pos = t.base + 64 * h + row0;
                    const bool in = pg >= 0 && pg < p.num_pages;
                    const uint8_t* src = p.kv_cache + ((int64_t)(in ? pg : 0) * 64 + row0) * 1152 + 512 * rank + 16 * lane;
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        v[h][k] = in && pos + k >= t.lo && pos + k < t.hi ? ld_input(reinterpret_cast<const uint4*>(src + 1152 * k))
                                                                          : make_uint4(0, 0, 0, 0);
                }
                uint32_t found = 0;  // an exponent of all ones carries into the sign bit's place
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const uint32_t c = 0x7F807F80u, one = 0x00800080u;
                        found |= ((v[h][k].x & c) + one) | ((v[h][k].y & c) + one) | ((v[h][k].z & c) + one) |
                                 ((v[h][k].w & c) + one);
                    }
                if (__any_sync(kAllLanes, (found & 0x80008000u) != 0)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const uint4 old = v[h][k];
                            v[h][k] = make_uint4(finite2(old.x), finite2(old.y), finite2(old.z), finite2(old.w));
                            if (((v[h][k].x ^ old.x) | (v[h][k].y ^ old.y) | (v[h][k].z ^ old.z) | (v[h][k].w ^ old.w)) != 0)
                                bad = min(bad, t.base + 64 * h + row0 + k);
                        }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!(ok = wait(&ctl->v_turn[h], turn & 1u))) break;
                    const uint32_t dst = smem_u32(v_s + h * kVSlot + (lane >> 3) * kAtom) + row0 * 128;
#pragma unroll
                    for (int k = 0; k < 16; ++k) st_shared_v4(dst + k * 128 + (((lane & 7) ^ (k & 7)) << 4), v[h][k]);
                }
                if (!ok) break;
                ++turn;
                if (bad != INT32_MAX) {  // for both CTAs' softmax; the slot's last segment has ended (its successor's weights
                                         // are behind this tile)
                    const unsigned long long mark = (unsigned long long)seg << 32 | (uint32_t)(INT32_MAX - bad);
                    for (int r = 0; r < 2; ++r)
                        red_max_cluster(mapa_shared(smem_u32(&ctl->cleaned[seg & 1u]), r), mark);
                    asm volatile("fence.acq_rel.cluster;" ::: "memory");
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(edge_full);
            }
        }
    }
    if constexpr (KVFP8) {
        // ---------------- FP8 rows: codes times scales, as f16, into the K and V rings ----------------
        // The codes of a row of two atoms (128 dims, one scale) come by TMA into that row's place in one of the two, so
        // that a row is expanded inside what it will fill: of four atoms, codes 0-127 lie in atom 1, 128-255 in atom
        // 2.  Eight lanes of a warp take a row, 16 codes each; they read, meet, and write.  Four warps expand K (this
        // CTA's page), four V (both pages, this CTA's 256 dims), a row of every 16 each; the rotary part and, at the
        // start of a segment, q go from bf16 to f16 where they are.  Tiles converted ahead pass by.
        const int cw = warp < kSoftmaxWarp ? warp - 2 : warp - kFillWarp + 2;  // 0-3: K, 4-7: V
        if (cw >= 0 && !softmax_warp) {
            const bool v_side = cw >= kFillWarps;
            const int row0 = 4 * (cw & 3) + (lane >> 3), c = lane & 7;  // rows row0 + 16 i; (row & 7) is row0 & 7
            const uint32_t done = leader(v_side ? &ctl->v_conv[0] : &ctl->k_conv[0]), q_done = leader(&ctl->q_conv);
            uint64_t* raw = v_side ? ctl->v_raw : ctl->k_raw;
            const uint32_t ring = smem_u32(v_side ? v_s : k_s) + row0 * 128;
            const uint32_t own16 = (c ^ (row0 & 7)) << 4;  // this lane's 16 bytes of a swizzled row
            // scales of this lane's rows in the order of use: K the four scale tiles of a row, V two of each page
            auto load_scales = [&](const Tile& t, float (&sc)[4][4]) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int pg = page_of(t, v_side ? h : rank);
                    const bool in = pg >= 0 && pg < p.num_pages;
                    const uint8_t* src = p.kv_cache + ((int64_t)(in ? pg : 0) * 64 + row0) * kKvFp8RowBytes + kKvFp8ScaleOff +
                                         (v_side ? 8 * rank : 8 * h);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 v = in ? ld_input(reinterpret_cast<const float2*>(src + 16 * i * kKvFp8RowBytes))
                                            : make_float2(0.f, 0.f);
                        sc[2 * h][i] = v.x;
                        sc[2 * h + 1][i] = v.y;
                    }
                }
            };
            Walk w = start;
            Segment s = ctl->first;
            uint32_t seg = 0, phase = 0;
            while (ok && next_segment<SEARCH>(p, w, s)) {
                // the first tile that is to be converted, and its scales, while q is on its way
                int u = p.ahead != nullptr ? max(s.u0, s.it.tiles_a) : s.u0;
                Tile t = tile_of(p, shared, s.it, min(u, s.u1 - 1));
                float next[4][4];
                if (u < s.u1) load_scales(t, next);
                if (!(ok = wait(&ctl->q_raw, seg++ & 1u))) break;
                uint32_t odd = 0;
#pragma unroll 3
                for (int i = 0; i < kQAtoms * 64 * 8 / (64 * kFillWarps); ++i) {  // 16-byte pieces, 256 lanes
                    const uint32_t at = smem_u32(q_s) + 16 * (32 * cw + lane + 256 * i);
                    const uint4 h = bf8_to_h8(ld_shared_v4(at), 1.f / kF16Gain);
                    odd |= not_finite(h);
                    st_shared_v4(at, h);
                }
                if (odd) {  // hardly ever: infinities and NaN, or values beyond the range
#pragma unroll 1
                    for (int i = 0; i < kQAtoms * 64 * 8 / (64 * kFillWarps); ++i) {
                        const int n = 32 * cw + lane + 256 * i, row = (n >> 3) & 63, piece = 8 * (n >> 9) + ((n ^ row) & 7);
                        const int tr = 64 * rank + row;
                        if (tr >= s.it.nrows) continue;
                        const uint16_t* src = p.q + ((int64_t)s.it.row0 + tr) * 576 + 8 * piece;
                        if (!values_over(ld_input(reinterpret_cast<const uint4*>(src)), 1.f / kF16Gain)) continue;
                        st_shared_v4(smem_u32(q_s) + 16 * n, make_uint4(kNaN2, kNaN2, kNaN2, kNaN2));
                        // (items of the prefix hold tokens of no sequence, too; the others every row of one)
                        if (s.it.b >= 0) raise_error(p.err, DSA_DEVERR_RANGE);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(q_done);
                for (; ok && u < s.u1; ++u) {
                    const Tile cur = t;
                    uint32_t sc[4][4];  // f16 pairs
                    float largest = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            sc[j][i] = f2_to_h2(next[j][i] * kScaleGain, next[j][i] * kScaleGain);
                            largest = fmaxf(largest, fabsf(next[j][i]));
                        }
                    if (u + 1 < s.u1) {
                        t = tile_of(p, shared, s.it, u + 1);
                        load_scales(t, next);
                    }
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {  // two atoms each
                        if (!(q & 1) && !(ok = wait(&raw[q >> 1], phase))) break;
                        const uint32_t at = ring + (4 * (q >> 1)) * kAtom;
                        const uint32_t from = at + ((q & 1) ? 2 : 1) * kAtom;
                        const uint32_t to = at + ((q & 1) ? 2 : 0) * kAtom + (c >> 2) * kAtom;
                        uint4 code[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) code[i] = ld_shared_v4(from + 16 * i * 128 + own16);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint4 lo = codes_to_h8(code[i].x, code[i].y, sc[0][i]);
                            uint4 hi = codes_to_h8(code[i].z, code[i].w, sc[0][i]);
                            if (v_side && cur.edge) {  // V of positions that do not exist is 0, and infinities and NaN are
                                const int pos = cur.base + 64 * (q >> 1) + row0 + 16 * i;
                                const uint32_t keep = pos >= cur.lo && pos < cur.hi ? 0xFFFFFFFFu : 0u;
                                auto clean = [&](uint32_t v) { return finite2<0x7C00u>(v) & keep; };
                                lo = make_uint4(clean(lo.x), clean(lo.y), clean(lo.z), clean(lo.w));
                                hi = make_uint4(clean(hi.x), clean(hi.y), clean(hi.z), clean(hi.w));
                            }
                            st_shared_v4(to + 16 * i * 128 + (((2 * (c & 3)) ^ (row0 & 7)) << 4), lo);
                            st_shared_v4(to + 16 * i * 128 + (((2 * (c & 3) + 1) ^ (row0 & 7)) << 4), hi);
                            sc[0][i] = sc[1][i];
                            sc[1][i] = sc[2][i];
                            sc[2][i] = sc[3][i];
                        }
                        if (q & 1) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster(done + 8 * (q >> 1));
                        }
                    }
                    if (ok && !v_side) {
                        if (!(ok = wait(&raw[2], phase))) break;
                        uint32_t odd = largest > kLargestScale ? 1u : 0u;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t at = ring + 8 * kAtom + 16 * i * 128 + own16;
                            const uint4 h = bf8_to_h8(ld_shared_v4(at), kF16Gain);
                            odd |= not_finite(h);
                            st_shared_v4(at, h);
                        }
                        if (odd) {  // hardly ever: this lane's pieces of its rows that are beyond the range, if any (the NaN
                                    // goes to the rotary part, which is handed over last)
                            const int pg = page_of(cur, rank);
#pragma unroll 1
                            for (int i = 0; i < 4; ++i) {
                                const int row = row0 + 16 * i, pos = cur.base + 64 * rank + row;
                                if (pg < 0 || pg >= p.num_pages || pos < cur.lo || pos >= cur.hi) continue;
                                const uint8_t* src = p.kv_cache + ((int64_t)pg * 64 + row) * kKvFp8RowBytes;
                                bool over = values_over(ld_input(reinterpret_cast<const uint4*>(src + kKvFp8RopeOff) + c), kF16Gain);
#pragma unroll 1
                                for (int q = 0; q < 4; ++q)
                                    over |= codes_over(ld_input(reinterpret_cast<const uint4*>(src) + 8 * q + c),
                                                       ld_input(reinterpret_cast<const float*>(src + kKvFp8ScaleOff) + q));
                                if (!over) continue;
                                st_shared_v4(ring + 8 * kAtom + 16 * i * 128 + own16, make_uint4(kNaN2, kNaN2, kNaN2, kNaN2));
                                raise_error(p.err, DSA_DEVERR_RANGE);
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(done + 16);
                    }
                    phase ^= 1u;
                }
            }
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
    cluster_sync();  // neither CTA leaves before the other's products, copies and arrivals are done
    tc_fence_after();
    if (warp == 2) tmem_pair_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------------------------------------
// FP8 rows of the prefix to f16 (times kF16Gain), once for all the tiles of rows that attend to them: a warp per
// position, in the order of the positions (rows behind the prefix in its last page are zeros).  Bound by L2 and HBM:
// 656 bytes read, 1152 written a row; 16000 rows take 6 to 8 us with the launch.
// ---------------------------------------------------------------------------------------------------------
constexpr int kAheadWarps = 8;

__global__ void __launch_bounds__(32 * kAheadWarps) prefix_ahead_kernel(const PrefixParams p) {
    const int lane = threadIdx.x & 31;
    const int pos = blockIdx.x * kAheadWarps + (threadIdx.x >> 5);
    if (pos >= (p.prefix_len + 63) / 64 * 64) return;
    grid_dependency_wait();
    allow_dependent_launch();
    uint4* dst = reinterpret_cast<uint4*>(p.ahead + (int64_t)pos * 1152);
    // sequence 0's entry is the one as a rule: loaded beside the lengths that say so
    int pg = pos < p.prefix_len ? ld_input(p.page_table + (pos >> 6)) : -1;
    const int64_t b = prefix_source(p, first_length(p, lane), lane);
    if (b > 0 && pos < p.prefix_len) pg = ld_input(p.page_table + b * p.max_pages + (pos >> 6));
    const bool in = pg >= 0 && pg < p.num_pages;
    if (!in && pos < p.prefix_len && lane == 0) raise_error(p.err, DSA_DEVERR_PAGE);
    uint4 code = make_uint4(0, 0, 0, 0), rot = code;
    float scale = 0.f;
    if (in) {
        const uint8_t* src = p.kv_cache + ((int64_t)pg * 64 + (pos & 63)) * kKvFp8RowBytes;
        code = ld_input(reinterpret_cast<const uint4*>(src) + lane);
        scale = ld_input(reinterpret_cast<const float*>(src + kKvFp8ScaleOff) + (lane >> 3));
        if (lane < 8) rot = ld_input(reinterpret_cast<const uint4*>(src + kKvFp8RopeOff) + lane);
    }
    const uint32_t scale2 = f2_to_h2(scale * kScaleGain, scale * kScaleGain);
    dst[2 * lane] = codes_to_h8(code.x, code.y, scale2);
    dst[2 * lane + 1] = codes_to_h8(code.z, code.w, scale2);
    uint4 turned = bf8_to_h8(rot, kF16Gain);
    const bool over = codes_over(code, scale) || values_over(rot, kF16Gain);
    if (over) raise_error(p.err, DSA_DEVERR_RANGE);
    if (__any_sync(kAllLanes, over)) turned = make_uint4(kNaN2, kNaN2, kNaN2, kNaN2);
    if (lane < 8) dst[64 + lane] = turned;
}

// ---------------------------------------------------------------------------------------------------------
// Combination of partial results: a warp per row, four parts' loads in flight (two: 1.5 us slower for rows of ten
// parts).  Bound by latency (offsets, then parts) and L2: some 20 MB in about 7 us.
//   M = max m_k, L = sum_k l_k 2^(m_k - M), out = sum_k 2^(m_k - M) O_k / L, lse = (M + log2 L) ln 2
// ---------------------------------------------------------------------------------------------------------
// The units of work are four rows, a warp each, or one row of an item in many parts, which the block's warps share.
constexpr int kCombineThreads = 128;
constexpr int kCombineWarps = kCombineThreads / 32;
constexpr int kCombineBlocks = 608;  // the four blocks that each of 152 SMs holds
constexpr int kManyParts = 8;
constexpr int kPartsInFlight = 4;
// Packed rows' parts are shared by four or two warps up to so many tiles of rows: the fewer tiles, the more parts each is
// cut in (16384 positions, 1, 4, 6, 12 tiles: a warp a row 28.4, 31.8, 35.2, 49.9 us; two 24.6, 29.8, 34.2, 52.2; four
// 22.6, 28.4, 35.6, 54.1; 32741 positions, 8 tiles: 61.2, 60.3, 62.5).
constexpr int kFourTiles = 5;
constexpr int kTwoTiles = 8;

// One row's parts: those of its own item, then of the packed item over the prefix.
struct RowParts {
    int item0, k0, count0, tr0;
    int item1, k1, count1, tr1;
};

__device__ __forceinline__ const float* part_of_row(const PrefixParams& p, const RowParts& r, int i, int* tr) {
    const bool own = i < r.count0;
    const int j = own ? i : i - r.count0;
    *tr = own ? r.tr0 : r.tr1;
    return p.partial + partial_slot(p, own ? r.item0 : r.item1, (own ? r.k0 : r.k1) + j, j == 0) * kPartialFloats;
}

// Parts sub, sub + step, ... of a row: acc = sum 2^(m - M) O (lane: float4 number 32 k + lane), returns the weighted
// sum of the l.  M: the maximum over all of the row's parts.
__device__ __forceinline__ float add_parts(const PrefixParams& p, const RowParts& r, int sub, int step, float (&acc)[16],
                                           float* M_out, int lane) {
    const int parts = r.count0 + r.count1;
    int tr;
    float M = -INFINITY;
    for (int i = lane; i < parts; i += 32) {
        const float* slot = part_of_row(p, r, i, &tr);
        M = fmaxf(M, __ldcg(reinterpret_cast<const float2*>(slot + 128 * 512) + tr).x);
    }
    float Ls = 0.f, mu = 0.f;
    bool first = true;
    for (int i = sub; i < parts; i += kPartsInFlight * step) {
        float2 ml[kPartsInFlight];
        float4 o[kPartsInFlight][4];
#pragma unroll
        for (int n = 0; n < kPartsInFlight; ++n) {
            ml[n] = make_float2(-INFINITY, 0.f);
            if (i + n * step >= parts) continue;
            const float* slot = part_of_row(p, r, i + n * step, &tr);
            ml[n] = __ldcg(reinterpret_cast<const float2*>(slot + 128 * 512) + tr);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[n][k] = __ldcg(reinterpret_cast<const float4*>(slot + tr * 512) + 32 * k + lane);
        }
        if (first) {  // while they are on their way
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kAllLanes, M, off));
            mu = M == -INFINITY ? 0.f : M;
            first = false;
        }
#pragma unroll
        for (int n = 0; n < kPartsInFlight; ++n) {
            if (i + n * step >= parts) continue;
            const float wgt = exp2f(ml[n].x - mu);  // 0 for a part without a score
            Ls += ml[n].y * wgt;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[4 * k] += wgt * o[n][k].x;
                acc[4 * k + 1] += wgt * o[n][k].y;
                acc[4 * k + 2] += wgt * o[n][k].z;
                acc[4 * k + 3] += wgt * o[n][k].w;
            }
        }
    }
    *M_out = M;
    return Ls;
}

__device__ __forceinline__ void write_row(const PrefixParams& p, int row, const float (&acc)[16], float M, float Ls, int lane) {
    const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        reinterpret_cast<uint2*>(p.out + (int64_t)row * 512)[32 * k + lane] =
            make_uint2(f2_to_bf2(acc[4 * k] * inv, acc[4 * k + 1] * inv), f2_to_bf2(acc[4 * k + 2] * inv, acc[4 * k + 3] * inv));
    if (lane == 0 && p.lse) p.lse[row] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * kLn2;
}

// The sums of the `of` neighbouring warps that share a row's parts, in their order, in the first of them.
struct WarpSums {
    float4 acc[kCombineWarps][128];
    float norm[kCombineWarps];
};
template <int OF>
__device__ __forceinline__ void add_warps(WarpSums& sums, float (&acc)[16], float& Ls, int warp, int lane) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k)
        sums.acc[warp][32 * k + lane] = make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
    if (lane == 0) sums.norm[warp] = Ls;
    __syncthreads();
    if (warp % OF != 0) return;
#pragma unroll
    for (int w = 1; w < OF; ++w) {
        Ls += sums.norm[warp + w];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 v = sums.acc[warp + w][32 * k + lane];
            acc[4 * k] += v.x;
            acc[4 * k + 1] += v.y;
            acc[4 * k + 2] += v.z;
            acc[4 * k + 3] += v.w;
        }
    }
}

// Packed: every row has parts in two items, which OF warps share.
template <int OF>
__global__ void __launch_bounds__(kCombineThreads) prefix_combine_packed_kernel(const PrefixParams p) {
    __shared__ WarpSums sums;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = (int)blockIdx.x * (kCombineWarps / OF) + warp / OF;
    const bool exists = row < p.total_q * p.heads;
    grid_dependency_wait();
    const int2* parts = reinterpret_cast<const int2*>(p.plan + 4 * kPrefixPairs);
    const int2 packed = exists ? __ldcg(parts + row / 128) : make_int2(0, 0);
    const int t = exists ? row / p.heads : -1;
    int b = -1, c0 = 0, n = 0, L = 0;
    for (int j0 = 0; j0 < p.batch && b < 0; j0 += 128) {  // four loads on their way
        int from[4], to[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + 32 * i + lane;
            from[i] = j < p.batch ? ld_input(p.cu_q_lens + j) : INT32_MAX;
            to[i] = j < p.batch ? ld_input(p.cu_q_lens + j + 1) : 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t hit = __ballot_sync(kAllLanes, from[i] <= t && t < to[i]);
            if (hit && b < 0) b = j0 + 32 * i + __ffs(hit) - 1;
        }
    }
    const bool ok = exists && b >= 0 && sequence(p, b, &c0, &n, &L);  // (if not: reported by the attention kernel)
    float acc[16], M = -INFINITY, Ls = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
    if (ok) {
        const int local = row - c0 * p.heads;
        RowParts r;
        r.item0 = p.packed_tiles + (int)first_item(p, b, c0) + local / 128;
        r.item1 = row / 128;
        const int2 own = __ldcg(parts + r.item0);
        r.k0 = own.x;
        r.count0 = own.y;
        r.tr0 = local & 127;
        r.k1 = packed.x;
        r.count1 = packed.y;
        r.tr1 = row & 127;
        Ls = add_parts(p, r, warp % OF, OF, acc, &M, lane);
    }
    if (OF > 1) add_warps<OF>(sums, acc, Ls, warp, lane);
    if (ok && warp % OF == 0) write_row(p, row, acc, M, Ls, lane);
}

// Merged: only items in several parts, each described by the part that begins inside it first.
__global__ void __launch_bounds__(kCombineThreads) prefix_combine_merged_kernel(const PrefixParams p) {
    __shared__ int4 cut[kCombineThreads];
    __shared__ int first_unit[kCombineThreads + 1];
    __shared__ WarpSums sums;
    static_assert(kPrefixPairs <= kCombineThreads, "one thread for each part");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dependency_wait();
    const int4 d = tid > 0 && tid < kPrefixPairs ? __ldcg(reinterpret_cast<const int4*>(p.plan) + tid) : make_int4(0, 0, 0, 0);
    cut[tid] = d;
    const int units = (d.z >> 8) > kManyParts ? d.y : (d.y + 3) / 4;
    int incl = units;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(kAllLanes, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) sums.norm[warp] = __int_as_float(incl);
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += __float_as_int(sums.norm[w]);
    first_unit[tid + 1] = incl;
    if (tid == 0) first_unit[0] = 0;
    __syncthreads();
    const int total = first_unit[kCombineThreads];
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
        int lo = 0, hi = kCombineThreads;  // first_unit[lo] <= u < first_unit[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (first_unit[mid] <= u) lo = mid;
            else hi = mid;
        }
        const int4 c = cut[lo];
        const bool many = (c.z >> 8) > kManyParts;
        const int tr = many ? u - first_unit[lo] : 4 * (u - first_unit[lo]) + warp;
        RowParts r = {};
        r.item0 = c.w;
        r.k0 = c.z & 255;
        r.count0 = tr < c.y ? c.z >> 8 : 0;
        r.tr0 = tr;
        float acc[16], M;
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[k] = 0.f;
        float Ls = add_parts(p, r, many ? warp : 0, many ? kCombineWarps : 1, acc, &M, lane);
        if (!many) {
            if (tr < c.y) write_row(p, c.x + tr, acc, M, Ls, lane);
            continue;
        }
        add_warps<kCombineWarps>(sums, acc, Ls, warp, lane);
        if (warp == 0) write_row(p, c.x + tr, acc, M, Ls, lane);
    }
}

}  // namespace

// Which items there are and how they are divided: of three ways the one whose time is the shortest by this estimate, in
// tiles (an FP8 tile that is converted in passing counts as two) summed over the pairs.
//   whole:   the pairs take whole merged items in turn; each round of them lasts as long as its longest item.
//   divided: the line of merged items in equal parts, and kDivideCost for finding the parts and the second launch.
//   packed:  the same with the prefix passed over by fewer tiles of rows, and all results written and read as partial
//            ones: kPartCost each.
// Measured, us (bf16 unless it says FP8; B sequences x heads, prefix + up to so many own positions):
//                            whole   divided  packed
//   38 x 128,    0 + 1024     17.5     24.5
//   8 x 128,     0 + 2048     26.3     20.5
//   100 x 128,   0 + 1024     32.9     35.8
//   100 x 128,   0 + 2048     52.8     49.9
//   64 x 16,   512 +  512     18.5     25.0     23.2
//   64 x 16,  2048 +  512     33.1     37.9     25.3
//   64 x 64,  1024 +  512     23.7     34.0     32.4
//   16 x 64,  2048 +  512     31.1     23.3     23.0
//   38 x 128,  512 +  512     27.3     30.8              FP8
//   100 x 128,   0 +  896     52.9     46.5              FP8
// The lengths are known to the device alone, so every own context counts as long as the table allows.  Whole items last
// as long as the longest whatever the others are: they are taken up to kWholeTiles own tiles only, so that a batch with
// one long sequence among short ones loses no more than about half of what an even one gains.
//
// FP8 rows of the prefix are converted ahead where that saves more than kAheadGain tiles' conversions in passing (less
// two passes, for the launch, the rows' writing and reading): 8 x 128 behind 2048 positions 27.5 us ahead, 25.6 in
// passing; behind 4096 28.6 and 32.6; 4 x 128 behind 4096 26.7 and 23.6, behind 8192 28.0 and 30.7.
void plan_prefix(PrefixParams* p, int max_pages) {
    const int64_t rows = (int64_t)p->total_q * p->heads;
    p->prefix_tiles = (p->prefix_len + 127) / 128;
    p->packed_tiles = (int)((rows + 127) / 128);
    p->tiles_per_seq = (int)(((int64_t)p->max_q_len * p->heads + 127) / 128);
    const int64_t each = (int64_t)p->batch * p->tiles_per_seq;
    const int64_t most = (int64_t)p->packed_tiles + p->batch;  // tiles of the sequences' rows, whatever their lengths
    const int64_t items = min(each, most);
    const int64_t alone = min(items, (int64_t)p->total_q);  // (no token's heads take more than a tile)
    if (most < each) p->tiles_per_seq = 0;  // (see first_item)
    const int64_t own_tiles = ((int64_t)max_pages * 64 - (p->prefix_len & ~63) + 127) / 128;
    const int64_t longest = p->prefix_tiles + own_tiles;
    const int64_t own = own_tiles * (p->kv_fp8 ? 2 : 1);
    auto ahead = [&](int64_t row_tiles) { return p->kv_fp8 && (row_tiles - 2) * p->prefix_tiles > kAheadGain; };
    auto prefix = [&](int64_t row_tiles) { return (int64_t)p->prefix_tiles * (p->kv_fp8 && !ahead(row_tiles) ? 2 : 1); };
    const int64_t rounds = (alone + kPrefixPairs - 1) / kPrefixPairs;
    const int64_t whole = own_tiles > kWholeTiles ? INT64_MAX : rounds * kPrefixPairs * (own + prefix(alone) + kItemCost);
    const int64_t divided = alone * (own + prefix(alone) + kItemCost) + kPrefixPairs * kDivideCost;
    const int64_t packed = alone * (own + kItemCost) + p->packed_tiles * (prefix(p->packed_tiles) + kItemCost) +
                           (alone + p->packed_tiles) * kPartCost + kPrefixPairs * kDivideCost;
    // Many items are even enough by themselves where their contexts are alike (1000 x 128 with up to 3000 positions: 368 us
    // whole, 339 divided; two prompts of 4000 tokens, 16 heads, 1000 items: 482 and 508; 4096 tokens x 128 heads at 65536,
    // 4096 items: 42.3 ms and 43.5, as the whole ones read the same rows at a time), and every CTA scans them all for a
    // plan.  Packing saves more (2048 x 16 heads behind 4096, 2304 items: 369 us, 1350 whole): its limit is the 1 GB that
    // the partial results take.  Places on the line are counted in 32 bits.  Batches of few queries but for one sequence:
    // 64 x 128 heads at 1000 positions and one of 131072, 33 queries for another: 77 us divided, 1265 whole; 64 x 16
    // behind 32768, 512 queries for one: 408 us packed, 1580 whole.
    const bool fits = (items + p->packed_tiles) * (3 * longest + kItemCost) <= INT32_MAX;
    p->packed = fits && p->packed_tiles < alone && items + p->packed_tiles <= kPackItems && packed < divided && packed < whole;
    p->planned = p->packed || (fits && items <= kPlanItems && divided < whole);
    p->n_items = (int)(items + (p->packed ? p->packed_tiles : 0));
    p->slot_by_item = p->packed || (p->heads < 128 && p->n_items < kPrefixPairs);
    p->row_tiles = (int)(p->packed ? p->packed_tiles : alone);
    p->convert_ahead = ahead(p->row_tiles);
}

namespace {
size_t plan_bytes(int64_t items) { return ((size_t)(2 * items + 4 * kPrefixPairs) * sizeof(int32_t) + 255) / 256 * 256; }
size_t ahead_bytes(int prefix_len) { return ((size_t)prefix_len + 63) / 64 * 64 * 1152; }
}  // namespace

size_t prefix_plan_bytes(const PrefixParams& p) { return p.planned ? plan_bytes(p.n_items) : 0; }
size_t prefix_partial_bytes(const PrefixParams& p) {
    if (!p.planned) return 0;
    return (size_t)(p.slot_by_item ? p.n_items + kPrefixPairs : 2 * kPrefixPairs) * kPartialFloats * sizeof(float);
}
size_t prefix_ahead_bytes(const PrefixParams& p) { return p.convert_ahead ? ahead_bytes(p.prefix_len) : 0; }

// Which way is taken jumps back and forth with the sizes (8 sequences of 2048 positions are divided, 38 are taken whole,
// without any partial result), and a program keeps one workspace for its largest step.  So what is asked for is the
// most that any call takes with no larger batch, total_q, max_q_len, prefix_len and max_pages: from the rules above,
//   divided: one item is the likeliest case (it leaves 75 pairs idle), and no way of splitting the longest context
//     into prefix and own positions has more than tiles + 1 tiles;
//   packed: with 128 heads there are as many packed tiles as tiles of sequences, so never; else, y being the prefix
//     tiles' cost, packed_tiles (y + 4) + alone < alone y and alone <= packed_tiles + batch leave fewer than
//     batch (y - 1) / 5 packed tiles;
//   converted ahead: for the longest prefix and the most row tiles, if at all.
size_t prefix_workspace_bound(const PrefixParams& p, int max_pages) {
    const int64_t each = (int64_t)p.batch * (((int64_t)p.max_q_len * p.heads + 127) / 128);
    const int64_t items = min(each, (int64_t)p.packed_tiles + p.batch);
    const int64_t tiles = ((int64_t)max_pages + 1) / 2, weight = p.kv_fp8 ? 2 : 1;
    const int64_t longest = weight * (tiles + (p.prefix_len > 0 ? 1 : 0)) + kItemCost;
    int64_t most_items = 0, slots = 0;
    if (tiles > kWholeTiles || (kPrefixPairs - 1) * longest > kPrefixPairs * kDivideCost) {
        most_items = min(items, (int64_t)kPlanItems);
        slots = p.heads == 128 ? 2 * kPrefixPairs : min(items + kPrefixPairs, (int64_t)2 * kPrefixPairs);
    }
    const int64_t y = weight * p.prefix_tiles;
    const int64_t packed = min((int64_t)p.packed_tiles, (p.batch * (y - 1) - 1) / 5);
    if (p.heads < 128 && y > 1 && packed > 0) {
        const int64_t n = min(packed + min(each, packed + p.batch), (int64_t)kPackItems);
        most_items = max(most_items, n);
        slots = max(slots, n + kPrefixPairs);
    }
    const bool ahead = p.kv_fp8 && (max(items, (int64_t)p.packed_tiles) - 2) * p.prefix_tiles > kAheadGain;
    return (slots > 0 ? plan_bytes(most_items) : 0) + (size_t)slots * kPartialFloats * sizeof(float) +
           (ahead ? ahead_bytes(p.prefix_len) : 0);
}

cudaError_t launch_prefix(const PrefixLaunch& L, cudaStream_t stream) {
    const PrefixParams& p = L.params;
    const bool search = p.tiles_per_seq == 0;
    auto kernel = p.kv_fp8 ? (search ? prefix_pair_kernel<true, true> : prefix_pair_kernel<true, false>)
                           : (search ? prefix_pair_kernel<false, true> : prefix_pair_kernel<false, false>);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int pairs = (int)(p.planned ? kPrefixPairs : (p.n_items < kPrefixPairs ? p.n_items : kPrefixPairs));
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.convert_ahead) {
        cfg.gridDim = dim3((unsigned)((p.prefix_len + 63) / 64 * 64 / kAheadWarps));
        cfg.blockDim = dim3(32 * kAheadWarps);
        e = cudaLaunchKernelEx(&cfg, prefix_ahead_kernel, p);
        if (e != cudaSuccess) return e;
    }
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3((unsigned)(p.kv_fp8 ? kThreads<true> : kThreads<false>));
    cfg.dynamicSmemBytes = kSmem;
    e = cudaLaunchKernelEx(&cfg, kernel, L.qmap, L.kmap, L.vmap, L.codemap, L.rotmap, p);
    if (e != cudaSuccess || !p.planned) return e;
    cfg.blockDim = dim3(kCombineThreads);
    cfg.dynamicSmemBytes = 0;
    if (p.packed) {
        const int of = p.packed_tiles <= kFourTiles ? 4 : p.packed_tiles <= kTwoTiles ? 2 : 1, rows = kCombineWarps / of;
        cfg.gridDim = dim3((unsigned)(((int64_t)p.total_q * p.heads + rows - 1) / rows));
        return cudaLaunchKernelEx(&cfg, of == 4   ? prefix_combine_packed_kernel<4>
                                        : of == 2 ? prefix_combine_packed_kernel<2>
                                                  : prefix_combine_packed_kernel<1>, p);
    }
    cfg.gridDim = dim3(kCombineBlocks);
    return cudaLaunchKernelEx(&cfg, prefix_combine_merged_kernel, p);
}

}  // namespace dsa
