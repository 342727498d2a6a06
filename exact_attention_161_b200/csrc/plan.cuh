// plan.cuh -- the work of a batch of packed sequences, cut into items on the device.
//
// The lengths of packed sequences are device data (offsets cu[0..S], and for the paged cache the
// lengths seq_lens), so the list of work items is built on the device by one CTA in front of the
// attention kernel, which then only walks the list:
//   forward   an item is a block of up to 2 TT consecutive tokens of one sequence (two 128-row query
//             tiles; TT = 128 / G tokens times the G query heads of a K/V head fill a tile) against a
//             range of 128-key tiles. Each item stands for every K/V head.
//   backward  an item is one 128-key tile of one sequence.
// Forward items are listed longest first (a counting sort by what they cost), and a CTA that is done with
// one takes the next, so that all finish together. Backward tiles are listed sequence by sequence, the
// longest first, so that the sequences' queries and dq sums stay in L2 while their tiles are worked on. Where the longest blocks would leave most CTAs idle at the end,
// long forward blocks are cut into parts along the keys; the warp that finishes a block's last part
// joins the parts' softmax states in ascending order, so the result depends on the lengths alone, not
// on timing.
//
// The index arithmetic is host code too, so that it can be checked without a GPU.
#pragma once
#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define ATTN_HD __host__ __device__ __forceinline__
#else
#define ATTN_HD inline
#endif

namespace attn {

constexpr int kPlanSms = 148;        // CTAs the split rule plans for (fixed: results never depend on the device)
// Parts per CTA the split rule aims at. Against 1: 8 tokens on 4,000 each 51 us (58), one on 32,000 63 us (54);
// against 4: one prompt of 4,000 tokens 139 us (209), 64 tokens of 512 to 16,384 and four chunks 336 us (380).
constexpr int kPlanWaves = 2;
constexpr int kPlanMinTiles = 4;     // no part is planned shorter than this many key tiles
constexpr int kPlanMaxParts = 1023;  // of one block (the record's part fields are 10 bits wide)
constexpr int kPlanBuckets = 1024;   // of the counting sort
// What cutting costs a call (partial states, joining them), in steps: one prompt of 1,500 tokens takes 41 us
// whole and 78 us cut (kPlanJoinTiles 3); one token on 2,000 takes 37 us whole and 29 us cut.
constexpr int kPlanJoinTiles = 6;
constexpr int kPlanJoinFew = 2;      // where no block that is cut has more than 32 rows

ATTN_HD int plan_min(int a, int b) { return a < b ? a : b; }
ATTN_HD int plan_max(int a, int b) { return a > b ? a : b; }
ATTN_HD int plan_ceil(int a, int b) { return (a + b - 1) / b; }
ATTN_HD int plan_ceil_div(long long a, int b) { return static_cast<int>((a + b - 1) / b); }

// One forward item: tokens [q_row, q_row + n_tok) of the packed queries, the first of them at
// position pos0 of its sequence, against key tiles [jb, jb + n_tiles) of the sequence.
struct PackedItem {
    int q_row;
    int pos0;
    int kv;       // packed: row of the sequence's first key; paged: the sequence's number
    int kv_len;   // keys of the sequence; -1: an invalid length, the rows are set to NaN
    int jb, n_tiles;
    int meta;     // n_tok | part << 10 | (parts - 1) << 20
    int slot;     // partial-state slot of part 0 (blocks of more than one part)
};
ATTN_HD int item_tokens(const PackedItem& x) { return x.meta & 1023; }
ATTN_HD int item_part(const PackedItem& x) { return (x.meta >> 10) & 1023; }
ATTN_HD int item_parts(const PackedItem& x) { return ((x.meta >> 20) & 1023) + 1; }
ATTN_HD int make_meta(int n_tok, int part, int parts) { return n_tok | (part << 10) | ((parts - 1) << 20); }

// One tile of 128 keys of a packed sequence, for the backward: rows [row0 + 128 t, ...) of a sequence of n
// rows that starts at row0; base is the number of the sequence's first query tile (of TT tokens).
struct PackedTile {
    int row0, n, t, base;
};

// Head of a plan in the workspace.
struct PlanHeader {
    int n_items;   // forward items (each for every K/V head); backward key tiles; 0 with invalid offsets
    int taken;     // items taken beyond the first of every CTA
    int pad[2];
};

// Key tiles visible to tokens [first, last] (positions) of a sequence of kv_len keys: [jb, jb + n).
struct KeyTiles {
    int jb, n;
};
ATTN_HD KeyTiles key_tiles(int first, int last, int kv_len, int causal, int window) {
    const int hi = causal ? plan_min(kv_len, last + 1) : kv_len;                  // exclusive
    const int lo = window > 0 ? plan_max(0, first - plan_min(window, first + 1) + 1) : 0;  // inclusive
    KeyTiles t;
    t.jb = lo / 128;
    t.n = plan_ceil(hi, 128) - t.jb;
    return t;
}

// Query tiles (TT tokens each) of a sequence of n tokens that see some key of key tile t: [ib, ie).
ATTN_HD void query_tiles(int t, int n, int TT, int causal, int window, int& ib, int& ie) {
    ib = causal ? t * 128 / TT : 0;
    ie = plan_ceil(n, TT);
    // the last query that sees the tile's last key is window - 1 rows after it
    if (window > 0 && window < n) ie = plan_min(ie, (t * 128 + 127 + window - 1) / TT + 1);
}

// What `tiles` key tiles cost, in steps of a CTA (one key tile for both query tiles): a block of one
// query tile (at most TT tokens) has both halves of its keys worked on at once, so a step takes two of
// its tiles; 5/8 and not 1/2, because it also reads two tiles a step.
ATTN_HD int plan_cost(int tiles, int one_tile) { return one_tile ? (5 * tiles + 7) / 8 : tiles; }

// Longest part the split rule leaves: the whole call's cost (every K/V head) over kPlanWaves
// parts per CTA, at least kPlanMinTiles.
ATTN_HD int plan_limit(long long cost_per_head, int Hkv) {
    const long long share = (cost_per_head * Hkv + kPlanWaves * kPlanSms - 1) / (kPlanWaves * kPlanSms);
    return share < kPlanMinTiles ? kPlanMinTiles : share > 0x3fffffff ? 0x3fffffff : static_cast<int>(share);
}
ATTN_HD int plan_parts(int cost, int limit) {
    const int p = cost > limit ? plan_ceil(cost, limit) : 1;
    return p > kPlanMaxParts ? kPlanMaxParts : p;
}
// Part i of `parts` over `tiles` tiles: [begin, end), sizes differing by at most one.
ATTN_HD void plan_part(int tiles, int parts, int i, int& begin, int& end) {
    const int q = tiles / parts, r = tiles % parts;
    begin = i * q + plan_min(i, r);
    end = begin + q + (i < r ? 1 : 0);
}

// Partial-state slots a plan can need (each for every K/V head): a block is cut only when it costs
// more than `limit`, and then into fewer than 2 cost / limit parts; summed over the blocks
// that is less than 2 kPlanWaves kPlanSms / Hkv. Nor can `blocks` blocks of at most max_tiles tiles
// be cut into more than blocks * ceil(max_tiles / kPlanMinTiles) parts.
// (No block costs more than its tiles.)
ATTN_HD long long plan_slots(long long blocks, long long max_tiles, int Hkv) {
    if (max_tiles <= kPlanMinTiles) return 0;
    const long long a = 2LL * kPlanWaves * kPlanSms / Hkv + 1;
    const long long b = blocks * ((max_tiles + kPlanMinTiles - 1) / kPlanMinTiles);
    return a < b ? a : b;
}

constexpr int kPlanWarps = 8;  // softmax warps, each with a counter of the parts it has finished
ATTN_HD size_t plan_up(size_t x) { return (x + 255) / 256 * 256; }

// Byte offsets of a forward plan in the workspace.
struct PlanLayout {
    size_t header, prefix, items, count, ml, o, total;
    long long max_items, max_slots;
};
// T packed query tokens in S sequences, TT tokens to a query tile, at most max_keys keys to a sequence.
ATTN_HD PlanLayout plan_layout(long long T, long long S, int TT, long long max_keys, int Hkv, int D) {
    PlanLayout L;
    const long long blocks = T / (2 * TT) + (S < T ? S : T);
    L.max_slots = plan_slots(blocks, (max_keys + 127) / 128, Hkv);
    L.max_items = blocks + L.max_slots;
    L.header = 0;
    L.prefix = 256;
    L.items = L.prefix + plan_up(static_cast<size_t>(S + 1) * sizeof(int));
    L.count = L.items + plan_up(static_cast<size_t>(L.max_items) * sizeof(PackedItem));
    L.ml = L.count + plan_up(static_cast<size_t>(L.max_slots) * Hkv * kPlanWarps * sizeof(int));
    const size_t rows = static_cast<size_t>(L.max_slots) * Hkv * 256;
    L.o = L.ml + plan_up(rows * 2 * sizeof(float));
    L.total = L.o + plan_up(rows * D * sizeof(float));
    return L;
}

// Byte offsets of a backward plan and its arrays: key tiles <= T / 128 + S, and query tiles of 128 rows
// (TT tokens times the query heads of a K/V head) for each K/V head, <= T / TT + S.
struct BwdPlanLayout {
    size_t header, prefix, start, base, tiles, order, vec, dqacc, total;
    long long max_tiles, max_q_tiles;
};
ATTN_HD BwdPlanLayout bwd_plan_layout(long long T, long long S, int TT, int Hkv, int D) {
    BwdPlanLayout L;
    L.max_tiles = T / 128 + (S < T ? S : T);
    L.max_q_tiles = T / TT + (S < T ? S : T);
    L.header = 0;
    L.prefix = 256;
    L.start = L.prefix + plan_up(static_cast<size_t>(S + 1) * sizeof(int));
    L.base = L.start + plan_up(static_cast<size_t>(S) * sizeof(int));
    L.tiles = L.base + plan_up(static_cast<size_t>(S) * sizeof(int));
    L.order = L.tiles + plan_up(static_cast<size_t>(L.max_tiles) * sizeof(PackedTile));
    L.vec = L.order + plan_up(static_cast<size_t>(L.max_tiles) * sizeof(int));
    const size_t rows = static_cast<size_t>(L.max_q_tiles) * Hkv * 128;
    L.dqacc = L.vec + plan_up(rows * 2 * sizeof(float));
    L.total = L.dqacc + plan_up(rows * D * sizeof(float));
    return L;
}

}  // namespace attn
