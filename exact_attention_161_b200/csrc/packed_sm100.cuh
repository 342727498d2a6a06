// packed_sm100.cuh -- attention over packed sequences of different lengths, and over chunks of new
// tokens on a paged KV cache, for sm_100a.
//
// Tokens of all sequences lie one behind the other (token-major [T, H, D] rows); sequence s owns
// rows [cu[s], cu[s+1]) of the queries. Its keys are its own rows (packed) or its pages of the cache
// (paged), of which its queries are the last ones. Per row the computation is the online softmax of
// fwd_sm100.cuh; what differs is how work is cut and fed:
//
//   Rows.  A query tile's 128 rows are TT = 128 / G tokens times the G query heads of one K/V head
//     (row r = token r / G, head r % G), loaded by one TMA box of {64 columns, G heads, TT tokens} per
//     128-byte region. Short sequences and single tokens then fill G times more of a tile, and a
//     K/V tile is read once for the whole group. (G that does not divide 128 leaves 128 - G TT rows
//     of every tile unused: 2 for G = 3, 8 for G = 5.)
//   Items. The list of plan.cuh, longest items first; one persistent CTA per SM takes the next when it is
//     nearly done with one.
//   Parts. A block whose keys were cut into parts writes fp32 partial states; of each group of 32 rows,
//     the warp that finishes last joins them in ascending order.
//   Sides. A block of at most TT tokens has one query tile. Both softmax warpgroups work on it, each with a
//     copy of the queries: steps alternate between the first and the second half of the item's key tiles,
//     and the first warpgroup joins both states out of Tensor Memory at the end. A tile of one warpgroup
//     alone takes as long as a tile of both, so this halves the time of single tokens and short chunks.
//   Pages. A 128-key tile of the cache is eight 16-token pages, each fetched by its own boxes; lane i
//     of a producer warp looks up and issues page i. K and V have a producer warp each.
//   Tails. A sequence ends inside a key tile; the rows behind its end belong to another sequence or
//     to nobody and may hold NaN. Scores are masked by selection. For P V, 0 * NaN would survive, so
//     the product stops at the last 16-key slice with a visible key (one MMA per slice), and the
//     rest of that slice's V rows are set to zero in shared memory by the softmax warps before P is
//     handed over.
//
// Roles: warps 0-3 and 4-7 softmax, 8 producer of Q, K and the work ring, 9 MMA issuer, then at D = 64 an
// issuer of the output products, then the producer of V. TMEM layout, issue order (D = 128) and softmax
// arithmetic are those of attn_fwd_kernel, but P is handed over in two halves, so that the product with the
// first runs while the second is computed (three long documents 2,243 -> 2,182 us; three quarters and one
// quarter measured the same at D = 128 and 10% slower at D = 64). P is rounded to bf16 because both operands of a
// product have one type and V is bf16: half a step, 2^-8 of each probability; its sum l is taken before the
// rounding. On normal inputs o is 0.0017 to 0.0023 from the fp64 result (2-norm, relative), where rounding the
// exact o once leaves 0.0017. All exponentials are the
// SFU's: an eighth or a sixteenth of them on the FMA pipe, as attn_fwd_kernel has it, measured the same or
// up to 5% slower here (with a polynomial of degree 4, as the sum of a few probabilities would show the
// error of one of degree 3), a quarter 10 to 18%.
//
// What bounds it (B200, measured with clock64 in a copy of the kernel):
//   D = 128, long sequences: the chain of one query tile from its scores through the softmax (1,900 clocks)
//     and its 16 products back to the next scores (1,500 to 1,650); two tiles share 2,048 clocks of tensor work
//     in a step of 3,300 to 3,500. Three documents of 4,000 to 12,000 tokens, 32 heads on 8: 2.68 TFLOP in
//     2,130 to 2,190 us, 1,220 to 1,260 TFLOP/s, 0.75 of the measured bf16 rate (attn_fwd_kernel 1,237 on one
//     sequence of 8,192).
//   Short sequences: 4,200 to 5,500 clocks an item outside its steps (the last tile's masks, the last
//     product, O to memory, the first scores): 24 prompts of 100 to 1,500 tokens 137 to 141 us, of which O's stores
//     cost 8 and the masks 4 (left out in copies).
//   D = 64: the exponentials (SFU 67% busy); 12 images of 200 to 3,300 patches 200 us, 590 TFLOP/s.
//   Single tokens: reading the keys, 64 on 16,000 tokens each 5.8 TB/s (0.89 of the copy rate).
// Registers: 168 a thread, all that 12 warps leave each other; 20 to 40 bytes a thread are spilled.
#pragma once
#include "common.cuh"
#include "fwd_sm100.cuh"
#include "plan.cuh"
#include "ptx.cuh"

namespace attn {

struct PlanParams {
    const int32_t* cu;        // [S + 1] offsets of the packed tokens
    const int32_t* seq_lens;  // paged: [S] keys of every sequence (its new tokens among them); packed: nullptr
    PlanHeader* header;
    int* prefix;              // [S + 1] blocks (backward: tiles) of the sequences before each
    PackedItem* items;
    int* count;               // finished parts of [slot of part 0][K/V head][softmax warp]
    PackedTile* tiles;        // backward: natural order
    int* order;               // backward: tile numbers, longest sequence first
    int* start;               // backward: [S] where each sequence's tiles stand in the order
    int* base;                // backward: [S] query tiles of the sequences before each
    int S, T, TT, Hkv, causal, window;
    int max_len;              // paged: tokens a block-table row can hold
};

constexpr int kPlanThreads = 1024;
constexpr int kPlanSmemSeqs = 2048;  // the prefix sums are searched in shared memory up to this many sequences

// Exclusive scan over the CTA; every thread gets the total. `warp_sums`: 33 ints of shared memory.
__device__ __forceinline__ int plan_scan(int x, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int v = warp_sums[lane];
        int w = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += y;
        }
        warp_sums[lane] = w - v;
        if (lane == 31) warp_sums[32] = w;
    }
    __syncthreads();
    total = warp_sums[32];
    const int out = warp_sums[warp] + inc - x;
    __syncthreads();
    return out;
}

// Builds the item list (one CTA). kBwd: the backward's tiles. Three or four walks over the blocks: the
// sum and the largest of their key tiles, the histogram (with and without cutting, where some block is
// long enough for it), the list. Runs in a few microseconds; what it costs is the latency of its steps,
// not the number of blocks.
//
// Whether to cut: taken in turns from the descending list, no CTA of G gets more than the sum of every
// G-th item. Blocks are cut when that sum with all parts within the limit, plus the cost of joining, is
// below the sum without.
template <bool kBwd>
__device__ void build_plan(const PlanParams& p) {
    __shared__ int s_hist[kPlanBuckets];
    __shared__ int s_prefix[kPlanSmemSeqs + 1];
    __shared__ int s_warp[33];
    __shared__ unsigned long long s_sum;
    __shared__ int s_max, s_slots, s_load[2], s_join;
    const int tid = threadIdx.x;
    const int tok = kBwd ? 128 : 2 * p.TT;  // tokens per block
    int* pre = p.S <= kPlanSmemSeqs ? s_prefix : p.prefix;
    if (tid == 0) {
        s_sum = 0;
        s_max = 1;
        s_slots = 0;
        s_load[0] = s_load[1] = 0;
        s_join = kPlanJoinFew;
    }
    int carry = 0, bad = 0, q_carry = 0;
    for (int base = 0; base < p.S; base += kPlanThreads) {
        const int s = base + tid;
        int blocks = 0, q_tiles = 0;
        if (s < p.S) {
            const int a = p.cu[s], b = p.cu[s + 1];
            if (a < 0 || b < a || b > p.T)
                bad = 1;
            else {
                blocks = plan_ceil(b - a, tok);
                q_tiles = plan_ceil(b - a, p.TT);
            }
        }
        int total;
        const int at = plan_scan(blocks, s_warp, total);
        if (s < p.S) pre[s] = carry + at;
        // T < 2^30 bounds the sum of valid offsets; with invalid ones it may pass 2^31, and the list is not built
        carry += total;
        if constexpr (kBwd) {
            const int q_at = plan_scan(q_tiles, s_warp, total);
            if (s < p.S) p.base[s] = q_carry + q_at;
            q_carry += total;
        }
    }
    bad = __syncthreads_or(bad);
    const int n_blocks = bad ? 0 : carry;
    if (tid == 0) pre[p.S] = n_blocks;
    if (bad) {
        if (tid == 0) {
            raise_status(kStatusBadOffsets);
            PlanHeader h{0, 0, {0, 0}};
            *p.header = h;
        }
        return;
    }
    __syncthreads();

    auto seq_of = [&](int b) {
        int lo = 0, hi = p.S - 1;  // the last sequence whose first block is <= b (empty ones never are the last)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= b)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo;
    };
    if constexpr (kBwd) {
        // sequences sorted by length (a counting sort by their tiles); a sequence's tiles in their own order,
        // which with a causal mask is most query tiles first
        s_hist[tid] = 0;
        __syncthreads();
        int most = 1;
        for (int s = tid; s < p.S; s += kPlanThreads) most = max(most, pre[s + 1] - pre[s]);
        most = __reduce_max_sync(0xffffffffu, most);
        if ((tid & 31) == 0) atomicMax(&s_max, most);
        __syncthreads();
        auto bucket = [&](int tiles) {
            return kPlanBuckets - 1 - static_cast<int>(static_cast<long long>(tiles) * (kPlanBuckets - 1) / s_max);
        };
        for (int s = tid; s < p.S; s += kPlanThreads) {
            const int tiles = pre[s + 1] - pre[s];
            if (tiles > 0) atomicAdd(&s_hist[bucket(tiles)], tiles);
        }
        __syncthreads();
        int total;
        const int first = plan_scan(s_hist[tid], s_warp, total);
        s_hist[tid] = first;
        __syncthreads();
        for (int s = tid; s < p.S; s += kPlanThreads) {
            const int tiles = pre[s + 1] - pre[s];
            if (tiles > 0) p.start[s] = atomicAdd(&s_hist[bucket(tiles)], tiles);
        }
        __syncthreads();
        for (int b = tid; b < n_blocks; b += kPlanThreads) {
            const int s = seq_of(b);
            PackedTile t;
            t.row0 = p.cu[s];
            t.n = p.cu[s + 1] - t.row0;
            t.base = p.base[s];
            t.t = b - pre[s];
            p.tiles[b] = t;
            p.order[p.start[s] + t.t] = b;
        }
        if (tid == 0) {
            PlanHeader h{n_blocks, 0, {0, 0}};
            *p.header = h;
        }
        return;
    }

    struct Block {
        int s, first, n, tiles, cost, kv_len;  // sequence, first token and tokens of the block, its tiles, keys
    };
    auto block_of = [&](int b) {
        const int lo = seq_of(b);
        Block x;
        x.s = lo;
        const int n = p.cu[lo + 1] - p.cu[lo];
        x.first = (b - pre[lo]) * tok;
        x.n = min(tok, n - x.first);
        int len = n;
        if (p.seq_lens != nullptr) {
            len = p.seq_lens[lo];
            if (len < n || len > p.max_len) len = -1;
        }
        x.kv_len = len;
        const int pos = len - n + x.first;
        x.tiles = len < 0 ? 0 : key_tiles(pos, pos + x.n - 1, len, p.causal, p.window).n;
        x.cost = plan_cost(x.tiles, x.n <= p.TT);
        return x;
    };
    Block mine{};  // this thread's first block is kept; further ones are looked up again in each walk
    if (tid < n_blocks) mine = block_of(tid);
    auto get = [&](int b) { return b == tid ? mine : block_of(b); };

    long long sum = 0;
    int most = 1;
    for (int b = tid; b < n_blocks; b += kPlanThreads) {
        const Block x = get(b);
        sum += x.cost;
        most = max(most, x.cost);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    most = __reduce_max_sync(0xffffffffu, most);
    if ((tid & 31) == 0 && tid < n_blocks) {
        atomicAdd(&s_sum, static_cast<unsigned long long>(sum));
        atomicMax(&s_max, most);
    }
    __syncthreads();
    const int limit = plan_limit(static_cast<long long>(s_sum), p.Hkv);
    const int longest = s_max;
    auto bucket = [&](const Block& x, int tiles) {  // of an item of block x
        const long long cost = plan_cost(tiles, x.n <= p.TT);
        return kPlanBuckets - 1 - static_cast<int>(cost * (kPlanBuckets - 1) / longest);
    };
    int n_items = 0;
    bool cut = false;
    // counts the items of each length into s_hist and turns that into the first position of each length
    auto sort_items = [&](bool with_parts) {
        s_hist[tid] = 0;
        __syncthreads();
        for (int b = tid; b < n_blocks; b += kPlanThreads) {
            const Block x = get(b);
            const int parts = with_parts ? plan_parts(x.cost, limit) : 1, q = x.tiles / parts, r = x.tiles % parts;
            if (parts > 1 && 4 * x.n > p.TT) s_join = kPlanJoinTiles;  // more than 32 rows
            if (r > 0) atomicAdd(&s_hist[bucket(x, q + 1)], r);
            atomicAdd(&s_hist[bucket(x, q)], parts - r);
        }
        __syncthreads();
        const int mine_n = s_hist[tid];
        const int start = plan_scan(mine_n, s_warp, n_items);
        s_hist[tid] = start;
        if (longest > limit && mine_n > 0) {
            // G-th items of this length
            const int first = plan_ceil_div(static_cast<long long>(start) * p.Hkv, kPlanSms);
            const int last = plan_ceil_div(static_cast<long long>(start + mine_n) * p.Hkv, kPlanSms);
            const int len = static_cast<int>(plan_ceil_div(static_cast<long long>(kPlanBuckets - 1 - tid) * longest, kPlanBuckets - 1));
            if (last > first) atomicAdd(&s_load[with_parts], (last - first) * len);
        }
        __syncthreads();
    };
    if (longest > limit) {
        sort_items(true);
        cut = true;
        const int with = s_load[1] + s_join;
        const int start = s_hist[tid], items_cut = n_items;
        sort_items(false);
        if (with < s_load[0]) {
            s_hist[tid] = start;
            n_items = items_cut;
        } else {
            cut = false;
        }
        __syncthreads();
    } else {
        sort_items(false);
    }

    for (int b = tid; b < n_blocks; b += kPlanThreads) {
        const Block x = get(b);
        const int parts = cut ? plan_parts(x.cost, limit) : 1;
        const int row0 = p.cu[x.s];
        const int n = p.cu[x.s + 1] - row0;
        PackedItem it;
        it.q_row = row0 + x.first;
        it.pos0 = x.kv_len < 0 ? 0 : x.kv_len - n + x.first;
        it.kv = p.seq_lens != nullptr ? x.s : row0;
        it.kv_len = x.kv_len;
        it.slot = 0;
        if (parts > 1) {
            it.slot = atomicAdd(&s_slots, parts);
            for (int i = 0; i < p.Hkv * kPlanWarps; ++i) p.count[static_cast<size_t>(it.slot) * p.Hkv * kPlanWarps + i] = 0;
        }
        const int jb =
            x.kv_len < 0 ? 0 : key_tiles(it.pos0, it.pos0 + x.n - 1, x.kv_len, p.causal, p.window).jb;
        for (int i = 0; i < parts; ++i) {
            int b0, b1;
            plan_part(x.tiles, parts, i, b0, b1);
            it.jb = jb + b0;
            it.n_tiles = b1 - b0;
            it.meta = make_meta(x.n, i, parts);
            p.items[atomicAdd(&s_hist[bucket(x, it.n_tiles)], 1)] = it;
        }
    }
    __syncthreads();
    if (tid == 0) {
        PlanHeader h{n_items, 0, {0, 0}};
        *p.header = h;
    }
}

// Chunks on the paged cache: new token t of sequence s goes to page block_table[s][pos / 16], slot
// pos % 16, pos = seq_lens[s] - n_s + t.
struct AppendParams {
    const __nv_bfloat16* k_new;  // [T, Hkv, D] (token stride ks), or nullptr (nothing to append)
    const __nv_bfloat16* v_new;
    __nv_bfloat16* k_pages;      // [num_pages, Hkv, 16, D]
    __nv_bfloat16* v_pages;
    const int32_t* block_table;
    long long ks, vs;
    int max_blocks, num_pages;
};

// Block 0 builds the plan; with kPaged the other blocks append the new tokens meanwhile, a warp per token:
// 2 D elements each way for every K/V head.
template <int D, bool kPaged, bool kBwd>
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const PlanParams p, const AppendParams a) {
    ptx::grid_launch_dependents();  // the attention kernel's set-up may overlap; it waits for this grid
    if (blockIdx.x == 0) {
        build_plan<kBwd>(p);
        return;
    }
    if constexpr (kPaged) {
        const int lane = threadIdx.x & 31;
        const int warps = static_cast<int>(gridDim.x - 1) * (kPlanThreads / 32);
        constexpr int LPR = D / 8;       // lanes per row of 16-byte pieces
        constexpr int HPW = 32 / (2 * LPR);  // heads a warp takes at a time (K and V rows)
        for (int t = static_cast<int>(blockIdx.x - 1) * (kPlanThreads / 32) + (threadIdx.x >> 5); t < p.T; t += warps) {
            // the sequence of token t: the last s with cu[s] <= t, 32 candidates a round (invalid offsets
            // end anywhere in [0, S))
            int lo = 0, n = p.S;
            while (n > 1) {
                const int step = plan_ceil(n, 32);
                const unsigned below = __ballot_sync(0xffffffffu, lane * step < n && p.cu[lo + min(lane * step, n - 1)] <= t);
                const int c = max(1, __popc(below)) - 1;
                lo += c * step;
                n = min(step, n - c * step);
            }
            const int c0 = p.cu[lo], c1 = p.cu[lo + 1], len = p.seq_lens[lo];
            if (t < c0 || t >= c1 || c0 < 0 || c1 > p.T) continue;       // behind the last sequence
            if (len < c1 - c0 || len > p.max_len) continue;              // flagged by the plan's user
            const int pos = len - (c1 - t);
            const int page = a.block_table[static_cast<size_t>(lo) * a.max_blocks + pos / kPageSize];
            if (page < 0 || page >= a.num_pages) {
                if (lane == 0) raise_status(kStatusBadPage);
                continue;
            }
            const int sub = lane / (2 * LPR), l = lane % (2 * LPR);
            const bool is_v = l >= LPR;
            const int c = is_v ? l - LPR : l;
            const __nv_bfloat16* src = is_v ? a.v_new + t * a.vs : a.k_new + t * a.ks;
            __nv_bfloat16* out = (is_v ? a.v_pages : a.k_pages) +
                                 (static_cast<size_t>(page) * p.Hkv * kPageSize + pos % kPageSize) * D;
#pragma unroll 4
            for (int g = sub; g < p.Hkv; g += HPW)
                reinterpret_cast<uint4*>(out + static_cast<size_t>(g) * kPageSize * D)[c] =
                    __ldg(reinterpret_cast<const uint4*>(src + static_cast<size_t>(g) * D) + c);
        }
    }
}

struct PackedParams {
    PlanHeader* header;
    const PackedItem* items;
    const int32_t* block_table;  // paged
    __nv_bfloat16* o;            // [T, Hq, D]
    float* lse;                  // element (token t, head h) at t * lse_t + h * lse_h, or nullptr
    int* count;                  // finished parts of [slot of part 0][Hkv][softmax warp]
    float* ws_ml;                // partial states: [slot][Hkv][256 rows][2] (max in log2 units, sum)
    float* ws_o;                 // [slot][Hkv][256 rows][D] unnormalised
    long long lse_t, lse_h;
    int Hq, Hkv, G, TT;
    int causal, window;
    int max_blocks, num_pages;   // paged
    float scale_log2;
    int debug_drop_copy;         // test hook: CTA 0 skips its first key-tile copy (see attn.h)
};

// An item of the list for one K/V head, with the key-tile range of each of its two query tiles. The
// producer decodes the items into a small ring in shared memory, ahead of the other warps: the record's
// load and the arithmetic are then off the path from one item's last product to the next one's first.
struct alignas(16) PackedWork {
    int q_row, pos0, kv, kv_len;
    int J0, T;          // key tiles of the item
    int g, parts;       // K/V head; parts of the block
    int tok[2];         // tokens of query tile i (0: absent)
    int slot, part;     // partial-state slot of part 0 (blocks of more than one part), and this part
    int a[2], e[2];     // steps of query tile i: [a, e), of a two-sided item every second of them
    int half;           // two-sided: key tiles of the first side; else 0
    int pad[3];
    // The key tile of step u, counted from J0.
    __device__ __forceinline__ int tile(int u) const { return half > 0 ? (u & 1) * half + (u >> 1) : u; }
};

__device__ __forceinline__ PackedWork decode_item(const PackedParams& p, const int4& lo, const int4& hi, int g) {
    PackedWork w;
    w.g = g;
    w.q_row = lo.x;
    w.pos0 = lo.y;
    w.kv = lo.z;
    w.kv_len = lo.w;
    w.J0 = hi.x;
    w.T = hi.y;
    const int n_tok = hi.z & 1023;
    w.parts = ((hi.z >> 20) & 1023) + 1;
    w.slot = hi.w;
    w.part = (hi.z >> 10) & 1023;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int n = min(p.TT, n_tok - i * p.TT);
        w.tok[i] = max(0, n);
        w.a[i] = w.e[i] = 0;
        if (n > 0 && w.T > 0) {
            const int first = w.pos0 + i * p.TT;
            const KeyTiles k = key_tiles(first, first + n - 1, w.kv_len, p.causal, p.window);
            const int a = max(0, k.jb - w.J0), e = min(w.T, k.jb + k.n - w.J0);
            if (e > a) {
                w.a[i] = a;
                w.e[i] = e;
            }
        }
    }
    w.half = 0;
    if (w.tok[1] == 0 && w.T > 1) {
        w.half = (w.T + 1) / 2;
        w.a[1] = 1;
        w.e[0] = ((w.T - 1) & ~1) + 1;
        w.e[1] = w.T - (w.T & 1);
    }
    return w;
}

constexpr int kWorkRing = 4;

template <int NK, int NV>
struct PackedBarriers : FwdBarriers<NK, NV> {
    uint64_t work_full[kWorkRing], work_empty[kWorkRing];
    uint64_t p_half[2];
    uint64_t s_free[2], pv_done[2], drain_outputs;  // kSplitP
    uint64_t side_full, side_empty;  // the second side's statistics
    PackedWork work[kWorkRing];
    float2 side_ml[128];
};

// Sets the columns of s outside [lo, hi] to -inf: a bit per column, 32 columns at a time (two
// instructions per score, where two compares and a select are three).
template <int N>
__device__ __forceinline__ void mask_columns(float (&s)[N], int lo, int hi) {
    auto low_bits = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
#pragma unroll
    for (int w = 0; w < N / 32; ++w) {
        const uint32_t m = low_bits(hi + 1 - 32 * w) & ~low_bits(lo - 32 * w);
#pragma unroll
        for (int k = 0; k < 32; ++k)
            if (!((m >> k) & 1u)) s[32 * w + k] = -INFINITY;
    }
}

// Called by a softmax warp that has stored its 32 rows' partial states of one part (rows of query tile
// wg from 32 quad on; q_row: the tile's first token): when it is the last of the block's parts, it joins them, M = max m_i,
// L = sum 2^(m_i - M) l_i, O = sum 2^(m_i - M) o_i / L, LSE = (M + log2 L) ln 2, in ascending order of i.
// The statistics go a row to a lane, the outputs a row to the warp, four rows and parts at a time: what
// counts is how many loads are in flight.
// A row that sees a NaN or a score of +inf has a sum of NaN in that part (beside a maximum of -inf or +inf)
// and comes out as NaN, as from a block that was not cut.
template <int D>
__device__ __noinline__ void join_parts(const PackedParams& p, int g, int q_row, int tok, int slot, int parts, int wg, int quad) {
    constexpr int PER = D / 32;  // columns of a lane
    const int lane = threadIdx.x & 31;
    if (tok * p.G <= quad * 32) return;  // none of its rows is live
    // the warp's states before the count, the count before the other parts' states
    __syncwarp();
    int last = 0;
    if (lane == 0)
        last = ptx::atomic_add_acq_rel(p.count + (static_cast<size_t>(slot) * p.Hkv + g) * kPlanWarps + wg * 4 + quad, 1) == parts - 1;
    if (!__shfl_sync(0xffffffffu, last, 0)) return;
    __syncwarp();  // lane 0 has acquired the other parts' states: the shuffle alone orders no memory
    const size_t step = static_cast<size_t>(p.Hkv) * 256;  // rows from one part's state to the next
    const int rows = min(32, tok * p.G - quad * 32);  // live rows of this warp
    const size_t row0 = (static_cast<size_t>(slot) * p.Hkv + g) * 256 + wg * 128 + quad * 32;
    const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + row0;
    constexpr int B = 8;  // parts at a time
    const int my_row = min(lane, rows - 1);
    float M = -INFINITY, L = 0.f;  // of row `lane`
    for (int base = 0; base < parts; base += B) {
        float2 x[B];
#pragma unroll
        for (int j = 0; j < B; ++j) x[j] = __ldcg(ml + my_row + min(base + j, parts - 1) * step);
        float top = M;
#pragma unroll
        for (int j = 0; j < B; ++j) top = fmaxf(top, x[j].x);
        L *= M == -INFINITY ? 0.f : ptx::ex2(M - top);
        M = top;
#pragma unroll
        for (int j = 0; j < B; ++j)  // a sum of 0: none of the row's keys, and no output
            if (base + j < parts && x[j].y != 0.f) L = fmaf(ptx::ex2(x[j].x - M), x[j].y, L);
    }
    const float inv = 1.f / L;  // (NaN of any part stays, whatever weight the part has)
    if (lane < rows && p.lse != nullptr) {
        const int r = quad * 32 + lane, t = r / p.G, h = g * p.G + r - t * p.G;
        const size_t row = static_cast<size_t>(q_row) + t;
        p.lse[row * p.lse_t + h * p.lse_h] = (M + ptx::lg2(L)) * kLn2;
    }
    constexpr int R = 4, P = 4;  // rows and parts at a time
    for (int r0 = 0; r0 < rows; r0 += R) {
        float acc[R][PER];
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int c = 0; c < PER; ++c) acc[j][c] = 0.f;
        for (int base = 0; base < parts; base += P) {
            float w[P], v[P][R][PER];  // w: of row `lane`
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const size_t part = min(base + i, parts - 1) * step;
                w[i] = __ldcg(ml + my_row + part).x;
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    const float* o = p.ws_o + (row0 + min(r0 + j, rows - 1) + part) * D + lane * PER;
                    if constexpr (PER == 4) {
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(o));
                        v[i][j][0] = y.x; v[i][j][1] = y.y; v[i][j][2] = y.z; v[i][j][3] = y.w;
                    } else {
                        const float2 y = __ldcg(reinterpret_cast<const float2*>(o));
                        v[i][j][0] = y.x; v[i][j][1] = y.y;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                w[i] = base + i < parts && w[i] != -INFINITY ? ptx::ex2(w[i] - M) : 0.f;
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    const float wr = __shfl_sync(0xffffffffu, w[i], min(r0 + j, rows - 1));
#pragma unroll
                    for (int c = 0; c < PER; ++c) acc[j][c] = wr > 0.f ? fmaf(wr, v[i][j][c], acc[j][c]) : acc[j][c];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const float iv = __shfl_sync(0xffffffffu, inv, min(r0 + j, rows - 1));
            if (r0 + j >= rows) continue;
            const int r = quad * 32 + r0 + j, t = r / p.G, h = g * p.G + r - t * p.G;
            uint32_t* out = reinterpret_cast<uint32_t*>(p.o + ((static_cast<size_t>(q_row) + t) * p.Hq + h) * D + lane * PER);
            if constexpr (PER == 4)
                *reinterpret_cast<uint2*>(out) = make_uint2(ptx::pack_bf16x2(acc[j][0] * iv, acc[j][1] * iv),
                                                            ptx::pack_bf16x2(acc[j][2] * iv, acc[j][3] * iv));
            else
                *out = ptx::pack_bf16x2(acc[j][0] * iv, acc[j][1] * iv);
        }
    }
}

template <int D>
struct PackedCfg {
    static constexpr bool kSplitP = D == 64;
    // beside the softmax warps: producer of Q and K, MMA issuer, (kSplitP) issuer of the outputs, producer of V
    static constexpr int V_WARP = kSplitP ? 11 : 10;
    static constexpr int THREADS = (V_WARP + 1) * 32;
    static constexpr int BAR_BYTES = 2048;
    // tiles, barriers, and the gap in front of the tiles' 1024-byte boundary
    static constexpr int SMEM_BYTES = FwdCfg<D>::SMEM_TILES * FwdCfg<D>::TILE_BYTES + BAR_BYTES + 1024;
    static_assert(SMEM_BYTES <= 232448, "shared memory above 227 KiB per CTA");
};

template <int D, bool kPaged>
__global__ void __launch_bounds__(PackedCfg<D>::THREADS, 1)
    attn_packed_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PackedParams p) {
    using C = FwdCfg<D>;
    constexpr int NK = C::NK, NV = C::NV;
    constexpr int kPages = C::BN / kPageSize;  // pages of a key tile
    // At D = 64 Tensor Memory has room for P beside S: see the MMA issuer.
    constexpr bool kSplitP = PackedCfg<D>::kSplitP;
    constexpr int kConsumers = kSplitP ? 11 : 10;  // warps that read the work ring: all but the producer of Q and K
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;
    uint8_t* sK = sQ + C::QT * C::TILE_BYTES;
    uint8_t* sV = sK + NK * C::TILE_BYTES;
    auto* bar = reinterpret_cast<PackedBarriers<NK, NV>*>(sV + NV * C::TILE_BYTES);
    static_assert(sizeof(PackedBarriers<NK, NV>) <= PackedCfg<D>::BAR_BYTES, "barrier block larger than its reserved bytes");
    volatile int* abort_flag = &bar->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bar->q_loaded[i], 1);
            ptx::mbar_init(&bar->q_empty[i], 1);
            ptx::mbar_init(&bar->s_full[i], 1);
            ptx::mbar_init(&bar->p_full[i], 128);
            ptx::mbar_init(&bar->o_final[i], 1);
            ptx::mbar_init(&bar->o_empty[i], 128);
            ptx::mbar_init(&bar->p_half[i], 128);
            ptx::mbar_init(&bar->s_free[i], 128);
            ptx::mbar_init(&bar->pv_done[i], 1);
        }
        for (int s = 0; s < kWorkRing; ++s) {
            ptx::mbar_init(&bar->work_full[s], 1);
            ptx::mbar_init(&bar->work_empty[s], kConsumers);
        }
        for (int s = 0; s < NK; ++s) {
            ptx::mbar_init(&bar->k_full[s], 1);
            ptx::mbar_init(&bar->k_empty[s], 1);
        }
        for (int s = 0; s < NV; ++s) {
            ptx::mbar_init(&bar->v_full[s], 1);
            ptx::mbar_init(&bar->v_empty[s], 1);
        }
        ptx::mbar_init(&bar->drain, 1);
        ptx::mbar_init(&bar->drain_outputs, 1);
        ptx::mbar_init(&bar->side_full, 128);
        ptx::mbar_init(&bar->side_empty, 128);
        bar->abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == C::PRODUCER_WARP && lane == 0) {
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
    }
    if (warp == C::MMA_WARP) {
        ptx::tmem_alloc(&bar->tmem_base, C::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();  // the plan (and the appended tokens)
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bar->tmem_base;
    const int n_items = p.header->n_items * p.Hkv;
    // TMEM columns of P: over the first half of S, or behind the accumulators
    auto tmem_p = [](int i) { return kSplitP ? 256u + 2u * D + 64u * i : C::tmem_s(i); };

    // Key tile of a step, loaded by a whole warp: lane 0 expects the bytes; a packed tile's boxes are issued
    // by lane 0, those of a paged tile by the lane that looked the page up (`page`; -1: none, read as zeros
    // by a box outside the tensor, so that what its memory holds cannot reach a product).
    auto load_tile = [&](const PackedWork& x, const CUtensorMap* tm, uint8_t* dst, uint64_t* full, int jt, int page, bool drop) {
        if constexpr (kPaged) {
            const int pages = min(kPages, (x.kv_len + kPageSize - 1) / kPageSize - jt * kPages);
            const int z = page >= 0 && page < p.num_pages ? page * p.Hkv + x.g : -1;
            if (lane == 0) ptx::mbar_arrive_expect_tx(full, pages * kPageSize * C::ROW_BYTES);
            __syncwarp();
            if (lane < pages && !drop) {
#pragma unroll
                for (int r = 0; r < C::NREG; ++r)
                    ptx::tma_load_3d(dst + r * C::REGION_BYTES + lane * kPageSize * 128, tm, full, r * 64, 0, z);
            }
        } else if (lane == 0) {
            ptx::mbar_arrive_expect_tx(full, C::TILE_BYTES);
            if (!drop) {
#pragma unroll
                for (int r = 0; r < C::NREG; ++r)
                    ptx::tma_load_3d(dst + r * C::REGION_BYTES, tm, full, r * 64, x.g, x.kv + jt * C::BN);
            }
        }
    };
    // lane i of a paged tile: page i of the tile of step u. Pages before the window of the item's first
    // token may have been given back: they are not looked up.
    auto look_up = [&](const PackedWork& x, int u) {
        if (!kPaged || lane >= kPages || u >= x.T) return -1;
        const int pg = (x.J0 + x.tile(u)) * kPages + lane;
        const int first_page = p.window > 0 ? max(0, x.pos0 - p.window + 1) / kPageSize : 0;
        if (pg < first_page || pg >= (x.kv_len + kPageSize - 1) / kPageSize) return -1;
        const int page = p.block_table[static_cast<size_t>(x.kv) * p.max_blocks + pg];
        if (page < 0 || page >= p.num_pages) raise_status(kStatusBadPage);
        return page;
    };

    if (warp == C::PRODUCER_WARP) {
        // ------------------------------------------------------------------ TMA producer
        // Decodes the items into the work ring and loads Q and K.
        int kq[2] = {0, 0};
        int sk = 0, issued = 0;
        uint32_t free_par = 1;  // (a fresh barrier passes parity 1)
        bool ok = true;
        int4 rec_lo{}, rec_hi{};  // the next item's record, loaded one item ahead
        auto load_record = [&](int it) {
            if (it >= n_items) return;
            const int4* rec = reinterpret_cast<const int4*>(p.items + it / p.Hkv);
            rec_lo = rec[0];
            rec_hi = rec[1];
        };
        int it = blockIdx.x;
        load_record(it);
        for (int rnd = 0; ok; ++rnd) {
            PackedWork x = decode_item(p, rec_lo, rec_hi, it % p.Hkv);
            if (it >= n_items) x.T = -1;  // the end, for every reader of the ring
            const int ws = rnd % kWorkRing;
            if (rnd >= kWorkRing && !ptx::mbar_wait_warp(&bar->work_empty[ws], (rnd / kWorkRing - 1) & 1, abort_flag)) { ok = false; break; }
            if (lane == 0) {
                bar->work[ws] = x;
                ptx::mbar_arrive(&bar->work_full[ws]);
            }
            if (x.T < 0) break;
            int page = look_up(x, 0);
            // the next item, taken a few tiles before this one's end: early enough to hide the latency, late
            // enough that CTAs with long items take fewer
            const int take = max(0, x.T - 4);
            auto take_next = [&]() {
                int n = 0;
                if (lane == 0) n = atomicAdd(&p.header->taken, 1);
                it = static_cast<int>(gridDim.x) + __shfl_sync(0xffffffffu, n, 0);
                load_record(it);
            };
            if (x.T == 0) take_next();
            for (int i = 0; i < 2 && ok; ++i) {
                if (x.e[i] == x.a[i]) continue;
                if (kq[i] > 0 && !ptx::mbar_wait_warp(&bar->q_empty[i], (kq[i] - 1) & 1, abort_flag)) { ok = false; break; }
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(&bar->q_loaded[i], static_cast<uint32_t>(p.G * p.TT * C::ROW_BYTES));
#pragma unroll
                    for (int r = 0; r < C::NREG; ++r)
                        ptx::tma_load_3d(sQ + i * C::TILE_BYTES + r * C::REGION_BYTES, &tm_q, &bar->q_loaded[i], r * 64,
                                         x.g * p.G, x.q_row + (x.half > 0 ? 0 : i * p.TT));
                }
                ++kq[i];
            }
            for (int u = 0; u < x.T && ok; ++u) {
                if (!ptx::mbar_wait_warp(&bar->k_empty[sk], free_par, abort_flag)) { ok = false; break; }
                const int now = page;
                page = look_up(x, u + 1);  // one tile ahead
                load_tile(x, &tm_k, sK + sk * C::TILE_BYTES, &bar->k_full[sk], x.J0 + x.tile(u), now,
                          p.debug_drop_copy && issued == 0 && blockIdx.x == 0);
                if (u == take) take_next();
                ++issued;
                if (++sk == NK) {
                    sk = 0;
                    free_par ^= 1;
                }
            }
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            raise_status(kStatusTimeout);
            // let the copies in flight land before the CTA's shared memory is released (bounded)
            volatile int never = 0;
            for (int i = 0; i < 2; ++i)
                if (kq[i] > 0) ptx::mbar_wait(&bar->q_loaded[i], (kq[i] - 1) & 1, &never);
            for (int u = max(0, issued - NK); u < issued; ++u) ptx::mbar_wait(&bar->k_full[u % NK], (u / NK) & 1, &never);
        }
        __syncwarp();
    } else if (warp == PackedCfg<D>::V_WARP) {
        // ------------------------------------------------------------------ producer of V
        // A warp of its own: the 16 boxes of a paged 128-key tile take 1,200 clocks to issue at D = 128,
        // and one warp issuing K and V bounded single tokens at 2,900 clocks a tile.
        int sv = 0, issued = 0;
        uint32_t free_par = 1;
        bool ok = true;
        for (int rnd = 0; ok; ++rnd) {
            const int ws = rnd % kWorkRing;
            if (!ptx::mbar_wait_warp(&bar->work_full[ws], (rnd / kWorkRing) & 1, abort_flag)) { ok = false; break; }
            const PackedWork x = bar->work[ws];
            if (x.T < 0) break;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bar->work_empty[ws]);
            int page = look_up(x, 0);
            for (int u = 0; u < x.T && ok; ++u) {
                if (!ptx::mbar_wait_warp(&bar->v_empty[sv], free_par, abort_flag)) { ok = false; break; }
                const int now = page;
                page = look_up(x, u + 1);
                load_tile(x, &tm_v, sV + sv * C::TILE_BYTES, &bar->v_full[sv], x.J0 + x.tile(u), now, false);
                ++issued;
                if (++sv == NV) {
                    sv = 0;
                    free_par ^= 1;
                }
            }
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            raise_status(kStatusTimeout);
            volatile int never = 0;  // as above
            for (int u = max(0, issued - NV); u < issued; ++u) ptx::mbar_wait(&bar->v_full[u % NV], (u / NV) & 1, &never);
        }
        __syncwarp();
    } else if (warp >= C::MMA_WARP) {
        // ------------------------------------------------------------------ MMA issuers
        // With P over S (D = 128) one warp issues, per key tile u: O_i += P_i(u) V(u), S_i(u+1) = Q_i K(u+1)^T
        // for i = 0, 1, in execution order. With P in columns of its own (D = 64) S_i(u + 1) only waits
        // until the softmax has read S_i(u), and a second warp issues the outputs: the scores run ahead,
        // across the items too. What a warp issues between two products counts (the softmax warps take most
        // issue slots): stages and parities are stepped, not computed.
        const bool scores = warp == C::MMA_WARP, outputs = !kSplitP || !scores;
        const uint32_t issue = ptx::elect_one() ? 1u : 0u;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        constexpr uint32_t IDESC_S = ptx::idesc_bf16_f32(128, C::BN, 0, 0);
        constexpr uint32_t IDESC_O = ptx::idesc_bf16_f32(128, D, 0, 1);
        constexpr uint32_t HI = ptx::sw128_desc_hi(1024);
        constexpr uint64_t TILE16 = C::TILE_BYTES >> 4;
        const uint64_t q_d = ptx::desc64(__shfl_sync(0xffffffffu, ptx::sw128_desc_lo(ptx::smem_u32(sQ), 16), 0), HI);
        const uint64_t k_d = ptx::desc64(__shfl_sync(0xffffffffu, ptx::sw128_desc_lo(ptx::smem_u32(sK), 16), 0), HI);
        const uint64_t v_d =
            ptx::desc64(__shfl_sync(0xffffffffu, ptx::sw128_desc_lo(ptx::smem_u32(sV), C::REGION_BYTES), 0), HI);
        bool ok = true, issued_any = false;
        int sk = 0, sv = 0;            // ring stages of the next K and V tile
        uint32_t pk = 0, pv = 0;       // and their parities
        uint32_t q_par[2] = {0, 0}, p_par[2] = {0, 0}, o_par[2] = {1, 1}, f_par[2] = {1, 1};
        int a[2], e[2], seen[2];       // of the current item: visible key tiles, keys the tile's last row sees
        auto score_tile = [&](int i, bool first, bool last) {
            if (first) {
                if (!ptx::mbar_wait_warp(&bar->q_loaded[i], q_par[i], abort_flag)) return false;
                q_par[i] ^= 1;
            }
            if (kSplitP) {  // the softmax has read the scores before (a fresh barrier passes parity 1)
                if (!ptx::mbar_wait_warp(&bar->s_free[i], f_par[i], abort_flag)) return false;
                f_par[i] ^= 1;
                ptx::tc_fence_after();
            }
            const uint64_t qa = q_d + i * TILE16, kb = k_d + sk * TILE16;
#pragma unroll
            for (int kk = 0; kk < C::S_KSTEPS; ++kk) {
                const uint64_t off = ((kk >> 2) * C::REGION_BYTES + (kk & 3) * 32) >> 4;
                ptx::mma_ss_if(issue, tm + C::tmem_s(i), qa + off, kb + off, IDESC_S, kk > 0);
            }
            ptx::mma_commit_if(issue, &bar->s_full[i]);
            if (last) ptx::mma_commit_if(issue, &bar->q_empty[i]);
            issued_any = true;
            return true;
        };
        // up to the last 16-key slice that a row of the tile sees; keys: how many from the tile's first key on
        auto output_tile = [&](int i, bool first, bool last, int keys) {
            if (first) {  // the epilogue before has read O (a fresh barrier passes parity 1)
                if (!ptx::mbar_wait_warp(&bar->o_empty[i], o_par[i], abort_flag)) return false;
                o_par[i] ^= 1;
            }
            if (!ptx::mbar_wait_warp(&bar->p_half[i], p_par[i], abort_flag)) return false;
            ptx::tc_fence_after();
            const uint32_t d_o = tm + C::tmem_o(i), d_p = tm + tmem_p(i);
            const uint64_t vb = v_d + sv * TILE16;
            const uint32_t acc = first ? 0u : 1u;
            auto slices = [&](int k0) {
                if (keys > 112) {
#pragma unroll
                    for (int kk = k0; kk < k0 + C::O_KSTEPS / 2; ++kk)
                        ptx::mma_ts_if(issue, d_o, d_p + kk * 8, vb + kk * ((C::O_ROWS * 128) >> 4), IDESC_O, kk > 0 ? 1u : acc);
                } else {
#pragma unroll
                    for (int kk = k0; kk < k0 + C::O_KSTEPS / 2; ++kk)
                        ptx::mma_ts_if(kk * 16 < keys ? issue : 0u, d_o, d_p + kk * 8, vb + kk * ((C::O_ROWS * 128) >> 4),
                                       IDESC_O, kk > 0 ? 1u : acc);
                }
            };
            slices(0);
            if (!ptx::mbar_wait_warp(&bar->p_full[i], p_par[i], abort_flag)) return false;
            p_par[i] ^= 1;
            ptx::tc_fence_after();
            slices(C::O_KSTEPS / 2);
            if (kSplitP)
                ptx::mma_commit_if(issue, &bar->pv_done[i]);
            else if (last)
                ptx::mma_commit_if(issue, &bar->o_final[i]);
            issued_any = true;
            return true;
        };
        for (int rnd = 0; ok; ++rnd) {
            const int ws = rnd % kWorkRing;
            if (!ptx::mbar_wait_warp(&bar->work_full[ws], (rnd / kWorkRing) & 1, abort_flag)) { ok = false; break; }
            const PackedWork& x = bar->work[ws];
            const int T = x.T, key0 = x.J0 * C::BN, half = x.half;
            if (T < 0) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i] = x.a[i];
                e[i] = x.e[i];
                const int q_tile = half > 0 ? 0 : i;
                seen[i] = (p.causal ? min(x.kv_len, x.pos0 + q_tile * p.TT + x.tok[q_tile]) : x.kv_len) - key0 -
                          (half > 0 && i == 1 ? half * C::BN : 0);
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bar->work_empty[ws]);
            // the scores run ahead of the outputs by one key tile of the same query tile
            const int ahead = kSplitP ? 0 : half > 0 ? 2 : 1;
            for (int u = -ahead; ok && u < T; ++u) {
                const int us = u + ahead;  // the step whose scores are due
                if (outputs && u >= 0) {
                    if (!ptx::mbar_wait_warp(&bar->v_full[sv], pv, abort_flag)) { ok = false; break; }
                }
                if (scores && us < T) {
                    if (!ptx::mbar_wait_warp(&bar->k_full[sk], pk, abort_flag)) { ok = false; break; }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (outputs && ok && u >= a[i] && u < e[i] && (half == 0 || (u & 1) == i))
                        ok = output_tile(i, u == a[i], u == e[i] - 1, seen[i] - (half > 0 ? u >> 1 : u) * C::BN);
                    if (scores && ok && us >= a[i] && us < e[i] && (half == 0 || (us & 1) == i))
                        ok = score_tile(i, us == a[i], us == e[i] - 1);
                }
                if (!ok) break;
                if (outputs && u >= 0) {
                    ptx::mma_commit_if(issue, &bar->v_empty[sv]);
                    if (++sv == NV) {
                        sv = 0;
                        pv ^= 1;
                    }
                }
                if (scores && us < T) {
                    ptx::mma_commit_if(issue, &bar->k_empty[sk]);
                    if (++sk == NK) {
                        sk = 0;
                        pk ^= 1;
                    }
                }
            }
        }
        if (!ok) {
            if (issue) {
                *abort_flag = 1;
                raise_status(kStatusTimeout);
                if (issued_any) {
                    uint64_t* drain = scores ? &bar->drain : &bar->drain_outputs;
                    ptx::mma_commit(drain);
                    volatile int never = 0;
                    ptx::mbar_wait(drain, 0, &never);
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------ softmax warpgroups
        const int wg = warp >> 2;
        const int r = threadIdx.x & 127;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_base + C::tmem_s(wg);
        const uint32_t t_o = tmem + lane_base + C::tmem_o(wg), t_p = tmem + lane_base + tmem_p(wg);
        const float sl = p.scale_log2;
        const int my_tok = r / p.G, my_head = r - my_tok * p.G;  // this row's token in the tile and head in the group
        bool ok = true;
        // Barrier parities, a bit each (a wait for the phase before is one for the other parity, which a
        // fresh barrier passes): this warpgroup's next key tile, its items; the second warpgroup's key
        // tiles and items; two-sided items.
        constexpr uint32_t kTiles = 1, kItems = 2, kTiles1 = 4, kItems1 = 8, kSides = 16;
        uint32_t par = 0;
        auto parity = [&](uint32_t bit) { return (par & bit) ? 1u : 0u; };
        int g = 0;  // key tiles of the items before
        for (int rnd = 0; ok; ++rnd) {
            const int ws = rnd % kWorkRing;
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->work_full[ws], (rnd / kWorkRing) & 1, abort_flag))) { ok = false; break; }
            const PackedWork& x = bar->work[ws];  // kept until the item is done: registers are scarce here
            if (x.T < 0) break;
            auto release_work = [&]() {
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bar->work_empty[ws]);
            };
            const bool two_sided = x.half > 0;
            const int q_tile = two_sided ? 0 : wg;
            const int a = x.a[wg], first = two_sided ? wg * x.half : a;  // first step and first key tile
            const int n1 = two_sided ? x.T - x.half : x.e[1] - x.a[1];
            const int n = wg ? n1 : two_sided ? x.half : x.e[0] - x.a[0];  // key tiles of this warpgroup
            const int jb = x.J0 + first, stride = two_sided ? 2 : 1;
            const int tok = x.tok[q_tile];
            const bool live = my_tok < tok;  // tok <= TT: rows past G * TT never are
            const int pos_first = x.pos0 + q_tile * p.TT, i_pos = pos_first + my_tok;
            float m_used = -INFINITY, l = 0.f;
            for (int c = 0; ok && c < n; ++c) {
                const int j0 = (jb + c) * C::BN;
                if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->s_full[wg], parity(kTiles), abort_flag))) { ok = false; break; }
                ptx::tc_fence_after();
                uint32_t sv[C::BN];
                ptx::tmem_ld128(t_s, sv);
                if constexpr (kSplitP) {
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&bar->s_free[wg]);
                }
                float s[C::BN];
#pragma unroll
                for (int k = 0; k < C::BN; ++k) s[k] = __uint_as_float(sv[k]);
                const bool need_mask = (j0 + C::BN > x.kv_len) || (p.causal && j0 + C::BN - 1 > pos_first) ||
                                       (p.window > 0 && pos_first + tok - 1 - j0 >= p.window);
                if (need_mask) {
                    const int lo = p.window > 0 ? i_pos - p.window + 1 : 0;
                    const int hi = live ? (p.causal ? i_pos : x.kv_len - 1) : -1;
                    // columns lo - j0 .. hi - j0; the first bound may pass -2^31 for a huge window
                    const int lo_c = p.window > i_pos ? 0 : lo - j0, hi_c = hi - j0;
                    mask_columns(s, lo_c, hi_c);
                }
                float mx0 = fmaxf(s[0], s[1]), mx1 = fmaxf(s[2], s[3]), mx2 = fmaxf(s[4], s[5]), mx3 = fmaxf(s[6], s[7]);
#pragma unroll
                for (int k = 8; k < C::BN; k += 8) {
                    mx0 = ptx::fmax3(mx0, s[k], s[k + 1]);
                    mx1 = ptx::fmax3(mx1, s[k + 2], s[k + 3]);
                    mx2 = ptx::fmax3(mx2, s[k + 4], s[k + 5]);
                    mx3 = ptx::fmax3(mx3, s[k + 6], s[k + 7]);
                }
                const float m_new = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * sl;
                float alpha = 1.f;
                bool rescale = false;
                if (m_new > m_used + C::RESCALE_THRESHOLD) {
                    alpha = ptx::ex2(m_used - m_new);
                    m_used = m_new;
                    rescale = true;
                }
                const float m_eff = (m_used == -INFINITY) ? 0.f : m_used;
                const float2 sl2 = make_float2(sl, sl), nm2 = make_float2(-m_eff, -m_eff);
                if constexpr (kSplitP) {
                    // P and O are free once the product before has completed
                    if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->pv_done[wg], parity(kTiles) ^ 1, abort_flag))) { ok = false; break; }
                    ptx::tc_fence_after();
                }
                // the end of the sequence inside a 16-key slice: zero the slice's other V rows (both
                // query tiles may do it: the same zeros, before either P is handed over)
                const int tail = x.kv_len - j0;
                if (tail < C::BN && (tail & 15)) {
                    const int gs = g + a + c * stride, sv_st = gs % NV;
                    if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->v_full[sv_st], (gs / NV) & 1, abort_flag))) { ok = false; break; }
                    const uint32_t base = ptx::smem_u32(sV + sv_st * C::TILE_BYTES) + tail * 128;
                    const int chunks = (16 - (tail & 15)) * 8;  // 16-byte pieces per region
                    for (int t = r; t < chunks * C::NREG; t += 128)
                        ptx::st_shared_v4(base + (t / chunks) * C::REGION_BYTES + (t % chunks) * 16, 0, 0, 0, 0);
                    ptx::fence_proxy_async_smem();
                }
                if (c > 0 && __any_sync(0xffffffffu, rescale)) {
                    const float2 al2 = make_float2(alpha, alpha);
#pragma unroll 1
                    for (int cc = 0; cc < D / 16; ++cc) {
                        uint32_t v[16];
                        ptx::tmem_ld16(t_o + cc * 16, v);
#pragma unroll
                        for (int k = 0; k < 16; k += 2) {
                            const float2 y =
                                ptx::fmul2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), al2);
                            v[k] = __float_as_uint(y.x);
                            v[k + 1] = __float_as_uint(y.y);
                        }
                        ptx::tmem_st16(t_o + cc * 16, v);
                    }
                }
                // P in two halves: the product starts on the first while the second is computed
                float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0, acc2 = acc0, acc3 = acc0;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[C::P_COLS / 2];
#pragma unroll
                    for (int k = 0; k < C::BN / 2; k += 8) {
                        const float* z = s + half * (C::BN / 2) + k;
                        float2 x0 = ptx::ffma2(make_float2(z[0], z[1]), sl2, nm2);
                        float2 x1 = ptx::ffma2(make_float2(z[2], z[3]), sl2, nm2);
                        float2 x2 = ptx::ffma2(make_float2(z[4], z[5]), sl2, nm2);
                        float2 x3 = ptx::ffma2(make_float2(z[6], z[7]), sl2, nm2);
                        x0 = make_float2(ptx::ex2(x0.x), ptx::ex2(x0.y));
                        x1 = make_float2(ptx::ex2(x1.x), ptx::ex2(x1.y));
                        x2 = make_float2(ptx::ex2(x2.x), ptx::ex2(x2.y));
                        x3 = make_float2(ptx::ex2(x3.x), ptx::ex2(x3.y));
                        acc0 = ptx::fadd2(acc0, x0);
                        acc1 = ptx::fadd2(acc1, x1);
                        acc2 = ptx::fadd2(acc2, x2);
                        acc3 = ptx::fadd2(acc3, x3);
                        pk[k / 2] = ptx::pack_bf16x2(x0.x, x0.y);
                        pk[k / 2 + 1] = ptx::pack_bf16x2(x1.x, x1.y);
                        pk[k / 2 + 2] = ptx::pack_bf16x2(x2.x, x2.y);
                        pk[k / 2 + 3] = ptx::pack_bf16x2(x3.x, x3.y);
                    }
                    ptx::tmem_st32(t_p + half * (C::P_COLS / 2), pk);
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(half ? &bar->p_full[wg] : &bar->p_half[wg]);
                }
                const float2 sum = ptx::fadd2(ptx::fadd2(acc0, acc1), ptx::fadd2(acc2, acc3));
                l = l * alpha + (sum.x + sum.y);
                par ^= kTiles;
            }
            if (!ok) break;
            g += x.T;
            if (n1 > 0) par ^= kItems1;
            if (n1 & 1) par ^= kTiles1;
            if (tok == 0) {
                release_work();
                continue;
            }
            const size_t prow =
                ((static_cast<size_t>(x.slot + x.part) * p.Hkv + x.g) * 256 + wg * 128 + r);  // partial-state row
            if (n == 0) {
                // an invalid length, or a part none of whose keys this query tile sees
                if (x.kv_len < 0) {
                    if (r == 0 && wg == 0 && x.g == 0) raise_status(kStatusBadSeqLen);
                    if (live) {
                        const size_t row = static_cast<size_t>(x.q_row + q_tile * p.TT + my_tok);
                        const int h = x.g * p.G + my_head;
                        uint4* dst = reinterpret_cast<uint4*>(p.o + (row * p.Hq + h) * D);
                        for (int k = 0; k < D / 8; ++k)
                            dst[k] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
                        if (p.lse != nullptr) p.lse[row * p.lse_t + h * p.lse_h] = __int_as_float(0x7fc00000);
                    }
                } else if (live) {
                    p.ws_ml[prow * 2] = -INFINITY;
                    p.ws_ml[prow * 2 + 1] = 0.f;
                }
                if (x.kv_len >= 0) join_parts<D>(p, x.g, x.q_row + wg * p.TT, tok, x.slot, x.parts, wg, warp & 3);
                release_work();
                continue;
            }
            if (two_sided && wg == 1) {
                // hand the statistics to the first warpgroup, which reads both accumulators
                if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->side_empty, parity(kSides) ^ 1, abort_flag))) { ok = false; break; }
                bar->side_ml[r] = make_float2(m_used, l);
                ptx::mbar_arrive(&bar->side_full);
                par ^= kSides | kItems;
                release_work();
                continue;
            }
            // ---- epilogue: O out of TMEM; normalised to the output, or as a partial state
            if (!__all_sync(0xffffffffu, kSplitP ? ptx::mbar_wait(&bar->pv_done[wg], parity(kTiles) ^ 1, abort_flag)
                                                 : ptx::mbar_wait(&bar->o_final[wg], parity(kItems), abort_flag))) { ok = false; break; }
            ptx::tc_fence_after();
            float w0 = 1.f, w1 = 0.f;  // weights of the sides' accumulators
            if (two_sided) {
                if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->side_full, parity(kSides), abort_flag))) { ok = false; break; }
                par ^= kSides;
                const float2 other = bar->side_ml[r];
                ptx::mbar_arrive(&bar->side_empty);
                if (!__all_sync(0xffffffffu, kSplitP ? ptx::mbar_wait(&bar->pv_done[1], parity(kTiles1) ^ 1, abort_flag)
                                                     : ptx::mbar_wait(&bar->o_final[1], parity(kItems1) ^ 1, abort_flag))) { ok = false; break; }
                ptx::tc_fence_after();
                const float m = fmaxf(m_used, other.x);
                w0 = m_used == -INFINITY ? 0.f : ptx::ex2(m_used - m);
                w1 = other.x == -INFINITY ? 0.f : ptx::ex2(other.x - m);
                l = l * w0 + other.y * w1;
                m_used = m;
            }
            // 32 columns of O, of a two-sided item both sides weighted
            auto load_output = [&](int c0, uint32_t (&v)[32]) {
                ptx::tmem_ld32(t_o + c0, v);
                if (two_sided) {
                    uint32_t v1[32];
                    ptx::tmem_ld32(tmem + lane_base + C::tmem_o(1) + c0, v1);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        v[k] = __float_as_uint(__uint_as_float(v[k]) * w0 + __uint_as_float(v1[k]) * w1);
                }
            };
            auto output_read = [&]() {
                ptx::tc_fence_before();
                ptx::mbar_arrive(&bar->o_empty[wg]);
                if (two_sided) ptx::mbar_arrive(&bar->o_empty[1]);
            };
            // (loops kept rolled: what runs once an item competes for instruction cache; 24 prompts 139 -> 137 us)
            if (x.parts > 1) {
                // rows lie at multiples of 256 bytes from the workspace's base, which may be 16 modulo 32
                const bool sectors = (reinterpret_cast<uintptr_t>(p.ws_o) & 31) == 0;
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t v[32];
                    load_output(cc * 32, v);
                    uint32_t* dst = reinterpret_cast<uint32_t*>(p.ws_o + prow * D + cc * 32);
                    if (live && sectors) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) ptx::st_global_v8(dst + k, v + k);
                    } else if (live) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<uint4*>(dst + k) = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    }
                }
                output_read();
                if (live) {
                    p.ws_ml[prow * 2] = m_used;
                    p.ws_ml[prow * 2 + 1] = l;
                }
                join_parts<D>(p, x.g, x.q_row + q_tile * p.TT, tok, x.slot, x.parts, wg, warp & 3);
            } else {
                const float inv_l = 1.f / l;
                const size_t row = static_cast<size_t>(x.q_row + q_tile * p.TT + my_tok);
                const int h = x.g * p.G + my_head;
                uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (row * p.Hq + h) * D);
                const bool sectors = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;  // whole 32-byte sectors
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t v[32], w[16];
                    load_output(cc * 32, v);
                    if (cc == D / 32 - 1) output_read();
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        w[k] = ptx::pack_bf16x2(__uint_as_float(v[2 * k]) * inv_l, __uint_as_float(v[2 * k + 1]) * inv_l);
                    if (!live) continue;
                    if (sectors) {
#pragma unroll
                        for (int k = 0; k < 16; k += 8) ptx::st_global_v8(dst + cc * 16 + k, w + k);
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            *reinterpret_cast<uint4*>(dst + cc * 16 + k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
                    }
                }
                if (live && p.lse != nullptr)
                    p.lse[row * p.lse_t + h * p.lse_h] = (m_used + ptx::lg2(l)) * kLn2;
            }
            par ^= kItems;
            release_work();
        }
        if (!ok) {
            *abort_flag = 1;
            raise_status(kStatusTimeout);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == C::MMA_WARP) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

}  // namespace attn
