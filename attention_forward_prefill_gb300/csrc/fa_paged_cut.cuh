// fa_paged_cut.cuh -- how the paged-attention kernels cut their work into equal
// ranges of key tiles, and how two passes over the same rows share the SMs.  Plain
// arithmetic: tests/test_paged_split_host.py compiles this file for the host.
//
// Work.  The cache keeps K and V as [page][kv head][slot][d]; sequence b's
// token j lives in page page_table[b][j / page_size], slot j % page_size.  A
// sequence with nq query tokens gives each kv head nq * G query rows
// (G = query heads per kv head), row r = (token r / G, head r % G), cut into
// blocks of block_rows.  A unit = (sequence, kv head, row block); it costs
// unit_steps for its own start and end and a step per key tile its rows can see,
// or a few (PagedCut; at least one tile, so that a unit without keys still writes its rows).  The W
// steps of the whole call, in the order (sequence, kv head, block), are cut
// into gridDim.x equal ranges, one per CTA, whatever the lengths are: they live
// on the device, so the cut is made there, by every CTA for itself (1 to 2 us,
// under the launch of what comes before).  A unit inside one range is written
// directly; the pieces of a unit that ranges cut keep (O, m, l) in fp32 and
// paged_join_kernel adds them in a fixed order, so a given shape and set of
// lengths gives the same bits on every run.
#pragma once

#include <cstdint>

namespace fa {

struct PagedParams {
    const uint16_t *q;     // [total_q][Hq][D]
    void *out;             // [total_q][Hq][D]
    float *lse;            // optional [total_q][Hq]: natural-log row log-sum-exp, -inf for a row without keys
    const int *page_table;  // [B][max_pages]
    const int *seq_lens;    // [B] keys of each sequence
    const int *cu_q;        // [B + 1] query token offsets, or null: nq_each tokens per sequence
    int nq_each;
    int B, Hq, Hkv, G;
    int total_q, max_q;
    int max_pages, max_len;
    int num_pages, page_shift;
    int block_rows;         // query rows of a unit
    int unit_steps;         // what a unit costs besides its key tiles, in steps
    int tile_tokens;        // paged_tiles_kernel: tokens of a query tile, of which a block has two
    int causal;             // query token i of nq sees keys j <= len - nq + i
    float scale_log2;       // scale * log2(e)
    int out_dtype;
    // paged_cluster_kernel alone: keys that every sequence has in front of its own
    const int *pre_table, *pre_lens;
    int pre_max_len;
    float *part_o;          // [gridDim.x][2][RB][D], RB >= block_rows the kernel's slot size
    float *part_ml;         // [gridDim.x][2][RB][2]: m (log2 units), l
    int4 *open;             // [gridDim.x][2]: the unit a CTA leaves unfinished
    // One of two passes over the same query rows, each over keys of its own (a shared
    // prefix, then the sequences'), that paged_pair_join_kernel joins: whole units'
    // rows go to dense_* as pieces do, and unit_note says where a unit's pieces are.
    float *dense_o, *dense_ml;  // [total_q][Hq][D] and [total_q][Hq][2], or null: rows go to out
    int2 *unit_note;            // [B][Hkv][row blocks]: the CTA that opened the unit, its pieces (1: dense)
    // Such a pass also leaves SMs to the other one, in proportion to their work.
    const int *peer_lens;       // the other pass's seq_lens
    int peer_B, peer_max_len, peer_tile, peer_unit_steps;
    // a kv head's blocks whose two query tiles, or one, have tokens, and what a key tile costs each
    int peer_both_blocks, peer_both_steps, peer_one_blocks, peer_one_steps;
    int step_ns, peer_step_ns;  // SM time of a step of this pass, and of the other
    int num_sms, per_sm, first; // first: the pass that is launched first
};

struct SeqView {
    int t0, nq, len;
};

__device__ __forceinline__ SeqView paged_seq(const PagedParams &p, int b) {
    SeqView s;
    const int raw = __ldg(p.seq_lens + b);
    s.len = min(max(raw, 0), p.max_len);
    if (p.cu_q) {
        s.t0 = min(max(__ldg(p.cu_q + b), 0), p.total_q);
        s.nq = min(min(max(__ldg(p.cu_q + b + 1), s.t0), p.total_q) - s.t0, p.max_q);
    } else {
        s.t0 = b * p.nq_each;
        s.nq = p.nq_each;
    }
    return s;
}

// Whether paged_seq had to clamp sequence b's length or offsets.
__device__ __forceinline__ bool paged_seq_bad(const PagedParams &p, int b) {
    const int raw = __ldg(p.seq_lens + b);
    bool bad = raw < 0 || raw > p.max_len;
    if (p.cu_q) {
        const int lo = __ldg(p.cu_q + b), hi = __ldg(p.cu_q + b + 1);
        bad |= lo < 0 || hi < lo || hi > p.total_q || hi - lo > p.max_q;
    }
    return bad;
}

// Key tiles (TK keys each) that rows up to last_row of a sequence must visit:
// at least one.
template <int TK>
__device__ __forceinline__ int paged_tiles_to_row(const PagedParams &p, const SeqView &s, int last_row) {
    int seen = s.len;
    if (p.causal) seen = max(0, s.len - s.nq + min(s.nq - 1, last_row / p.G) + 1);
    return max(1, (seen + TK - 1) / TK);
}

__device__ __forceinline__ int paged_blocks(const PagedParams &p, const SeqView &s) {
    return (s.nq * p.G + p.block_rows - 1) / p.block_rows;
}

// How a kernel's work is cut: keys of a tile, and what a key tile costs in steps.  Of
// paged_tiles_kernel's two query tiles (KEYS = 128) a causal or short block has key tiles
// that one alone visits, ONE steps against BOTH.
template <int KEYS, int BOTH, int ONE>
struct PagedCut {
    static constexpr int kKeys = KEYS, kBoth = BOTH, kOne = ONE;
};

using RowsCut = PagedCut<64, 1, 1>;
// (Per CTA of 4 chunks of 700 to 2048 tokens at d = 128 and 3 prompts of 3500 to 5000 at d = 64,
// fitted: a key tile 1.80 us for both and 1.60 for one, and 1.60 and 1.10; a piece 2.64 and 2.39.)
template <int D>
using TilesCut = PagedCut<128, D == 64 ? 3 : 1, D == 64 ? 2 : 1>;

// What row block rb costs, in steps: its unit_steps, then its key tiles in order, those
// that both query tiles visit first.
template <typename C>
struct UnitSteps {
    int tiles, both;  // key tiles, and those for both query tiles
    int total;

    __device__ __forceinline__ UnitSteps(const PagedParams &p, const SeqView &s, int rb) {
        if constexpr (C::kKeys == 128) {
            // (no division by G: the plan goes through all blocks of a causal sequence, and with
            // two divisions each its CTAs started 5 us later for 32 blocks)
            const int tok1 = (2 * rb + 1) * p.tile_tokens;  // the second query tile's first token
            const int past = s.len - s.nq;
            auto tiles_to = [&](int tok) {  // that tokens before tok visit: at least one
                return max(1, ((p.causal ? max(0, past + min(s.nq, tok)) : s.len) + C::kKeys - 1) / C::kKeys);
            };
            tiles = tiles_to(tok1 + p.tile_tokens);
            both = C::kBoth == C::kOne ? tiles : (tok1 < s.nq ? tiles_to(tok1) : 0);
        } else {
            tiles = both = paged_tiles_to_row<C::kKeys>(p, s, rb * p.block_rows + p.block_rows - 1);
        }
        total = before(p, tiles);
    }
    // Steps before key tile j.
    __device__ __forceinline__ int before(const PagedParams &p, int j) const {
        return p.unit_steps + j * C::kOne + min(j, both) * (C::kBoth - C::kOne);
    }
    // Key tiles that start before step v: a range has those that start in it.
    __device__ __forceinline__ int tiles_before(const PagedParams &p, int v) const {
        const int e = max(0, v - p.unit_steps), b = both * C::kBoth;
        return e <= b ? (e + C::kBoth - 1) / C::kBoth : min(tiles, both + (e - b + C::kOne - 1) / C::kOne);
    }
};

// Steps of one kv head of a sequence.
template <typename C>
__device__ __forceinline__ long long paged_head_steps(const PagedParams &p, const SeqView &s) {
    const int n = paged_blocks(p, s);
    if (n == 0) return 0;
    long long sum = UnitSteps<C>(p, s, n - 1).total;
    if (n == 1) return sum;
    if (!p.causal) return sum + static_cast<long long>(n - 1) * UnitSteps<C>(p, s, 0).total;
    for (int rb = 0; rb < n - 1; ++rb) sum += UnitSteps<C>(p, s, rb).total;
    return sum;
}

// ---------------------------------------------------------------- two passes
// Steps of one kv head of the other pass's sequence b: what paged_head_steps gives there
// (neither is causal, and every sequence of a pass has the same number of query tokens).
__device__ __forceinline__ long long paged_peer_steps(const PagedParams &p, int b) {
    const int len = min(max(__ldg(p.peer_lens + b), 0), p.peer_max_len);
    const long long tiles = max(1, (len + p.peer_tile - 1) / p.peer_tile);
    return p.peer_both_blocks * (p.peer_unit_steps + tiles * p.peer_both_steps) +
           p.peer_one_blocks * (p.peer_unit_steps + tiles * p.peer_one_steps);
}

// SMs of the first pass, in proportion to the two passes' work; at least one each.  Both
// passes come to the same number: each one's `theirs` is the other's `mine`.
__device__ __forceinline__ int paged_first_sms(const PagedParams &p, long long mine, long long theirs) {
    const long long mine_ns = mine * p.step_ns, their_ns = theirs * p.peer_step_ns;
    const long long first_ns = p.first ? mine_ns : their_ns;
    return static_cast<int>(min(max(p.num_sms * first_ns / (mine_ns + their_ns), 1LL),
                                static_cast<long long>(max(p.num_sms - 1, 1))));
}

// ---------------------------------------------------------------- host side
// How a call runs, from its sizes alone.
struct PagedPlan {
    bool tiles;      // 128-row tensor-memory tiles (paged_tiles_kernel), else paged_rows_kernel
    int block_rows;  // query rows of a unit
    int slot_rows;   // rows of a partial slot
    int tile;        // keys of a tile
    int per_sm;      // CTAs per SM
    int both_steps, one_steps;  // what a key tile costs (PagedCut)
    int unit_steps;  // what a unit costs besides its key tiles
};

inline PagedPlan plan_paged(int max_q, int group, int d) {
    const long long rows = static_cast<long long>(max_q) * group;
    if (rows > 64 && group <= 128) {
        const int block = 2 * (128 / group) * group;
        return d == 64 ? PagedPlan{true, block, 256, 128, 1, TilesCut<64>::kBoth, TilesCut<64>::kOne, 5}
                       : PagedPlan{true, block, 256, 128, 1, TilesCut<128>::kBoth, TilesCut<128>::kOne, 2};
    }
    const int rb = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
    return {false, rb, rb, RowsCut::kKeys, 2, RowsCut::kBoth, RowsCut::kOne, 2};
}

// CTAs per cluster for a call of `units` units that paged_cluster_kernel serves best, or 0 for
// the split form.  The sizes are bounds: lengths are known on the device only.
//
// A cluster's CTAs take their unit's key tiles one after another, and no other CTA helps them,
// so that the longest sequence sets the time alone, where the split form shares it among all
// SMs but costs a plan and a join (7 us more, and 12 to 17 us with a prefix, whose two passes
// and join it replaces).  So the bound is on the tiles in a row, whatever the number of units, by
// what one takes: at most 10 us, which loses 3 us when one sequence has the
// bound's length and gains 5 when none comes near it.  Measured on 32 units, one sequence of that
// length among short ones, clusters against split: 16 rows of 128, 12 tiles in a row 12.8 us
// against 12.6 and 16 tiles 15.4 against 13.3; 32 rows of 128, 4 tiles 11.8 against 14.5 and 8
// tiles 16.6 against 15.1; 64 rows of 64, 8 tiles 12.5 against 12.2 and 10 tiles 14.3 against
// 12.4.  All of that length: 18.2 against 22.6, 25.5 against 26.3, 12.9 against 18.3, 17.9 against
// 24.2, 15.8 against 20.5, 18.2 against 22.8.  None: 4 sequences of 1000 tokens, 8 kv heads of
// 128, in tables of 8192, 7.0 against 11.9.
inline int paged_cluster_size(const PagedPlan &pl, int d, long long units, long long max_len, long long prefix_max,
                              int num_sms) {
    if (pl.tiles) return 0;
    const long long tiles = (max_len + pl.tile - 1) / pl.tile + (prefix_max + pl.tile - 1) / pl.tile;
    const long long all = static_cast<long long>(pl.per_sm) * num_sms;  // CTAs at a time
    // Clusters of 8 or 4 do not fill the last SMs of every group of SMs: 36 and 74 ran at a time
    // on 152 SMs, and one more made a second wave (16 rows of 128: 8.7 to 13.1 us).
    auto fit = [&](int size) { return units * size <= (size > 2 ? all - all / 20 : all); };
    int size = 8;
    while (size > 1 && (size / 2 >= tiles || !fit(size))) size /= 2;
    if (!fit(size)) return 0;
    const long long tile_ns = pl.block_rows == 16 ? (d == 128 ? 580 : 450) : pl.block_rows == 32 ? (d == 128 ? 950 : 580)
                                                                                               : (d == 128 ? 1700 : 870);
    const long long in_a_row = (tiles + size - 1) / size;
    if (in_a_row * tile_ns <= (prefix_max ? 12000 : 10000)) return size;
    // A prefix is as long for every unit, so that its tiles are shared evenly where the units fill
    // the GPU: up to 18 us of them (36 units of 40 tiles in a row: 20 us, 30 in two passes).
    return prefix_max && in_a_row - units * tiles / all <= 6 && in_a_row * tile_ns <= 18000 ? size : 0;
}

// What a step of a pass costs an SM, in ns; only the ratio of two passes counts.  At d = 128
// measured on runs confined to a few SMs (shared prefix of 16500 tokens for 256 sequences of
// 16 to 1024 own ones, 64 query heads: 202 us with the SMs split so, 228 one after the other).
// At d = 64 what 11 calls of 18 to 256 sequences behind 500 to 30000 tokens took least with:
// 128 sequences of 500 behind 16000, 12 heads: 73 us with 1400, 58 with 2400, 52 with 2600, 54
// with 3000; 256 of them behind 16500, 64 over 8 heads: 165, 145, 152 and 166.
inline int paged_step_ns(const PagedPlan &pl, int d) {
    if (pl.tiles) return (d == 128 ? 1900 : 2400) / pl.both_steps;
    const int ns = pl.block_rows == 16 ? 420 : (pl.block_rows == 32 ? 800 : 1150);
    return d == 128 ? ns : ns * 5 / 6;
}

// p: one of two passes; o: the other, planned so.
inline void paged_set_peer(PagedParams &p, const PagedParams &o, const PagedPlan &plan) {
    const int blocks = static_cast<int>((static_cast<long long>(o.nq_each) * o.G + o.block_rows - 1) / o.block_rows);
    // only the last block's second query tile may be empty
    const bool one = plan.tiles && (2LL * blocks - 1) * o.tile_tokens >= o.nq_each;
    p.peer_lens = o.seq_lens;
    p.peer_B = o.B;
    p.peer_max_len = o.max_len;
    p.peer_tile = plan.tile;
    p.peer_unit_steps = plan.unit_steps;
    p.peer_both_blocks = blocks - (one ? 1 : 0);
    p.peer_both_steps = plan.both_steps;
    p.peer_one_blocks = one ? 1 : 0;
    p.peer_one_steps = plan.one_steps;
    p.peer_step_ns = o.step_ns;
}

}  // namespace fa
