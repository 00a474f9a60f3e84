// fa_paged.cuh -- what the paged-attention kernels share: the launch
// parameters, the cut of the work into equal ranges of key tiles, and the
// writing and joining of rows.
//
// Work.  The cache keeps K and V as [page][kv head][slot][d]; sequence b's
// token j lives in page page_table[b][j / page_size], slot j % page_size.  A
// sequence with nq query tokens gives each kv head nq * G query rows
// (G = query heads per kv head), row r = (token r / G, head r % G), cut into
// blocks of block_rows.  A unit = (sequence, kv head, row block); it costs
// unit_steps for its own start and end and a step per key tile its rows can see
// (at least one, so that a unit without keys still writes its rows).  The W steps of the whole call, in the order
// (sequence, kv head, block), are cut into gridDim.x equal ranges, one per
// CTA, whatever the lengths are: they live on the device, so the cut is made
// there, by every CTA for itself.  A unit inside one range is written
// directly; the pieces of a unit that ranges cut keep (O, m, l) in fp32 and
// paged_join_kernel adds them in CTA order, so a given shape and set of
// lengths gives the same bits on every run.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <algorithm>
#include <atomic>
#include <cstdint>

#include "fa_internal.h"
#include "fa_tiles.cuh"
#include "sm103_ptx.cuh"

namespace fa {

struct PagedParams {
    const uint16_t *q;     // [total_q][Hq][D]
    void *out;             // [total_q][Hq][D]
    float *lse;            // optional [total_q][Hq]: natural-log row log-sum-exp, -inf for a row without keys
    // Optional result over other keys that the rows also see (a shared prefix):
    // normalised fp32 rows and their natural-log log-sum-exp, joined at the end.
    const float *init_o, *init_lse;
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
    int causal;             // query token i of nq sees keys j <= len - nq + i
    float scale_log2;       // scale * log2(e)
    int out_dtype;
    float *part_o;          // [gridDim.x][2][RB][D], RB >= block_rows the kernel's slot size
    float *part_ml;         // [gridDim.x][2][RB][2]: m (log2 units), l
    int4 *open;             // [gridDim.x][2]: the unit a CTA leaves unfinished
};

// Bounded wait in which every lane polls the barrier itself, so that every lane's
// loads come after the phase it waited for (one lane's wait and a shuffle order
// nothing for the loads of the other lanes).
__device__ __forceinline__ bool lanes_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, kWatchdogNs));
}

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

// Key tiles (TK keys each) that rows up to last_row of a sequence, or row block rb, must
// visit: at least one.
template <int TK>
__device__ __forceinline__ int paged_tiles_to_row(const PagedParams &p, const SeqView &s, int last_row) {
    int seen = s.len;
    if (p.causal) seen = max(0, s.len - s.nq + min(s.nq - 1, last_row / p.G) + 1);
    return max(1, (seen + TK - 1) / TK);
}

template <int TK>
__device__ __forceinline__ int paged_tiles(const PagedParams &p, const SeqView &s, int rb) {
    return paged_tiles_to_row<TK>(p, s, rb * p.block_rows + p.block_rows - 1);
}

__device__ __forceinline__ int paged_blocks(const PagedParams &p, const SeqView &s) {
    return (s.nq * p.G + p.block_rows - 1) / p.block_rows;
}

// Steps of one kv head of a sequence.
template <int TK>
__device__ __forceinline__ long long paged_head_steps(const PagedParams &p, const SeqView &s) {
    const int n = paged_blocks(p, s);
    if (n == 0) return 0;
    long long sum = static_cast<long long>(n) * p.unit_steps;
    if (!p.causal || n == 1) return sum + static_cast<long long>(n) * paged_tiles<TK>(p, s, n - 1);
    for (int rb = 0; rb < n; ++rb) sum += paged_tiles<TK>(p, s, rb);
    return sum;
}

// Where a CTA's range of steps starts.
struct PagedStart {
    long long W;    // steps of the call
    long long rem;  // steps of sequence b before the range
    long long first, end;
    int b;
    int G;          // CTAs with work: every one of them has at least one step
};

// The whole CTA (NT threads) adds up the sequences' steps and finds its range.
template <int TK, int NT>
__device__ __forceinline__ void paged_plan(const PagedParams &p, PagedStart &st, long long *warp_sum, int *status) {
    constexpr int NW = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + NT - 1) / NT;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long mine = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        mine += paged_head_steps<TK>(p, paged_seq(p, b)) * p.Hkv;
        bad |= paged_seq_bad(p, b);
    }
    if (bad && blockIdx.x == 0) atomicCAS(status, 0, static_cast<int>(FA_ERR_SEQ_LEN));
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long before = incl - mine, W = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const long long v = warp_sum[w];
        if (w < warp) before += v;
        W += v;
    }
    const int c = blockIdx.x;
    const int G = static_cast<int>(min(static_cast<long long>(gridDim.x), max(W, 1LL)));
    const long long first = c < G ? c * W / G : W;
    const long long end = c < G ? (c + 1) * W / G : W;
    if (tid == 0) {
        st.W = W;
        st.G = G;
        st.first = first;
        st.end = end;
    }
    if (first < end && before <= first && first < before + mine) {
        long long rem = first - before;
        int b = b0;
        for (; b < b1 - 1; ++b) {
            const long long c = paged_head_steps<TK>(p, paged_seq(p, b)) * p.Hkv;
            if (rem < c) break;
            rem -= c;
        }
        st.b = b;
        st.rem = rem;
    }
    __syncthreads();
}

// One piece of a unit, as the producer hands it to the other warps.
struct PagedPiece {
    int b, t0, nq, len;
    int hk, row0;   // row0: first row of the block among the nq * G rows
    int j0, j1;     // key tiles
    int kind;       // 0 whole unit, 1 opens a unit that the next CTA continues, 2 continues one, -1 no more work
};

// Walks a CTA's pieces in order.  A unit's steps are its unit_steps, then its key
// tiles: a range that ends among the former leaves the whole unit to the next CTA.
template <int TK>
struct PagedCursor {
    SeqView s;
    int b, hk, rb, blocks, v;  // v: the next step of unit (b, hk, rb)
    long long left;

    __device__ __forceinline__ void begin(const PagedParams &p, const PagedStart &st) {
        left = st.end - st.first;
        if (left <= 0) return;
        b = st.b;
        s = paged_seq(p, b);
        blocks = paged_blocks(p, s);
        const long long per_head = paged_head_steps<TK>(p, s);
        hk = static_cast<int>(st.rem / per_head);
        long long rem = st.rem - hk * per_head;
        if (!p.causal) {
            const int c = paged_tiles<TK>(p, s, 0) + p.unit_steps;
            rb = static_cast<int>(rem / c);
            v = static_cast<int>(rem - static_cast<long long>(rb) * c);
            return;
        }
        for (rb = 0; rb < blocks - 1; ++rb) {
            const int c = paged_tiles<TK>(p, s, rb) + p.unit_steps;
            if (rem < c) break;
            rem -= c;
        }
        v = static_cast<int>(rem);
    }

    // The next piece with key tiles; false when the range is used up.  tiles: the whole unit's.
    __device__ __forceinline__ bool next(const PagedParams &p, PagedPiece &u, int &tiles) {
        while (left > 0) {
            const int t = paged_tiles<TK>(p, s, rb), cost = t + p.unit_steps;
            const int end = static_cast<int>(min(static_cast<long long>(cost), v + left));
            const int j0 = max(0, v - p.unit_steps), j1 = max(0, end - p.unit_steps);
            const bool some = j1 > j0;
            if (some) {
                tiles = t;
                u.b = b;
                u.t0 = s.t0;
                u.nq = s.nq;
                u.len = s.len;
                u.hk = hk;
                u.row0 = rb * p.block_rows;
                u.j0 = j0;
                u.j1 = j1;
                u.kind = j0 > 0 ? 2 : (j1 < t ? 1 : 0);
            }
            left -= end - v;
            v = 0;
            if (left > 0 && ++rb == blocks) {
                rb = 0;
                if (++hk == p.Hkv) {
                    hk = 0;
                    do {  // steps are left, so a later sequence has rows
                        s = paged_seq(p, ++b);
                        blocks = paged_blocks(p, s);
                    } while (blocks == 0);
                }
            }
            if (some) return true;
        }
        return false;
    }
};

// The CTA whose range holds `step`.
__device__ __forceinline__ int paged_cta_of(long long step, long long W, int G) {
    long long c = ((step + 1) * G - 1) / W;
    if (c >= G) c = G - 1;
    while (c > 0 && c * W / G > step) --c;
    while (c + 1 < G && (c + 1) * W / G <= step) ++c;
    return static_cast<int>(c);
}

// What a CTA notes about the unit it leaves unfinished (or that there is none): u, its
// last piece, ended where the CTA's range does.
__device__ __forceinline__ void paged_note_open(const PagedParams &p, const PagedPiece *u, int tiles, long long end,
                                                long long W, int G) {
    int4 *o = p.open + 2 * blockIdx.x;
    if (!u || u->kind != 1) {
        o[0] = make_int4(-1, 0, 0, 0);
        return;
    }
    o[0] = make_int4(paged_cta_of(end + (tiles - u->j1) - 1, W, G), u->t0, u->hk, u->row0);
    o[1] = make_int4(u->nq, 0, 0, 0);
}

// ---------------------------------------------------------------- rows out
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2_from(float m, float M) { return m == -INFINITY ? 0.f : ex2_approx(m - M); }

// N consecutive columns of a finished row at element offset `off`.
template <int N>
__device__ __forceinline__ void paged_store(const PagedParams &p, long long off, const float (&v)[N]) {
    if (p.out_dtype == FA_F32) {
        float *o = reinterpret_cast<float *>(p.out) + off;
        if constexpr (N == 4) *reinterpret_cast<float4 *>(o) = make_float4(v[0], v[1], v[2], v[3]);
        else *reinterpret_cast<float2 *>(o) = make_float2(v[0], v[1]);
    } else {
        const int bf = p.out_dtype == FA_BF16;
        uint16_t *o = reinterpret_cast<uint16_t *>(p.out) + off;
        if constexpr (N == 4)
            *reinterpret_cast<uint2 *>(o) = make_uint2(pack2(v[0], v[1], bf), pack2(v[2], v[3], bf));
        else
            *reinterpret_cast<uint32_t *>(o) = pack2(v[0], v[1], bf);
    }
}

// N columns of the earlier result of a row, loaded ahead of their use.
template <int N>
struct PagedInit {
    float o[N], m;  // m: log2 units
    __device__ __forceinline__ void load(const PagedParams &p, int D, long long row, int col) {
        if (!p.init_o) return;
        const float *src = p.init_o + row * D + col;
        m = p.init_lse[row] * kLog2e;
        if constexpr (N == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(src);
            o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(src);
            o[0] = v.x; o[1] = v.y;
        }
    }
};

// A whole row's (or all pieces') unnormalised columns acc with (m, l), m in log2
// units: joins the optional earlier result and writes out, and the row's lse once.
template <int N>
__device__ __forceinline__ void paged_finish(const PagedParams &p, int D, long long row, int col, float (&acc)[N],
                                             float m, float l, const PagedInit<N> &init) {
    const long long off = row * D + col;
    float inv;
    if (p.init_o) {
        const float M = fmaxf(m, init.m);
        const float w = ex2_from(m, M), wi = ex2_from(init.m, M);
        const float total = fmaf(w, l, wi);
        inv = total > 0.f ? 1.f / total : 0.f;
        const float a = w * inv, c = wi * inv;
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = fmaf(a, acc[e], c * init.o[e]);
        if (p.lse && col == 0) p.lse[row] = total > 0.f ? (M + __log2f(total)) * kLn2 : -INFINITY;
    } else {
        inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] *= inv;
        if (p.lse && col == 0) p.lse[row] = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
    }
    paged_store<N>(p, off, acc);
}

// Row r of a block among the rows of the output.
__device__ __forceinline__ long long paged_row(const PagedParams &p, const PagedPiece &u, int r) {
    const int rr = u.row0 + r;
    return (static_cast<long long>(u.t0) + rr / p.G) * p.Hq + u.hk * p.G + rr % p.G;
}

// N columns of a row of the current piece: finished rows go to out, cut ones to the CTA's partial slot.
template <int D, int RB, int N>
__device__ __forceinline__ void paged_emit(const PagedParams &p, const PagedPiece &u, int r, long long row, int col,
                                           float (&acc)[N], float m, float l, const PagedInit<N> &init) {
    if (u.kind == 0) {
        paged_finish<N>(p, D, row, col, acc, m, l, init);
    } else {
        const size_t rec = (static_cast<size_t>(blockIdx.x) * 2 + (u.kind == 1 ? 1 : 0)) * RB + r;
        float *o = p.part_o + rec * D + col;
        if constexpr (N == 4) *reinterpret_cast<float4 *>(o) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        else *reinterpret_cast<float2 *>(o) = make_float2(acc[0], acc[1]);
        if (col == 0) *reinterpret_cast<float2 *>(p.part_ml + rec * 2) = make_float2(m, l);
    }
}

// Joins the pieces of the units that ranges cut: the unit that CTA c of the main
// kernel left open has its pieces in slot 1 of c and slot 0 of the CTAs after it, up
// to the one that closed the unit.  They are added in CTA order.
// All latency.  Every CTA reads all notes at once and numbers the items (two rows
// of a unit of at most four pieces, or one row of one with more), the warps of the
// grid take the items in turn, and an item's loads (2 rows x 4 pieces, or 12
// pieces) are in flight together.
constexpr int kJoinThreads = 256;
constexpr int kJoinMax = 512;  // CTAs of the main kernel

template <int D, int RB, int R, int F>
__device__ __forceinline__ void paged_join_rows(const PagedParams &p, int c, const int4 &a, int r0, int rows, int lane) {
    constexpr int N = D / 32;
    using Vec = typename std::conditional<N == 4, float4, float2>::type;
    const int n = a.x - c + 1;  // pieces
    auto rec = [&](int k, int r) { return (static_cast<size_t>(c + k) * 2 + (k == 0 ? 1 : 0)) * RB + r; };
    float M[R], L[R], acc[R][N];
    PagedInit<N> init[R];
    long long row[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        M[r] = -INFINITY;
        L[r] = 0.f;
        const int rr = a.w + min(r0 + r, rows - 1);
        row[r] = (static_cast<long long>(a.y) + rr / p.G) * p.Hq + a.z * p.G + rr % p.G;
        init[r].load(p, D, row[r], lane * N);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[r][e] = 0.f;
    }
    for (int k0 = 0; k0 < n; k0 += F) {
        Vec x[R][F];
        // lane i * R + r holds the (m, l) of piece k0 + i and row r
        const int lk = k0 + lane / R, lr = r0 + lane % R;
        const float2 ml = lane < R * F && lk < n && lr < rows
                              ? *reinterpret_cast<const float2 *>(p.part_ml + rec(lk, lr) * 2)
                              : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (k0 + i < n && r0 + r < rows)
                    x[r][i] = reinterpret_cast<const Vec *>(p.part_o + rec(k0 + i, r0 + r) * D)[lane];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float next = M[r], mi[F];
#pragma unroll
            for (int i = 0; i < F; ++i) {
                mi[i] = __shfl_sync(0xffffffffu, ml.x, i * R + r);
                next = fmaxf(next, mi[i]);
            }
            const float keep = ex2_from(M[r], next);
            M[r] = next;
            L[r] *= keep;
#pragma unroll
            for (int e = 0; e < N; ++e) acc[r][e] *= keep;
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const float w = ex2_from(mi[i], next), li = __shfl_sync(0xffffffffu, ml.y, i * R + r);
                if (w > 0.f) {  // 0: the row saw no key in this piece, whose columns may be unwritten
                    const float *xv = reinterpret_cast<const float *>(&x[r][i]);
                    L[r] = fmaf(w, li, L[r]);
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[r][e] = fmaf(w, xv[e], acc[r][e]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (r0 + r < rows) paged_finish<N>(p, D, row[r], lane * N, acc[r], M[r], L[r], init[r]);
}

template <int D, int RB>
__global__ void __launch_bounds__(kJoinThreads, 2) paged_join_kernel(const PagedParams p, const int ctas) {
    __shared__ int4 note[kJoinMax];
    __shared__ int first[kJoinMax];  // items before CTA c's unit
    __shared__ int rows_of[kJoinMax];
    __shared__ int warp_items[kJoinThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kEach = kJoinMax / kJoinThreads;
    int items[kEach], mine = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int c = tid * kEach + i;
        items[i] = 0;
        if (c < ctas) {
            const int4 a = p.open[2 * c], b = p.open[2 * c + 1];
            note[c] = a;
            if (a.x >= 0) {
                const int rows = min(p.block_rows, b.x * p.G - a.w);
                rows_of[c] = rows;
                items[i] = a.x - c < 4 ? (rows + 1) / 2 : rows;
            }
        }
        mine += items[i];
    }
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) warp_items[warp] = incl;
    __syncthreads();
    int before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
        if (w < warp) before += warp_items[w];
        total += warp_items[w];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (tid * kEach + i < ctas) first[tid * kEach + i] = before;
        before += items[i];
    }
    __syncthreads();
    for (int item = blockIdx.x * (kJoinThreads / 32) + warp; item < total; item += gridDim.x * (kJoinThreads / 32)) {
        int lo = 0, hi = ctas - 1;  // the last c with first[c] <= item (those without a unit have none after it)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= item) lo = mid; else hi = mid - 1;
        }
        const int4 a = note[lo];
        const int i = item - first[lo];
        if (a.x - lo < 4) paged_join_rows<D, RB, 2, 4>(p, lo, a, i * 2, rows_of[lo], lane);
        else paged_join_rows<D, RB, 1, 12>(p, lo, a, i, rows_of[lo], lane);
    }
}

// ---------------------------------------------------------------- host side
// Pages [page][head][slot][d] with any strides as (d, slots, heads, pages), copied
// in boxes of 64 columns x min(page size, tile) slots, 128-byte swizzled.  A page
// index of num_pages reads as zeros.
inline int make_page_map(CUtensorMap *map, const void *base, const fa_paged_cache &c, int tile) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cuda_fail(cudaErrorNotSupported);
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.num_heads,
                                (cuuint64_t)c.num_pages};
    // the stride of an extent of one is never used, and may be anything in a view
    const cuuint64_t row = (cuuint64_t)c.head_dim * 2;
    const cuuint64_t strides[3] = {(cuuint64_t)c.slot_stride * 2,
                                   c.num_heads > 1 ? (cuuint64_t)c.head_stride * 2 : row,
                                   c.num_pages > 1 ? (cuuint64_t)c.page_stride * 2 : row};
    const cuuint32_t box[4] = {64, (cuuint32_t)(c.page_size < tile ? c.page_size : tile), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = enc(map, c.dtype == FA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                     const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cuda_fail(cudaErrorInvalidValue);
    return FA_OK;
}

int launch_paged_tiles(const PagedLaunch &a, const PagedParams &p, int grid, cudaStream_t stream);

// Launch attributes of the paged kernels; `early`: may start before the kernels
// ahead of it in the stream have finished (it waits for them where it must).
struct PagedConfig {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[1];
    PagedConfig(dim3 grid, int threads, size_t smem, bool early, cudaStream_t stream) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        c.gridDim = grid;
        c.blockDim = dim3(threads);
        c.dynamicSmemBytes = smem;
        c.stream = stream;
        c.attrs = attr;
        c.numAttrs = early ? 1 : 0;
    }
    PagedConfig(const PagedConfig &) = delete;
};

// Dynamic shared memory of a kernel allowed on a device, once (`ready`: a static
// array of the kernel's own); min_regs: registers at launch that its setmaxnreg
// split needs (it would wait forever with fewer).
template <typename K>
int ready_kernel(K kernel, int smem, int min_regs, int device, std::atomic<bool> *ready) {
    if (ready[device].load(std::memory_order_acquire)) return FA_OK;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_fail(e);
    cudaFuncAttributes f;
    if ((e = cudaFuncGetAttributes(&f, kernel)) != cudaSuccess) return cuda_fail(e);
    if (f.numRegs < min_regs) return cuda_fail(cudaErrorInvalidConfiguration);
    ready[device].store(true, std::memory_order_release);
    return FA_OK;
}

// ctas: the main kernel's; units: no more units than this exist.
template <int D, int RB>
int launch_join(const PagedParams &p, int ctas, long long units, int num_sms, cudaStream_t stream) {
    if (ctas > kJoinMax) return cuda_fail(cudaErrorInvalidConfiguration);
    const long long items = std::min<long long>(ctas, units) * p.block_rows, warps = kJoinThreads / 32;
    const int grid = static_cast<int>(std::min<long long>(2LL * num_sms, (items + warps - 1) / warps));
    PagedConfig cfg(grid, kJoinThreads, 0, true, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, paged_join_kernel<D, RB>, p, ctas);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

}  // namespace fa
