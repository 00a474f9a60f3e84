// fa_paged.cuh -- what the paged-attention kernels share: the launch
// parameters, the cut of the work into equal ranges of key tiles, and the
// writing and joining of rows.
//
// Work.  The cache keeps K and V as [page][kv head][slot][d]; sequence b's
// token j lives in page page_table[b][j / page_size], slot j % page_size.  A
// sequence with nq query tokens gives each kv head nq * G query rows
// (G = query heads per kv head), row r = (token r / G, head r % G), cut into
// blocks of block_rows.  A unit = (sequence, kv head, row block); it costs one
// step per key tile its rows can see (at least one, so that a unit without
// keys still writes its rows).  The W steps of the whole call, in the order
// (sequence, kv head, block), are cut into gridDim.x equal ranges, one per
// CTA, whatever the lengths are: they live on the device, so the cut is made
// there, by every CTA for itself.  A unit inside one range is written
// directly; the pieces of a unit that ranges cut keep (O, m, l) in fp32 and
// paged_join_kernel adds them in CTA order, so a given shape and set of
// lengths gives the same bits on every run.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
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
    if (!p.causal || n == 1) return static_cast<long long>(n) * paged_tiles<TK>(p, s, n - 1);
    long long sum = 0;
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

// Walks a CTA's pieces in order.
template <int TK>
struct PagedCursor {
    SeqView s;
    int b, hk, rb, blocks, j;
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
            const int c = paged_tiles<TK>(p, s, 0);
            rb = static_cast<int>(rem / c);
            j = static_cast<int>(rem - static_cast<long long>(rb) * c);
            return;
        }
        for (rb = 0; rb < blocks - 1; ++rb) {
            const int c = paged_tiles<TK>(p, s, rb);
            if (rem < c) break;
            rem -= c;
        }
        j = static_cast<int>(rem);
    }

    // The next piece; false when the range is used up.  cost: the whole unit's steps.
    __device__ __forceinline__ bool next(const PagedParams &p, PagedPiece &u, int &cost) {
        if (left <= 0) return false;
        cost = paged_tiles<TK>(p, s, rb);
        u.b = b;
        u.t0 = s.t0;
        u.nq = s.nq;
        u.len = s.len;
        u.hk = hk;
        u.row0 = rb * p.block_rows;
        u.j0 = j;
        u.j1 = static_cast<int>(min(static_cast<long long>(cost), j + left));
        u.kind = u.j0 > 0 ? 2 : (u.j1 < cost ? 1 : 0);
        left -= u.j1 - u.j0;
        j = 0;
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
        return true;
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

// What a CTA notes about the unit it leaves unfinished (or that there is none).
__device__ __forceinline__ void paged_note_open(const PagedParams &p, const PagedPiece *u, int cost, long long end,
                                                long long W, int G) {
    int4 *o = p.open + 2 * blockIdx.x;
    if (!u || u->kind != 1) {
        o[0] = make_int4(-1, 0, 0, 0);
        return;
    }
    o[0] = make_int4(paged_cta_of(end + (cost - u->j1) - 1, W, G), u->t0, u->hk, u->row0);
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

// A whole row's (or all pieces') unnormalised columns acc with (m, l), m in log2
// units: joins the optional earlier result and writes out, and the row's lse once.
template <int N>
__device__ __forceinline__ void paged_finish(const PagedParams &p, int D, long long row, int col, float (&acc)[N],
                                             float m, float l) {
    const long long off = row * D + col;
    float inv;
    if (p.init_o) {
        const float mi = p.init_lse[row] * kLog2e;
        const float M = fmaxf(m, mi);
        const float w = ex2_from(m, M), wi = ex2_from(mi, M);
        const float total = fmaf(w, l, wi);
        inv = total > 0.f ? 1.f / total : 0.f;
        const float a = w * inv, c = wi * inv;
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = fmaf(a, acc[e], c * p.init_o[off + e]);
        if (p.lse && col == 0) p.lse[row] = total > 0.f ? (M + __log2f(total)) * kLn2 : -INFINITY;
    } else {
        inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] *= inv;
        if (p.lse && col == 0) p.lse[row] = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
    }
    paged_store<N>(p, off, acc);
}

// N columns of a row of the current piece: finished rows go to out, cut ones to the CTA's partial slot.
template <int D, int RB, int N>
__device__ __forceinline__ void paged_emit(const PagedParams &p, const PagedPiece &u, int r, int col, float (&acc)[N],
                                           float m, float l) {
    const int rr = u.row0 + r;
    if (u.kind == 0) {
        const long long row = (static_cast<long long>(u.t0) + rr / p.G) * p.Hq + u.hk * p.G + rr % p.G;
        paged_finish<N>(p, D, row, col, acc, m, l);
    } else {
        const size_t rec = (static_cast<size_t>(blockIdx.x) * 2 + (u.kind == 1 ? 1 : 0)) * RB + r;
        float *o = p.part_o + rec * D + col;
        if constexpr (N == 4) *reinterpret_cast<float4 *>(o) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        else *reinterpret_cast<float2 *>(o) = make_float2(acc[0], acc[1]);
        if (col == 0) *reinterpret_cast<float2 *>(p.part_ml + rec * 2) = make_float2(m, l);
    }
}

// Joins the pieces of the units that ranges cut.  CTA (c, y): the unit that CTA c
// of the main kernel left open (slot 1 of c, slot 0 of the CTAs after it up to the
// one that closed the unit), rows [y * kJoinRows, ...).  A warp takes a row, its
// lanes D / 32 columns each; pieces are added in CTA order.
constexpr int kJoinWarps = 4;
constexpr int kJoinRows = 8;

template <int D, int RB>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const PagedParams p) {
    constexpr int N = D / 32;
    constexpr int U = 4;  // pieces in flight
    using Vec = typename std::conditional<N == 4, float4, float2>::type;
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 a = p.open[2 * c];
    if (a.x < 0) return;
    const int4 b = p.open[2 * c + 1];
    const int n = a.x - c + 1;  // pieces
    const int rows = min(p.block_rows, b.x * p.G - a.w);
    auto rec = [&](int k, int r) { return (static_cast<size_t>(c + k) * 2 + (k == 0 ? 1 : 0)) * RB + r; };
    for (int r = blockIdx.y * kJoinRows + warp; r < min(rows, (blockIdx.y + 1) * kJoinRows); r += kJoinWarps) {
        float M = -INFINITY;
        for (int k = lane; k < n; k += 32) M = fmaxf(M, p.part_ml[rec(k, r) * 2]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        float acc[N] = {}, L = 0.f;
        for (int k0 = 0; k0 < n; k0 += U) {
            Vec x[U];
            float2 ml[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int k = min(k0 + i, n - 1);
                x[i] = reinterpret_cast<const Vec *>(p.part_o + rec(k, r) * D)[lane];
                ml[i] = *reinterpret_cast<const float2 *>(p.part_ml + rec(k, r) * 2);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float w = k0 + i < n ? ex2_from(ml[i].x, M) : 0.f;
                const float *xv = reinterpret_cast<const float *>(&x[i]);
                if (w > 0.f) {  // a piece without visible keys leaves l = 0 and no weight
                    L = fmaf(w, ml[i].y, L);
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[e] = fmaf(w, xv[e], acc[e]);
                }
            }
        }
        const int rr = a.w + r;
        const long long row = (static_cast<long long>(a.y) + rr / p.G) * p.Hq + a.z * p.G + rr % p.G;
        paged_finish<N>(p, D, row, lane * N, acc, M, L);
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

template <int D, int RB>
int launch_join(const PagedParams &p, int grid, cudaStream_t stream) {
    PagedConfig cfg(dim3(grid, (p.block_rows + kJoinRows - 1) / kJoinRows), kJoinWarps * 32, 0, true, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, paged_join_kernel<D, RB>, p);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

}  // namespace fa
