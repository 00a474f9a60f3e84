// fa_paged.cuh -- what the paged-attention kernels share: a CTA's walk through
// its range of the work (fa_paged_cut.cuh), and the writing and joining of rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <algorithm>
#include <atomic>
#include <cstdint>

#include "fa_internal.h"
#include "fa_paged_cut.cuh"
#include "fa_status.cuh"
#include "fa_tiles.cuh"
#include "sm103_ptx.cuh"

namespace fa {

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar,
                                            int c0, int c1, int c2, int c3, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
        "l"(policy)
        : "memory");
}

// Bounded wait in which every lane polls the barrier itself, so that every lane's
// loads come after the phase it waited for (one lane's wait and a shuffle order
// nothing for the loads of the other lanes).
__device__ __forceinline__ bool lanes_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, kWatchdogNs));
}

// Every paged kernel may be launched while the kernels ahead of it in the stream
// still run; it sets itself up and touches nothing in global memory before they
// are done.  What follows it is let go only after that, so whatever is launched
// early behind it may read what was complete before it.  The second of two passes
// over the same rows is the exception: it reads nothing that the first one writes,
// and the first one has been through here.
__device__ __forceinline__ void paged_wait(const PagedParams &p) {
    if (!p.peer_lens || p.first) asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void paged_let_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void paged_enter(const PagedParams &p) {
    paged_wait(p);
    paged_let_go();
}

// Whoever waits for the second of two passes also waits for the first: one CTA of it stays
// until the first has finished.  (While all of them stayed, those of its CTAs that had no
// room yet, though nothing to do, came after the first pass, and the join after them: 67 us
// against 65 for a prefix of 32801 and 64 sequences.)
__device__ __forceinline__ void paged_leave(const PagedParams &p) {
    if (p.peer_lens && !p.first && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
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
template <typename C, int NT>
__device__ __forceinline__ void paged_plan(const PagedParams &p, PagedStart &st, long long *warp_sum, int *status) {
    constexpr int NW = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + NT - 1) / NT;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long mine = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        mine += paged_head_steps<C>(p, paged_seq(p, b)) * p.Hkv;
        bad |= paged_seq_bad(p, b);
    }
    if (bad && blockIdx.x == 0) record_status(status, FA_ERR_SEQ_LEN);
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
    int most = gridDim.x;
    if (p.peer_lens) {  // SMs in proportion to the two passes' work, at least one each
        long long theirs = 0;
        for (int b = tid; b < p.peer_B; b += NT) {
            theirs += paged_peer_steps(p, b);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) theirs += __shfl_xor_sync(0xffffffffu, theirs, off);
        __syncthreads();
        if (lane == 0) warp_sum[warp] = theirs;
        __syncthreads();
        theirs = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) theirs += warp_sum[w];
        const int first_sms = paged_first_sms(p, W, theirs * p.Hkv);
        most = min(most, p.per_sm * (p.first ? first_sms : max(p.num_sms - first_sms, 1)));
    }
    const int c = blockIdx.x;
    // (a range holds a key tile at least, but for those in a unit's first steps)
    const int G = static_cast<int>(min(static_cast<long long>(most), max(W / C::kBoth, 1LL)));
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
            const long long c = paged_head_steps<C>(p, paged_seq(p, b)) * p.Hkv;
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
    int end0, end1; // paged_tiles_kernel: the piece's key tiles for its two query tiles are [j0, end0), [j0, end1)
    int kind;       // 0 whole unit, 1 opens a unit that the next CTA continues, 2 continues one, -1 no more work
};

// True never, and known only when a piece is in registers, in every lane: what hands its
// place back hangs on it (see PagedRows::loads_pending).  zero: a mask that is zero, which the
// compiler does not know.
__device__ __forceinline__ bool paged_pending(const PagedPiece &u, int zero) {
    const int x = u.b | u.t0 | u.nq | u.len | u.hk | u.row0 | u.j0 | u.j1 | u.end0 | u.end1 | u.kind;
    return __any_sync(0xffffffffu, (x & zero) != 0);
}

// Walks a CTA's pieces in order (UnitSteps: a range that ends among a unit's unit_steps
// leaves the whole unit to the next CTA).
template <typename C>
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
        const long long per_head = max(paged_head_steps<C>(p, s), 1LL);
        hk = static_cast<int>(st.rem / per_head);
        long long rem = st.rem - hk * per_head;
        if (!p.causal) {
            const int c = UnitSteps<C>(p, s, 0).total;  // (the last block's may be less)
            rb = static_cast<int>(rem / c);
            v = static_cast<int>(rem - static_cast<long long>(rb) * c);
            return;
        }
        for (rb = 0; rb < blocks - 1; ++rb) {
            const int c = UnitSteps<C>(p, s, rb).total;
            if (rem < c) break;
            rem -= c;
        }
        v = static_cast<int>(rem);
    }

    // The next piece with key tiles; false when the range is used up.  to_last: steps from
    // the piece's end to the start of the unit's last tile (of a piece that opens a unit).
    __device__ __forceinline__ bool next(const PagedParams &p, PagedPiece &u, int &to_last) {
        while (left > 0) {
            const UnitSteps<C> c(p, s, rb);
            const int end = static_cast<int>(min(static_cast<long long>(c.total), v + left));
            const int j0 = c.tiles_before(p, v), j1 = c.tiles_before(p, end);
            const bool some = j1 > j0;
            if (some) {
                to_last = c.before(p, c.tiles - 1) - end;
                u.b = b;
                u.t0 = s.t0;
                u.nq = s.nq;
                u.len = s.len;
                u.hk = hk;
                u.row0 = rb * p.block_rows;
                u.j0 = j0;
                u.j1 = j1;
                u.kind = j0 > 0 ? 2 : (j1 < c.tiles ? 1 : 0);
            }
            left -= end - v;
            v = 0;
            if (left > 0 && ++rb == blocks) {
                rb = 0;
                if (++hk == p.Hkv) {
                    hk = 0;
                    blocks = 0;
                    while (blocks == 0 && b + 1 < p.B) {  // steps are left, so a later sequence has rows
                        s = paged_seq(p, ++b);
                        blocks = paged_blocks(p, s);
                    }
                    if (blocks == 0) left = 0;
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

// Where a unit's pieces are, for paged_pair_join_kernel: noted by the CTA whose piece starts it.
__device__ __forceinline__ void paged_note_unit(const PagedParams &p, const PagedPiece &u, int to_last, const PagedStart &st) {
    if (!p.unit_note || u.kind == 2) return;
    const int blocks = (u.nq * p.G + p.block_rows - 1) / p.block_rows;
    int2 *note = p.unit_note + (static_cast<long long>(u.b) * p.Hkv + u.hk) * blocks + u.row0 / p.block_rows;
    const int c = blockIdx.x;
    *note = u.kind == 0 ? make_int2(c, 1)
                        : make_int2(c, paged_cta_of(st.end + to_last, st.W, st.G) - c + 1);
}

// What a CTA notes about the unit it leaves unfinished: u, its last piece, ended where the
// CTA's range does.  Without one (and while there is none: a CTA that gives up notes no
// more) the note says so.
__device__ __forceinline__ void paged_note_none(const PagedParams &p) {
    p.open[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
}
__device__ __forceinline__ void paged_note_open(const PagedParams &p, const PagedPiece &u, int to_last, const PagedStart &st) {
    int4 *o = p.open + 2 * blockIdx.x;
    o[1] = make_int4(u.nq, 0, 0, 0);
    o[0] = make_int4(paged_cta_of(st.end + to_last, st.W, st.G), u.t0, u.hk, u.row0);
}

// ---------------------------------------------------------------- drafted trees
// Which of a sequence's keys k0 .. k0 + 31 query token `token` sees, as bits; bits of nodes behind
// the sequence's last one count for nothing.
__device__ __forceinline__ uint32_t tree_seen32(const PagedParams &p, const SeqView &s, const uint32_t *row, int k0) {
    const int n = k0 - (s.len - s.nq);  // the node whose key is k0; below 0 lies the context
    if (n <= -32) return 0xffffffffu;
    const int w = n >> 5;
    const uint32_t lo = w >= 0 && w < p.tree_words ? __ldg(row + w) : 0u;
    const uint32_t hi = w + 1 < p.tree_words ? __ldg(row + w + 1) : 0u;
    uint32_t seen = __funnelshift_r(lo, hi, n & 31);
    if (n < 0) seen |= (1u << -n) - 1u;
    const int left = s.nq - n;
    if (left < 32) seen &= left <= 0 ? 0u : (1u << left) - 1u;
    return seen;
}
// The mask row of query row rr of a sequence (rows behind its last token: that token's).
__device__ __forceinline__ const uint32_t *tree_row(const PagedParams &p, const SeqView &s, int rr) {
    return p.tree + static_cast<long long>(s.t0 + min(rr / p.G, s.nq - 1)) * p.tree_words;
}
// The same for keys k0 .. k0 + 63 and query row rr.
__device__ __forceinline__ uint64_t tree_seen64(const PagedParams &p, const SeqView &s, int rr, int k0) {
    if (k0 + 64 <= s.len - s.nq) return ~0ull;  // context alone
    const uint32_t *row = tree_row(p, s, rr);
    return tree_seen32(p, s, row, k0) | static_cast<uint64_t>(tree_seen32(p, s, row, k0 + 32)) << 32;
}

// ---------------------------------------------------------------- rows out
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2_from(float m, float M) { return m == -INFINITY ? 0.f : ex2_approx(m - M); }

// Whether a row has seen a key, by its sum, to which the key whose score is m added 1 or more.
// (m does not tell: a maximum passes NaN over, so a row of NaN scores has m = -inf like one without
// keys.  Its l is NaN, as is that of a row with a score of +inf, and has to reach the output.)
__device__ __forceinline__ bool saw_key(float l) { return l != 0.f; }

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
// units: writes out, and the row's lse once.
template <int N>
__device__ __forceinline__ void paged_finish(const PagedParams &p, int D, long long row, int col, float (&acc)[N],
                                             float m, float l) {
    const float inv = saw_key(l) ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] *= inv;
    if (p.lse && col == 0) p.lse[row] = saw_key(l) ? (m + __log2f(l)) * kLn2 : -INFINITY;
    paged_store<N>(p, row * D + col, acc);
}

// Row r of a block among the rows of the output.
__device__ __forceinline__ long long paged_row(const PagedParams &p, const PagedPiece &u, int r) {
    const int rr = u.row0 + r;
    return (static_cast<long long>(u.t0) + rr / p.G) * p.Hq + u.hk * p.G + rr % p.G;
}

// Whether a piece's rows are kept as they are (unnormalised, with their m and l) for a
// join, and the record of its row r in part_* or, for a whole unit, of row `row` in dense_*.
__device__ __forceinline__ bool paged_keeps(const PagedParams &p, const PagedPiece &u) {
    return u.kind != 0 || p.dense_o != nullptr;
}
template <int RB>
__device__ __forceinline__ long long paged_record(const PagedPiece &u, int r, long long row) {
    return u.kind == 0 ? row : (static_cast<long long>(blockIdx.x) * 2 + (u.kind == 1 ? 1 : 0)) * RB + r;
}

// N columns of row r of the current piece, row `row` of the output.
template <int D, int RB, int N>
__device__ __forceinline__ void paged_emit(const PagedParams &p, const PagedPiece &u, int r, long long row, int col,
                                           float (&acc)[N], float m, float l) {
    if (!paged_keeps(p, u)) {
        paged_finish<N>(p, D, row, col, acc, m, l);
        return;
    }
    const long long rec = paged_record<RB>(u, r, row);
    float *o = (u.kind == 0 ? p.dense_o : p.part_o) + rec * D + col;
    if constexpr (N == 4) *reinterpret_cast<float4 *>(o) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    else *reinterpret_cast<float2 *>(o) = make_float2(acc[0], acc[1]);
    if (col == 0) *reinterpret_cast<float2 *>((u.kind == 0 ? p.dense_ml : p.part_ml) + rec * 2) = make_float2(m, l);
}

// Joins the pieces of the units that ranges cut: the unit that CTA c of the main
// kernel left open has its pieces in slot 1 of c and slot 0 of the CTAs after it, up
// to the one that closed the unit.  O = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k.
// All latency.  Every CTA reads all notes at once and numbers the items (four rows of
// a unit of two pieces, as most are that hold many rows, two of one of three or four, or
// one row of one with more), the warps of the grid share the items out, and an item's
// loads (4 rows x 2 pieces, 2 x 4, or 8 pieces) are in flight together.  Where the items
// leave most warps idle, a CTA takes an item and its warps a share of the pieces each
// (one long sequence: 300 pieces of 64 rows took 26 us a warp per row).  8 us for 303 units
// of 4 rows, 13.5 us for 151 of 256 (39 MB of pieces, out of L2).
constexpr int kJoinThreads = 256;
// CTAs per SM (d = 64: 3 take 2.5 us less than 2 for 151 units of 256 rows; d = 128 at 3: spills, 7 us more)
template <int D>
constexpr int kJoinPerSm = D == 64 ? 3 : 2;
constexpr int kJoinMax = 512;  // CTAs of the main kernel

// The sums of R rows over n pieces, F pieces at a time: ml_at(k, r) and row_at(k, r)
// give a piece's (m, l) and its columns.  Lanes hold D / 32 columns each.
template <int D, int R, int F, typename MlAt, typename RowAt>
__device__ __forceinline__ void paged_add_pieces(int n, int rows, int lane, MlAt ml_at, RowAt row_at, float (&M)[R],
                                                 float (&L)[R], float (&acc)[R][D / 32]) {
    constexpr int N = D / 32;
    using Vec = typename std::conditional<N == 4, float4, float2>::type;
    static_assert(R * F <= 32, "a lane per (m, l)");
#pragma unroll
    for (int r = 0; r < R; ++r) {
        M[r] = -INFINITY;
        L[r] = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) acc[r][e] = 0.f;
    }
    for (int k0 = 0; k0 < n; k0 += F) {
        Vec x[R][F];
        // lane i * R + r holds the (m, l) of piece k0 + i and row r
        const int lk = k0 + lane / R, lr = lane % R;
        const float2 ml = lane < R * F && lk < n && lr < rows ? ml_at(lk, lr) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (k0 + i < n && r < rows) x[r][i] = reinterpret_cast<const Vec *>(row_at(k0 + i, r))[lane];
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
                if (saw_key(li)) {  // else the piece's columns may be unwritten
                    const float *xv = reinterpret_cast<const float *>(&x[r][i]);
                    L[r] = fmaf(w, li, L[r]);
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[r][e] = fmaf(w, xv[e], acc[r][e]);
                }
            }
        }
    }
}

template <int D, int RB, int R, int F>
__device__ __forceinline__ void paged_join_rows(const PagedParams &p, int c, const int4 &a, int r0, int rows, int lane,
                                                int k0, int n, float (&M)[R], float (&L)[R], float (&acc)[R][D / 32]) {
    auto rec = [&](int k, int r) { return (static_cast<size_t>(c + k0 + k) * 2 + (k0 + k == 0 ? 1 : 0)) * RB + r0 + r; };
    paged_add_pieces<D, R, F>(
        n, rows - r0, lane, [&](int k, int r) { return *reinterpret_cast<const float2 *>(p.part_ml + rec(k, r) * 2); },
        [&](int k, int r) { return p.part_o + rec(k, r) * D; }, M, L, acc);
}

// The output row of row r of the unit that note a describes.
__device__ __forceinline__ long long paged_noted_row(const PagedParams &p, const int4 &a, int r) {
    const int rr = a.w + r;
    return (static_cast<long long>(a.y) + rr / p.G) * p.Hq + a.z * p.G + rr % p.G;
}

// R rows of a unit of at most F pieces, all at once.
template <int D, int RB, int R, int F>
__device__ __forceinline__ void paged_join_few(const PagedParams &p, int c, const int4 &a, int r0, int rows, int lane) {
    constexpr int N = D / 32;
    using Vec = typename std::conditional<N == 4, float4, float2>::type;
    const int n = a.x - c + 1;
    Vec x[R][F];
    float2 ml[R][F];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < F; ++k) {  // (behind the last piece or row: that one again)
            const int kk = min(k, n - 1);
            const size_t rec = (static_cast<size_t>(c + kk) * 2 + (kk == 0 ? 1 : 0)) * RB + min(r0 + r, rows - 1);
            x[r][k] = reinterpret_cast<const Vec *>(p.part_o + rec * D)[lane];
            ml[r][k] = *reinterpret_cast<const float2 *>(p.part_ml + rec * 2);
        }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r0 + r >= rows) break;
        float M = -INFINITY, L = 0.f, acc[N] = {};
#pragma unroll
        for (int k = 0; k < F; ++k) M = fmaxf(M, ml[r][k].x);
#pragma unroll
        for (int k = 0; k < F; ++k) {
            const float w = ex2_from(ml[r][k].x, M);
            const float *xv = reinterpret_cast<const float *>(&x[r][k]);
            const bool adds = k < n && saw_key(ml[r][k].y);  // else the piece's columns may be unwritten
            L += adds ? w * ml[r][k].y : 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] += adds ? w * xv[e] : 0.f;
        }
        paged_finish<N>(p, D, paged_noted_row(p, a, r0 + r), lane * N, acc, M, L);
    }
}

__device__ __forceinline__ int join_rows_each(int pieces) { return pieces <= 2 ? 4 : (pieces <= 4 ? 2 : 1); }

template <int D, int RB>
__global__ void __launch_bounds__(kJoinThreads, kJoinPerSm<D>) paged_join_kernel(const PagedParams p, const int ctas) {
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
                const int per = join_rows_each(a.x - c + 1);
                items[i] = (rows + per - 1) / per;
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
    constexpr int N = D / 32, kWarps = kJoinThreads / 32;
    auto unit_of = [&](int item) {  // the last c with first[c] <= item (those without a unit have none after it)
        int lo = 0, hi = ctas - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= item) lo = mid; else hi = mid - 1;
        }
        return lo;
    };
    if (total <= static_cast<int>(gridDim.x)) {
        __shared__ __align__(16) float part[kWarps][D];
        __shared__ float2 part_ml[kWarps];
        if (static_cast<int>(blockIdx.x) >= total) return;
        const int c = unit_of(blockIdx.x), i = blockIdx.x - first[c];
        const int4 a = note[c];
        const int n = a.x - c + 1, rows = rows_of[c], per = join_rows_each(n);
        for (int r = i * per; r < min(rows, i * per + per); ++r) {
            const int k0 = warp * n / kWarps, k1 = (warp + 1) * n / kWarps;
            float M[1], L[1], acc[1][N];
            paged_join_rows<D, RB, 1, 8>(p, c, a, r, rows, lane, k0, k1 - k0, M, L, acc);
#pragma unroll
            for (int e = 0; e < N; ++e) part[warp][lane * N + e] = acc[0][e];
            if (lane == 0) part_ml[warp] = make_float2(M[0], L[0]);
            __syncthreads();
            if (warp == 0) {
                float top = -INFINITY, sum = 0.f, o[N] = {};
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_ml[w].x);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = ex2_from(part_ml[w].x, top);
                    sum = fmaf(f, part_ml[w].y, sum);
#pragma unroll
                    for (int e = 0; e < N; ++e) o[e] = fmaf(f, part[w][lane * N + e], o[e]);
                }
                paged_finish<N>(p, D, paged_noted_row(p, a, r), lane * N, o, top, sum);
            }
            __syncthreads();
        }
        return;
    }
    // a warp takes neighbouring items: one search, then on from unit to unit
    const int each = (total + gridDim.x * kWarps - 1) / (gridDim.x * kWarps);
    const int item0 = (blockIdx.x * kWarps + warp) * each, item1 = min(item0 + each, total);
    if (item0 >= item1) return;
    int c = unit_of(item0);
    for (int item = item0; item < item1; ++item) {
        while (c + 1 < ctas && first[c + 1] <= item) ++c;
        const int i = item - first[c];
        const int4 a = note[c];
        const int n = a.x - c + 1, rows = rows_of[c];
        if (n > 4) {
            float M[1], L[1], acc[1][N];
            paged_join_rows<D, RB, 1, 8>(p, c, a, i, rows, lane, 0, n, M, L, acc);
            paged_finish<N>(p, D, paged_noted_row(p, a, i), lane * N, acc[0], M[0], L[0]);
        } else if (n > 2) {
            paged_join_few<D, RB, 2, 4>(p, c, a, i * 2, rows, lane);
        } else {
            paged_join_few<D, RB, 4, 2>(p, c, a, i * 4, rows, lane);
        }
    }
}

// Joins two passes over the same rows, one query token per sequence: a over keys that
// all sequences share (one sequence of B tokens), b over each sequence's own.  A warp
// takes R rows at a time; their notes, then their pieces, a's first and in CTA order.
// 8 us for 2048 rows of 20 and 1 to 2 pieces, 15.5 us for 16384 of 2 to 4 and 1 to 2 (d = 128).
template <int D, int R, int F>
__device__ __forceinline__ void paged_pair_rows(const PagedParams &a, const PagedParams &b, int slot_a, int slot_b,
                                                int blocks_a, int blocks_b, int ctas_a, int ctas_b, int row0, int rows,
                                                int lane) {
    constexpr int N = D / 32;
    // lane 2 r: row r's note in a; lane 2 r + 1: in b
    int2 note = make_int2(0, 0);
    int off = 0;
    if (lane < 2 * R && lane / 2 < rows) {
        const int row = row0 + lane / 2, s = row / b.Hq, h = row % b.Hq, hk = h / b.G, g = h % b.G;
        if (lane & 1) {
            note = b.unit_note[(static_cast<long long>(s) * b.Hkv + hk) * blocks_b + g / b.block_rows];
            off = g % b.block_rows;
        } else {
            const int r = s * b.G + g;
            note = a.unit_note[static_cast<long long>(hk) * blocks_a + r / a.block_rows];
            off = r % a.block_rows;
        }
        // (a CTA that gave up has left notes unwritten)
        if (note.x < 0 || note.y < 1 || note.y > (lane & 1 ? ctas_b : ctas_a) - note.x) note = make_int2(0, 0);
    }
    int ca[R], na[R], oa[R], cb[R], nb[R], ob[R], most = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        ca[r] = __shfl_sync(0xffffffffu, note.x, 2 * r);
        na[r] = __shfl_sync(0xffffffffu, note.y, 2 * r);
        oa[r] = __shfl_sync(0xffffffffu, off, 2 * r);
        cb[r] = __shfl_sync(0xffffffffu, note.x, 2 * r + 1);
        nb[r] = __shfl_sync(0xffffffffu, note.y, 2 * r + 1);
        ob[r] = __shfl_sync(0xffffffffu, off, 2 * r + 1);
        most = max(most, na[r] + nb[r]);
    }
    // Piece k of row r: in pass a or b, and its record there; false behind the row's last one.
    auto find = [&](int k, int r, bool &in_a, bool &dense, long long &rec) {
        int c = ca[0], n = na[0], o = oa[0], c2 = cb[0], n2 = nb[0], o2 = ob[0];
#pragma unroll
        for (int i = 1; i < R; ++i)
            if (r == i) { c = ca[i]; n = na[i]; o = oa[i]; c2 = cb[i]; n2 = nb[i]; o2 = ob[i]; }
        in_a = k < n;
        if (!in_a) { k -= n; c = c2; n = n2; o = o2; }
        dense = n == 1;
        rec = dense ? row0 + r : (static_cast<long long>(c + k) * 2 + (k == 0 ? 1 : 0)) * (in_a ? slot_a : slot_b) + o;
        return k < n;
    };
    float M[R], L[R], acc[R][N];
    paged_add_pieces<D, R, F>(
        most, rows, lane,
        [&](int k, int r) {
            bool in_a, dense;
            long long rec;
            if (!find(k, r, in_a, dense, rec)) return make_float2(-INFINITY, 0.f);
            const PagedParams &x = in_a ? a : b;
            return *reinterpret_cast<const float2 *>((dense ? x.dense_ml : x.part_ml) + rec * 2);
        },
        [&](int k, int r) -> const float * {
            bool in_a, dense;
            long long rec;
            if (!find(k, r, in_a, dense, rec)) return b.dense_o;  // any row: it has no weight
            const PagedParams &x = in_a ? a : b;
            return (dense ? x.dense_o : x.part_o) + rec * D;
        },
        M, L, acc);
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (r < rows) paged_finish<N>(b, D, row0 + r, lane * N, acc[r], M[r], L[r]);
}

template <int D>
__global__ void __launch_bounds__(kJoinThreads, 2)
    paged_pair_join_kernel(const PagedParams a, const PagedParams b, const int slot_a, const int slot_b,
                           const int blocks_a, const int blocks_b, const int ctas_a, const int ctas_b) {
    const int lane = threadIdx.x & 31;
    const int rows = b.total_q * b.Hq;
    const int warps = gridDim.x * (kJoinThreads / 32), w = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // rows enough for every warp: two at a time, few pieces each; else one with more of its pieces in flight
    if (rows >= 2 * warps)
        for (int r = 2 * w; r < rows; r += 2 * warps)
            paged_pair_rows<D, 2, 4>(a, b, slot_a, slot_b, blocks_a, blocks_b, ctas_a, ctas_b, r, rows - r, lane);
    else
        for (int r = w; r < rows; r += warps)
            paged_pair_rows<D, 1, 12>(a, b, slot_a, slot_b, blocks_a, blocks_b, ctas_a, ctas_b, r, 1, lane);
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

// One launch of a main kernel, with its join or without.
struct PagedPass {
    fa_paged_cache c;
    PagedParams p;
    PagedPlan plan;
    int grid, blocks;  // CTAs; row blocks of the longest sequence, per kv head
    long long units;   // no more units than this exist
    int device, num_sms;
    bool early, join;  // see PagedConfig; followed by paged_join_kernel
};

int launch_paged_tiles(const PagedPass &a, cudaStream_t stream);
int launch_paged_cluster(const PagedPass &a, int size, cudaStream_t stream);

// Launch attributes of the paged kernels; `early`: may start before the kernels ahead of
// it in the stream have finished (see paged_enter).
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

template <int D, int RB>
int launch_join(const PagedPass &a, cudaStream_t stream) {
    if (a.grid > kJoinMax) return cuda_fail(cudaErrorInvalidConfiguration);
    const long long rows = std::min<long long>(a.grid, a.units) * std::min<long long>(a.p.block_rows, 1LL * a.p.max_q * a.p.G);
    const int grid = static_cast<int>(std::min<long long>(1LL * kJoinPerSm<D> * a.num_sms, rows));
    PagedConfig cfg(grid, kJoinThreads, 0, true, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, paged_join_kernel<D, RB>, a.p, a.grid);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

}  // namespace fa
