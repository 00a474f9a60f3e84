// fa_paged_sm103.cu -- attention of few query rows over a paged key/value
// cache: the next token of every sequence, a handful of drafted tokens.
//
// O = softmax(scale Q K^T [causal]) V for the nq * G query rows that share a
// kv head, one pass over the keys with a running maximum m and sum l per row
// (fp32), O rescaled when m moves by more than 2^kTau.
//
// What bounds it: every K and V row is read once and used for RT * 16 rows at
// most, so the HBM sets the time as long as enough bytes are in flight and
// the products keep up.  The products go through the 16 x 8 x 16 warp
// instruction: with 1 to 64 rows a 128-row tensor-memory tile would be mostly
// padding, and S and P stay in registers between the two products.
//
// CTA: four consumer warps and one producer warp.  The producer's lanes copy
// 64-key tiles of K and V page by page with TMA (128-byte swizzle) into a ring
// of shared-memory stages, and each unit's query rows with bulk copies.  The
// consumers split a tile by row tiles of 16 (RT) and by keys (4 / RT groups,
// each with its own m, l, O, joined once per unit), so nothing in the loop
// over tiles waits for another consumer.
#include <algorithm>

#include "fa_paged.cuh"

namespace fa {

namespace {

constexpr int kConsumers = 4;
constexpr int kPagedThreads = 32 * (kConsumers + 1);
constexpr int kTile = 64;             // keys per stage
constexpr float kTau = 8.0f;          // lazy-rescale threshold, log2 units
constexpr int kJoinCols = 32;         // columns per pass of the join between key groups

__device__ int g_paged_status = 0;

template <int D, int RT>
struct PagedLayout {
    static constexpr int kRows = 16 * RT;
    static constexpr int kGroups = kConsumers / RT;   // key groups
    static constexpr int kSlab = kTile * 128;         // 64 keys x 64 columns
    static constexpr int kOperand = (D / 64) * kSlab;  // a K or V tile
    static constexpr int kStage = 2 * kOperand;
    static constexpr int kStages = 98304 / kStage;    // 96 KB in flight per CTA, two CTAs per SM
    // Query rows 16 bytes apart in banks where there is room, so that the fragment
    // loads do not conflict (32 or 64 rows of 256 bytes leave none; it is once per unit).
    static constexpr int kQPitch = D * 2 + (RT == 1 ? 16 : 0);
    static constexpr int kQOff = kStages * kStage;
    static constexpr int kJoinOff = kQOff + kRows * kQPitch;
    static constexpr int kJoinBytes = kGroups > 1 ? kConsumers * 16 * (kJoinCols * 4 + 8) : 0;
    static constexpr int kBarOff = kJoinOff + kJoinBytes;
    static constexpr int kNumBars = 2 * kStages + 2 + 2 * RT;  // full, empty, unit full, unit empty, join full, join empty
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kPieceOff = kMiscOff + 8;
    static constexpr int kStartOff = kPieceOff + ((int)sizeof(PagedPiece) + 7) / 8 * 8;
    static constexpr int kSumOff = kStartOff + (int)sizeof(PagedStart);
    static constexpr int kSmemBytes = kSumOff + 8 * (kConsumers + 1);
    static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
};

template <int D, int RT, bool BF16>
__global__ void __launch_bounds__(kPagedThreads, 2)
    paged_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                      const PagedParams p) {
    using L = PagedLayout<D, RT>;
    constexpr int RB = L::kRows;
    constexpr int KG = L::kGroups;
    constexpr int NK = kTile / KG;  // keys of a tile per warp
    // fp16 weights keep 7 bits of headroom below the largest (2^kTau), which
    // pushes the smallest ones that do not vanish down to 2^-31 of the reference
    constexpr float kShift = BF16 ? 0.f : 7.f;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *empty = full + L::kStages;
    uint64_t *u_full = empty + L::kStages;
    uint64_t *u_empty = u_full + 1;
    uint64_t *j_full = u_empty + 1, *j_empty = j_full + RT;  // [RT] each
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMiscOff);
    PagedPiece *piece = reinterpret_cast<PagedPiece *>(smem + L::kPieceOff);
    PagedStart *start = reinterpret_cast<PagedStart *>(smem + L::kStartOff);
    long long *warp_sum = reinterpret_cast<long long *>(smem + L::kSumOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, kConsumers);
        }
        mbar_init(u_full, 1);
        mbar_init(u_empty, kConsumers);
        for (int t = 0; t < RT; ++t) {
            mbar_init(j_full + t, KG);
            mbar_init(j_empty + t, KG);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kConsumers && lane == 0) {
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    paged_plan<kTile, kPagedThreads>(p, *start, warp_sum, &g_paged_status);
    uint32_t units = 0, tiles = 0;  // handed over / taken so far

    if (warp == kConsumers) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = l2_policy_evict_first();
        const int page = 1 << p.page_shift;
        const int box = min(page, kTile), boxes = kTile / box;  // pages (or parts of one) per tile
        // lane -> (operand, slab, box) of a tile's copies
        const int my_box = lane % boxes, my_slab = lane / boxes % (D / 64), my_op = lane / boxes / (D / 64);
        bool ok = true;
        PagedCursor<kTile> cur;
        cur.begin(p, *start);
        PagedPiece u;
        int unit_tiles = 0;
        bool any = false;
        while (ok) {
            const bool more = cur.next(p, u, unit_tiles);
            if (more) {
                if (lane == 0) paged_note_unit(p, u, unit_tiles, *start);
            } else {
                if (lane == 0) paged_note_open(p, any ? &u : nullptr, unit_tiles, start->end, start->W, start->G);
                u.kind = -1;
            }
            any = true;
            if (units > 0 && !lanes_wait(u_empty, (units - 1) & 1, abort_flag)) { ok = false; break; }
            const int rows = u.kind < 0 ? 0 : min(RB, u.nq * p.G - u.row0);
            if (lane == 0) {
                *piece = u;
                mbar_arrive_expect_tx(u_full, rows * D * 2);
            }
            __syncwarp();
            ++units;
            if (u.kind < 0) break;
            for (int r = lane; r < rows; r += 32) {
                const int rr = u.row0 + r;
                const long long row = (static_cast<long long>(u.t0) + rr / p.G) * p.Hq + u.hk * p.G + rr % p.G;
                bulk_load(smem + L::kQOff + r * L::kQPitch, p.q + row * D, D * 2, u_full);
            }
            const int *table = p.page_table + static_cast<long long>(u.b) * p.max_pages;
            auto page_of = [&](int j) {
                const int key = j * kTile + my_box * box;
                return my_op < 2 && key < u.len ? __ldg(table + (key >> p.page_shift)) : -1;
            };
            int id = page_of(u.j0);
            for (int j = u.j0; j < u.j1; ++j) {
                const int next = j + 1 < u.j1 ? page_of(j + 1) : -1;
                const int st = tiles % L::kStages;
                if (tiles >= L::kStages &&
                    !lanes_wait(empty + st, (tiles / L::kStages - 1) & 1, abort_flag)) { ok = false; break; }
                const int key = j * kTile + my_box * box;
                const bool live = my_op < 2 && key < u.len;
                const int copies = __popc(__ballot_sync(0xffffffffu, live));
                if (lane == 0) mbar_arrive_expect_tx(full + st, copies * box * 128);
                __syncwarp();
                if (live) {
                    if (id < 0 || id >= p.num_pages) {
                        atomicCAS(&g_paged_status, 0, static_cast<int>(FA_ERR_PAGE));
                        id = p.num_pages;  // outside the tensor: the copy writes zeros
                    }
                    tma_load_4d(smem + st * L::kStage + my_op * L::kOperand + my_slab * L::kSlab + my_box * box * 128,
                                my_op ? &map_v : &map_k, full + st, my_slab * 64, key & (page - 1), u.hk, id, pol);
                }
                id = next;
                ++tiles;
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ consumers
        const int rw = warp % RT, kw = warp / RT;  // row tile, key group
        const int quad = lane & 3, qrow = lane >> 2;
        const uint32_t q_addr = smem_u32(smem + L::kQOff) +
                                (rw * 16 + (lane & 7) + ((lane >> 3) & 1) * 8) * L::kQPitch + (lane >> 4) * 16;
        const uint32_t ring = smem_u32(smem);
        // K fragments: lane = key row lane % 8 of an 8-key block, 16-byte chunk lane / 8 of four
        const uint32_t k_row = (lane & 7) * 128;
        // V fragments (transposed): lane = key row of a 16-key block, chunk lane / 16 of two
        const uint32_t v_row = ((lane & 7) + ((lane >> 3) & 1) * 8) * 128;
        float *join = reinterpret_cast<float *>(smem + L::kJoinOff);
        float2 *join_ml = reinterpret_cast<float2 *>(smem + L::kJoinOff + kConsumers * 16 * kJoinCols * 4);
        uint32_t joins = 0;
        bool ok = true;
        while (ok) {
            if (!lanes_wait(u_full, units & 1, abort_flag)) { ok = false; break; }
            ++units;
            const PagedPiece u = *piece;
            if (u.kind < 0) break;
            uint32_t qf[D / 16][4];
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) ldmatrix4(q_addr + kk * 32, qf[kk]);
            __syncwarp();
            if (lane == 0) mbar_arrive(u_empty);
            // the last key each of this thread's two rows sees
            const int r0 = rw * 16 + qrow;
            int lim0 = u.len - 1, lim1 = u.len - 1;
            if (p.causal) {
                lim0 = min(lim0, u.len - u.nq + (u.row0 + r0) / p.G);
                lim1 = min(lim1, u.len - u.nq + (u.row0 + r0 + 8) / p.G);
            }
            float o[D / 8][4];
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
            float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
            // kShift - m once a key has been seen; before, masked scores (-inf) still give weight 0
            float n0 = 0.f, n1 = 0.f;

            for (int j = u.j0; j < u.j1; ++j) {
                const int st = tiles % L::kStages;
                if (!lanes_wait(full + st, (tiles / L::kStages) & 1, abort_flag)) { ok = false; break; }
                ++tiles;
                const uint32_t kt = ring + st * L::kStage + kw * NK * 128;
                const uint32_t vt = kt + L::kOperand;
                const int key0 = j * kTile + kw * NK;  // this warp's first key
                // ---- S = Q K^T
                float s[NK / 8][4];
#pragma unroll
                for (int nb = 0; nb < NK / 8; ++nb) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[nb][e] = 0.f;
#pragma unroll
                    for (int k2 = 0; k2 < D / 32; ++k2) {
                        uint32_t kb[4];
                        const int chunk = (k2 & 1) * 4 + (lane >> 3);
                        ldmatrix4(kt + (k2 >> 1) * L::kSlab + nb * 1024 + k_row + ((chunk ^ (lane & 7)) << 4), kb);
                        mma_16816<BF16>(s[nb], qf[2 * k2], kb[0], kb[1]);
                        mma_16816<BF16>(s[nb], qf[2 * k2 + 1], kb[2], kb[3]);
                    }
                }
                // ---- scores in log2 units, masked; the tile's row maxima
                const bool tail = min(lim0, lim1) < key0 + NK - 1;
                float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
                for (int nb = 0; nb < NK / 8; ++nb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = key0 + nb * 8 + quad * 2 + e;
                        s[nb][e] *= p.scale_log2;
                        s[nb][2 + e] *= p.scale_log2;
                        if (tail) {
                            if (key > lim0) s[nb][e] = -INFINITY;
                            if (key > lim1) s[nb][2 + e] = -INFINITY;
                        }
                        x0 = fmaxf(x0, s[nb][e]);
                        x1 = fmaxf(x1, s[nb][2 + e]);
                    }
                __syncwarp();
#pragma unroll
                for (int off = 1; off < 4; off <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
                }
                const bool up0 = x0 > m0 + kTau, up1 = x1 > m1 + kTau;
                if (__any_sync(0xffffffffu, up0 || up1)) {
                    float a0 = 1.f, a1 = 1.f;
                    if (up0) { a0 = ex2_approx(m0 - x0); m0 = x0; n0 = kShift - x0; }
                    if (up1) { a1 = ex2_approx(m1 - x1); m1 = x1; n1 = kShift - x1; }
                    l0 *= a0;
                    l1 *= a1;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        o[i][0] *= a0;
                        o[i][1] *= a0;
                        o[i][2] *= a1;
                        o[i][3] *= a1;
                    }
                }
                // ---- weights 2^(s - m), rounded to the 16-bit type of V; l adds the rounded ones,
                // so a row that one key dominates returns that key's value row
                uint32_t pf[NK / 16][4];
#pragma unroll
                for (int nb = 0; nb < NK / 8; ++nb) {
                    const uint32_t lo = pack2t<BF16>(ex2_approx(s[nb][0] + n0), ex2_approx(s[nb][1] + n0));
                    const uint32_t hi = pack2t<BF16>(ex2_approx(s[nb][2] + n1), ex2_approx(s[nb][3] + n1));
                    float e0 = 0.f, e1 = 0.f;
                    add_pair16<BF16>(l0, e0, lo);
                    add_pair16<BF16>(l1, e1, hi);
                    l0 += e0;
                    l1 += e1;
                    pf[nb >> 1][(nb & 1) * 2] = lo;
                    pf[nb >> 1][(nb & 1) * 2 + 1] = hi;
                }
                // ---- O += P V.  Slots behind the last key hold anything at all, so
                // their V rows are read as zero (0 x NaN would be NaN).
                const int valid = u.len - key0;  // keys of this warp that exist
#pragma unroll
                for (int kb = 0; kb < NK / 16; ++kb) {
                    uint32_t mask0 = 0xffffffffu, mask1 = 0xffffffffu;
                    if (valid < NK) {
                        const int a = kb * 16 + quad * 2;
                        mask0 = (a < valid ? 0xffffu : 0u) | (a + 1 < valid ? 0xffff0000u : 0u);
                        mask1 = (a + 8 < valid ? 0xffffu : 0u) | (a + 9 < valid ? 0xffff0000u : 0u);
                    }
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t vb[4];
                        const int chunk = (c & 3) * 2 + (lane >> 4);
                        ldmatrix4_trans(vt + (c >> 2) * L::kSlab + kb * 2048 + v_row + ((chunk ^ (lane & 7)) << 4), vb);
                        mma_16816<BF16>(o[2 * c], pf[kb], vb[0] & mask0, vb[1] & mask1);
                        mma_16816<BF16>(o[2 * c + 1], pf[kb], vb[2] & mask0, vb[3] & mask1);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + st);
            }
            if (!ok) break;
            // ---- the unit's rows
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, off);
                l1 += __shfl_xor_sync(0xffffffffu, l1, off);
            }
            m0 -= kShift;  // (-inf stays)
            m1 -= kShift;
            const int rows = min(RB, u.nq * p.G - u.row0);
            if constexpr (KG == 1) {
                auto write = [&](int r, float m, float l, auto half) {
                    constexpr int H = decltype(half)::value;
                    if (r >= rows) return;
                    const long long row = paged_row(p, u, r);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        float a[2] = {o[i][2 * H], o[i][2 * H + 1]};
                        paged_emit<D, RB, 2>(p, u, r, row, i * 8 + quad * 2, a, m, l);
                    }
                };
                write(r0, m0, l0, std::integral_constant<int, 0>{});
                write(r0 + 8, m1, l1, std::integral_constant<int, 1>{});
            } else {
                // join the KG key groups of row tile rw through shared memory: as many columns per
                // pass as the unit's rows leave room for
                float *buf = join + rw * KG * 16 * kJoinCols;
                float2 *buf_ml = join_ml + rw * KG * 16;
                auto passes = [&](auto used) {
                    constexpr int RU = decltype(used)::value;    // rows that exist, rounded up
                    constexpr int C = kJoinCols * 16 / RU < D ? kJoinCols * 16 / RU : D;  // columns per pass
                    constexpr int kCells = RU * C / 4, kPer = (kCells + KG * 32 - 1) / (KG * 32);
                    const int cell = kw * 32 + lane;
                    auto cell_row = [&](int i) { return (cell + i * KG * 32) / (C / 4); };
                    const int cell_col = cell % (C / 4) * 4;
                    // 16-byte chunks of a row change places by row, against bank conflicts
                    auto at = [&](int g, int r, int col) {
                        return buf + (g * RU + r) * C + (((col >> 2) ^ (r & 7)) << 2) + (col & 3);
                    };
                    long long row[kPer];
                    bool live[kPer];
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        live[i] = cell + i * KG * 32 < kCells && rw * 16 + cell_row(i) < rows;
                        row[i] = paged_row(p, u, rw * 16 + cell_row(i));
                    }
#pragma unroll
                    for (int pass = 0; pass < D / C; ++pass) {
                        if (joins > 0 && !lanes_wait(j_empty + rw, (joins - 1) & 1, abort_flag)) { ok = false; return; }
#pragma unroll
                        for (int i = 0; i < C / 8; ++i) {
                            const int nb = pass * (C / 8) + i, col = i * 8 + quad * 2;
                            if (RU >= 8 || qrow < RU)
                                *reinterpret_cast<float2 *>(at(kw, qrow, col)) = make_float2(o[nb][0], o[nb][1]);
                            if constexpr (RU == 16)
                                *reinterpret_cast<float2 *>(at(kw, qrow + 8, col)) = make_float2(o[nb][2], o[nb][3]);
                        }
                        if (pass == 0 && quad == 0) {
                            buf_ml[kw * 16 + qrow] = make_float2(m0, l0);
                            buf_ml[kw * 16 + qrow + 8] = make_float2(m1, l1);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(j_full + rw);
                        if (!lanes_wait(j_full + rw, joins & 1, abort_flag)) { ok = false; return; }
                        ++joins;
#pragma unroll
                        for (int i = 0; i < kPer; ++i) {
                            if (!live[i]) continue;
                            const int r = cell_row(i);
                            float acc[4] = {0.f, 0.f, 0.f, 0.f};
                            float M = -INFINITY, Ls = 0.f;
#pragma unroll
                            for (int g = 0; g < KG; ++g) M = fmaxf(M, buf_ml[g * 16 + r].x);
#pragma unroll
                            for (int g = 0; g < KG; ++g) {
                                const float4 v = *reinterpret_cast<const float4 *>(at(g, r, cell_col));
                                const float2 ml = buf_ml[g * 16 + r];
                                const float w = ex2_from(ml.x, M);
                                Ls = fmaf(w, ml.y, Ls);
                                acc[0] = fmaf(w, v.x, acc[0]);
                                acc[1] = fmaf(w, v.y, acc[1]);
                                acc[2] = fmaf(w, v.z, acc[2]);
                                acc[3] = fmaf(w, v.w, acc[3]);
                            }
                            paged_emit<D, RB, 4>(p, u, rw * 16 + r, row[i], pass * C + cell_col, acc, M, Ls);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(j_empty + rw);
                    }
                };
                const int used = rows - rw * 16;
                if (RT == 1 && used <= 8) passes(std::integral_constant<int, 8>{});
                else passes(std::integral_constant<int, 16>{});
                if (!ok) break;
            }
        }
        __syncwarp();
    }
    // Whoever waits for this grid also waits for the grids before it.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    if (*abort_flag && warp == kConsumers && lane == 0) {
        // let every copy already issued land before the CTA goes away
        constexpr uint64_t kDrainNs = 200ull * 1000ull * 1000ull;
        int dummy = 0;
        if (units > 0) mbar_wait(u_full, (units - 1) & 1, &dummy, kDrainNs);
        for (uint32_t i = tiles > L::kStages ? tiles - L::kStages : 0; i < tiles; ++i)
            mbar_wait(full + i % L::kStages, (i / L::kStages) & 1, &dummy, kDrainNs);
        atomicCAS(&g_paged_status, 0, static_cast<int>(FA_ERR_WATCHDOG));
    }
}

// How a call runs, from its sizes alone.
PagedPlan plan_paged(int max_q, int group) {
    const long long rows = static_cast<long long>(max_q) * group;
    if (rows > 64 && group <= 128) return {true, 2 * (128 / group) * group, 256, 128, 1, 2};
    const int rb = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
    return {false, rb, rb, kTile, 2, 2};
}

template <int D, int RT, bool BF16>
int launch_rows(const PagedPass &a, cudaStream_t stream) {
    using L = PagedLayout<D, RT>;
    CUtensorMap mk, mv;
    int rc;
    if ((rc = make_page_map(&mk, a.c.k_pages, a.c, kTile)) != FA_OK) return rc;
    if ((rc = make_page_map(&mv, a.c.v_pages, a.c, kTile)) != FA_OK) return rc;
    const auto kernel = paged_rows_kernel<D, RT, BF16>;
    static std::atomic<bool> ready[kMaxDevices];
    if ((rc = ready_kernel(kernel, L::kSmemBytes, 0, a.device, ready)) != FA_OK) return rc;
    PagedConfig cfg(a.grid, kPagedThreads, L::kSmemBytes, a.early, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, kernel, mk, mv, a.p);
    if (e != cudaSuccess) return cuda_fail(e);
    return a.join ? launch_join<D, L::kRows>(a, stream) : FA_OK;
}

template <int D, bool BF16>
int launch_rows_d(const PagedPass &a, cudaStream_t stream) {
    switch (a.plan.block_rows) {
        case 16: return launch_rows<D, 1, BF16>(a, stream);
        case 32: return launch_rows<D, 2, BF16>(a, stream);
        default: return launch_rows<D, 4, BF16>(a, stream);
    }
}

int launch_pass(const PagedPass &a, cudaStream_t stream) {
    if (a.plan.tiles) return launch_paged_tiles(a, stream);
    const bool bf16 = a.c.dtype == FA_BF16;
    if (a.c.head_dim == 64) return bf16 ? launch_rows_d<64, true>(a, stream) : launch_rows_d<64, false>(a, stream);
    return bf16 ? launch_rows_d<128, true>(a, stream) : launch_rows_d<128, false>(a, stream);
}

// What a step of a pass costs an SM, in ns, measured on runs confined to a few SMs; only
// the ratio of two passes counts.  (Shared prefix of 16500 tokens for 256 sequences of
// 16 to 1024 own ones, 64 query heads: 202 us with the SMs split so, 228 one after the other.)
int step_ns(const PagedPlan &pl, int d) {
    if (pl.tiles) return d == 128 ? 1900 : 1400;
    const int ns = pl.block_rows == 16 ? 420 : (pl.block_rows == 32 ? 800 : 1150);
    return d == 128 ? ns : ns * 5 / 6;
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Partial rows, (m, l) and notes of one pass with the largest grid.
size_t pass_bytes(const PagedPlan &pl, int d, int num_sms) {
    const size_t slots = static_cast<size_t>(pl.per_sm) * num_sms * 2, rec = slots * pl.slot_rows;
    return rec * d * 4 + rec * 8 + slots * sizeof(int4);
}

PagedPass make_pass(const PagedLaunch &a, const DeviceInfo &dev, void *scratch) {
    PagedPass x;
    x.c = a.c;
    x.device = dev.device;
    x.num_sms = dev.num_sms;
    x.early = false;
    x.join = true;
    PagedParams &p = x.p;
    p = PagedParams{};
    p.q = static_cast<const uint16_t *>(a.q);
    p.out = a.out;
    p.lse = a.lse;
    p.page_table = a.page_table;
    p.seq_lens = a.seq_lens;
    p.cu_q = a.cu_q;
    p.nq_each = a.cu_q ? 0 : a.max_q;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.c.num_heads;
    p.G = a.Hq / a.c.num_heads;
    p.total_q = a.total_q;
    p.max_q = a.max_q;
    p.max_pages = a.max_pages;
    p.max_len = a.max_pages * a.c.page_size;
    p.num_pages = a.c.num_pages;
    p.page_shift = 0;
    while ((1 << p.page_shift) < a.c.page_size) ++p.page_shift;
    p.causal = a.causal;
    p.scale_log2 = a.scale * kLog2e;
    p.out_dtype = a.out_dtype;
    const PagedPlan pl = x.plan = plan_paged(a.max_q, p.G);
    p.block_rows = pl.block_rows;
    p.unit_steps = pl.unit_steps;
    const int most = pl.per_sm * dev.num_sms;
    const size_t slots = static_cast<size_t>(most) * 2, rec = slots * pl.slot_rows;
    p.part_o = static_cast<float *>(scratch);
    p.part_ml = p.part_o + rec * a.c.head_dim;
    p.open = reinterpret_cast<int4 *>(p.part_ml + rec * 2);
    // no more CTAs than the call can have steps
    const long long rows = static_cast<long long>(a.max_q) * p.G;
    x.blocks = static_cast<int>((rows + pl.block_rows - 1) / pl.block_rows);
    x.units = static_cast<long long>(a.B) * p.Hkv * x.blocks;
    x.grid = static_cast<int>(std::min<long long>(most, x.units * ((p.max_len + pl.tile - 1) / pl.tile)));
    return x;
}

}  // namespace

size_t paged_scratch_bytes(int max_q, int group, int d, int num_sms) {
    return pass_bytes(plan_paged(max_q, group), d, num_sms);
}

int launch_paged(const PagedLaunch &a, const DeviceInfo &dev, cudaStream_t stream) {
    return launch_pass(make_pass(a, dev, a.scratch), stream);
}

size_t paged_pair_scratch_bytes(int B, int Hq, int Hkv, int d, int num_sms) {
    const size_t rows = static_cast<size_t>(B) * Hq;
    size_t total = 0;
    for (int i = 0; i < 2; ++i) {
        const PagedPlan pl = plan_paged(i ? 1 : B, Hq / Hkv);
        const size_t per = static_cast<size_t>(i ? 1 : B) * (Hq / Hkv);
        const size_t units = static_cast<size_t>(i ? B : 1) * Hkv * ((per + pl.block_rows - 1) / pl.block_rows);
        total += align256(pass_bytes(pl, d, num_sms)) + align256(rows * d * 4) + align256(rows * 8) +
                 align256(units * sizeof(int2));
    }
    return total;
}

// The two passes share the SMs: the second starts on those that the first leaves,
// and neither waits for the other; the join waits for both.
int launch_paged_pair(const PagedLaunch &pre, const PagedLaunch &own, void *scratch, const DeviceInfo &dev,
                      cudaStream_t stream) {
    const size_t rows = static_cast<size_t>(own.B) * own.Hq;
    const int d = own.c.head_dim;
    char *at = static_cast<char *>(scratch);
    PagedPass pass[2];
    for (int i = 0; i < 2; ++i) {
        PagedPass &x = pass[i] = make_pass(i ? own : pre, dev, at);
        at += align256(pass_bytes(x.plan, d, dev.num_sms));
        x.p.dense_o = reinterpret_cast<float *>(at);
        at += align256(rows * d * 4);
        x.p.dense_ml = reinterpret_cast<float *>(at);
        at += align256(rows * 8);
        x.p.unit_note = reinterpret_cast<int2 *>(at);
        at += align256(x.units * sizeof(int2));
        x.join = false;
        x.early = i == 1;
        x.p.first = i == 0;
        x.p.num_sms = dev.num_sms;
        x.p.per_sm = x.plan.per_sm;
        x.p.step_ns = step_ns(x.plan, d);
    }
    for (int i = 0; i < 2; ++i) {
        const PagedPass &o = pass[1 - i];
        PagedParams &p = pass[i].p;
        p.peer_lens = o.p.seq_lens;
        p.peer_B = o.p.B;
        p.peer_max_len = o.p.max_len;
        p.peer_blocks = o.blocks;
        p.peer_tile = o.plan.tile;
        p.peer_unit_steps = o.plan.unit_steps;
        p.peer_step_ns = o.p.step_ns;
    }
    int rc;
    for (const PagedPass &x : pass)
        if ((rc = launch_pass(x, stream)) != FA_OK) return rc;
    constexpr long long kWarps = kJoinThreads / 32;
    const int grid = static_cast<int>(std::min<long long>(2LL * dev.num_sms, (static_cast<long long>(rows) + kWarps - 1) / kWarps));
    PagedConfig cfg(grid, kJoinThreads, 0, true, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, d == 64 ? paged_pair_join_kernel<64> : paged_pair_join_kernel<128>,
                                             pass[0].p, pass[1].p, pass[0].plan.slot_rows, pass[1].plan.slot_rows,
                                             pass[0].blocks, pass[1].blocks);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

int read_paged_status(int reset) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_paged_status, sizeof(int)) != cudaSuccess) return -1;
    if (reset && v) {
        int z = 0;
        if (cudaMemcpyToSymbol(g_paged_status, &z, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace fa
