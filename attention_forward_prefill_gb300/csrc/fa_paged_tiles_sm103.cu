// fa_paged_tiles_sm103.cu -- attention of many query rows over a paged cache:
// chunks of prompts, and the prefix that a whole batch shares.
//
// The same sums as paged_rows_kernel, for calls whose sequences have more rows
// per kv head than its registers hold: here the tensor cores set the time
// (4 rows x keys x d operations against 4 keys x d bytes), so the products run
// on 128-row tiles with accumulators in tensor memory.
//
// A kv head's query heads lie side by side in a token's row, so one tensor copy
// with a box of (64 channels, G heads, 128 / G tokens) brings a query tile of
// whole tokens, and every key tile is read once for all G heads.  Keys and
// values come page by page as in paged_rows_kernel.
//
// CTA (one per SM, 12 warps = 3 warpgroups):
//   warps 0-3   softmax of query tile 0 (thread = row = TMEM lane)
//   warps 4-7   softmax of query tile 1
//   warp  8     producer: pieces of work, then Q, K and V by TMA, a lane per box
//   warp  9     issues the products (one thread), owns the tensor memory
//   warps 10-11 clear the V rows behind a sequence's last key: the slots there
//               may hold anything, and 0 x NaN would reach O
// Key and value tiles travel in groups, one per step of the products: {K_j0},
// then {V_j, K_j+1}, the last {V_j1-1}; a group is two slots of a ring of four.
// While the softmax of one query tile works on its weights, the tensor core
// runs the other tile's products.  (A unit's start and end cost 2.7 to 3.5 us at
// d = 128, a step 1.75 us.)  Measured: 4 chunks of 700 to 2048 tokens on up to 12048, 32
// heads over 8 of 128, bf16, causal: 287 us, 1205 TFLOP/s, tensor pipe 54% active, and
// 13.5 us of join; 8192 tokens, 16 heads, full: 421 us against the dense kernel's 410.
// TMEM: S0 | S1 | O0 | O1; at d = 128 the
// weights overwrite S, at d = 64 they have columns of their own and the next
// S starts as soon as the last one is in registers.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fa_paged.cuh"

namespace fa {

namespace {

constexpr int kThreads = 384;
// setmaxnreg split of the launch's registers (checked at launch, as a sum above
// them would wait forever)
constexpr int kRegsSoftmax = 176;
constexpr int kRegsOther = 152;
constexpr int kMinLaunchRegs = (2 * 128 * kRegsSoftmax + 128 * kRegsOther + kThreads - 1) / kThreads;
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kM = 128;          // rows of a query tile
constexpr int kKeys = 128;       // keys of a tile
constexpr float kTau = 8.0f;     // lazy-rescale threshold, log2 units
constexpr uint32_t kTmemCols = 512;
constexpr int kReaders = 11;     // warps that read a piece: 8 softmax, 1 products, 2 clearing

__device__ int g_tiles_status = 0;

template <int D>
struct TilesLayout {
    static constexpr int kSlab = kM * 128;  // 128 rows x 64 columns
    static constexpr int kSlabs = D / 64;
    static constexpr int kTileBytes = kSlabs * kSlab;
    static constexpr int kGroups = 2;
    static constexpr int kQOff = 0;
    static constexpr int kRingOff = 2 * kTileBytes;
    static constexpr int kBarOff = kRingOff + 2 * kGroups * kTileBytes;
    // q_full, q_empty, s_full[2], p_full[2], o_done[2], s_free[2], pv_done[2], kv_full[2],
    // kv_empty[2], u_full[2], u_empty[2], v_clean, drain, v_dirty
    static constexpr int kNumBars = 23;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kPieceOff = kMiscOff + 8;
    static constexpr int kStartOff = kPieceOff + 2 * (((int)sizeof(PagedPiece) + 7) / 8 * 8);
    static constexpr int kSumOff = kStartOff + (int)sizeof(PagedStart);
    static constexpr int kStageOff = (kSumOff + 8 * (kThreads / 32) + 127) / 128 * 128;  // rows on their way out
    static constexpr int kSmemBytes = kStageOff + 8 * 32 * 32 * 4;
    static constexpr uint32_t kS0 = 0, kS1 = 128, kO0 = 256, kO1 = 256 + D;
    static constexpr bool kSepP = D == 64;
    static constexpr uint32_t kP0 = kSepP ? 256 + 2 * D : kS0;
    static constexpr uint32_t kP1 = kSepP ? 256 + 2 * D + 64 : kS1;
};

// Key tiles that the piece holds for query tile t (rows from row_t): [j0, end).
__device__ __forceinline__ int tile_end(const PagedParams &p, const PagedPiece &u, int row_t, int tile_rows) {
    if (row_t >= u.nq * p.G) return 0;
    const SeqView s{u.t0, u.nq, u.len};
    return min(paged_tiles_to_row<kKeys>(p, s, row_t + tile_rows - 1), u.j1);
}

// The last step of a piece reads V rows behind the sequence's last key.
__device__ __forceinline__ bool has_tail(const PagedPiece &u) { return u.j1 * kKeys > u.len; }

template <int D, bool BF16, bool TREE>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tiles_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const PagedParams p, const int scale_neg) {
    using L = TilesLayout<D>;
    constexpr float kShift = BF16 ? 0.f : 7.f;  // fp16 weights: as in paged_rows_kernel
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *q_full = bars, *q_empty = bars + 1, *s_full = bars + 2, *p_full = bars + 4, *o_done = bars + 6,
             *s_free = bars + 8, *pv_done = bars + 10, *kv_full = bars + 12, *kv_empty = bars + 14,
             *u_full = bars + 16, *u_empty = bars + 18, *v_clean = bars + 20, *drain = bars + 21, *v_dirty = bars + 22;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMiscOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMiscOff + 4);
    PagedStart *start = reinterpret_cast<PagedStart *>(smem + L::kStartOff);
    long long *warp_sum = reinterpret_cast<long long *>(smem + L::kSumOff);
    auto piece_at = [&](uint32_t i) {
        return reinterpret_cast<PagedPiece *>(smem + L::kPieceOff + (i & 1) * (((int)sizeof(PagedPiece) + 7) / 8 * 8));
    };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile_tokens = p.tile_tokens, tile_rows = tile_tokens * p.G;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full + t, 1);
            mbar_init(p_full + t, 4);  // one arrival per softmax warp
            mbar_init(o_done + t, 1);
            mbar_init(s_free + t, 4);
            mbar_init(pv_done + t, 1);
            mbar_init(kv_full + t, 1);
            mbar_init(kv_empty + t, 1);
            mbar_init(u_full + t, 1);
            mbar_init(u_empty + t, kReaders);
        }
        mbar_init(v_clean, 2);
        mbar_init(v_dirty, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kTmaWarp && lane == 0) {
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    paged_wait(p);
    if (warp == kMmaWarp) {
        // behind the wait and before followers start: a kernel ahead of this one, or this one, may
        // still need columns that a kernel which waits for it would hold
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
        paged_let_go();
    }
    tc_fence_before();
    paged_plan<TilesCut<D>, kThreads>(p, *start, warp_sum, &g_tiles_status);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint32_t pieces = 0;  // handed over / taken so far
    uint32_t gc = 0;      // key/value groups so far
    uint32_t qc = 0;      // query loads so far
    bool ok = true;
    // The next piece of work for a reading warp; kind -1: no more, or the wait ran out.
    auto take_piece = [&]() {
        const uint32_t slot = pieces & 1;
        PagedPiece u;
        u.kind = -1;
        if (lanes_wait(u_full + slot, (pieces >> 1) & 1, abort_flag)) {
            u = *piece_at(pieces);
            const bool pending = paged_pending(u, p.unit_steps >> 30);
            __syncwarp();
            if (lane == 0) mbar_arrive(u_empty + slot + pending);
            ++pieces;
        } else {
            ok = false;
        }
        return u;
    };

    if (warp == kTmaWarp) {
        // ------------------------------------------------------------ producer
        regs_shrink<kRegsOther>();
        const uint64_t pol_kv = l2_policy_evict_last(), pol_q = l2_policy_evict_first();
        const int page = 1 << p.page_shift;
        const int box = min(page, kKeys), boxes = kKeys / box;
        // lane -> (half of a group: V_j or K_j+1, slab, page) of its copies: up to 2 x 2 x 8
        const int my_box = lane % boxes, my_slab = lane / boxes % L::kSlabs, my_half = lane / boxes / L::kSlabs;
        PagedCursor<TilesCut<D>> cur;
        if (lane == 0) paged_note_none(p);
        cur.begin(p, *start);
        PagedPiece u = {};
        int to_last = 0;
        bool any = false;
        while (ok) {
            const bool more = cur.next(p, u, to_last);
            if (more) {
                if (lane == 0) paged_note_unit(p, u, to_last, *start);
            } else {
                if (lane == 0 && any && u.kind == 1) paged_note_open(p, u, to_last, *start);
                u.kind = -1;
            }
            any = true;
            u.end0 = tile_end(p, u, u.row0, tile_rows);
            u.end1 = tile_end(p, u, u.row0 + tile_rows, tile_rows);
            const uint32_t slot = pieces & 1;
            if (pieces >= 2 && !lanes_wait(u_empty + slot, ((pieces >> 1) - 1) & 1, abort_flag)) { ok = false; break; }
            if (lane == 0) {
                *piece_at(pieces) = u;
                mbar_arrive(u_full + slot);
            }
            ++pieces;
            if (!more) break;
            // ---- groups {K_j0}, {V_j, K_j+1} ...: group i holds V_(j0 + i - 1) and K_(j0 + i)
            const int *table = p.page_table + static_cast<long long>(u.b) * p.max_pages;
            const int steps = u.j1 - u.j0;
            auto key_of = [&](int i) { return (u.j0 + i - (my_half == 0 ? 1 : 0)) * kKeys + my_box * box; };
            auto mine = [&](int i) {
                return my_half < 2 && (my_half == 0 ? i > 0 : i < steps) && key_of(i) < u.len;
            };
            auto page_of = [&](int i) { return mine(i) ? __ldg(table + (key_of(i) >> p.page_shift)) : -1; };
            int id = page_of(0);  // (on its way while the query tiles become free)
            // ---- query tiles with key tiles in this piece
            const bool need0 = u.end0 > u.j0, need1 = u.end1 > u.j0;
            if (qc > 0 && !lanes_wait(q_empty, (qc - 1) & 1, abort_flag)) { ok = false; break; }
            if (lane == 0) {
                mbar_arrive_expect_tx(q_full, ((need0 ? 1 : 0) + (need1 ? 1 : 0)) * tile_rows * 128 * L::kSlabs);
                for (int t = 0; t < 2; ++t) {
                    if (!(t ? need1 : need0)) continue;
                    for (int c = 0; c < L::kSlabs; ++c)
                        tma_load_3d(smem + L::kQOff + t * L::kTileBytes + c * L::kSlab, &map_q, q_full, c * 64, u.hk * p.G,
                                    u.t0 + u.row0 / p.G + t * tile_tokens, pol_q);
                }
            }
            __syncwarp();
            ++qc;
            for (int i = 0; i <= steps; ++i) {
                const int next = i < steps ? page_of(i + 1) : -1;
                const uint32_t st = gc % L::kGroups;
                if (gc >= L::kGroups && !lanes_wait(kv_empty + st, (gc / L::kGroups - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                const bool live = mine(i);
                const int copies = __popc(__ballot_sync(0xffffffffu, live));
                if (lane == 0) mbar_arrive_expect_tx(kv_full + st, copies * box * 128);
                __syncwarp();
                if (live) {
                    if (id < 0 || id >= p.num_pages) {
                        record_status(&g_tiles_status, FA_ERR_PAGE);
                        id = p.num_pages;  // outside the tensor: the copy writes zeros
                    }
                    // slot 2 st: V_j (or the first K); slot 2 st + 1: K_j+1
                    const int half = i == 0 ? 0 : my_half;
                    tma_load_4d(smem + L::kRingOff + (2 * st + half) * L::kTileBytes + my_slab * L::kSlab + my_box * box * 128,
                                my_half == 0 ? &map_v : &map_k, kv_full + st, my_slab * 64, key_of(i) & (page - 1), u.hk, id,
                                pol_kv);
                }
                id = next;
                ++gc;
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ products
        regs_shrink<kRegsOther>();
        const uint32_t idesc_qk = idesc_f16(BF16, kM, kKeys, false, false);
        const uint32_t idesc_pv = idesc_f16(BF16, kM, D, false, true);
        const uint32_t q_addr = smem_u32(smem + L::kQOff), ring = smem_u32(smem + L::kRingOff);
        const uint64_t q_desc[2] = {sdesc_sw128(q_addr, 16, 1024), sdesc_sw128(q_addr + L::kTileBytes, 16, 1024)};
        const uint32_t s_tm[2] = {tmem + L::kS0, tmem + L::kS1};
        const uint32_t o_tm[2] = {tmem + L::kO0, tmem + L::kO1};
        const uint32_t p_tm[2] = {tmem + L::kP0, tmem + L::kP1};
        uint32_t pc[2] = {0, 0}, qk[2] = {0, 0}, tails = 0;
        while (ok) {
            const PagedPiece u = take_piece();
            if (u.kind < 0) break;
            const int j0 = u.j0, j1 = u.j1;
            const int end[2] = {u.end0, u.end1};
            if (lane == 0) {
                do {
                    if (!mbar_wait(q_full, qc & 1, abort_flag, kWatchdogNs)) { ok = false; break; }
                    uint32_t st = gc % L::kGroups;
                    if (!mbar_wait(kv_full + st, (gc / L::kGroups) & 1, abort_flag, kWatchdogNs)) { ok = false; break; }
                    tc_fence_after();
                    // S_t = Q_t K_j0^T, once the softmax has the last piece's final S in registers
                    auto first_qk = [&](auto tile) {
                        constexpr int T = decltype(tile)::value;
                        if (end[T] <= j0) return true;
                        if constexpr (L::kSepP) {
                            if (qk[T] > 0 && !mbar_wait(s_free + T, (qk[T] - 1) & 1, abort_flag, kWatchdogNs)) return false;
                            tc_fence_after();
                            ++qk[T];
                        }
                        issue_qk<D>(s_tm[T], q_desc[T], sdesc_sw128(ring + 2 * st * L::kTileBytes, 16, 1024), idesc_qk);
                        umma_commit(s_full + T);
                        return true;
                    };
                    if (!first_qk(std::integral_constant<int, 0>{}) || !first_qk(std::integral_constant<int, 1>{})) {
                        ok = false;
                        break;
                    }
                    umma_commit(kv_empty + st);
                    ++gc;
                    if (j1 - j0 == 1) umma_commit(q_empty);
                    for (int j = j0; j < j1; ++j) {
                        st = gc % L::kGroups;
                        if (!mbar_wait(kv_full + st, (gc / L::kGroups) & 1, abort_flag, kWatchdogNs)) { ok = false; break; }
                        if (j == j1 - 1 && has_tail(u)) {
                            mbar_arrive(v_dirty);  // the rows are here: the clearing warps may go
                            if (!mbar_wait(v_clean, tails & 1, abort_flag, kWatchdogNs)) { ok = false; break; }
                            ++tails;
                        }
                        tc_fence_after();
                        const uint64_t v_desc = sdesc_sw128(ring + 2 * st * L::kTileBytes, L::kSlab, 1024);
                        const uint64_t k_desc = sdesc_sw128(ring + (2 * st + 1) * L::kTileBytes, 16, 1024);
                        auto next_qk = [&](auto tile) {  // S_t = Q_t K_j+1^T
                            constexpr int T = decltype(tile)::value;
                            if (j + 1 >= end[T]) return true;
                            if constexpr (L::kSepP) {
                                if (!mbar_spin(s_free + T, (qk[T] - 1) & 1, abort_flag, kWatchdogNs)) return false;
                                tc_fence_after();
                                ++qk[T];
                            }
                            issue_qk<D>(s_tm[T], q_desc[T], k_desc, idesc_qk);
                            umma_commit(s_full + T);
                            return true;
                        };
                        auto pv = [&](auto tile) {  // O_t (+)= P_t V_j
                            constexpr int T = decltype(tile)::value;
                            if (j >= end[T]) return true;
                            // polled: the product should start the moment P is in
                            if (!mbar_spin(p_full + T, pc[T] & 1, abort_flag, kWatchdogNs)) return false;
                            ++pc[T];
                            tc_fence_after();
                            issue_pv<D>(o_tm[T], p_tm[T], v_desc, idesc_pv, j > j0);
                            if constexpr (L::kSepP) umma_commit(pv_done + T);
                            else if (j == end[T] - 1) umma_commit(o_done + T);
                            return true;
                        };
                        constexpr std::integral_constant<int, 0> t0{};
                        constexpr std::integral_constant<int, 1> t1{};
                        // at d = 128 a tile's next S overwrites the weights that its P V reads
                        if constexpr (L::kSepP) ok = next_qk(t0) && next_qk(t1) && pv(t0) && pv(t1);
                        else ok = pv(t0) && next_qk(t0) && pv(t1) && next_qk(t1);
                        if (!ok) break;
                        umma_commit(kv_empty + st);
                        ++gc;
                        if (j + 1 == j1 - 1) umma_commit(q_empty);
                    }
                } while (false);
            }
            ok = __all_sync(0xffffffffu, ok);
            ++qc;
        }
        if (lane == 0) {  // nothing may still run on the tensor core at teardown
            umma_commit(drain);
            int dummy = 0;
            mbar_wait(drain, 0, &dummy, kWatchdogNs);
        }
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------------------ softmax
        regs_grow<kRegsSoftmax>();
        const int t = warp >> 2, wq = warp & 3;
        const int r = wq * 32 + lane;  // row of the tile
        const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t s_addr = tmem + lanes + (t ? L::kS1 : L::kS0);
        const uint32_t o_addr = tmem + lanes + (t ? L::kO1 : L::kO0);
        const uint32_t p_addr = tmem + lanes + (t ? L::kP1 : L::kP0);
        const float cexp = p.scale_log2, cabs = fabsf(p.scale_log2);
        uint32_t sc = 0, oc = 0, pvc = 0;
        while (ok) {
            const PagedPiece u = take_piece();
            if (u.kind < 0) break;
            const int j0 = u.j0;
            const int row_t = u.row0 + t * tile_rows;
            const int end = t ? u.end1 : u.end0;
            const int rr = row_t + r;  // row among the sequence's nq * G
            const bool row_ok = r < tile_rows && rr < u.nq * p.G;
            const long long row = paged_row(p, u, t * tile_rows + r);
            const bool keep = paged_keeps(p, u);
            const long long rec = paged_record<2 * kM>(u, t * tile_rows + r, row);
            if (end <= j0) {
                // a cut unit's piece without keys for this tile: nothing to add
                if (u.kind != 0 && row_ok) *reinterpret_cast<float2 *>(p.part_ml + rec * 2) = make_float2(-INFINITY, 0.f);
                continue;
            }
            int lim = u.len - 1;  // last key that the row sees
            const SeqView view{u.t0, u.nq, u.len};
            const uint32_t *see = nullptr;
            if constexpr (TREE) see = tree_row(p, view, rr);
            else if (p.causal) lim = min(lim, u.len - u.nq + rr / p.G);
            float m_ref = -INFINITY, l = 0.f;
            // kShift - m_ref once a key has been seen; before, masked scores still give weight 0
            float neg_m = 0.f;
            for (int j = j0; j < end; ++j) {
                if (!warp_wait(s_full + t, sc & 1, abort_flag)) { ok = false; break; }
                ++sc;
                tc_fence_after();
                uint32_t sr[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(s_addr + q * 32, sr[q]);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 4; ++q) reg_fence32(sr[q]);
                if constexpr (L::kSepP) {
                    tc_fence_before();  // S is in registers: the next one may start
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_free + t);
                }
                const uint32_t fill = __float_as_uint(scale_neg ? INFINITY : -INFINITY);
                if constexpr (TREE) {
                    if ((j + 1) * kKeys > u.len - u.nq) {  // not context alone
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t seen = tree_seen32(p, view, see, j * kKeys + q * 32);
#pragma unroll
                            for (int c = 0; c < 32; ++c) sr[q][c] = seen >> c & 1 ? sr[q][c] : fill;
                        }
                    }
                } else {
                    const int cmax = lim - j * kKeys;  // columns behind it are masked
                    if (cmax < kKeys - 1) {
#pragma unroll
                        for (int c = 0; c < 128; ++c) sr[c >> 5][c & 31] = c > cmax ? fill : sr[c >> 5][c & 31];
                    }
                }
                const float mx = scale_neg ? row_max128<true>(sr) : row_max128<false>(sr);
                const float m_tile = mx == -INFINITY ? -INFINITY : mx * cabs;
                __syncwarp();  // the masked branch may diverge per lane
                const bool need = m_tile > m_ref + kTau;
                float alpha = 1.f;
                if (need) {
                    alpha = ex2_approx(m_ref - m_tile);  // 0 on the first tile
                    l *= alpha;
                    m_ref = m_tile;
                    neg_m = kShift - m_tile;
                }
                const uint64_t c2 = f2_pack(cexp, cexp), nm2 = f2_pack(neg_m, neg_m);
                float sum_lo[4] = {0.f, 0.f, 0.f, 0.f}, sum_hi[4] = {0.f, 0.f, 0.f, 0.f};
                // weights in 32-key quarters, rounded to V's 16-bit type; l adds the rounded ones
                uint32_t pk[4][16];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const uint64_t x = ffma2(f2_pack(__uint_as_float(sr[q][2 * c]), __uint_as_float(sr[q][2 * c + 1])),
                                                 c2, nm2);
                        pk[q][c] = pack2t<BF16>(ex2_approx(f2_lo(x)), ex2_approx(f2_hi(x)));
                        add_pair16<BF16>(sum_lo[c & 3], sum_hi[c & 3], pk[q][c]);
                    }
                    if constexpr (!L::kSepP) tmem_st16(p_addr + q * 16, pk[q]);
                }
                if constexpr (L::kSepP) {
                    if (j > j0) {  // the last P V has read its weights, and O is complete
                        if (!warp_wait(pv_done + t, pvc & 1, abort_flag)) { ok = false; break; }
                        ++pvc;
                        tc_fence_after();
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_st16(p_addr + q * 16, pk[q]);
                }
                const uint64_t s01 = fadd2(f2_pack(sum_lo[0], sum_hi[0]), f2_pack(sum_lo[1], sum_hi[1]));
                const uint64_t s23 = fadd2(f2_pack(sum_lo[2], sum_hi[2]), f2_pack(sum_lo[3], sum_hi[3]));
                const uint64_t sum = fadd2(s01, s23);
                l += f2_lo(sum) + f2_hi(sum);
                if (j > j0 && __any_sync(0xffffffffu, need)) {
                    // O is complete up to tile j - 1 (the commit behind S covers that product)
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t o[32];
                        tmem_ld32(o_addr + q * 32, o);
                        tmem_ld_wait();
                        reg_fence32(o);
#pragma unroll
                        for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                        tmem_st32(o_addr + q * 32, o);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + t);
            }
            if (!ok) break;
            // ---- rows out
            if constexpr (L::kSepP) {
                if (!warp_wait(pv_done + t, pvc & 1, abort_flag)) { ok = false; break; }
                ++pvc;
            } else {
                if (!warp_wait(o_done + t, oc & 1, abort_flag)) { ok = false; break; }
                ++oc;
            }
            tc_fence_after();
            const float m = m_ref - kShift;  // (-inf stays)
            const float inv = keep ? 1.f : (saw_key(l) ? 1.f / l : 0.f);
            if (row_ok) {
                if (keep)
                    *reinterpret_cast<float2 *>((u.kind == 0 ? p.dense_ml : p.part_ml) + rec * 2) = make_float2(m, l);
                else if (p.lse)
                    p.lse[row] = saw_key(l) ? (m + __log2f(l)) * kLn2 : -INFINITY;
            }
            // A lane holds a row, and a row's neighbours in memory are its columns: 32 rows x 32
            // words at a time turn in shared memory, so that eight lanes write a row's 128 bytes.
            // (Lanes writing rows of their own took 4 us per piece, as 16-byte stores far apart.)
            const bool wide = keep || p.out_dtype == FA_F32;
            const int bf = p.out_dtype == FA_BF16;
            uint8_t *base = reinterpret_cast<uint8_t *>(keep ? (u.kind == 0 ? p.dense_o : p.part_o) : p.out);
            const long long offset = row_ok ? (keep ? rec : row) * D * (wide ? 4 : 2) : -1;
            uint32_t *stage = reinterpret_cast<uint32_t *>(smem + L::kStageOff) + warp * 32 * 32;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                tmem_ld32(o_addr + q * 32, o);
                tmem_ld_wait();
                reg_fence32(o);
                // 16-byte chunks of a row change places by row, against bank conflicts
                auto put = [&](int chunk, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
                    *reinterpret_cast<uint4 *>(stage + lane * 32 + ((chunk ^ (lane & 7)) << 2)) = make_uint4(x, y, z, w);
                };
                auto f = [&](int c) { return __uint_as_float(o[c]) * inv; };
                if (wide) {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        put(c, __float_as_uint(f(4 * c)), __float_as_uint(f(4 * c + 1)), __float_as_uint(f(4 * c + 2)),
                            __float_as_uint(f(4 * c + 3)));
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        put((q & 1) * 4 + c, pack2(f(8 * c), f(8 * c + 1), bf), pack2(f(8 * c + 2), f(8 * c + 3), bf),
                            pack2(f(8 * c + 4), f(8 * c + 5), bf), pack2(f(8 * c + 6), f(8 * c + 7), bf));
                    if ((q & 1) == 0) continue;  // two quarters make a row's 128 bytes
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int from = i * 4 + (lane >> 3), chunk = lane & 7;
                    const long long to = __shfl_sync(0xffffffffu, offset, from);
                    const uint4 v = *reinterpret_cast<const uint4 *>(stage + from * 32 + ((chunk ^ (from & 7)) << 2));
                    if (to >= 0)
                        *reinterpret_cast<uint4 *>(base + to + (wide ? q : q >> 1) * 128 + chunk * 16) = v;
                }
                __syncwarp();
            }
            tc_fence_before();
        }
    } else {
        // ------------------------------------------------------------ clearing (warps 10, 11)
        regs_shrink<kRegsOther>();
        // (They wait for the products' thread, not for the ring's own barrier, whose phases
        // they do not follow one by one.)
        uint32_t tails = 0;
        while (ok) {
            const PagedPiece u = take_piece();
            if (u.kind < 0) break;
            gc += u.j1 - u.j0 + 1;
            if (!has_tail(u)) continue;
            const uint32_t g = gc - 1, st = g % L::kGroups;  // the piece's last group holds V_j1-1 in its first slot
            if (!lanes_wait(v_dirty, tails & 1, abort_flag)) { ok = false; break; }
            ++tails;
            const int first = max(0, u.len - (u.j1 - 1) * kKeys);
            uint8_t *v = smem + L::kRingOff + 2 * st * L::kTileBytes;
            for (int i = first * 8 + (warp - 10) * 32 + lane; i < kKeys * 8; i += 64)
#pragma unroll
                for (int c = 0; c < L::kSlabs; ++c)
                    *reinterpret_cast<uint4 *>(v + c * L::kSlab + i * 16) = make_uint4(0, 0, 0, 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(v_clean);
        }
    }

    // Whoever waits for this grid also waits for the grids before it.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    if (warp == kTmaWarp && lane == 0 && *abort_flag) {
        // let every copy already issued land before the CTA goes away
        constexpr uint64_t kDrainNs = 200ull * 1000ull * 1000ull;
        int dummy = 0;
        if (qc > 0) mbar_wait(q_full, (qc - 1) & 1, &dummy, kDrainNs);
        for (uint32_t i = gc > L::kGroups ? gc - L::kGroups : 0; i < gc; ++i)
            mbar_wait(kv_full + i % L::kGroups, (i / L::kGroups) & 1, &dummy, kDrainNs);
        record_status(&g_tiles_status, FA_ERR_WATCHDOG);
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, bool BF16, bool TREE>
int launch_tiles_m(const PagedPass &a, cudaStream_t stream) {
    PagedParams p = a.p;
    using L = TilesLayout<D>;
    static_assert(L::kSmemBytes <= 227 * 1024, "shared memory budget");
    CUtensorMap mq, mk, mv;
    int rc;
    // queries [token][head][d], a box of the G heads of a kv head and tile_tokens tokens
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cuda_fail(cudaErrorNotSupported);
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.total_q};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * p.Hq};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)p.tile_tokens};
    const cuuint32_t estr[3] = {1, 1, 1};
    if (enc(&mq, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t *>(p.q),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cuda_fail(cudaErrorInvalidValue);
    if ((rc = make_page_map(&mk, a.c.k_pages, a.c, kKeys)) != FA_OK) return rc;
    if ((rc = make_page_map(&mv, a.c.v_pages, a.c, kKeys)) != FA_OK) return rc;
    // scale == 0 runs as 2^-100: every weight is then exactly 1 as well, and masked
    // scores (+-inf) never meet a zero multiplier
    // (below 2^-126 the packed products would take it for 0)
    if (p.scale_log2 == 0.f) p.scale_log2 = 0x1p-100f;
    else if (std::fabs(p.scale_log2) < 0x1p-126f) p.scale_log2 = std::copysign(0x1p-126f, p.scale_log2);
    const auto kernel = paged_tiles_kernel<D, BF16, TREE>;
    static std::atomic<bool> ready[kMaxDevices];
    if ((rc = ready_kernel(kernel, L::kSmemBytes, kMinLaunchRegs, a.device, ready)) != FA_OK) return rc;
    PagedConfig cfg(a.grid, kThreads, L::kSmemBytes, a.early, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, kernel, mq, mk, mv, p, p.scale_log2 < 0.f ? 1 : 0);
    if (e != cudaSuccess) return cuda_fail(e);
    return a.join ? launch_join<D, 2 * kM>(a, stream) : FA_OK;
}

template <int D, bool BF16>
int launch_tiles_d(const PagedPass &a, cudaStream_t stream) {
    return a.p.tree ? launch_tiles_m<D, BF16, true>(a, stream) : launch_tiles_m<D, BF16, false>(a, stream);
}

}  // namespace

int launch_paged_tiles(const PagedPass &a, cudaStream_t stream) {
    const bool bf16 = a.c.dtype == FA_BF16;
    if (a.c.head_dim == 64) return bf16 ? launch_tiles_d<64, true>(a, stream) : launch_tiles_d<64, false>(a, stream);
    return bf16 ? launch_tiles_d<128, true>(a, stream) : launch_tiles_d<128, false>(a, stream);
}

int read_tiles_status(int reset) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_tiles_status, sizeof(int)) != cudaSuccess) return -1;
    if (reset && v) {
        int z = 0;
        if (cudaMemcpyToSymbol(g_tiles_status, &z, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace fa
