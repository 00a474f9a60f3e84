// fa_weigh_tiles_sm103.cu -- what cached tokens got of the attention of many query rows.
//
// The sums of fa_weigh_sm103.cu, S^T = K Q^T on tiles of 128 keys x 128 rows in tensor memory: a
// thread holds a key (a lane of the accumulator) and goes through the rows (its columns), so that
// the sum over the rows stays in the thread.  One product and one exponential per pair of key and
// row: at d = 128 the tensor core and the exponential unit (32 a clock and SM) take as long.
//
// CTA (one per SM, 20 warps):
//   warps 0-15  exponentials and sums, four warps for each key tile of the unit and parity of the
//               chunk (thread = key = TMEM lane)
//   warp  16    producer: both key tiles of a unit, then its chunks of query rows, by TMA
//   warps 17-18 issue the products of a key tile each (one thread); the first owns the tensor memory
//   warp  19    the chunks' log-sum-exps, four chunks at a time
// A unit's 256 keys stay in shared memory while the chunks of rows go by, so that a chunk is
// loaded once for two products, and the next unit's are on their way.  A wait costs 200 to 350
// clocks under sixteen busy warps, whether there is anything to wait for or not: hence a thread for
// each tile's products, and log-sum-exps in lots.  Every warp walks through the CTA's pieces
// (fa_weigh_cut.cuh) by itself.  TMEM: S of (tile, parity).
//
// 4 chunks of 700 to 2048 tokens on up to 11048, 32 heads over 8, d = 128: 115 us (1234 TFLOP/s; tensor pipe
// 56% active, exponential unit 55%, issue 57%) again and again on the same inputs, whose keys stay in L2, and 131 among
// calls on others; the start takes 8 of them and the join 5.  Before: eight
// summing warps 230, a branch for every quarter of a chunk 159, sixteen warps and eight columns at a
// time 145, a product thread for each tile 138, hidden quarters
// passed over 124, a whole chunk without a loop 118, two units' keys and two chunks of rows held instead
// of one and four 116.
// Rows whose log-sum-exp is infinite add nothing, whatever their products are: bits for the rows that count come with the
// log-sum-exps, and chunks in which some do not are summed under them (4 chunks of 1024 tokens on 5000, 32 heads over 8,
// d = 128, 115 us, with one row in a hundred left out 183).
// One chunk a unit (up to 128 rows), 16 sequences of 4096 tokens: 34 to 36 us for 134 MB (40 with one
// unit's keys, 37 where the warps of both parities still met at every unit, 36 to 39 where the log-sum-exps' warp went
// through four chunks whether they were there or not: it is in the way of short units).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "fa_weigh.cuh"

namespace fa {

namespace {

constexpr int kThreads = 640;
constexpr int kTmaWarp = 16;
constexpr int kMmaWarp = 17;  // and the next
constexpr int kOffWarp = 19;
constexpr int kM = 128;          // keys of a tile
constexpr int kRows = kWeighRows;  // rows of a chunk
constexpr uint32_t kTmemCols = 512;
constexpr int kOffStages = 2, kOffChunks = 4;  // lots of log-sum-exps, and chunks of a lot

constexpr int kKeySets = 2;  // units whose keys are in shared memory

__device__ int g_weigh_tiles_status = 0;

template <int D>
struct WeighLayout {
    static constexpr int kSlabs = D / 64, kSlab = 128 * 128;
    static constexpr int kTileBytes = kSlabs * kSlab;
    static constexpr int kRowStages = D == 128 ? 2 : 8;
    static constexpr int kRowsOff = 2 * kKeySets * kTileBytes;
    static constexpr int kOffOff = kRowsOff + kRowStages * kTileBytes;  // [kOffStages][kOffChunks][kRows] floats
    static constexpr int kOddOff = kOffOff + kOffStages * kOffChunks * kRows * 4;    // [2][kM]: sums over the odd chunks
    static constexpr int kCountOff = kOddOff + 2 * kM * 4;  // [kOffStages][kOffChunks]: which of a chunk's rows count
    static constexpr int kLiveOff = kCountOff + kOffStages * kOffChunks * 16;  // and how many it has; below 0: not all of them count
    static constexpr int kBarOff = kLiveOff + kOffStages * kOffChunks * 4;
    // k_full[set][tile], k_empty[set][tile], q_full, q_empty, off_full, off_empty, s_full[tile][parity], s_free[tile][parity],
    // sum_full[tile], sum_free[tile], drain[tile]
    static constexpr int kNumBars = 4 * kKeySets + 2 * kRowStages + 2 * kOffStages + 8 + 4 + 2;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kStartOff = kMiscOff + 8;
    static constexpr int kSumOff = kStartOff + (int)sizeof(WeighStart);
    static constexpr int kSmemBytes = kSumOff + 8 * (kThreads / 32);
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

// The weights of 8 rows' columns s, added to two pairs of sums; MASKED: of the columns whose bits are set.
// (Written stage by stage, so that eight exponentials are in flight: column by column, each waited for its
// own chain of a load, a product and an exponential.)
template <bool MASKED>
__device__ __forceinline__ void add_weights(const uint32_t *s, const ulonglong2 *off, uint64_t scale2, uint32_t bits,
                                            uint64_t (&acc)[2]) {
    uint64_t x[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const ulonglong2 o = off[i];
        x[2 * i] = o.x;
        x[2 * i + 1] = o.y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = ffma2(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), scale2, x[i]);
    float e[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        e[2 * i] = ex2_approx(f2_lo(x[i]));
        e[2 * i + 1] = ex2_approx(f2_hi(x[i]));
    }
    if constexpr (MASKED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = bits >> i & 1 ? e[i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i & 1] = fadd2(acc[i & 1], f2_pack(e[2 * i], e[2 * i + 1]));
}

// RAGGED: tile_rows < kRows, as whole tokens leave some columns of a chunk without rows.  (Only the last quarter of
// its whole chunks is masked: 4 chunks of 1024 tokens on 5000, 14 heads over 2 of 64, 58 us, and 96 with every quarter.)
template <int D, bool BF16, bool RAGGED>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_tiles_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k, const WeighParams p) {
    using L = WeighLayout<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + L::kBarOff), *k_empty = k_full + 2 * kKeySets, *q_full = k_empty + 2 * kKeySets,
             *q_empty = q_full + L::kRowStages, *off_full = q_empty + L::kRowStages, *off_empty = off_full + kOffStages,
             *s_full = off_empty + kOffStages, *s_free = s_full + 4, *sum_full = s_free + 4, *sum_free = sum_full + 2,
             *drain = sum_free + 2;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMiscOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMiscOff + 4);
    WeighStart *start = reinterpret_cast<WeighStart *>(smem + L::kStartOff);
    long long *warp_sum = reinterpret_cast<long long *>(smem + L::kSumOff);
    float *offs = reinterpret_cast<float *>(smem + L::kOffOff);
    uint32_t *counts = reinterpret_cast<uint32_t *>(smem + L::kCountOff);
    int *live_rows = reinterpret_cast<int *>(smem + L::kLiveOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile_rows = p.tile_tokens * p.G;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kKeySets; ++i) {
            mbar_init(k_full + i, 1);
            mbar_init(k_empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(drain + i, 1);
        for (int i = 0; i < L::kRowStages; ++i) {
            mbar_init(q_full + i, 1);
            mbar_init(q_empty + i, 2);  // both tiles' products
        }
        for (int i = 0; i < kOffStages; ++i) {
            mbar_init(off_full + i, 1);
            mbar_init(off_empty + i, 16);  // one arrival per summing warp
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_free + i, 4);
            mbar_init(sum_full + i, 4);  // (sum_full, then sum_free)
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kTmaWarp && lane == 0) {
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) p.open[blockIdx.x] = make_int4(-1, 0, 0, 0);  // (the plan's barriers are between this and another)
    if (warp == kMmaWarp) {
        // behind the wait and before followers start, as in paged_tiles_kernel
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    tc_fence_before();
    weigh_plan<kThreads>(p, *start, warp_sum, kWeighUnit + 1, &g_weigh_tiles_status,
                         [&](const WeighSeq &s) { return weigh_head_steps(p, s); });
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint32_t kc = 0;  // pieces with rows so far (the producer: their key tiles, two each)
    auto key_set = [](uint32_t piece, int t) { return static_cast<int>(piece % kKeySets * 2 + t); };
    uint32_t ch = 0;  // chunks so far
    bool ok = true;
    WeighCursor cur;
    WeighPiece u;
    cur.begin(p, *start);

    if (warp == kTmaWarp) {
        // ------------------------------------------------------------ producer
        const uint64_t pol_k = l2_policy_evict_first(), pol_q = l2_policy_evict_last();
        const int page = 1 << p.page_shift;
        const int box = min(page, kM), boxes = kM / box;
        // lane -> (key tile, slab, page) of a unit's copies: up to 2 x 2 x 8
        const int my_box = lane % boxes, my_slab = lane / boxes % L::kSlabs, my_tile = lane / boxes / L::kSlabs;
        while (ok && cur.next(p, u)) {
            if (u.s.nq == 0) continue;
            const int key = u.u * kWeighKeys + my_tile * kM + my_box * box;
            const bool live = my_tile < 2 && key < u.s.len;
            int id = live ? __ldg(p.page_table + static_cast<long long>(u.b) * p.max_pages + (key >> p.page_shift)) : 0;
            for (int t = 0; t < 2 && ok; ++t) {
                const uint32_t piece = kc / 2;
                const int set = key_set(piece, t);
                if (piece >= kKeySets && !lanes_wait(k_empty + set, (piece / kKeySets - 1) & 1, abort_flag)) { ok = false; break; }
                const bool mine = live && my_tile == t;
                const int copies = __popc(__ballot_sync(0xffffffffu, mine));
                if (lane == 0) mbar_arrive_expect_tx(k_full + set, copies * box * 128);  // (a tile without keys: none)
                __syncwarp();
                if (mine) {
                    if (id < 0 || id >= p.num_pages) {
                        record_status(&g_weigh_tiles_status, FA_ERR_PAGE);
                        id = p.num_pages;  // outside the tensor: the copy writes zeros
                    }
                    tma_load_4d(smem + set * L::kTileBytes + my_slab * L::kSlab + my_box * box * 128, &map_k, k_full + set, my_slab * 64,
                                key & (page - 1), u.h, id, pol_k);
                }
                ++kc;
            }
            if (!ok) break;
            for (int c = u.c0; c < u.c1; ++c) {
                const uint32_t qs = ch % L::kRowStages;
                if (ch >= L::kRowStages && !lanes_wait(q_empty + qs, (ch / L::kRowStages - 1) & 1, abort_flag)) { ok = false; break; }
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full + qs, tile_rows * 128 * L::kSlabs);
                    for (int i = 0; i < L::kSlabs; ++i)
                        tma_load_3d(smem + L::kRowsOff + qs * L::kTileBytes + i * L::kSlab, &map_q, q_full + qs, i * 64, u.h * p.G,
                                    u.s.t0 + c * p.tile_tokens, pol_q);
                }
                __syncwarp();
                ++ch;
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        // ------------------------------------------------------------ products
        const uint32_t idesc = idesc_f16(BF16, kM, kRows, false, false);
        const int t = warp - kMmaWarp;  // the key tile
        const uint32_t rows = smem_u32(smem) + L::kRowsOff, acc = tmem + t * 2 * kRows;
        while (ok && cur.next(p, u)) {
            if (u.s.nq == 0) continue;
            if (lane == 0) {
                const bool has_keys = u.u * kWeighKeys + t * kM < u.s.len;
                const int set = key_set(kc, t);
                const uint64_t k_desc = sdesc_sw128(smem_u32(smem) + set * L::kTileBytes, 16, 1024);
                ok = mbar_wait(k_full + set, (kc / kKeySets) & 1, abort_flag, kWatchdogNs);
                for (int c = u.c0; ok && c < u.c1; ++c) {  // (a tile without keys goes through the same steps)
                    const uint32_t qs = ch % L::kRowStages, buf = ch & 1;
                    // polled: the product should start the moment the accumulator is free
                    if (ch >= 2 && !mbar_spin(s_free + t * 2 + buf, (ch / 2 - 1) & 1, abort_flag, kWatchdogNs)) { ok = false; break; }
                    if (!mbar_wait(q_full + qs, (ch / L::kRowStages) & 1, abort_flag, kWatchdogNs)) { ok = false; break; }
                    tc_fence_after();
                    if (has_keys) issue_qk<D>(acc + buf * kRows, k_desc, sdesc_sw128(rows + qs * L::kTileBytes, 16, 1024), idesc);
                    umma_commit(s_full + t * 2 + buf);
                    umma_commit(q_empty + qs);
                    ++ch;
                }
                if (ok) umma_commit(k_empty + set);
            }
            ++kc;
            ok = __all_sync(0xffffffffu, ok);
        }
        if (lane == 0) {  // nothing may still run on the tensor core at teardown
            umma_commit(drain + t);
            int dummy = 0;
            mbar_wait(drain + t, 0, &dummy, kWatchdogNs);
        }
        __syncwarp();
    } else if (warp >= kOffWarp) {
        // ------------------------------------------------------------ log-sum-exps
        int at[4];  // this lane's four rows of a chunk
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = i * 32 + lane;
            at[i] = c < tile_rows ? c / p.G * p.Hq + c % p.G : -1;
        }
        while (ok && cur.next(p, u)) {
            if (u.s.nq == 0) continue;
            // (a lot is of one piece: the last of a piece may have fewer chunks)
            const int rows = u.s.nq * p.G;
            for (int c0 = u.c0; c0 < u.c1; c0 += kOffChunks, ++ch) {
                float v[kOffChunks][4];
#pragma unroll
                for (int k = 0; k < kOffChunks; ++k) {
                    const int c = c0 + k;
                    if (c >= u.c1) break;
                    const float *lse = p.lse + (static_cast<long long>(u.s.t0) + c * p.tile_tokens) * p.Hq + u.h * p.G;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[k][i] = at[i] >= 0 && c * tile_rows + i * 32 + lane < rows ? __ldg(lse + at[i]) : -INFINITY;
                }
                const uint32_t os = ch % kOffStages;
                if (ch >= kOffStages && !lanes_wait(off_empty + os, (ch / kOffStages - 1) & 1, abort_flag)) { ok = false; break; }
#pragma unroll
                for (int k = 0; k < kOffChunks; ++k) {
                    if (c0 + k >= u.c1) break;
                    uint32_t is[4];  // the rows that count, as bits
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float off = weigh_off(v[k][i]);
                        offs[(os * kOffChunks + k) * kRows + i * 32 + lane] = off;
                        is[i] = __ballot_sync(0xffffffffu, off != -INFINITY);
                    }
                    const int live = min(rows - (c0 + k) * tile_rows, tile_rows);
                    const bool all = __popc(is[0]) + __popc(is[1]) + __popc(is[2]) + __popc(is[3]) == live;
                    if (lane == 0) {
                        reinterpret_cast<uint4 *>(counts)[os * kOffChunks + k] = make_uint4(is[0], is[1], is[2], is[3]);
                        live_rows[os * kOffChunks + k] = all ? live : -live;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(off_full + os);
            }
        }
    } else {
        // ------------------------------------------------------------ exponentials and sums
        const int t = warp >> 3;
        const uint32_t odd = warp >> 2 & 1;
        float *odd_sum = reinterpret_cast<float *>(smem + L::kOddOff) + t * kM + (warp & 3) * 32 + lane;
        uint32_t pieces = 0, lots = 0;  // pieces of several chunks, lots of log-sum-exps
        const int in_unit = t * kM + (warp & 3) * 32 + lane;
        const uint32_t s_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (t * 2 + odd) * kRows;
        const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2);
        while (ok && cur.next(p, u)) {
            const int key = u.u * kWeighKeys + in_unit;
            const bool tile_live = u.u * kWeighKeys + t * kM < u.s.len;
            float sum = 0.f;
            bool mine = !odd;  // whose sums are written
            if (u.s.nq > 0) {
                const uint32_t ch0 = ch;
                const int see = weigh_first_token(p, u.s, key) * p.G;  // the first row that sees the key
                uint64_t acc[2] = {};  // two pairs of sums
                const int c1 = u.c1;
                for (int c0 = u.c0; ok && c0 < c1; c0 += kOffChunks, ++lots) {
                    const uint32_t os = lots % kOffStages;
                    if (!lanes_wait(off_full + os, (lots / kOffStages) & 1, abort_flag)) { ok = false; break; }
                    for (int c = c0; c < min(c1, c0 + kOffChunks); ++c, ++ch) {
                        if ((ch & 1) != odd) continue;
                        const int live = live_rows[os * kOffChunks + c - c0];
                        if (!warp_wait(s_full + t * 2 + odd, (ch / 2) & 1, abort_flag)) { ok = false; break; }
                        tc_fence_after();
                        auto load = [&](int q, uint32_t (&s)[32]) {
                            tmem_ld32(s_addr + q * 32, s);
                            tmem_ld_wait();
                            reg_fence32(s);
                        };
                        auto release = [&] {  // S is in registers: the next one may start
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(s_free + t * 2 + odd);
                        };
                        // Columns [first, live) of the chunk are rows that see the key; what lies outside may be anything.
                        const int first = see - c * tile_rows;
                        const ulonglong2 *off = reinterpret_cast<const ulonglong2 *>(offs + (os * kOffChunks + c - c0) * kRows);
                        if (__all_sync(0xffffffffu, first <= 0) && tile_live && live >= (RAGGED ? max(tile_rows, kRows - 32) : kRows)) {
#pragma unroll
                            for (int q = 0; q < kRows / 32; ++q) {
                                uint32_t s[32];
                                load(q, s);
                                if (q == kRows / 32 - 1) release();
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    if (RAGGED && q == kRows / 32 - 1)
                                        add_weights<true>(&s[i * 8], off + q * 8 + i * 2, scale2, ~(~0u << max(0, min(live - q * 32 - i * 8, 8))), acc);
                                    else
                                        add_weights<false>(&s[i * 8], off + q * 8 + i * 2, scale2, ~0u, acc);
                                }
                            }
                        } else {
                            // the quarters that any of the warp's keys are seen from; of the rows those that count
                            const uint32_t *is = counts + (os * kOffChunks + c - c0) * 4;
                            const int q0 = max(0, __reduce_min_sync(0xffffffffu, first)) / 32, q1 = tile_live ? (abs(live) + 31) / 32 : 0;
#pragma unroll 1
                            for (int q = q0; q < q1; ++q) {
                                uint32_t s[32];
                                load(q, s);
                                const int hidden = first - q * 32;
                                const uint32_t bits = hidden >= 32 ? 0u : is[q] & (~0u << max(hidden, 0));
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    add_weights<true>(&s[i * 8], off + q * 8 + i * 2, scale2, bits >> i * 8, acc);
                            }
                            release();
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(off_empty + os);
                }
                if (!ok) break;
                const uint64_t both = fadd2(acc[0], acc[1]);
                sum = f2_lo(both) + f2_hi(both);
                // the odd chunks' sums go to the even ones' warps (of a single chunk to nobody: neither waits for the other)
                if (c1 - u.c0 == 1) {
                    mine = (ch0 & 1) == odd;
                } else if (odd) {
                    if (pieces > 0 && !lanes_wait(sum_free + t, (pieces - 1) & 1, abort_flag)) { ok = false; break; }
                    *odd_sum = sum;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sum_full + t);
                } else {
                    if (!lanes_wait(sum_full + t, pieces & 1, abort_flag)) { ok = false; break; }
                    sum += *odd_sum;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sum_free + t);
                }
                pieces += c1 - u.c0 > 1;
            }
            if (!mine) continue;
            if (u.opens && u.closes) {
                if (key < u.s.len) weigh_store(p, u.b, u.h, u.s.nq, key, sum);
            } else {
                p.part[(static_cast<long long>(blockIdx.x) * 2 + (u.opens ? 1 : 0)) * kWeighKeys + in_unit] = sum;
                if (u.opens && in_unit == 0)
                    p.open[blockIdx.x] = make_int4(weigh_cta_of(start->end + u.to_last, start->W, start->G), u.b, u.h, u.u * kWeighKeys);
            }
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
        for (uint32_t i = kc > 2 * kKeySets ? kc - 2 * kKeySets : 0; i < kc; ++i)
            mbar_wait(k_full + key_set(i / 2, i & 1), (i / 2 / kKeySets) & 1, &dummy, kDrainNs);
        for (uint32_t i = ch > L::kRowStages ? ch - L::kRowStages : 0; i < ch; ++i)
            mbar_wait(q_full + i % L::kRowStages, (i / L::kRowStages) & 1, &dummy, kDrainNs);
        record_status(&g_weigh_tiles_status, FA_ERR_WATCHDOG);
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// The units that ranges cut: the one that CTA c left open has its sums in place 1 of c and place 0 of the
// CTAs after it, up to the one that closed it.
__global__ void __launch_bounds__(kWeighKeys) weigh_join_kernel(const WeighParams p) {
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    const int c = blockIdx.x;
    const int4 open = p.open[c];
    if (open.x < 0) return;
    float sum = p.part[(static_cast<long long>(c) * 2 + 1) * kWeighKeys + threadIdx.x];
    for (int k = c + 1; k <= open.x; ++k) sum += p.part[static_cast<long long>(k) * 2 * kWeighKeys + threadIdx.x];
    const WeighSeq s = weigh_seq(p, open.y);
    const int key = open.w + threadIdx.x;
    if (key < s.len) weigh_store(p, open.y, open.z, s.nq, key, sum);
}

template <int D, bool BF16, bool RAGGED>
int launch_d(const WeighLaunch &a, const WeighParams &p, const DeviceInfo &dev, cudaStream_t stream) {
    using L = WeighLayout<D>;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cuda_fail(cudaErrorNotSupported);
    CUtensorMap mq, mk;
    // queries [token][head][d], a box of the G heads of a kv head and tile_tokens tokens
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.total_q};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * p.Hq};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)p.tile_tokens};
    const cuuint32_t estr[3] = {1, 1, 1};
    if (enc(&mq, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t *>(p.q), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cuda_fail(cudaErrorInvalidValue);
    int rc = make_page_map(&mk, a.c.k_pages, a.c, kM);
    if (rc != FA_OK) return rc;
    const auto kernel = weigh_tiles_kernel<D, BF16, RAGGED>;
    static std::atomic<bool> ready[kMaxDevices];
    if ((rc = ready_kernel(kernel, L::kSmemBytes, 0, dev.device, ready)) != FA_OK) return rc;
    PagedConfig cfg(dev.num_sms, kThreads, L::kSmemBytes, true, stream);
    cudaError_t e = cudaLaunchKernelEx(&cfg.c, kernel, mq, mk, p);
    if (e != cudaSuccess) return cuda_fail(e);
    PagedConfig join(dev.num_sms, kWeighKeys, 0, true, stream);
    e = cudaLaunchKernelEx(&join.c, weigh_join_kernel, p);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

size_t part_bytes(int num_sms) { return static_cast<size_t>(num_sms) * 2 * kWeighKeys * 4; }

}  // namespace

// Which kernel: the tiles' takes about as long for one row of a kv head as for 128, the warp products' some more with
// every eight.  In us, theirs against the tiles':
//   16 sequences of 4096, 32 heads over 8, d = 128:   8 rows 28 : 34, 16 rows 46 : 34, 32 rows 66 : 34, 128 rows 189 : 36
//   4 of 16384, 12 heads, d = 64:                     8 rows 24 : 37, 12 rows 45 : 37, 24 rows 57 : 37, 128 rows 217 : 38
//   32 of 1000, 64 over 8, d = 128:                   8 rows 13 : 22, 16 rows 22 : 21, 32 rows 33 : 21, 128 rows 96 : 25
//   1 of 4096, 32 over 8, d = 128 (its start counts): 8 rows  6 : 11, 32 rows  9 : 11, 48 rows 11 : 11, 64 rows 13 : 11
bool weigh_in_tiles(const WeighLaunch &a, int num_sms) {
    const int group = a.Hq / a.c.num_heads;
    const long long rows = static_cast<long long>(a.max_q) * group;
    const int max_len = std::min(a.max_pages * a.c.page_size, a.weights_len);
    const long long units = static_cast<long long>(a.B) * a.c.num_heads * ((max_len + kWeighKeys - 1) / kWeighKeys);
    return rows > (units >= 2LL * num_sms ? 8 : 48) && group <= kRows && a.total_q > 0;
}

size_t weigh_scratch_bytes(int num_sms) { return part_bytes(num_sms) + static_cast<size_t>(num_sms) * sizeof(int4); }

int launch_weigh_tiles(const WeighLaunch &a, WeighParams p, const DeviceInfo &dev, cudaStream_t stream) {
    p.tile_tokens = kRows / p.G;
    p.part = static_cast<float *>(a.scratch);
    p.open = reinterpret_cast<int4 *>(static_cast<char *>(a.scratch) + part_bytes(dev.num_sms));
    const bool bf16 = a.c.dtype == FA_BF16;
    const bool ragged = p.tile_tokens * p.G < kRows;
    auto launch = [&](auto d, auto is_bf16) {
        constexpr int D = decltype(d)::value;
        constexpr bool BF16 = decltype(is_bf16)::value;
        return ragged ? launch_d<D, BF16, true>(a, p, dev, stream) : launch_d<D, BF16, false>(a, p, dev, stream);
    };
    const std::integral_constant<int, 64> d64;
    const std::integral_constant<int, 128> d128;
    if (a.c.head_dim == 64) return bf16 ? launch(d64, std::true_type()) : launch(d64, std::false_type());
    return bf16 ? launch(d128, std::true_type()) : launch(d128, std::false_type());
}

int read_weigh_tiles_status(int reset) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_weigh_tiles_status, sizeof(int)) != cudaSuccess) return -1;
    if (reset && v) {
        int z = 0;
        if (cudaMemcpyToSymbol(g_weigh_tiles_status, &z, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace fa
