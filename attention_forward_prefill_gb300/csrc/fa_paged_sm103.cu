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
//
// Measured: 32 sequences of 200 to 8192 tokens, 32 heads over 8 of 128, bf16: 97 us
// for 603 MB of DRAM reads, 6.28 TB/s (92.4% of the copy rate).  A CTA alone on an SM
// takes 0.73 us a tile with 16 rows, 1.41 with 32, 2.03 with 64 (d = 128), and 1.6 us
// per unit.
#include <algorithm>

#include "fa_paged_rows.cuh"

namespace fa {

namespace {

__device__ int g_paged_status = 0;

template <int D, int RT>
struct PagedLayout {
    using R = PagedRows<D, RT, false>;  // (sizes are the same for both types)
    static constexpr int kRows = 16 * RT;
    static constexpr int kStage = 2 * R::kOperand;
    static constexpr int kStages = 98304 / kStage;    // 96 KB in flight per CTA, two CTAs per SM
    // Query rows 16 bytes apart in banks where there is room, so that the fragment
    // loads do not conflict (32 or 64 rows of 256 bytes leave none; it is once per unit).
    static constexpr int kQPitch = D * 2 + (RT == 1 ? 16 : 0);
    static constexpr int kQOff = kStages * kStage;
    static constexpr int kJoinOff = kQOff + kRows * kQPitch;
    static constexpr int kBarOff = kJoinOff + R::kJoinBytes;
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
    using R = PagedRows<D, RT, BF16>;
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
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, kConsumers);
        }
        mbar_init(u_full, 1);
        mbar_init(u_empty, kConsumers);
        for (int t = 0; t < RT; ++t) {
            mbar_init(j_full + t, R::KG);
            mbar_init(j_empty + t, R::KG);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kConsumers && lane == 0) {
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    paged_enter(p);
    paged_plan<RowsCut, kPagedThreads>(p, *start, warp_sum, &g_paged_status);
    if (static_cast<int>(blockIdx.x) >= start->G) {  // no work: makes room for a CTA that has some
        if (threadIdx.x == 0) paged_note_none(p);
        return;
    }
    uint32_t units = 0, tiles = 0;  // handed over / taken so far

    if (warp == kConsumers) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = l2_policy_evict_first();
        const int page = 1 << p.page_shift;
        const int box = min(page, kTile), boxes = kTile / box;  // pages (or parts of one) per tile
        // lane -> (operand, slab, box) of a tile's copies
        const int my_box = lane % boxes, my_slab = lane / boxes % (D / 64), my_op = lane / boxes / (D / 64);
        bool ok = true;
        PagedCursor<RowsCut> cur;
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
                        record_status(&g_paged_status, FA_ERR_PAGE);
                        id = p.num_pages;  // outside the tensor: the copy writes zeros
                    }
                    tma_load_4d(smem + st * L::kStage + my_op * R::kOperand + my_slab * R::kSlab + my_box * box * 128,
                                my_op ? &map_v : &map_k, full + st, my_slab * 64, key & (page - 1), u.hk, id, pol);
                }
                id = next;
                ++tiles;
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ consumers
        R rows(warp, lane);
        const uint32_t zero = static_cast<uint32_t>(p.unit_steps) >> 30;
        const uint32_t ring = smem_u32(smem);
        bool ok = true;
        while (ok) {
            if (!lanes_wait(u_full, units & 1, abort_flag)) { ok = false; break; }
            ++units;
            const PagedPiece u = *piece;
            if (u.kind < 0) break;
            rows.begin(smem_u32(smem + L::kQOff), L::kQPitch);
            const bool pending = rows.loads_pending(zero) || paged_pending(u, static_cast<int>(zero));
            __syncwarp();
            if (lane == 0) mbar_arrive(u_empty + pending);
            // the last key that each of this thread's two rows sees
            int lim0 = u.len - 1, lim1 = u.len - 1;
            if (p.causal) {
                const int r0 = u.row0 + rows.rw * 16 + rows.qrow;
                lim0 = min(lim0, u.len - u.nq + r0 / p.G);
                lim1 = min(lim1, u.len - u.nq + (r0 + 8) / p.G);
            }
            for (int j = u.j0; j < u.j1; ++j) {
                const int st = tiles % L::kStages;
                if (!lanes_wait(full + st, (tiles / L::kStages) & 1, abort_flag)) { ok = false; break; }
                ++tiles;
                rows.tile(ring + st * L::kStage, lim0 - j * kTile, lim1 - j * kTile, u.len - j * kTile, p.scale_log2);
                const bool pending = rows.loads_pending(zero);
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + st + pending);
            }
            if (!ok) break;
            rows.end();
            ok = rows.write(
                min(RB, u.nq * p.G - u.row0), smem + L::kJoinOff, j_full, j_empty, abort_flag,
                [&](int r) { return paged_row(p, u, r); },
                [&](int r, long long row, int col, auto &acc, float m, float l) {
                    paged_emit<D, RB>(p, u, r, row, col, acc, m, l);
                });
        }
        __syncwarp();
    }
    paged_leave(p);
    __syncthreads();
    if (*abort_flag && warp == kConsumers && lane == 0) {
        // let every copy already issued land before the CTA goes away
        constexpr uint64_t kDrainNs = 200ull * 1000ull * 1000ull;
        int dummy = 0;
        if (units > 0) mbar_wait(u_full, (units - 1) & 1, &dummy, kDrainNs);
        for (uint32_t i = tiles > L::kStages ? tiles - L::kStages : 0; i < tiles; ++i)
            mbar_wait(full + i % L::kStages, (i / L::kStages) & 1, &dummy, kDrainNs);
        record_status(&g_paged_status, FA_ERR_WATCHDOG);
    }
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

// CTAs per cluster when the call (prefix_max: and the keys in front of it) goes to paged_cluster_kernel, or 0.
int cluster_size(const PagedPass &x, long long prefix_max) {
    return paged_cluster_size(x.plan, x.c.head_dim, x.units, x.p.max_len, prefix_max, x.num_sms);
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
    x.early = true;
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
    const PagedPlan pl = x.plan = plan_paged(a.max_q, p.G, a.c.head_dim);
    p.block_rows = pl.block_rows;
    p.unit_steps = pl.unit_steps;
    p.tile_tokens = pl.tiles ? pl.block_rows / p.G / 2 : 0;
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
    return pass_bytes(plan_paged(max_q, group, d), d, num_sms);
}

bool paged_needs_scratch(const PagedLaunch &a, const DeviceInfo &dev) {
    return cluster_size(make_pass(a, dev, nullptr), 0) == 0;
}

int launch_paged(const PagedLaunch &a, const DeviceInfo &dev, cudaStream_t stream) {
    const PagedPass x = make_pass(a, dev, a.scratch);
    const int size = cluster_size(x, 0);
    return size ? launch_paged_cluster(x, size, stream) : launch_pass(x, stream);
}

bool paged_pair_needs_scratch(const PagedLaunch &pre, const PagedLaunch &own, const DeviceInfo &dev) {
    return cluster_size(make_pass(own, dev, nullptr), 1LL * pre.max_pages * pre.c.page_size) == 0;
}

size_t paged_pair_scratch_bytes(int B, int Hq, int Hkv, int d, int num_sms) {
    const size_t rows = static_cast<size_t>(B) * Hq;
    size_t total = 0;
    for (int i = 0; i < 2; ++i) {
        const PagedPlan pl = plan_paged(i ? 1 : B, Hq / Hkv, d);
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
    PagedPass one = make_pass(own, dev, nullptr);
    one.p.pre_table = pre.page_table;
    one.p.pre_lens = pre.seq_lens;
    one.p.pre_max_len = pre.max_pages * pre.c.page_size;
    if (const int size = cluster_size(one, one.p.pre_max_len)) return launch_paged_cluster(one, size, stream);
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
        // (One call right behind another: 192 us with the first pass launched when the last
        // call's join is through, 208 with it waiting on the SMs under that join.)
        x.early = i == 1;
        x.p.first = i == 0;
        x.p.num_sms = dev.num_sms;
        x.p.per_sm = x.plan.per_sm;
        x.p.step_ns = paged_step_ns(x.plan, d);
    }
    for (int i = 0; i < 2; ++i) paged_set_peer(pass[i].p, pass[1 - i].p, pass[1 - i].plan);
    int rc;
    for (const PagedPass &x : pass)
        if ((rc = launch_pass(x, stream)) != FA_OK) return rc;
    constexpr long long kWarps = kJoinThreads / 32;
    const int grid = static_cast<int>(std::min<long long>(2LL * dev.num_sms, (static_cast<long long>(rows) + kWarps - 1) / kWarps));
    PagedConfig cfg(grid, kJoinThreads, 0, true, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, d == 64 ? paged_pair_join_kernel<64> : paged_pair_join_kernel<128>,
                                             pass[0].p, pass[1].p, pass[0].plan.slot_rows, pass[1].plan.slot_rows,
                                             pass[0].blocks, pass[1].blocks, pass[0].grid, pass[1].grid);
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
