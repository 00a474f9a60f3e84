// fa_weigh_tiles_sm103.cu -- what cached tokens got of the attention of many query rows.
//
// The sums of fa_weigh_sm103.cu, S^T = K Q^T on 128 x 128 tiles in tensor memory: a thread holds
// a key (a lane of the accumulator) and goes through the rows (its columns), so that the sum over
// the rows stays in the thread.  One product and one exponential per pair of key and row: at
// d = 128 a tile takes the tensor core 256 clocks and the 16384 exponentials 512 at 32 a clock
// and SM, which sets the time.
//
// CTA (one per SM, 12 warps):
//   warps 0-3   exponentials and sums of the unit's keys 0 .. 127 (thread = key = TMEM lane)
//   warps 4-7   of keys 128 .. 255
//   warp  8     producer: both key tiles of a unit, then its chunks of query rows, by TMA
//   warp  9     issues the products (one thread), owns the tensor memory
//   warps 10-11 the chunks' log-sum-exps, in turn
// A unit's 256 keys stay in shared memory while the chunks of 128 rows go by, so that a chunk is
// loaded once for two products.  Every warp walks through the CTA's pieces (fa_weigh_cut.cuh) by
// itself.  TMEM: two accumulators for each key tile, so that a product runs under the other's
// exponentials.
#include <algorithm>
#include <atomic>

#include "fa_weigh.cuh"

namespace fa {

namespace {

constexpr int kThreads = 384;
constexpr int kRegsSums = 176;
constexpr int kRegsOther = 152;
constexpr int kMinLaunchRegs = (2 * 128 * kRegsSums + 128 * kRegsOther + kThreads - 1) / kThreads;
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kM = 128;  // keys of a tile, rows of a chunk
constexpr uint32_t kTmemCols = 512;
constexpr int kKeyStages = 2, kOffStages = 4;

__device__ int g_weigh_tiles_status = 0;

template <int D>
struct WeighLayout {
    static constexpr int kSlab = kM * 128;
    static constexpr int kSlabs = D / 64;
    static constexpr int kTileBytes = kSlabs * kSlab;
    static constexpr int kRowStages = D == 128 ? 3 : 4;
    static constexpr int kRowsOff = 2 * kKeyStages * kTileBytes;
    static constexpr int kOffOff = kRowsOff + kRowStages * kTileBytes;  // [kOffStages][kM] floats
    static constexpr int kBarOff = kOffOff + kOffStages * kM * 4;
    // k_full, k_empty, q_full, q_empty, off_full, off_empty, s_full[tile][buffer], s_free[tile][buffer], drain
    static constexpr int kNumBars = 2 * kKeyStages + 2 * kRowStages + 2 * kOffStages + 8 + 1;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kStartOff = kMiscOff + 8;
    static constexpr int kSumOff = kStartOff + (int)sizeof(WeighStart);
    static constexpr int kSmemBytes = kSumOff + 8 * (kThreads / 32);
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_tiles_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k, const WeighParams p) {
    using L = WeighLayout<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + L::kBarOff), *k_empty = k_full + kKeyStages,
             *q_full = k_empty + kKeyStages, *q_empty = q_full + L::kRowStages, *off_full = q_empty + L::kRowStages,
             *off_empty = off_full + kOffStages, *s_full = off_empty + kOffStages, *s_free = s_full + 4, *drain = s_free + 4;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMiscOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMiscOff + 4);
    WeighStart *start = reinterpret_cast<WeighStart *>(smem + L::kStartOff);
    long long *warp_sum = reinterpret_cast<long long *>(smem + L::kSumOff);
    float *offs = reinterpret_cast<float *>(smem + L::kOffOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile_rows = p.tile_tokens * p.G;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kKeyStages; ++i) {
            mbar_init(k_full + i, 1);
            mbar_init(k_empty + i, 1);
        }
        for (int i = 0; i < L::kRowStages; ++i) {
            mbar_init(q_full + i, 1);
            mbar_init(q_empty + i, 1);
        }
        for (int i = 0; i < kOffStages; ++i) {
            mbar_init(off_full + i, 1);
            mbar_init(off_empty + i, 8);  // one arrival per summing warp
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_free + i, 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kTmaWarp && lane == 0) {
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
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
    uint32_t kc = 0;  // pieces with rows so far
    uint32_t ch = 0;  // chunks so far
    bool ok = true;
    WeighCursor cur;
    cur.begin(p, *start);
    WeighPiece u;

    if (warp == kTmaWarp) {
        // ------------------------------------------------------------ producer
        regs_shrink<kRegsOther>();
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
            const uint32_t st = kc % kKeyStages;
            if (kc >= kKeyStages && !lanes_wait(k_empty + st, (kc / kKeyStages - 1) & 1, abort_flag)) { ok = false; break; }
            const int copies = __popc(__ballot_sync(0xffffffffu, live));
            if (lane == 0) mbar_arrive_expect_tx(k_full + st, copies * box * 128);
            __syncwarp();
            if (live) {
                if (id < 0 || id >= p.num_pages) {
                    record_status(&g_weigh_tiles_status, FA_ERR_PAGE);
                    id = p.num_pages;  // outside the tensor: the copy writes zeros
                }
                tma_load_4d(smem + (2 * st + my_tile) * L::kTileBytes + my_slab * L::kSlab + my_box * box * 128, &map_k, k_full + st,
                            my_slab * 64, key & (page - 1), u.h, id, pol_k);
            }
            ++kc;
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
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ products
        regs_shrink<kRegsOther>();
        const uint32_t idesc = idesc_f16(BF16, kM, kM, false, false);
        const uint32_t base = smem_u32(smem);
        while (ok && cur.next(p, u)) {
            if (u.s.nq == 0) continue;
            if (lane == 0) {
                const uint32_t st = kc % kKeyStages;
                const int tiles = u.u * kWeighKeys + kM < u.s.len ? 2 : 1;
                do {
                    if (!mbar_wait(k_full + st, (kc / kKeyStages) & 1, abort_flag, kWatchdogNs)) { ok = false; break; }
                    for (int c = u.c0; c < u.c1; ++c) {
                        const uint32_t qs = ch % L::kRowStages, buf = ch & 1;
                        if (!mbar_wait(q_full + qs, (ch / L::kRowStages) & 1, abort_flag, kWatchdogNs)) { ok = false; break; }
                        const uint64_t q_desc = sdesc_sw128(base + L::kRowsOff + qs * L::kTileBytes, 16, 1024);
                        for (int t = 0; t < 2; ++t) {  // (a tile without keys goes through the same steps)
                            if (ch >= 2 && !mbar_wait(s_free + t * 2 + buf, (ch / 2 - 1) & 1, abort_flag, kWatchdogNs)) { ok = false; break; }
                            tc_fence_after();
                            if (t < tiles)
                                issue_qk<D>(tmem + (t * 2 + buf) * kM, sdesc_sw128(base + (2 * st + t) * L::kTileBytes, 16, 1024), q_desc, idesc);
                            umma_commit(s_full + t * 2 + buf);
                        }
                        if (!ok) break;
                        umma_commit(q_empty + qs);
                        ++ch;
                    }
                    if (!ok) break;
                    umma_commit(k_empty + st);
                } while (false);
                ++kc;
            }
            ok = __all_sync(0xffffffffu, ok);
        }
        if (lane == 0) {  // nothing may still run on the tensor core at teardown
            umma_commit(drain);
            int dummy = 0;
            mbar_wait(drain, 0, &dummy, kWatchdogNs);
        }
        __syncwarp();
    } else if (warp >= 10) {
        // ------------------------------------------------------------ log-sum-exps (warps 10, 11)
        regs_shrink<kRegsOther>();
        int at[4];  // this lane's four rows of a chunk
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = lane * 4 + i;
            at[i] = c < tile_rows ? c / p.G * p.Hq + c % p.G : -1;
        }
        while (ok && cur.next(p, u)) {
            if (u.s.nq == 0) continue;
            for (int c = u.c0; c < u.c1; ++c, ++ch) {
                if ((ch & 1) != (warp & 1)) continue;
                const float *lse = p.lse + (static_cast<long long>(u.s.t0) + c * p.tile_tokens) * p.Hq + u.h * p.G;
                const int rows = u.s.nq * p.G - c * tile_rows;
                float4 v;
                v.x = at[0] >= 0 && lane * 4 < rows ? weigh_off(__ldg(lse + at[0])) : -INFINITY;
                v.y = at[1] >= 0 && lane * 4 + 1 < rows ? weigh_off(__ldg(lse + at[1])) : -INFINITY;
                v.z = at[2] >= 0 && lane * 4 + 2 < rows ? weigh_off(__ldg(lse + at[2])) : -INFINITY;
                v.w = at[3] >= 0 && lane * 4 + 3 < rows ? weigh_off(__ldg(lse + at[3])) : -INFINITY;
                const uint32_t os = ch % kOffStages;
                if (ch >= kOffStages && !lanes_wait(off_empty + os, (ch / kOffStages - 1) & 1, abort_flag)) { ok = false; break; }
                *reinterpret_cast<float4 *>(offs + os * kM + lane * 4) = v;
                __syncwarp();
                if (lane == 0) mbar_arrive(off_full + os);
            }
        }
    } else {
        // ------------------------------------------------------------ exponentials and sums
        regs_grow<kRegsSums>();
        const int t = warp >> 2;
        const int in_unit = t * kM + (warp & 3) * 32 + lane;
        const uint32_t s_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + t * 2 * kM;
        const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2);
        if (threadIdx.x == 0) p.open[blockIdx.x] = make_int4(-1, 0, 0, 0);
        while (ok && cur.next(p, u)) {
            const int key = u.u * kWeighKeys + in_unit;
            const bool tile_live = u.u * kWeighKeys + t * kM < u.s.len;
            float sum = 0.f;
            if (u.s.nq > 0) {
                const int see = weigh_first_token(p, u.s, key) * p.G;  // the first row that sees the key
                // two sums of two each
                uint64_t acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
                for (int c = u.c0; c < u.c1; ++c, ++ch) {
                    const uint32_t buf = ch & 1, os = ch % kOffStages;
                    if (!warp_wait(off_full + os, (ch / kOffStages) & 1, abort_flag)) { ok = false; break; }
                    if (!warp_wait(s_full + t * 2 + buf, (ch / 2) & 1, abort_flag)) { ok = false; break; }
                    if (tile_live) {
                        tc_fence_after();
                        // columns of the chunk that the key is seen from: what lies outside may be anything
                        const int first = see - c * tile_rows, end = min(u.s.nq * p.G - c * tile_rows, tile_rows);
                        const bool all = __all_sync(0xffffffffu, first <= 0);
                        const float4 *off4 = reinterpret_cast<const float4 *>(offs + os * kM);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t s[32];
                            tmem_ld32(s_addr + buf * kM + q * 32, s);
                            tmem_ld_wait();
                            reg_fence32(s);
                            if (q == 3) {  // S is in registers: the next one may start
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(s_free + t * 2 + buf);
                            }
                            const bool plain = all && end >= q * 32 + 32;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 o = off4[q * 8 + i];
                                const uint64_t x = ffma2(f2_pack(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), scale2,
                                                         f2_pack(o.x, o.y));
                                const uint64_t y = ffma2(f2_pack(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), scale2,
                                                         f2_pack(o.z, o.w));
                                float e[4] = {ex2_approx(f2_lo(x)), ex2_approx(f2_hi(x)), ex2_approx(f2_lo(y)), ex2_approx(f2_hi(y))};
                                if (!plain) {
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        const int column = q * 32 + i * 4 + k;
                                        if (column < first || column >= end) e[k] = 0.f;
                                    }
                                }
                                acc[0] = fadd2(acc[0], f2_pack(e[0], e[1]));
                                acc[1] = fadd2(acc[1], f2_pack(e[2], e[3]));
                            }
                        }
                    } else {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(s_free + t * 2 + buf);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(off_empty + os);
                }
                if (!ok) break;
                const uint64_t both = fadd2(acc[0], acc[1]);
                sum = f2_lo(both) + f2_hi(both);
            }
            if (u.opens && u.closes) {
                if (key < u.s.len) weigh_store(p, u.b, u.h, u.s.nq, key, sum);
            } else {
                p.part[(static_cast<long long>(blockIdx.x) * 2 + (u.opens ? 1 : 0)) * kWeighKeys + in_unit] = sum;
                if (u.opens && threadIdx.x == 0)
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
        for (uint32_t i = kc > kKeyStages ? kc - kKeyStages : 0; i < kc; ++i)
            mbar_wait(k_full + i % kKeyStages, (i / kKeyStages) & 1, &dummy, kDrainNs);
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

template <int D, bool BF16>
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
    const auto kernel = weigh_tiles_kernel<D, BF16>;
    static std::atomic<bool> ready[kMaxDevices];
    if ((rc = ready_kernel(kernel, L::kSmemBytes, kMinLaunchRegs, dev.device, ready)) != FA_OK) return rc;
    PagedConfig cfg(dev.num_sms, kThreads, L::kSmemBytes, true, stream);
    cudaError_t e = cudaLaunchKernelEx(&cfg.c, kernel, mq, mk, p);
    if (e != cudaSuccess) return cuda_fail(e);
    PagedConfig join(dev.num_sms, kWeighKeys, 0, true, stream);
    e = cudaLaunchKernelEx(&join.c, weigh_join_kernel, p);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

size_t part_bytes(int num_sms) { return static_cast<size_t>(num_sms) * 2 * kWeighKeys * 4; }

}  // namespace

bool weigh_in_tiles(const WeighLaunch &a) {
    const int group = a.Hq / a.c.num_heads;
    return static_cast<long long>(a.max_q) * group > 64 && group <= kM && a.total_q > 0;
}

size_t weigh_scratch_bytes(int num_sms) { return part_bytes(num_sms) + static_cast<size_t>(num_sms) * sizeof(int4); }

int launch_weigh_tiles(const WeighLaunch &a, WeighParams p, const DeviceInfo &dev, cudaStream_t stream) {
    p.tile_tokens = kM / p.G;
    p.part = static_cast<float *>(a.scratch);
    p.open = reinterpret_cast<int4 *>(static_cast<char *>(a.scratch) + part_bytes(dev.num_sms));
    const bool bf16 = a.c.dtype == FA_BF16;
    if (a.c.head_dim == 64) return bf16 ? launch_d<64, true>(a, p, dev, stream) : launch_d<64, false>(a, p, dev, stream);
    return bf16 ? launch_d<128, true>(a, p, dev, stream) : launch_d<128, false>(a, p, dev, stream);
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
