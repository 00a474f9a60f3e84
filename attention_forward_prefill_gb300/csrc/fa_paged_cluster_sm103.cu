// fa_paged_cluster_sm103.cu -- attention over a paged cache for calls that are all
// latency: few units, few keys.
//
// The cut into equal ranges that paged_rows_kernel makes costs such a call a scan
// of the lengths, a scratch allocation and a second kernel that joins the pieces.
// Here a unit (sequence, kv head, row block) belongs to a thread-block cluster, its
// key tiles are dealt to the cluster's CTAs, and the CTAs join their rows through
// each other's shared memory: one launch and no scratch.  One token of one sequence
// of 1000, 12 heads of 64: 9.0 us by the split form, 4.5 us here (back to back in a
// graph), of which the launch and four loads that wait for one another (length, page
// id, tile, the other CTAs' rows) are most.  The balance is only as good as the lengths
// are alike, and a cluster has no more than eight CTAs, so launch_paged takes this
// form only where no sequence can be long (paged_cluster_size).
//
// A shared prefix is read by every sequence's clusters in front of its own keys: at
// these sizes its keys come from L2, and one kernel replaces three (four sequences
// behind 777 tokens, 12 heads of 64: 10.9 to 6.0 us).
#include <algorithm>

#include "fa_paged_rows.cuh"

namespace fa {

namespace {

constexpr int kMaxCluster = 8;

__device__ int g_cluster_status = 0;

template <int D, int RT>
struct ClusterLayout {
    using R = PagedRows<D, RT, false>;
    static constexpr int kRows = 16 * RT;
    static constexpr int kStage = 2 * R::kOperand;
    static constexpr int kStages = 65536 / kStage;
    static constexpr int kQPitch = D * 2 + (RT == 4 ? 0 : 16);
    static constexpr int kQOff = kStages * kStage;
    static constexpr int kJoinOff = kQOff + kRows * kQPitch;
    static constexpr int kOutOff = kJoinOff + R::kJoinBytes;     // this CTA's rows, for the cluster
    static constexpr int kOutMlOff = kOutOff + kRows * D * 4;
    static constexpr int kBarOff = kOutMlOff + kRows * 8;
    static constexpr int kNumBars = 2 * kStages + 1 + 2 * RT;    // full, empty, queries, join full, join empty
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kSmemBytes = kMiscOff + 16;
    static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
};

// (.aligned: all lanes of a warp at once, whatever branch they come from)
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}
__device__ __forceinline__ float2 cluster_load2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

template <int D, int RT, bool BF16, bool TREE>
__global__ void __launch_bounds__(kPagedThreads, 2)
    paged_cluster_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                         const PagedParams p, const int blocks, const int size) {
    using L = ClusterLayout<D, RT>;
    using R = PagedRows<D, RT, BF16>;
    constexpr int RB = L::kRows;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *empty = full + L::kStages, *q_full = empty + L::kStages, *j_full = q_full + 1, *j_empty = j_full + RT;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMiscOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % size, unit = blockIdx.x / size;
    PagedPiece u;
    u.row0 = unit % blocks * RB;
    u.hk = unit / blocks % p.Hkv;
    u.b = unit / blocks / p.Hkv;
    u.kind = 0;
    if (warp == kConsumers && lane == 0) {
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, kConsumers);
        }
        mbar_init(q_full, 1);
        for (int t = 0; t < RT; ++t) {
            mbar_init(j_full + t, R::KG);
            mbar_init(j_empty + t, R::KG);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    paged_enter(p);
    const SeqView s = paged_seq(p, u.b);
    u.t0 = s.t0;
    u.nq = s.nq;
    u.len = s.len;
    int prefix = 0;
    if (p.pre_lens) prefix = min(max(__ldg(p.pre_lens), 0), p.pre_max_len);
    if (threadIdx.x == 0 && rank == 0 && u.hk == 0 && u.row0 == 0 &&
        (paged_seq_bad(p, u.b) || (p.pre_lens && __ldg(p.pre_lens) != prefix)))
        record_status(&g_cluster_status, FA_ERR_SEQ_LEN);
    const int rows = min(RB, u.nq * p.G - u.row0);
    if (rows <= 0) return;  // (the whole cluster)
    // key tiles: the prefix's, then the sequence's own that the rows can see
    const int pre_tiles = (prefix + kTile - 1) / kTile;
    int seen = u.len;
    if (p.causal) seen = max(0, u.len - u.nq + min(u.nq - 1, (u.row0 + RB - 1) / p.G) + 1);
    const int tiles = pre_tiles + (seen + kTile - 1) / kTile;
    const int j0 = rank * tiles / size, j1 = (rank + 1) * tiles / size;
    __syncthreads();
    float2 *out_ml = reinterpret_cast<float2 *>(smem + L::kOutMlOff);
    uint32_t issued = 0;

    if (j0 == j1) {
        // no tile for this CTA: its rows have seen no key
        if (threadIdx.x < rows) out_ml[threadIdx.x] = make_float2(-INFINITY, 0.f);
    } else if (warp == kConsumers) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = l2_policy_evict_last();
        const int page = 1 << p.page_shift;
        const int box = min(page, kTile), boxes = kTile / box;
        const int my_box = lane % boxes, my_slab = lane / boxes % (D / 64), my_op = lane / boxes / (D / 64);
        const int *own = p.page_table + static_cast<long long>(u.b) * p.max_pages;
        // this lane's key of tile j within the prefix or the sequence, and whether it has one
        auto key_of = [&](int j) { return (j < pre_tiles ? j : j - pre_tiles) * kTile + my_box * box; };
        auto mine = [&](int j) { return my_op < 2 && key_of(j) < (j < pre_tiles ? prefix : u.len); };
        auto page_of = [&](int j) {
            return mine(j) ? __ldg((j < pre_tiles ? p.pre_table : own) + (key_of(j) >> p.page_shift)) : -1;
        };
        int id = page_of(j0);
        if (lane == 0) mbar_arrive_expect_tx(q_full, rows * D * 2);
        __syncwarp();
        for (int r = lane; r < rows; r += 32)
            bulk_load(smem + L::kQOff + r * L::kQPitch, p.q + paged_row(p, u, r) * D, D * 2, q_full);
        for (int j = j0; j < j1; ++j) {
            const int next = j + 1 < j1 ? page_of(j + 1) : -1;
            const int st = issued % L::kStages;
            if (issued >= L::kStages && !lanes_wait(empty + st, (issued / L::kStages - 1) & 1, abort_flag)) break;
            const bool live = mine(j);
            const int copies = __popc(__ballot_sync(0xffffffffu, live));
            if (lane == 0) mbar_arrive_expect_tx(full + st, copies * box * 128);
            __syncwarp();
            if (live) {
                if (id < 0 || id >= p.num_pages) {
                    record_status(&g_cluster_status, FA_ERR_PAGE);
                    id = p.num_pages;  // outside the tensor: the copy writes zeros
                }
                tma_load_4d(smem + st * L::kStage + my_op * R::kOperand + my_slab * R::kSlab + my_box * box * 128,
                            my_op ? &map_v : &map_k, full + st, my_slab * 64, key_of(j) & (page - 1), u.hk, id, pol);
            }
            id = next;
            ++issued;
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ consumers
        R r(warp, lane);
        const uint32_t ring = smem_u32(smem);
        bool ok = lanes_wait(q_full, 0, abort_flag);
        if (ok) {
            r.begin(smem_u32(smem + L::kQOff), L::kQPitch);
            int lim0 = u.len - 1, lim1 = u.len - 1;  // last own key of this thread's two rows
            const int r0 = u.row0 + r.rw * 16 + r.qrow;
            if (!TREE && p.causal) {
                lim0 = min(lim0, u.len - u.nq + r0 / p.G);
                lim1 = min(lim1, u.len - u.nq + (r0 + 8) / p.G);
            }
            for (int j = j0; j < j1; ++j) {
                const int i = j - j0, st = i % L::kStages;
                if (!lanes_wait(full + st, (i / L::kStages) & 1, abort_flag)) { ok = false; break; }
                if constexpr (TREE) {  // (trees have no prefix)
                    r.tile_seen(ring + st * L::kStage, tree_seen64(p, s, r0, j * kTile), tree_seen64(p, s, r0 + 8, j * kTile),
                                u.len - j * kTile, p.scale_log2);
                } else if (j < pre_tiles) {
                    const int keys = prefix - j * kTile;
                    r.tile(ring + st * L::kStage, keys - 1, keys - 1, keys, p.scale_log2);
                } else {
                    const int k0 = (j - pre_tiles) * kTile;
                    r.tile(ring + st * L::kStage, lim0 - k0, lim1 - k0, u.len - k0, p.scale_log2);
                }
                const bool pending = r.loads_pending(static_cast<uint32_t>(p.unit_steps) >> 30);
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + st + pending);
            }
        }
        if (ok) {
            r.end();
            float *out = reinterpret_cast<float *>(smem + L::kOutOff);
            r.write(
                rows, smem + L::kJoinOff, j_full, j_empty, abort_flag, [](int) { return 0; },
                [&](int row, int, int col, auto &acc, float m, float l) {
                    constexpr int N = sizeof(acc) / sizeof(float);
                    float *o = out + row * D + col;
                    if constexpr (N == 4) *reinterpret_cast<float4 *>(o) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    else *reinterpret_cast<float2 *>(o) = make_float2(acc[0], acc[1]);
                    if (col == 0) out_ml[row] = make_float2(m, l);
                });
        }
    }

    cluster_sync();
    // Every CTA finishes a share of the rows' columns, four at a time.
    const uint32_t out_addr = smem_u32(smem + L::kOutOff), ml_addr = smem_u32(smem + L::kOutMlOff);
    for (int i = rank * kPagedThreads + threadIdx.x; i < rows * (D / 4); i += size * kPagedThreads) {
        const int r = i / (D / 4), col = i % (D / 4) * 4;
        float2 ml[kMaxCluster];
        float4 v[kMaxCluster];
        float M = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
            ml[k] = k < size ? cluster_load2(cluster_addr(ml_addr + r * 8, k)) : make_float2(-INFINITY, 0.f);
            if (k < size) v[k] = cluster_load4(cluster_addr(out_addr + (r * D + col) * 4, k));
        }
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) M = fmaxf(M, ml[k].x);
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
            if (saw_key(ml[k].y)) {  // else the columns may be unwritten
                const float w = ex2_from(ml[k].x, M);
                sum = fmaf(w, ml[k].y, sum);
                acc[0] = fmaf(w, v[k].x, acc[0]);
                acc[1] = fmaf(w, v[k].y, acc[1]);
                acc[2] = fmaf(w, v[k].z, acc[2]);
                acc[3] = fmaf(w, v[k].w, acc[3]);
            }
        }
        paged_finish<4>(p, D, paged_row(p, u, r), col, acc, M, sum);
    }
    if (*abort_flag && warp == kConsumers && lane == 0) {
        // let every copy already issued land before the CTA goes away
        constexpr uint64_t kDrainNs = 200ull * 1000ull * 1000ull;
        int dummy = 0;
        if (j1 > j0) mbar_wait(q_full, 0, &dummy, kDrainNs);
        for (uint32_t i = issued > L::kStages ? issued - L::kStages : 0; i < issued; ++i)
            mbar_wait(full + i % L::kStages, (i / L::kStages) & 1, &dummy, kDrainNs);
        record_status(&g_cluster_status, FA_ERR_WATCHDOG);
    }
    cluster_sync();  // nobody leaves while its rows are read
}

template <int D, int RT, bool BF16, bool TREE>
int launch_cluster(const PagedPass &a, int size, cudaStream_t stream) {
    using L = ClusterLayout<D, RT>;
    CUtensorMap mk, mv;
    int rc;
    if ((rc = make_page_map(&mk, a.c.k_pages, a.c, kTile)) != FA_OK) return rc;
    if ((rc = make_page_map(&mv, a.c.v_pages, a.c, kTile)) != FA_OK) return rc;
    const auto kernel = paged_cluster_kernel<D, RT, BF16, TREE>;
    static std::atomic<bool> ready[kMaxDevices];
    if ((rc = ready_kernel(kernel, L::kSmemBytes, 0, a.device, ready)) != FA_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(a.units) * size);
    cfg.blockDim = dim3(kPagedThreads);
    cfg.dynamicSmemBytes = L::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, mk, mv, a.p, a.blocks, size);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

template <int D, int RT, bool BF16>
int launch_cluster_m(const PagedPass &a, int size, cudaStream_t stream) {
    return a.p.tree ? launch_cluster<D, RT, BF16, true>(a, size, stream) : launch_cluster<D, RT, BF16, false>(a, size, stream);
}

template <int D, bool BF16>
int launch_cluster_d(const PagedPass &a, int size, cudaStream_t stream) {
    switch (a.plan.block_rows) {
        case 16: return launch_cluster_m<D, 1, BF16>(a, size, stream);
        case 32: return launch_cluster_m<D, 2, BF16>(a, size, stream);
        default: return launch_cluster_m<D, 4, BF16>(a, size, stream);
    }
}

}  // namespace

int launch_paged_cluster(const PagedPass &a, int size, cudaStream_t stream) {
    const bool bf16 = a.c.dtype == FA_BF16;
    if (a.c.head_dim == 64)
        return bf16 ? launch_cluster_d<64, true>(a, size, stream) : launch_cluster_d<64, false>(a, size, stream);
    return bf16 ? launch_cluster_d<128, true>(a, size, stream) : launch_cluster_d<128, false>(a, size, stream);
}

int read_cluster_status(int reset) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_cluster_status, sizeof(int)) != cudaSuccess) return -1;
    if (reset && v) {
        int z = 0;
        if (cudaMemcpyToSymbol(g_cluster_status, &z, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace fa
