// fa_evict_sm103.cu -- which tokens of a paged cache stay, and moving those that do.
//
// Selection.  Of a row (sequence, head) of n accumulated weights the first `sink` and
// the last `recent` tokens stay, and of the ones between them those with the largest
// weights, budget = k in all.  With keys u(w) in the order of the weights the smallest
// key T that stays is found digit by digit from the top (11, 11 and 10 bits): the
// counts of a digit's values, summed from above, say which value holds the k-th key.
// All keys above T stay, and of those equal to T the ones at the lowest positions.
//
// Moving.  Token keep[i] goes to place first + i.  In place, keep[i] >= first + i, so
// that the place a token comes from is written by the token of the same or a later i
// alone: whoever reads a column of a row in the order of i, ahead of what it writes, can
// move it without a copy.
#include <algorithm>
#include <atomic>

#include "fa_internal.h"
#include "fa_status.cuh"
#include "sm103_ptx.cuh"

namespace fa {

namespace {

__device__ int g_evict_status = 0;

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;

struct SelectParams {
    const float *weights;
    const int *seq_lens;
    int *keep, *counts;
    float *kept;
    int B, heads, len, budget, sink, recent;
    int resident;  // floats of a CTA's slice that its shared memory holds
};

// Larger for larger weights; -0 is 0, and NaN comes above all.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xfffffffeu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_load(const uint32_t *at, int rank) {
    uint32_t a, v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t scan_up(uint32_t v, int lane) {  // over the lanes, inclusive
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    return v;
}

// A cluster of `size` CTAs per row, a slice of the row's tokens each.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p, const int size) {
    extern __shared__ __align__(16) float slice[];  // [p.resident]
    __shared__ uint32_t hist[2][kBins];
    __shared__ uint32_t warp_sum[kSelWarps], found[2], cta_above, cta_equal;
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % size, row = blockIdx.x / size;
    const int b = row / p.heads;
    const int raw = __ldg(p.seq_lens + b), n = min(max(raw, 0), p.len);
    const int count = min(n, p.budget);
    if (tid == 0 && rank == 0 && row % p.heads == 0) {
        p.counts[b] = count;
        if (raw != n) record_status(&g_evict_status, FA_ERR_SEQ_LEN);
    }
    const float *w = p.weights + static_cast<long long>(row) * p.len;
    int *keep = p.keep + static_cast<long long>(row) * p.budget;
    float *kept = p.kept ? p.kept + static_cast<long long>(row) * p.len : nullptr;
    const int t = rank * kSelThreads + tid, threads = size * kSelThreads;
    for (int i = count + t; i < p.budget; i += threads) keep[i] = -1;
    if (kept)
        for (int i = count + t; i < p.len; i += threads) kept[i] = 0.f;
    if (n <= p.budget) {  // all of them stay (the whole cluster)
        for (int i = t; i < n; i += threads) {
            keep[i] = i;
            if (kept) kept[i] = __ldg(w + i);
        }
        return;
    }
    // this CTA's tokens, and each warp's among them, in runs of whole warps
    const int per = ((n + size - 1) / size + kSelThreads - 1) / kSelThreads * kSelThreads;
    const int lo = min(rank * per, n), hi = min(lo + per, n);
    const float *from = w + lo;
    if (per <= p.resident) {
        for (int i = tid; i < hi - lo; i += kSelThreads) slice[i] = __ldg(w + lo + i);
        from = slice;
    }
    for (int i = tid; i < kBins; i += kSelThreads) hist[0][i] = 0;
    __syncthreads();
    auto key_of = [&](int i) {  // of token lo + i
        const int at = lo + i;
        return at < p.sink || at >= n - p.recent ? 0xffffffffu : weight_key(from[i]);
    };
    uint32_t top = 0, left = count;  // the digits found, and how many keys of that prefix stay
    int shift = 32;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass == 2 ? 10 : 11, above = shift;
        shift -= bits;
        uint32_t *h = hist[pass & 1];
        for (int i0 = warp * 32; i0 < hi - lo; i0 += kSelThreads) {
            const int i = i0 + lane;
            const uint32_t key = i < hi - lo ? key_of(i) : 0u;
            const bool in = i < hi - lo && (pass == 0 || key >> above == top);
            const uint32_t bin = key >> shift & ((1u << bits) - 1u);
            const uint32_t who = __ballot_sync(0xffffffffu, in);
            if (!who) continue;
            const int one = __ffs(who) - 1;
            const uint32_t its = __shfl_sync(0xffffffffu, bin, one);
            // (many equal weights, zeros above all: one addition for the warp)
            if (__all_sync(0xffffffffu, !in || bin == its)) {
                if (lane == one) atomicAdd(h + bin, __popc(who));
            } else if (in) {
                atomicAdd(h + bin, 1u);
            }
        }
        cluster_sync();
        // bins from above, four a thread, of all CTAs
        uint32_t c[4] = {0, 0, 0, 0};
        for (int r = 0; r < size; ++r)
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] += cluster_load(h + kBins - 1 - (tid * 4 + k), r);
        const uint32_t mine = c[0] + c[1] + c[2] + c[3], incl = scan_up(mine, lane);
        if (lane == 31) warp_sum[warp] = incl;
        // (the other CTAs have read the other table before they came here)
        for (int i = tid; i < kBins; i += kSelThreads) hist[~pass & 1][i] = 0;
        __syncthreads();
        uint32_t sum = incl - mine;
        for (int k = 0; k < warp; ++k) sum += warp_sum[k];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (sum < left && left <= sum + c[k]) {
                found[0] = kBins - 1 - (tid * 4 + k);
                found[1] = left - sum;
            }
            sum += c[k];
        }
        __syncthreads();
        top = pass == 0 ? found[0] : top << bits | found[0];
        left = found[1];
    }
    // top: the smallest key that stays; left: how many of those equal to it
    const int run = per / kSelWarps;  // a multiple of 32
    const int w0 = min(warp * run, hi - lo), w1 = min(w0 + run, hi - lo);
    uint32_t above = 0, equal = 0;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const uint32_t key = i0 + lane < w1 ? key_of(i0 + lane) : 0u;
        above += __popc(__ballot_sync(0xffffffffu, i0 + lane < w1 && key > top));
        equal += __popc(__ballot_sync(0xffffffffu, i0 + lane < w1 && key == top));
    }
    __shared__ uint32_t warp_above[kSelWarps], warp_equal[kSelWarps];
    if (lane == 0) {
        warp_above[warp] = above;
        warp_equal[warp] = equal;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t x = 0, y = 0;
        for (int k = 0; k < kSelWarps; ++k) {
            x += warp_above[k];
            y += warp_equal[k];
        }
        cta_above = x;
        cta_equal = y;
    }
    cluster_sync();
    above = equal = 0;
    for (int r = 0; r < rank; ++r) {
        above += cluster_load(&cta_above, r);
        equal += cluster_load(&cta_equal, r);
    }
    for (int k = 0; k < warp; ++k) {
        above += warp_above[k];
        equal += warp_equal[k];
    }
    const uint32_t before = (1u << lane) - 1u;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t key = i < w1 ? key_of(i) : 0u;
        const uint32_t is_above = __ballot_sync(0xffffffffu, i < w1 && key > top);
        const uint32_t is_equal = __ballot_sync(0xffffffffu, i < w1 && key == top);
        const uint32_t a = above + __popc(is_above & before), e = equal + __popc(is_equal & before);
        const bool stays = i < w1 && (key > top || (key == top && e < left));
        if (stays) {
            const uint32_t to = a + min(e, left);
            keep[to] = lo + i;
            if (kept) kept[to] = from[i];
        }
        above += __popc(is_above);
        equal += __popc(is_equal);
    }
    cluster_sync();  // nobody leaves while its counts are read
}

// ---------------------------------------------------------------- moving
constexpr int kKeepThreads = 256;

struct KeepParams {
    uint16_t *k_pages, *v_pages;
    long long page_stride, head_stride, slot_stride;
    const int *page_table, *seq_lens, *keep, *counts, *first, *out_table;
    int B, Hkv, heads, keep_len, max_pages, out_max_pages, num_pages, page_shift, chunks;
    int in_place;
};

// A thread moves a column of 16 bytes of a row (sequence, kv head, keys or values), kDeep tokens at a time.
constexpr int kDeep = 8;
__global__ void __launch_bounds__(kKeepThreads) keep_columns_kernel(const KeepParams p) {
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    const long long column = static_cast<long long>(blockIdx.x) * kKeepThreads + threadIdx.x;
    const int chunk = column % p.chunks;
    const long long pair = column / p.chunks;  // ((b, h), keys or values)
    if (pair >= 2LL * p.B * p.Hkv) return;
    const int h = pair / 2 % p.Hkv, b = pair / 2 / p.Hkv;
    uint16_t *base = (pair & 1 ? p.v_pages : p.k_pages) + h * p.head_stride + chunk * 8;
    const int raw_len = __ldg(p.seq_lens + b), raw_count = __ldg(p.counts + b), raw_first = p.first ? __ldg(p.first + b) : 0;
    const int max_len = p.max_pages << p.page_shift, out_len = p.out_max_pages << p.page_shift;
    const int len = min(max(raw_len, 0), max_len);
    const int first = min(max(raw_first, 0), out_len);
    const int count = min(min(max(raw_count, 0), p.keep_len), out_len - first);
    int status = len != raw_len || count != raw_count || first != raw_first ? FA_ERR_SEQ_LEN : 0;
    const int *list = p.keep + (static_cast<long long>(b) * p.heads + (p.heads > 1 ? h : 0)) * p.keep_len;
    const int *table = p.page_table + static_cast<long long>(b) * p.max_pages;
    const int *out_table = p.out_table + static_cast<long long>(b) * p.out_max_pages;
    const int mask = (1 << p.page_shift) - 1;
    for (int i0 = 0; i0 < count; i0 += kDeep) {
        uint4 data[kDeep];
        uint16_t *to[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            to[k] = nullptr;
            const int i = i0 + k;
            if (i >= count) continue;
            const int src = __ldg(list + i), dst = first + i;
            if (src < (p.in_place ? dst : 0) || src >= len) {
                if (!status) status = FA_ERR_INDEX;
                continue;
            }
            const int page = __ldg(table + (src >> p.page_shift)), out_page = __ldg(out_table + (dst >> p.page_shift));
            if (out_page < 0 || out_page >= p.num_pages) {
                if (!status) status = FA_ERR_PAGE;
                continue;
            }
            uint16_t *at = base + out_page * p.page_stride + (dst & mask) * p.slot_stride;
            if (page < 0 || page >= p.num_pages) {  // its tokens are zeros
                if (!status) status = FA_ERR_PAGE;
                data[k] = make_uint4(0, 0, 0, 0);
            } else {
                const uint16_t *s = base + page * p.page_stride + (src & mask) * p.slot_stride;
                if (s == at) continue;
                data[k] = *reinterpret_cast<const uint4 *>(s);
            }
            to[k] = at;
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            if (to[k]) *reinterpret_cast<uint4 *>(to[k]) = data[k];
    }
    if (status && chunk == 0) record_status(&g_evict_status, status);
}

// ---------------------------------------------------------------- host side
struct Launch {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[2];
    Launch(unsigned grid, int threads, size_t smem, int cluster, cudaStream_t stream) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        c.gridDim = dim3(grid);
        c.blockDim = dim3(threads);
        c.dynamicSmemBytes = smem;
        c.stream = stream;
        c.attrs = attr;
        c.numAttrs = cluster ? 2 : 1;
    }
    Launch(const Launch &) = delete;
};

}  // namespace

int launch_select(const SelectLaunch &a, const DeviceInfo &dev, cudaStream_t stream) {
    const long long rows = static_cast<long long>(a.B) * a.heads;
    int size = 1;
    while (size < kMaxCluster && a.weights_len > 4096LL * size && rows * size < 2LL * dev.num_sms) size *= 2;
    constexpr int kMostResident = 180 * 1024 / 4;
    static std::atomic<bool> ready[kMaxDevices];
    if (!ready[dev.device].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostResident * 4);
        if (e != cudaSuccess) return cuda_fail(e);
        ready[dev.device].store(true, std::memory_order_release);
    }
    const long long per = (a.weights_len + size - 1) / size;
    const int want = static_cast<int>(std::min<long long>(kMostResident, (per + kSelThreads - 1) / kSelThreads * kSelThreads));
    const SelectParams p = {a.weights, a.seq_lens, a.keep, a.counts, a.kept, a.B, a.heads, a.weights_len,
                            a.budget, a.sink, a.recent, want};
    Launch cfg(static_cast<unsigned>(rows * size), kSelThreads, want * 4, size, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, select_kernel, p, size);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

int launch_keep(const KeepLaunch &a, const DeviceInfo &, cudaStream_t stream) {
    KeepParams p;
    p.k_pages = static_cast<uint16_t *>(a.c.k_pages);
    p.v_pages = static_cast<uint16_t *>(a.c.v_pages);
    p.page_stride = a.c.page_stride;
    p.head_stride = a.c.head_stride;
    p.slot_stride = a.c.slot_stride;
    p.page_table = a.page_table;
    p.seq_lens = a.seq_lens;
    p.keep = a.keep;
    p.counts = a.counts;
    p.first = a.first;
    p.out_table = a.out_table;
    p.B = a.B;
    p.Hkv = a.c.num_heads;
    p.heads = a.heads;
    p.keep_len = a.keep_len;
    p.max_pages = a.max_pages;
    p.out_max_pages = a.out_max_pages;
    p.num_pages = a.c.num_pages;
    p.page_shift = 0;
    while ((1 << p.page_shift) < a.c.page_size) ++p.page_shift;
    p.chunks = a.c.head_dim / 8;
    p.in_place = a.in_place ? 1 : 0;
    const long long columns = 2LL * a.B * p.Hkv * p.chunks;
    Launch cfg(static_cast<unsigned>((columns + kKeepThreads - 1) / kKeepThreads), kKeepThreads, 0, 0, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, keep_columns_kernel, p);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

int read_evict_status(int reset) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_evict_status, sizeof(int)) != cudaSuccess) return -1;
    if (reset && v) {
        int z = 0;
        if (cudaMemcpyToSymbol(g_evict_status, &z, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace fa
