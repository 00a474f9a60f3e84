// fa_tree_sm103.cu -- the nodes of drafted trees: which nodes each one sees, and at
// which position it stands.
//
// Node i of a sequence's tree has a parent parents[i] < i, or -1 where it follows the
// sequence's context.  It sees itself and its ancestors,
//   row_i = bit i + (parent < 0 ? 0 : row_parent),   position_i = len - nq + depth_i.
// A thread walks up from its node: the nodes on the way come in falling order, so that
// the words of its row are finished, and written, one after another.
//
// The bytes are nothing (256 trees of 20 to 256 nodes: 1.3 MB, 0.2 us); the depth of the trees, a
// load from shared memory for every ancestor, and the launch set the time.  That batch takes 4.3 us
// (8.1 with the parents read from L1 and the words kept until the walk's end), a tree of 8 nodes 1.6.
#include <algorithm>

#include "fa_internal.h"
#include "fa_status.cuh"

namespace fa {

namespace {

constexpr int kThreads = 128;
constexpr int kShared = 4096;  // parents of a sequence kept in shared memory; more are read from L1

__device__ int g_tree_status = 0;

struct TreeParams {
    const int *parents, *seq_lens, *cu;
    uint32_t *mask;
    int *positions;
    int words, total, max_q;
    int blocks;  // CTAs per sequence
};

__global__ void __launch_bounds__(kThreads) tree_mask_kernel(const TreeParams p) {
    __shared__ int up[kShared];
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x / p.blocks, first = blockIdx.x % p.blocks * kThreads;
    const int lo = __ldg(p.cu + b), hi = __ldg(p.cu + b + 1);
    const int t0 = min(max(lo, 0), p.total);
    const int nq = min(min(max(hi, t0), p.total) - t0, p.max_q);
    if (threadIdx.x == 0 && first == 0 && (lo < 0 || hi < lo || hi > p.total || hi - lo > p.max_q))
        record_status(&g_tree_status, FA_ERR_SEQ_LEN);
    if (first >= nq) return;
    const int *parent = p.parents + t0;
    if (nq <= kShared) {
        const int last = min(nq, first + kThreads);  // (ancestors stand in front of a node)
        for (int i = threadIdx.x; i < last; i += kThreads) up[i] = __ldg(parent + i);
        __syncthreads();
    }
    const int i = first + threadIdx.x;
    if (i >= nq) return;
    uint32_t *row = p.mask + static_cast<long long>(t0 + i) * p.words;
    int depth = -1;
    bool bad = false;
    auto walk = [&](auto parent_of) {
        int at = i;
        for (int w = p.words - 1; w >= 0; --w) {
            uint32_t bits = 0;
            while (at >> 5 == w) {  // (-1 is of no word)
                bits |= 1u << (at & 31);
                ++depth;
                int next = parent_of(at);
                if (next >= at || next < -1) {
                    bad = true;
                    next = -1;
                }
                at = next;
            }
            row[w] = bits;
        }
    };
    if (nq <= kShared) walk([&](int at) { return up[at]; });
    else walk([&](int at) { return __ldg(parent + at); });
    if (p.positions) p.positions[t0 + i] = __ldg(p.seq_lens + b) - nq + depth;
    if (bad) record_status(&g_tree_status, FA_ERR_INDEX);
}

}  // namespace

int launch_tree_mask(const TreeLaunch &a, cudaStream_t stream) {
    const int blocks = (std::min(a.max_q, a.total_q) + kThreads - 1) / kThreads;
    const TreeParams p = {a.parents, a.seq_lens, a.cu_seqlens_q, a.mask, a.positions, a.mask_words, a.total_q, a.max_q, blocks};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_mask_kernel, p);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

int read_tree_status(int reset) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_tree_status, sizeof(int)) != cudaSuccess) return -1;
    if (reset && v) {
        int z = 0;
        if (cudaMemcpyToSymbol(g_tree_status, &z, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace fa
