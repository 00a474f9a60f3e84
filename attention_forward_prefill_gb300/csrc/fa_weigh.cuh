// fa_weigh.cuh -- what the kernels that weigh cached tokens share.
#pragma once

#include <algorithm>
#include <cstdint>

#include "fa_paged_rows.cuh"
#include "fa_weigh_cut.cuh"

namespace fa {

// The whole CTA (NT threads) adds up the sequences' steps, steps_of(sequence) for each kv head, and
// finds its range; no more CTAs get one than there are lots of `least` steps.
template <int NT, typename StepsOf>
__device__ __forceinline__ void weigh_plan(const WeighParams &p, WeighStart &st, long long *warp_sum, int least, int *status,
                                           StepsOf steps_of) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const WeighShare share = weigh_share(p, tid, NT);
    bool bad = false;
    const long long mine = weigh_sum(p, share, steps_of, bad);
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
    for (int w = 0; w < NT / 32; ++w) {
        const long long v = warp_sum[w];
        if (w < warp) before += v;
        W += v;
    }
    const WeighStart range = weigh_range(W, blockIdx.x, gridDim.x, least);
    if (tid == 0) {
        st.W = range.W;
        st.G = range.G;
        st.first = range.first;
        st.end = range.end;
    }
    weigh_find(p, range, share, before, mine, steps_of, st);
    __syncthreads();
}

// Key j's weight from the sum over its rows; without rows it keeps its bits (-0 + 0 would be 0).
__device__ __forceinline__ void weigh_store(const WeighParams &p, int b, int h, int nq, int key, float sum) {
    const long long at = (static_cast<long long>(b) * p.Hkv + h) * p.len + key;
    p.out[at] = !p.in ? sum : nq > 0 ? fmaf(p.decay, p.in[at], sum) : p.in[at];
}
// -lse in log2 units.  -inf: the row adds nothing, whatever its products are.
__device__ __forceinline__ float weigh_off(float lse) { return lse == -INFINITY ? -INFINITY : -lse * kLog2e; }

int launch_weigh_tiles(const WeighLaunch &a, WeighParams p, const DeviceInfo &dev, cudaStream_t stream);

}  // namespace fa
