// fa_weigh_sm103.cu -- what the tokens of a paged cache got of some queries' attention.
//
// For key j of a sequence and kv head, over the query rows i (token, head of the group)
// that see it,
//   out_j = decay in_j + sum_i exp(scale q_i.k_j - lse_i)
// with the row log-sum-exp that the attention has returned: one product and one
// exponential per pair of row and key, and a sum over the rows, which a key's thread or
// warp holds alone.  No atomics: the same arguments give the same bits.
//
// weigh_rows_kernel: a warp holds 16 keys as the left operand of 16 x 8 x 16 products,
// straight from global memory (a lane's eight channels of 16 bytes take the places of two
// products' channels; the order of the channels does not matter to q.k), and goes through
// the query rows eight at a time.
#include <algorithm>
#include <cmath>

#include "fa_internal.h"
#include "fa_paged_rows.cuh"

namespace fa {

namespace {

__device__ int g_weigh_status = 0;

struct WeighParams {
    const uint16_t *q, *k_pages;
    const float *lse, *in;
    float *out;
    long long page_stride, head_stride, slot_stride;
    const int *page_table, *seq_lens, *cu_q;
    int B, Hq, Hkv, G, total_q, max_q, nq_each;
    int max_pages, max_len, num_pages, page_shift, len;  // len: of a row of weights
    int causal;
    float scale_log2, decay;
};

struct WeighSeq {
    int t0, nq, len;
};

__device__ __forceinline__ WeighSeq weigh_seq(const WeighParams &p, int b) {
    WeighSeq s;
    s.len = min(max(__ldg(p.seq_lens + b), 0), p.max_len);
    if (p.cu_q) {
        s.t0 = min(max(__ldg(p.cu_q + b), 0), p.total_q);
        s.nq = min(min(max(__ldg(p.cu_q + b + 1), s.t0), p.total_q) - s.t0, p.max_q);
    } else {
        s.t0 = b * p.nq_each;
        s.nq = p.nq_each;
    }
    return s;
}
__device__ __forceinline__ bool weigh_seq_bad(const WeighParams &p, int b) {
    const int raw = __ldg(p.seq_lens + b);
    bool bad = raw < 0 || raw > p.max_len;
    if (p.cu_q) {
        const int lo = __ldg(p.cu_q + b), hi = __ldg(p.cu_q + b + 1);
        bad |= lo < 0 || hi < lo || hi > p.total_q || hi - lo > p.max_q;
    }
    return bad;
}

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kWarpKeys = 16;
constexpr int kStepKeys = kWarps * kWarpKeys;  // keys of a CTA's step

// A CTA's range of the call's steps, an equal share: the sequence that it starts in and the
// steps of that sequence before it.
struct WeighStart {
    long long first, end, rem;
    int b;
};
__device__ __forceinline__ int weigh_steps(const WeighParams &p, const WeighSeq &s) {
    return (s.len + kStepKeys - 1) / kStepKeys;
}
__device__ void weigh_plan(const WeighParams &p, WeighStart &st, long long *warp_sum) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long mine = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        mine += static_cast<long long>(weigh_steps(p, weigh_seq(p, b))) * p.Hkv;
        bad |= weigh_seq_bad(p, b);
    }
    if (bad && blockIdx.x == 0) record_status(&g_weigh_status, FA_ERR_SEQ_LEN);
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
    for (int w = 0; w < kWarps; ++w) {
        const long long v = warp_sum[w];
        if (w < warp) before += v;
        W += v;
    }
    const long long first = blockIdx.x * W / gridDim.x, end = (blockIdx.x + 1LL) * W / gridDim.x;
    if (tid == 0) {
        st.first = first;
        st.end = end;
    }
    if (first < end && before <= first && first < before + mine) {
        long long rem = first - before;
        int b = b0;
        for (; b < b1 - 1; ++b) {
            const long long c = static_cast<long long>(weigh_steps(p, weigh_seq(p, b))) * p.Hkv;
            if (rem < c) break;
            rem -= c;
        }
        st.b = b;
        st.rem = rem;
    }
    __syncthreads();
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 2) weigh_rows_kernel(const WeighParams p) {
    __shared__ WeighStart st;
    __shared__ long long warp_sum[kWarps];
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    weigh_plan(p, st, warp_sum);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
    long long left = st.end - st.first;
    if (left <= 0) return;
    int b = st.b;
    WeighSeq s = weigh_seq(p, b);
    int steps = weigh_steps(p, s);  // (of this sequence: at least one)
    int h = static_cast<int>(st.rem / steps), j = static_cast<int>(st.rem % steps);
    for (; left > 0; --left) {
        const int k0 = j * kStepKeys + warp * kWarpKeys, key[2] = {k0 + g, k0 + g + 8};
        if (k0 < s.len) {
            // the keys, eight channels a lane and 32 channels: places 2 quad, 2 quad + 1, 2 quad + 8, 2 quad + 9
            // of two products
            uint4 kf[2][D / 32];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint16_t *row = nullptr;
                if (key[r] < s.len) {
                    const int page = __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + (key[r] >> p.page_shift));
                    if (page < 0 || page >= p.num_pages) record_status(&g_weigh_status, FA_ERR_PAGE);  // zeros
                    else row = p.k_pages + page * p.page_stride + h * p.head_stride +
                               (key[r] & ((1 << p.page_shift) - 1)) * p.slot_stride + quad * 8;
                }
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    kf[r][c] = row ? __ldg(reinterpret_cast<const uint4 *>(row + c * 32)) : make_uint4(0, 0, 0, 0);
            }
            // rows from `see` on see the key
            const int rows = s.nq * p.G, past = s.len - s.nq;
            int see[2] = {0, 0};
            if (p.causal) {
                see[0] = min(max(key[0] - past, 0), s.nq) * p.G;
                see[1] = min(max(key[1] - past, 0), s.nq) * p.G;
            }
            const int r_first = p.causal ? min(max(k0 - past, 0), s.nq) * p.G & ~7 : 0;
            float sum[2] = {0.f, 0.f};
            for (int r0 = r_first; r0 < rows; r0 += 8) {
                const int rq = min(r0 + g, rows - 1);
                const uint16_t *qr = p.q + ((static_cast<long long>(s.t0) + rq / p.G) * p.Hq + h * p.G + rq % p.G) * D + quad * 8;
                float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint4 z = __ldg(reinterpret_cast<const uint4 *>(qr + i * 32));
                    const uint32_t lo[4] = {kf[0][i].x, kf[1][i].x, kf[0][i].y, kf[1][i].y};
                    const uint32_t hi[4] = {kf[0][i].z, kf[1][i].z, kf[0][i].w, kf[1][i].w};
                    mma_16816<BF16>(c, lo, z.x, z.y);
                    mma_16816<BF16>(c, hi, z.z, z.w);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = r0 + quad * 2 + e;
                    if (r >= rows) continue;
                    const float lse = __ldg(p.lse + (static_cast<long long>(s.t0) + r / p.G) * p.Hq + h * p.G + r % p.G);
                    // (a row that saw no key adds nothing)
                    const float off = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
                    if (r >= see[0]) sum[0] += ex2_approx(fmaf(c[e], p.scale_log2, off));
                    if (r >= see[1]) sum[1] += ex2_approx(fmaf(c[2 + e], p.scale_log2, off));
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
                sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
                if (quad == 0 && key[r] < s.len) {
                    const long long at = (static_cast<long long>(b) * p.Hkv + h) * p.len + key[r];
                    const float decay = s.nq > 0 ? p.decay : 1.f;
                    p.out[at] = p.in ? fmaf(decay, p.in[at], sum[r]) : sum[r];
                }
            }
        }
        if (left > 1 && ++j == steps) {
            j = 0;
            if (++h == p.Hkv) {
                h = 0;
                do {
                    s = weigh_seq(p, ++b);  // steps are left, so a later sequence has some
                    steps = weigh_steps(p, s);
                } while (steps == 0 && b + 1 < p.B);
                if (steps == 0) return;
            }
        }
    }
}

template <int D, bool BF16>
int launch_rows(const WeighParams &p, const DeviceInfo &dev, cudaStream_t stream) {
    const long long most = static_cast<long long>(p.B) * p.Hkv * ((p.max_len + kStepKeys - 1) / kStepKeys);
    PagedConfig cfg(static_cast<unsigned>(std::min<long long>(most, 2LL * dev.num_sms)), kThreads, 0, true, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, weigh_rows_kernel<D, BF16>, p);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

}  // namespace

int launch_weigh(const WeighLaunch &a, const DeviceInfo &dev, cudaStream_t stream) {
    WeighParams p;
    p.q = static_cast<const uint16_t *>(a.q);
    p.k_pages = static_cast<const uint16_t *>(a.c.k_pages);
    p.lse = a.lse;
    p.in = a.weights;
    p.out = a.out;
    p.page_stride = a.c.page_stride;
    p.head_stride = a.c.head_stride;
    p.slot_stride = a.c.slot_stride;
    p.page_table = a.page_table;
    p.seq_lens = a.seq_lens;
    p.cu_q = a.cu_q;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.c.num_heads;
    p.G = a.Hq / a.c.num_heads;
    p.total_q = a.total_q;
    p.max_q = a.max_q;
    p.nq_each = a.cu_q ? 0 : a.max_q;
    p.max_pages = a.max_pages;
    p.max_len = std::min(a.max_pages * a.c.page_size, a.weights_len);
    p.num_pages = a.c.num_pages;
    p.page_shift = 0;
    while ((1 << p.page_shift) < a.c.page_size) ++p.page_shift;
    p.len = a.weights_len;
    p.causal = a.causal;
    p.scale_log2 = a.scale * kLog2e;
    p.decay = a.decay;
    const bool bf16 = a.c.dtype == FA_BF16;
    if (a.c.head_dim == 64) return bf16 ? launch_rows<64, true>(p, dev, stream) : launch_rows<64, false>(p, dev, stream);
    return bf16 ? launch_rows<128, true>(p, dev, stream) : launch_rows<128, false>(p, dev, stream);
}

int read_weigh_status(int reset) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_weigh_status, sizeof(int)) != cudaSuccess) return -1;
    if (reset && v) {
        int z = 0;
        if (cudaMemcpyToSymbol(g_weigh_status, &z, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace fa
