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

#include "fa_weigh.cuh"

namespace fa {

namespace {

__device__ int g_weigh_status = 0;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kWarpKeys = 16;
constexpr int kStepKeys = kWarps * kWarpKeys;  // keys of a CTA's step

__device__ __forceinline__ int weigh_steps(const WeighSeq &s) { return (s.len + kStepKeys - 1) / kStepKeys; }

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 2) weigh_rows_kernel(const WeighParams p) {
    __shared__ WeighStart st;
    __shared__ long long warp_sum[kWarps];
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    weigh_plan<kThreads>(p, st, warp_sum, 1, &g_weigh_status, [&](const WeighSeq &s) { return static_cast<long long>(weigh_steps(s)); });
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
    long long left = st.end - st.first;
    if (left <= 0) return;
    int b = st.b;
    WeighSeq s = weigh_seq(p, b);
    int steps = weigh_steps(s);  // (of this sequence: at least one)
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
                    const float off = weigh_off(lse);
                    if (r >= see[0]) sum[0] += ex2_approx(fmaf(c[e], p.scale_log2, off));
                    if (r >= see[1]) sum[1] += ex2_approx(fmaf(c[2 + e], p.scale_log2, off));
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
                sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
                if (quad == 0 && key[r] < s.len) weigh_store(p, b, h, s.nq, key[r], sum[r]);
            }
        }
        if (left > 1 && ++j == steps) {
            j = 0;
            if (++h == p.Hkv) {
                h = 0;
                do {
                    s = weigh_seq(p, ++b);  // steps are left, so a later sequence has some
                    steps = weigh_steps(s);
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
    WeighParams p = {};
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
    if (weigh_in_tiles(a)) return launch_weigh_tiles(a, p, dev, stream);
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
