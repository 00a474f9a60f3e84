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
// the query rows eight at a time.  HBM-bound with up to eight rows of a kv head, whose next keys are
// on their way while one step is computed: 32 sequences of 200 to 8192 tokens, 32 heads over 8, d = 128:
// 40 us (5.8 TB/s; 54 with a step's keys loaded when it starts).  With more rows the products of a
// warp of 16 keys count, 9 us for every eight rows of 16 sequences of 4096 tokens.
#include <algorithm>
#include <climits>

#include "fa_weigh.cuh"

namespace fa {

namespace {

__device__ int g_weigh_status = 0;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kWarpKeys = 16;
constexpr int kStepKeys = kWarps * kWarpKeys;  // keys of a CTA's step

__device__ __forceinline__ int weigh_steps(const WeighParams &p, const WeighSeq &s) {
    return weigh_stays(p, s) ? 0 : (s.len + kStepKeys - 1) / kStepKeys;
}

// A warp's 16 keys of a step: where they are, and what they bring.
template <int D>
struct WeighKeys {
    uint4 k[2][D / 32];  // keys k0 + lane / 4 and the one 8 behind it: eight channels a lane and 32 channels
    float old[2];        // their weights so far, in the lanes that write them
    int b, h, k0;
    WeighSeq s;
};

// Walks through a CTA's steps.
struct WeighWalk {
    WeighSeq s;
    int b, h, j, steps;
    long long left;

    __device__ __forceinline__ void begin(const WeighParams &p, const WeighStart &st) {
        left = st.end - st.first;
        if (left <= 0) return;
        b = st.b;
        s = weigh_seq(p, b);
        steps = weigh_steps(p, s);  // (at least one)
        h = static_cast<int>(st.rem / steps);
        j = static_cast<int>(st.rem % steps);
    }
    __device__ __forceinline__ void next(const WeighParams &p) {
        if (--left <= 0 || ++j < steps) return;
        j = 0;
        if (++h < p.Hkv) return;
        h = 0;
        do {
            s = weigh_seq(p, ++b);  // steps are left, so a later sequence has some
            steps = weigh_steps(p, s);
        } while (steps == 0 && b + 1 < p.B);
        if (steps == 0) left = 0;
    }
};

// FEW: at most 8 rows a kv head (one token of up to 8 heads), which stay in registers while the warp's
// keys are of one sequence and head.  HBM-bound: the next step's keys are on their way while a step is
// computed, and its page's number while they are.
template <int D, bool BF16, bool FEW>
__global__ void __launch_bounds__(kThreads, 2) weigh_rows_kernel(const WeighParams p) {
    __shared__ WeighStart st;
    __shared__ long long warp_sum[kWarps];
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    weigh_plan<kThreads>(p, st, warp_sum, 1, &g_weigh_status, [&](const WeighSeq &s) { return static_cast<long long>(weigh_steps(p, s)); });
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
    WeighWalk walk;
    walk.begin(p, st);
    if (walk.left <= 0) return;
    // the page of a step's keys (16 of one page), or -1 without keys
    auto page_of = [&](const WeighWalk &w) {
        const int k0 = w.j * kStepKeys + warp * kWarpKeys;
        return w.left > 0 && k0 < w.s.len ? __ldg(p.page_table + static_cast<long long>(w.b) * p.max_pages + (k0 >> p.page_shift)) : -1;
    };
    auto load = [&](const WeighWalk &w, int page, WeighKeys<D> &x) {
        x.b = w.b;
        x.h = w.h;
        x.s = w.s;
        x.k0 = w.left > 0 ? w.j * kStepKeys + warp * kWarpKeys : INT_MAX / 2;
        const bool asked = x.k0 < x.s.len && x.s.nq > 0, there = page >= 0 && page < p.num_pages;
        if (asked && !there) record_status(&g_weigh_status, FA_ERR_PAGE);  // zeros
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int key = x.k0 + g + 8 * r;
            // the eight channels take places 2 quad, 2 quad + 1, 2 quad + 8 and 2 quad + 9 of two products
            const uint16_t *row = p.k_pages + page * p.page_stride + w.h * p.head_stride +
                                  (key & ((1 << p.page_shift) - 1)) * p.slot_stride + quad * 8;
            const bool live = asked && there && key < x.s.len;
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                x.k[r][c] = live ? __ldg(reinterpret_cast<const uint4 *>(row + c * 32)) : make_uint4(0, 0, 0, 0);
            x.old[r] = p.in && quad == 0 && key < x.s.len
                           ? __ldcg(p.in + (static_cast<long long>(w.b) * p.Hkv + w.h) * p.len + key) : 0.f;
        }
    };
    uint4 z[FEW ? D / 32 : 1];
    float lse[2] = {-INFINITY, -INFINITY};
    int z_of = -1;  // the sequence and head of z
    auto rows_of = [&](const WeighKeys<D> &x, int r0, uint4 (&q)[D / 32]) {  // 8 rows from r0 on, eight channels a lane
        const int rq = min(r0 + g, x.s.nq * p.G - 1);
        const uint16_t *qr = p.q + ((static_cast<long long>(x.s.t0) + rq / p.G) * p.Hq + x.h * p.G + rq % p.G) * D + quad * 8;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) q[i] = __ldg(reinterpret_cast<const uint4 *>(qr + i * 32));
    };
    auto off_of = [&](const WeighKeys<D> &x, int r) {
        return r < x.s.nq * p.G ? weigh_off(__ldg(p.lse + (static_cast<long long>(x.s.t0) + r / p.G) * p.Hq + x.h * p.G + r % p.G)) : -INFINITY;
    };
    auto products = [&](const WeighKeys<D> &x, const uint4 (&q)[D / 32], float (&c)[4]) {
        c[0] = c[1] = c[2] = c[3] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t lo[4] = {x.k[0][i].x, x.k[1][i].x, x.k[0][i].y, x.k[1][i].y};
            const uint32_t hi[4] = {x.k[0][i].z, x.k[1][i].z, x.k[0][i].w, x.k[1][i].w};
            mma_16816<BF16>(c, lo, q[i].x, q[i].y);
            mma_16816<BF16>(c, hi, q[i].z, q[i].w);
        }
    };
    auto compute = [&](const WeighKeys<D> &x) {
        if (x.k0 >= x.s.len) return;
        const int rows = x.s.nq * p.G, key[2] = {x.k0 + g, x.k0 + g + 8};
        if (rows == 0) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (quad == 0 && key[r] < x.s.len) p.out[(static_cast<long long>(x.b) * p.Hkv + x.h) * p.len + key[r]] = x.old[r];
            return;
        }
        // rows from `see` on see the key
        const int see[2] = {weigh_first_token(p, x.s, key[0]) * p.G, weigh_first_token(p, x.s, key[1]) * p.G};
        float sum[2] = {0.f, 0.f}, c[4];
        auto add = [&](int r0, float off0, float off1) {
            const float off[2] = {off0, off1};
            const bool counts[2] = {off0 != -INFINITY, off1 != -INFINITY};  // (rows that there are not have it too)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = r0 + quad * 2 + e;
                if (counts[e] && r >= see[0]) sum[0] += ex2_approx(fmaf(c[e], p.scale_log2, off[e]));
                if (counts[e] && r >= see[1]) sum[1] += ex2_approx(fmaf(c[2 + e], p.scale_log2, off[e]));
            }
        };
        if constexpr (FEW) {
            if (z_of != x.b * p.Hkv + x.h) {
                z_of = x.b * p.Hkv + x.h;
                rows_of(x, 0, z);
                lse[0] = off_of(x, quad * 2);
                lse[1] = off_of(x, quad * 2 + 1);
            }
            products(x, z, c);
            add(0, lse[0], lse[1]);
        } else {
            for (int r0 = weigh_first_token(p, x.s, x.k0) * p.G & ~7; r0 < rows; r0 += 8) {
                uint4 q[D / 32];
                rows_of(x, r0, q);
                const float off0 = off_of(x, r0 + quad * 2), off1 = off_of(x, r0 + quad * 2 + 1);
                products(x, q, c);
                add(r0, off0, off1);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
            if (quad == 0 && key[r] < x.s.len)
                p.out[(static_cast<long long>(x.b) * p.Hkv + x.h) * p.len + key[r]] =
                    p.in ? fmaf(p.decay, x.old[r], sum[r]) : sum[r];
        }
    };
    WeighKeys<D> one, two;
    load(walk, page_of(walk), one);
    walk.next(p);
    int page = page_of(walk);
    for (;;) {
        load(walk, page, two);
        if (walk.left > 0) walk.next(p);
        page = page_of(walk);
        compute(one);
        if (two.k0 == INT_MAX / 2) break;
        load(walk, page, one);
        if (walk.left > 0) walk.next(p);
        page = page_of(walk);
        compute(two);
        if (one.k0 == INT_MAX / 2) break;
    }
}

template <int D, bool BF16>
int launch_rows(const WeighParams &p, const DeviceInfo &dev, cudaStream_t stream) {
    const long long most = static_cast<long long>(p.B) * p.Hkv * ((p.max_len + kStepKeys - 1) / kStepKeys);
    PagedConfig cfg(static_cast<unsigned>(std::min<long long>(most, 2LL * dev.num_sms)), kThreads, 0, true, stream);
    const bool few = static_cast<long long>(p.max_q) * p.G <= 8 && static_cast<long long>(p.B) * p.Hkv <= INT_MAX;
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, few ? weigh_rows_kernel<D, BF16, true> : weigh_rows_kernel<D, BF16, false>, p);
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
    p.in_place = a.weights == a.out ? 1 : 0;
    if (weigh_in_tiles(a, dev.num_sms)) return launch_weigh_tiles(a, p, dev, stream);
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
