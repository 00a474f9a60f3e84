// fa_cache_sm103.cu -- appending tokens to a paged key/value cache, with the
// rotary position rotation of q and k on the way.
//
// Token i of sequence b's n new ones has position pos = seq_lens[b] - n + i and
// goes to slot pos % page_size of page page_table[b][pos / page_size].  The
// first rope_dim channels of q and k turn in pairs,
//   (x1, x2) -> (x1 cos a - x2 sin a, x1 sin a + x2 cos a),
// with cos a and sin a of the position's row of an fp32 table; the arithmetic
// is fp32 and each value is rounded once, to its 16-bit type.
//
// Bound by the HBM for prompts (every element is read once and written once)
// and by the chain of dependent loads for single tokens (offsets, length, page
// id, then the data).  A warp works on one token and keeps that token's slice
// of the table in registers while it walks over the heads, D / 16 lanes a head,
// 32 bytes a lane: a pair's two halves are then always in one lane.  38 thousand
// tokens of 32 + 8 + 8 heads of 128: 141 us, 6.4 TB/s of DRAM traffic (95% of the copy
// rate); 256 single tokens: 3.3 us, one token 2.2 us (back to back in a graph).
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_internal.h"
#include "fa_tiles.cuh"
#include "sm103_ptx.cuh"

namespace fa {

namespace {

constexpr int kWarps = 4;

__device__ int g_append_status = 0;

struct AppendParams {
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *k_pages, *v_pages;
    long long q_stride, k_stride, v_stride, q_out_stride;
    long long page_stride, head_stride, slot_stride;
    const int *page_table, *seq_lens, *cu, *positions;
    const float *rope;
    int B, Hq, Hkv, total, max_pages, num_pages, page_shift;
    int max_positions, rope_dim;
    int heads_each;  // heads per warp
};

// The sequence that owns token t: the last b with cu[b] <= t (empty sequences in
// between own nothing).  The warp narrows the range 32-fold per step.
__device__ __forceinline__ int find_seq(const int *cu, int B, int t, int lane) {
    int lo = 0, n = B;  // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool below = lane * step < n && __ldg(cu + i) <= t;
        // (cu[lo] <= t is known or checked by the caller; lane 0 counts regardless)
        const int last = max(0, 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u));
        const int off = last * step;
        lo += off;
        n = min(step, n - off);
    }
    return lo;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t t = unpack2<BF16>(u[i]);
        f[2 * i] = f2_lo(t);
        f[2 * i + 1] = f2_hi(t);
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2t<BF16>(f[0], f[1]), pack2t<BF16>(f[2], f[3]), pack2t<BF16>(f[4], f[5]),
                      pack2t<BF16>(f[6], f[7]));
}

template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const AppendParams p) {
    constexpr int LPH = D / 16;      // lanes per head
    constexpr int HPW = 32 / LPH;    // heads per warp and step
    // launched while the kernels ahead of it still run; nothing in global memory before they are done
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= p.total) return;
    int b = t, first = t, last = t + 1;
    if (p.cu) {
        if (t < __ldg(p.cu) || t >= __ldg(p.cu + p.B)) return;  // behind the last sequence
        b = find_seq(p.cu, p.B, t, lane);
        first = __ldg(p.cu + b);
        last = __ldg(p.cu + b + 1);
    }
    const long long at = static_cast<long long>(__ldg(p.seq_lens + b)) - last + t;
    const long long max_len = static_cast<long long>(p.max_pages) << p.page_shift;
    bool slot_ok = at >= 0 && at < max_len && t >= first && t < last;
    const int pos = static_cast<int>(min(max(at, -1LL), max_len));
    int status = slot_ok ? 0 : FA_ERR_SEQ_LEN;
    int page = 0;
    if (slot_ok) {
        page = __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + (pos >> p.page_shift));
        if (page < 0 || page >= p.num_pages) {
            slot_ok = false;
            status = FA_ERR_PAGE;
        }
    }
    int angle = p.positions ? __ldg(p.positions + t) : pos;
    if (p.rope_dim && (angle < 0 || angle >= p.max_positions)) {
        if (!status) status = FA_ERR_SEQ_LEN;
        angle = min(max(angle, 0), p.max_positions - 1);
    }
    if (status && lane == 0 && blockIdx.y == 0) atomicCAS(&g_append_status, 0, status);

    // This lane's two 8-channel pieces, and whether they turn.
    const int c = lane % LPH;
    const int half = p.rope_dim / 2;
    const bool turns = c < p.rope_dim / 16;
    int ca, cb;
    if (!INTER && turns) {
        ca = 8 * c;
        cb = half + 8 * c;
    } else {
        ca = 16 * c;
        cb = 16 * c + 8;
    }
    float cs[8], sn[8];
    if (turns) {  // pair i of this lane: half-split 8 c + i, interleaved likewise
        const float4 *row = reinterpret_cast<const float4 *>(p.rope + static_cast<long long>(angle) * p.rope_dim);
        const float4 c0 = __ldg(row + 2 * c), c1 = __ldg(row + 2 * c + 1);
        const float4 s0 = __ldg(row + half / 4 + 2 * c), s1 = __ldg(row + half / 4 + 2 * c + 1);
        cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w;
        cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
        sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w;
        sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
    }
    const long long slot = static_cast<long long>(page) * p.page_stride +
                           (pos & ((1 << p.page_shift) - 1)) * p.slot_stride;
    const int heads = p.Hq + 2 * p.Hkv;
    const int h0 = blockIdx.y * p.heads_each, h1 = min(h0 + p.heads_each, heads);
    constexpr int U = 4;
    for (int hb = h0 + lane / LPH; hb < h1; hb += U * HPW) {
        uint4 a[U], e[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = hb + i * HPW;
            if (h < h1) {
                const uint16_t *src = h < p.Hq             ? p.q + t * p.q_stride + h * D
                                      : h < p.Hq + p.Hkv ? p.k + t * p.k_stride + (h - p.Hq) * D
                                                         : p.v + t * p.v_stride + (h - p.Hq - p.Hkv) * D;
                const bool v = h >= p.Hq + p.Hkv;
                a[i] = *reinterpret_cast<const uint4 *>(src + (v ? 16 * c : ca));
                e[i] = *reinterpret_cast<const uint4 *>(src + (v ? 16 * c + 8 : cb));
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = hb + i * HPW;
            if (h >= h1) break;
            const bool v = h >= p.Hq + p.Hkv;
            if (turns && !v) {
                float x[8], y[8];
                unpack8<BF16>(a[i], x);
                unpack8<BF16>(e[i], y);
                if constexpr (INTER) {
                    // pieces a, e hold pairs 8 c .. 8 c + 3 and 8 c + 4 .. 8 c + 7
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float x1 = x[2 * k], x2 = x[2 * k + 1], y1 = y[2 * k], y2 = y[2 * k + 1];
                        x[2 * k] = x1 * cs[k] - x2 * sn[k];
                        x[2 * k + 1] = x1 * sn[k] + x2 * cs[k];
                        y[2 * k] = y1 * cs[4 + k] - y2 * sn[4 + k];
                        y[2 * k + 1] = y1 * sn[4 + k] + y2 * cs[4 + k];
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float x1 = x[k], x2 = y[k];
                        x[k] = x1 * cs[k] - x2 * sn[k];
                        y[k] = x1 * sn[k] + x2 * cs[k];
                    }
                }
                a[i] = pack8<BF16>(x);
                e[i] = pack8<BF16>(y);
            }
            uint16_t *dst;
            if (h < p.Hq) dst = p.q_out + t * p.q_out_stride + h * D;
            else if (!slot_ok) continue;
            else if (!v) dst = p.k_pages + slot + (h - p.Hq) * p.head_stride;
            else dst = p.v_pages + slot + (h - p.Hq - p.Hkv) * p.head_stride;
            *reinterpret_cast<uint4 *>(dst + (v ? 16 * c : ca)) = a[i];
            *reinterpret_cast<uint4 *>(dst + (v ? 16 * c + 8 : cb)) = e[i];
        }
    }
}

template <int D, bool BF16>
cudaError_t launch_append_d(const AppendParams &p, dim3 grid, bool inter, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, inter ? append_kernel<D, BF16, true> : append_kernel<D, BF16, false>, p);
}

}  // namespace

int launch_append(const AppendLaunch &a, const DeviceInfo &dev, cudaStream_t stream) {
    AppendParams p;
    p.q = static_cast<const uint16_t *>(a.q);
    p.k = static_cast<const uint16_t *>(a.k);
    p.v = static_cast<const uint16_t *>(a.v);
    p.q_out = static_cast<uint16_t *>(a.q_out);
    p.k_pages = static_cast<uint16_t *>(a.c.k_pages);
    p.v_pages = static_cast<uint16_t *>(a.c.v_pages);
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.q_out_stride = a.q_out_stride;
    p.page_stride = a.c.page_stride;
    p.head_stride = a.c.head_stride;
    p.slot_stride = a.c.slot_stride;
    p.page_table = a.page_table;
    p.seq_lens = a.seq_lens;
    p.cu = a.cu_seqlens;
    p.positions = a.positions;
    p.rope = a.rope;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.c.num_heads;
    p.total = a.total;
    p.max_pages = a.max_pages;
    p.num_pages = a.c.num_pages;
    p.page_shift = 0;
    while ((1 << p.page_shift) < a.c.page_size) ++p.page_shift;
    p.max_positions = a.max_positions;
    p.rope_dim = a.rope_dim;
    // A warp takes all of a token's heads when there are tokens enough, and down to
    // one step of them (four or eight heads) when there are few.
    const int heads = a.Hq + 2 * p.Hkv, step = 32 / (a.c.head_dim / 16);
    const long long want = 16LL * dev.num_sms;  // warps
    const int most = (heads + step - 1) / step;
    const int slices = static_cast<int>(std::min<long long>(most, std::max<long long>(1, want / a.total)));
    p.heads_each = ((heads + slices - 1) / slices + step - 1) / step * step;
    const dim3 grid((a.total + kWarps - 1) / kWarps, (heads + p.heads_each - 1) / p.heads_each);
    const bool bf16 = a.c.dtype == FA_BF16, inter = a.interleaved != 0;
    const auto launch = a.c.head_dim == 64 ? (bf16 ? launch_append_d<64, true> : launch_append_d<64, false>)
                                           : (bf16 ? launch_append_d<128, true> : launch_append_d<128, false>);
    const cudaError_t e = launch(p, grid, inter, stream);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

int read_append_status(int reset) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_append_status, sizeof(int)) != cudaSuccess) return -1;
    if (reset && v) {
        int z = 0;
        if (cudaMemcpyToSymbol(g_append_status, &z, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace fa
