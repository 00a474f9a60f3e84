// fa_paged_api.cu -- the extern "C" calls on a paged key/value cache (declared
// in include/fa.h): argument checks before any CUDA call, scratch, launches.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kMaxPageSize = 1 << 20;
constexpr float kLog2eHost = 1.4426950408889634f;

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// Bytes [base, base + size) of an argument.
struct Span {
    const void *base;
    size_t size;
};

bool meet(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.base), y = reinterpret_cast<uintptr_t>(b.base);
    return a.base && b.base && a.size && b.size && x < y + b.size && y < x + a.size;
}

size_t out_size(fa_dtype dt) { return dt == FA_F32 ? 4 : 2; }

// Elements from the first to the last of H heads of d over `rows` rows `stride` apart.
size_t strided(long long rows, long long stride, int H, int d) {
    return rows < 1 || H < 1 ? 0 : static_cast<size_t>(rows - 1) * stride + static_cast<size_t>(H) * d;
}

struct Dim {
    long long n, stride;
};

// The dimensions of a page tensor that are stepped over, shortest stride first; how many.
int page_dims(const fa_paged_cache &c, Dim (&dims)[3]) {
    int n = 0;
    for (const Dim &m : {Dim{c.page_size, c.slot_stride}, Dim{c.num_heads, c.head_stride}, Dim{c.num_pages, c.page_stride}})
        if (m.n > 1) dims[n++] = m;  // (the stride of an extent of one may be anything)
    std::sort(dims, dims + n, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
    return n;
}

long long floor_div(long long a, long long b) { return a / b - (a % b < 0 ? 1 : 0); }

// Whether two tensors of these dimensions over rows of `row` elements, `delta` elements apart, share a
// place.  Every stride is at least what the dimensions below it span, so two steps of one come into question.
bool share_place(const Dim *dims, int n, long long row, long long delta) {
    if (n == 0) return delta > -row && delta < row;
    const Dim &m = dims[n - 1];
    const long long step = floor_div(delta, m.stride);
    for (long long i = step; i <= step + 1; ++i)
        if (i > -m.n && i < m.n && share_place(dims, n - 1, row, delta - i * m.stride)) return true;
    return false;
}

// `row` elements every `stride`.
struct Rows {
    const void *base;
    long long row, stride;
};
// Whether any of `total` rows of either meet.  (At different strides: whether their spans do.)
bool rows_meet(const Rows &a, const Rows &b, long long total) {
    const auto span = [&](const Rows &r) {
        return Span{r.base, static_cast<size_t>((total < 1 ? 0 : (total - 1) * r.stride + r.row) * 2)};
    };
    if (total < 1 || !meet(span(a), span(b))) return false;
    if (total < 2 || a.stride != b.stride) return true;
    const long long delta = (reinterpret_cast<intptr_t>(b.base) - reinterpret_cast<intptr_t>(a.base)) / 2;
    const long long step = floor_div(delta, a.stride), off = delta - step * a.stride;
    return (off < a.row && step > -total && step < total) ||
           (off + b.row > a.stride && step + 1 > -total && step + 1 < total);
}

// The pages themselves; *elements: from the first to the last element of either tensor.
int check_cache(const fa_paged_cache *c, size_t *elements) {
    if (!c || !c->k_pages || !c->v_pages) return FA_ERR_NULL;
    if (c->num_pages < 1 || c->num_heads < 1) return FA_ERR_SHAPE;
    if (c->page_size < 16 || c->page_size > kMaxPageSize || (c->page_size & (c->page_size - 1))) return FA_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128) return FA_ERR_HEAD_DIM;
    if (c->dtype != FA_F16 && c->dtype != FA_BF16) return FA_ERR_DTYPE;
    if (off16(c->k_pages) || off16(c->v_pages)) return FA_ERR_ALIGN;
    Dim dims[3];
    const int n = page_dims(*c, dims);
    for (int i = 0; i < n; ++i) {
        const Dim &m = dims[i];
        if (m.stride < c->head_dim || m.stride >= (1LL << 39)) return FA_ERR_SHAPE;
        if (m.stride % 8) return FA_ERR_ALIGN;
    }
    unsigned long long span = c->head_dim;  // no two elements share a place
    for (int i = 0; i < n; ++i) {
        const Dim &m = dims[i];
        if (static_cast<unsigned long long>(m.stride) < span) return FA_ERR_SHAPE;
        span += static_cast<unsigned long long>(m.n - 1) * m.stride;
        if (span > (1ULL << 46)) return FA_ERR_SHAPE;
    }
    *elements = static_cast<size_t>(span);
    return FA_OK;
}

struct Attention {
    const fa_paged_cache *c;
    const void *q;
    void *out;
    float *lse;
    const int32_t *page_table;
    int max_pages;
    const int32_t *seq_lens, *cu;
    int B, Hq, total, max_q;
    float scale;
    fa_dtype out_dtype;
    const void *workspace;
};

int check_attention(const Attention &a) {
    size_t elements = 0;
    if (!a.c || !a.q || !a.out || !a.page_table || !a.seq_lens) return FA_ERR_NULL;
    const int rc = check_cache(a.c, &elements);
    if (rc != FA_OK) return rc;
    if (a.B < 1 || a.Hq < 1 || a.Hq % a.c->num_heads != 0 || a.max_pages < 1 || a.total < 0 || a.max_q < 1)
        return FA_ERR_SHAPE;
    if (static_cast<long long>(a.max_pages) * a.c->page_size > INT_MAX / 2 ||
        static_cast<long long>(a.B) * a.Hq > INT_MAX / 2 || static_cast<long long>(a.total) * a.Hq > INT_MAX / 2 ||
        static_cast<long long>(a.max_q) * a.Hq > INT_MAX / 2)
        return FA_ERR_SHAPE;
    if (a.out_dtype != FA_F16 && a.out_dtype != FA_BF16 && a.out_dtype != FA_F32) return FA_ERR_DTYPE;
    if (off16(a.q) || off16(a.out) || off4(a.lse) || off4(a.page_table) || off4(a.seq_lens) || off4(a.cu) ||
        off16(a.workspace))
        return FA_ERR_ALIGN;
    if (!std::isfinite(a.scale * kLog2eHost)) return FA_ERR_SCALE;  // (the kernels' scores are in log2 units)
    const size_t rows = static_cast<size_t>(a.total) * a.Hq;
    const Span outs[2] = {{a.out, rows * a.c->head_dim * out_size(a.out_dtype)}, {a.lse, a.lse ? rows * 4 : 0}};
    const Span ins[6] = {{a.q, rows * a.c->head_dim * 2},
                         {a.c->k_pages, elements * 2},
                         {a.c->v_pages, elements * 2},
                         {a.page_table, static_cast<size_t>(a.B) * a.max_pages * 4},
                         {a.seq_lens, static_cast<size_t>(a.B) * 4},
                         {a.cu, a.cu ? (static_cast<size_t>(a.B) + 1) * 4 : 0}};
    for (const Span &o : outs)
        for (const Span &i : ins)
            if (meet(o, i)) return FA_ERR_ALIAS;
    if (meet(outs[0], outs[1])) return FA_ERR_ALIAS;
    return FA_OK;
}

PagedLaunch launch_of(const Attention &a, int causal) {
    PagedLaunch l = {};
    l.c = *a.c;
    l.q = a.q;
    l.out = a.out;
    l.lse = a.lse;
    l.page_table = a.page_table;
    l.seq_lens = a.seq_lens;
    l.cu_q = a.cu;
    l.B = a.B;
    l.Hq = a.Hq;
    l.total_q = a.total;
    l.max_q = a.max_q;
    l.max_pages = a.max_pages;
    l.causal = causal ? 1 : 0;
    l.scale = a.scale;
    l.out_dtype = a.out_dtype;
    return l;
}

// The caller's workspace, or the library's pool.
struct Scratch {
    void *ptr = nullptr;
    bool ours = false;
    cudaStream_t stream;
    explicit Scratch(cudaStream_t s) : stream(s) {}
    // used: whether this call writes it (a workspace that is given has to be large enough either way)
    int take(void *given, size_t given_bytes, size_t need, bool used) {
        if (given) {
            ptr = given;
            return given_bytes < need ? FA_ERR_WORKSPACE : FA_OK;
        }
        if (!used) return FA_OK;
        const cudaError_t e = scratch_alloc(&ptr, need, stream);
        if (e != cudaSuccess) {
            cuda_fail(e);
            return FA_ERR_WORKSPACE;
        }
        ours = true;
        return FA_OK;
    }
    int done(int rc) {
        if (ours) {
            const cudaError_t e = scratch_free(ptr, stream);
            if (rc == FA_OK && e != cudaSuccess) rc = cuda_fail(e);
        }
        return rc;
    }
};

int run_attention(const Attention &a, int causal, void *workspace, size_t workspace_bytes, void *stream) {
    DeviceInfo dev;
    int rc = current_device_info(&dev);
    if (rc != FA_OK) return rc;
    if (a.total == 0) return FA_OK;
    PagedLaunch l = launch_of(a, causal);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    Scratch s(st);
    // (a workspace is sized for max_seqlen_q, which fewer tokens than that do not change)
    const size_t need = paged_scratch_bytes(a.max_q, a.Hq / a.c->num_heads, a.c->head_dim, dev.num_sms);
    if ((rc = s.take(workspace, workspace_bytes, need, paged_needs_scratch(l, dev))) != FA_OK) return rc;
    l.scratch = s.ptr;
    return s.done(launch_paged(l, dev, st));
}

int sms_of(int device) {
    cudaError_t e;
    if (device < 0 && (e = cudaGetDevice(&device)) != cudaSuccess) return -cuda_fail(e);
    int sms = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device)) != cudaSuccess) return -cuda_fail(e);
    return sms;
}

bool head_sizes_ok(int Hq, int Hkv, int d) { return Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && (d == 64 || d == 128); }

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_cache_append(const fa_paged_cache *cache, const void *q, const void *k, const void *v, void *q_out,
                    long long q_stride, long long k_stride, long long v_stride, long long q_out_stride,
                    const int32_t *page_table, int max_pages, const int32_t *seq_lens, const int32_t *cu_seqlens,
                    const int32_t *positions, int B, int Hq, int total, const float *rope, int max_positions,
                    int rope_dim, int interleaved, void *stream) {
    if (!cache || !k || !v || !page_table || !seq_lens) return FA_ERR_NULL;
    size_t elements = 0;
    int rc = check_cache(cache, &elements);
    if (rc != FA_OK) return rc;
    const int d = cache->head_dim, Hkv = cache->num_heads;
    if (B < 1 || Hq < 0 || total < 0 || max_pages < 1) return FA_ERR_SHAPE;
    if ((Hq > 0) != (q != nullptr) || (Hq > 0) != (q_out != nullptr)) return FA_ERR_NULL;
    if (!cu_seqlens && total != B) return FA_ERR_SHAPE;
    if (static_cast<long long>(max_pages) * cache->page_size > INT_MAX / 2 ||
        static_cast<long long>(total) * (Hq + 2LL * Hkv) > INT_MAX || Hq + 2LL * Hkv > 65536)
        return FA_ERR_SHAPE;
    if (rope_dim < 0 || rope_dim > d || rope_dim % 16) return FA_ERR_SHAPE;
    if (rope_dim > 0) {
        if (!rope) return FA_ERR_NULL;
        if (max_positions < 1) return FA_ERR_SHAPE;
        if (off16(rope)) return FA_ERR_ALIGN;
    }
    if (off16(q) || off16(k) || off16(v) || off16(q_out) || off4(page_table) || off4(seq_lens) || off4(cu_seqlens) ||
        off4(positions))
        return FA_ERR_ALIGN;
    struct {
        long long stride;
        int H;
    } const rows[4] = {{q_stride, Hq}, {k_stride, Hkv}, {v_stride, Hkv}, {q_out_stride, Hq}};
    for (const auto &r : rows) {
        if (r.H == 0 || total < 2) continue;
        if (r.stride < static_cast<long long>(r.H) * d || r.stride >= (1LL << 39)) return FA_ERR_SHAPE;
        if (r.stride % 8) return FA_ERR_ALIGN;
    }
    // What is written: the pages and q_out.  q_out may be q itself (in place).
    const Span in[3] = {{q, strided(total, q_stride, Hq, d) * 2},
                        {k, strided(total, k_stride, Hkv, d) * 2},
                        {v, strided(total, v_stride, Hkv, d) * 2}};
    const Span aux[5] = {{page_table, static_cast<size_t>(B) * max_pages * 4},
                         {seq_lens, static_cast<size_t>(B) * 4},
                         {cu_seqlens, (static_cast<size_t>(B) + 1) * 4},
                         {positions, static_cast<size_t>(total) * 4},
                         {rope_dim ? rope : nullptr, static_cast<size_t>(std::max(max_positions, 0)) * rope_dim * 4}};
    const Span pages[2] = {{cache->k_pages, elements * 2}, {cache->v_pages, elements * 2}};
    const Span qo = {q_out, strided(total, q_out_stride, Hq, d) * 2};
    const bool in_place = q_out == q && (q_out_stride == q_stride || total < 2);
    for (const Span &w : pages) {
        if (meet(w, qo)) return FA_ERR_ALIAS;
        for (const Span &i : in)
            if (meet(w, i)) return FA_ERR_ALIAS;
        for (const Span &x : aux)
            if (meet(w, x)) return FA_ERR_ALIAS;
    }
    if (in_place) {  // (k and v may lie between q's rows, as in a fused projection)
        const Rows rq = {q, 1LL * Hq * d, q_stride};
        if (rows_meet(rq, {k, 1LL * Hkv * d, k_stride}, q ? total : 0) ||
            rows_meet(rq, {v, 1LL * Hkv * d, v_stride}, q ? total : 0))
            return FA_ERR_ALIAS;
    } else {
        for (const Span &i : in)
            if (meet(qo, i)) return FA_ERR_ALIAS;
    }
    // a slot's key and its value are two places
    Dim dims[3];
    const int n = page_dims(*cache, dims);
    if (share_place(dims, n, d, (reinterpret_cast<intptr_t>(cache->v_pages) - reinterpret_cast<intptr_t>(cache->k_pages)) / 2))
        return FA_ERR_ALIAS;
    for (const Span &x : aux)
        if (meet(qo, x)) return FA_ERR_ALIAS;
    DeviceInfo dev;
    if ((rc = current_device_info(&dev)) != FA_OK) return rc;
    if (total == 0) return FA_OK;
    AppendLaunch a;
    a.c = *cache;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.cu_seqlens = cu_seqlens;
    a.positions = positions;
    a.B = B;
    a.Hq = Hq;
    a.total = total;
    a.max_pages = max_pages;
    a.rope = rope;
    a.max_positions = max_positions;
    a.rope_dim = rope_dim;
    a.interleaved = interleaved;
    return launch_append(a, dev, static_cast<cudaStream_t>(stream));
}

size_t fa_paged_workspace_bytes(int Hq, int Hkv, int max_seqlen_q, int d, int device) {
    if (!head_sizes_ok(Hq, Hkv, d) || max_seqlen_q < 1) return 0;
    const int sms = sms_of(device);
    return sms < 0 ? 0 : paged_scratch_bytes(max_seqlen_q, Hq / Hkv, d, sms);
}

size_t fa_shared_workspace_bytes(int B, int Hq, int Hkv, int d, int device) {
    if (!head_sizes_ok(Hq, Hkv, d) || B < 1) return 0;
    const int sms = sms_of(device);
    return sms < 0 ? 0 : paged_pair_scratch_bytes(B, Hq, Hkv, d, sms);
}

int fa_prefill_paged(const fa_paged_cache *cache, const void *q, void *out, float *lse, const int32_t *page_table,
                     int max_pages, const int32_t *seq_lens, const int32_t *cu_seqlens_q, int B, int Hq, int total_q,
                     int max_seqlen_q, int causal, float scale, fa_dtype out_dtype, void *workspace,
                     size_t workspace_bytes, void *stream) {
    if (!cu_seqlens_q) return FA_ERR_NULL;
    const Attention a = {cache,        q, out, lse, page_table, max_pages, seq_lens, cu_seqlens_q, B, Hq, total_q,
                         max_seqlen_q, scale, out_dtype, workspace};
    const int rc = check_attention(a);
    return rc != FA_OK ? rc : run_attention(a, causal, workspace, workspace_bytes, stream);
}

int fa_decode_paged(const fa_paged_cache *cache, const void *q, void *out, const int32_t *page_table, int max_pages,
                    const int32_t *seq_lens, int B, int Hq, float scale, fa_dtype out_dtype, void *workspace,
                    size_t workspace_bytes, void *stream) {
    const Attention a = {cache, q, out, nullptr, page_table, max_pages, seq_lens, nullptr, B, Hq, B, 1, scale,
                         out_dtype, workspace};
    const int rc = check_attention(a);
    return rc != FA_OK ? rc : run_attention(a, 0, workspace, workspace_bytes, stream);
}

int fa_decode_shared(const fa_paged_cache *cache, const void *q, void *out, const int32_t *prefix_table,
                     int max_prefix_pages, const int32_t *prefix_len, const int32_t *page_table, int max_pages,
                     const int32_t *seq_lens, int B, int Hq, float scale, fa_dtype out_dtype, void *workspace,
                     size_t workspace_bytes, void *stream) {
    const Attention own = {cache, q, out, nullptr, page_table, max_pages, seq_lens, nullptr, B, Hq, B, 1, scale,
                           out_dtype, workspace};
    int rc = check_attention(own);
    if (rc != FA_OK) return rc;
    // the prefix as one sequence that every row of the batch reads in full
    Attention pre = own;
    pre.page_table = prefix_table;
    pre.max_pages = max_prefix_pages;
    pre.seq_lens = prefix_len;
    pre.B = 1;
    pre.max_q = B;
    if ((rc = check_attention(pre)) != FA_OK) return rc;
    DeviceInfo dev;
    if ((rc = current_device_info(&dev)) != FA_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    Scratch s(st);
    const size_t need = paged_pair_scratch_bytes(B, Hq, cache->num_heads, cache->head_dim, dev.num_sms);
    const PagedLaunch first = launch_of(pre, 0), second = launch_of(own, 0);
    if ((rc = s.take(workspace, workspace_bytes, need, paged_pair_needs_scratch(first, second, dev))) != FA_OK) return rc;
    return s.done(launch_paged_pair(first, second, s.ptr, dev, st));
}

}  // extern "C"
