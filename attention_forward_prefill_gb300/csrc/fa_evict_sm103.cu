// fa_evict_sm103.cu -- which tokens of a paged cache stay, and moving those that do.
//
// Selection.  Of a row (sequence, head) of n accumulated weights the first `sink` and
// the last `recent` tokens stay, and of the ones between them those with the largest
// weights, budget = k in all.  With keys u(w) in the order of the weights the smallest
// key T that stays is found digit by digit from the top (11, 11 and 10 bits): the
// counts of a digit's values, summed from above, say which value holds the k-th key.
// All keys above T stay, and of those equal to T the ones at the lowest positions.
// Latency: a digit costs a pass over the row in shared memory and two exchanges between the CTAs
// of its cluster.  4 x 8 rows of 90001 to 131071 weights, 16384 to keep: 26 us (110 with the weights
// read again for every digit, 90 with them in shared memory, 35 with all CTAs' counts read by every CTA and the
// whole row looked at again for every digit and twice for the lists; the weights and lists take 4.9 us at 6.8 TB/s).
// A CTA of those, by its clock: the start 2.4 thousand clocks, the weights' load with the first digit's counts 6 to 8, and
// 13 where two CTAs share an SM; the second digit's sweep 4.5 to 6, the third's 1 to 2; a digit's exchanges 3.5 to
// 7, with the wait for the slowest CTA in the first; a digit's value 1 to 1.8; the places 2.7; the lists 2.5; 36 to 50 in
// all.  Weights whose first digits are spread evenly over the bins take as long for the first digit (and 10% less in all).
// 155648 weights, the most that shared memory holds: 32 us for as many rows; 155649 54, 500001 140.
// 2 x 2 rows of 1000 weights: 5.9 us.
//
// Moving.  Token keep[i] goes to place first + i.  In place, keep[i] >= first + i, so
// that the place a token comes from is written by the token of the same or a later i
// alone: whoever reads a column of a row in the order of i, ahead of what it writes, can
// move it without a copy.  HBM-bound: 8 sequences of up to 32768 tokens, 8192 to keep, 8 heads
// of 128: 93 us for 539 MB (5.8 TB/s); with one token after another 2279.
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
    int heads, len, budget, sink, recent;
};

constexpr uint32_t kZeroKey = 0x80000000u;
// Larger for larger weights; -0 is 0, and NaN comes above all.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xfffffffeu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void *at, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
    return a;
}
// 16 or 8 bytes to shared memory of a CTA of the cluster, whose barrier counts them as they come in.
__device__ __forceinline__ void cluster_send(void *at, int rank, uint64_t *bar, uint4 v) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];" ::
                 "r"(cluster_addr(at, rank)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(cluster_addr(bar, rank)) : "memory");
}
__device__ __forceinline__ void cluster_send(void *at, int rank, uint64_t *bar, uint2 v) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1,%2}, [%3];" ::
                 "r"(cluster_addr(at, rank)), "r"(v.x), "r"(v.y), "r"(cluster_addr(bar, rank)) : "memory");
}
__device__ __forceinline__ bool cluster_received(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return done;
}
constexpr uint64_t kReceiveNs = 1500ull * 1000ull * 1000ull, kLandNs = 1000ull * 1000ull;
// False: it has not come within the limit.
__device__ __forceinline__ bool cluster_receive(uint64_t *bar, uint32_t parity) {
    if (cluster_received(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    do {
        if (cluster_received(bar, parity)) return true;
    } while (globaltimer_ns() - t0 <= kReceiveNs);
    return false;
}
__device__ __forceinline__ uint4 add4(uint4 a, uint4 b) { return make_uint4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

__device__ __forceinline__ uint32_t scan_up(uint32_t v, int lane) {  // over the lanes, inclusive
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    return v;
}

// A cluster of `size` CTAs per row, a slice of the row's tokens each, and a run of the slice
// each warp.  HOLDS: the slice's keys stay in shared memory, and after the first digit a lane holds
// bits for up to 32 tokens side by side, or twice 32: whether a key is above those that share the
// digits found, or one of them.  Only the latter are looked at again.  Else, for rows of any length,
// the weights are read again for every digit.
constexpr int kHeld = 19456;  // two CTAs per SM
constexpr int kWords = 2;     // words of such bits a lane
static_assert(kHeld / kSelWarps <= kWords * 32 * 32);
template <bool HOLDS>
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const SelectParams p, const int size) {
    extern __shared__ __align__(16) uint32_t held[];
    // counts by digit, the highest first, in two tables (and for the first digit in a third, the sums'), as additions
    // to one bin go one by one; what the cluster's CTAs sent for the bins that this one adds up; and the sums of all
    __shared__ __align__(16) uint32_t hist[2][kBins];
    __shared__ __align__(16) uint4 sent[kBins / 4], sums[kBins / 4];
    __shared__ uint32_t warp_sum[kSelWarps], found[2];
    __shared__ uint2 warp_has[kSelWarps], cta_has[kMaxCluster];  // keys above, and equal to, the last that stays
    __shared__ uint64_t sent_bar, sums_bar, has_bar;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0 && size > 1) {
        mbar_init(&sent_bar, 1);
        mbar_init(&sums_bar, 1);
        mbar_init(&has_bar, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(&sent_bar, sizeof(sent));
        mbar_arrive_expect_tx(&sums_bar, sizeof(sums));
        mbar_arrive_expect_tx(&has_bar, blockIdx.x % size * sizeof(uint2));
    }
    for (int i = tid; i < 2 * kBins; i += kSelThreads) hist[0][i] = 0;
    sums[tid] = make_uint4(0, 0, 0, 0);
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    const int rank = blockIdx.x % size, row = blockIdx.x / size;
    const int b = row / p.heads;
    const int raw = __ldg(p.seq_lens + b), n = min(max(raw, 0), p.len);
    const int count = min(n, p.budget);
    const float *w = p.weights + static_cast<long long>(row) * p.len;
    int *keep = p.keep + static_cast<long long>(row) * p.budget;
    float *kept = p.kept ? p.kept + static_cast<long long>(row) * p.len : nullptr;
    const int t = rank * kSelThreads + tid, threads = size * kSelThreads;
    // this CTA's tokens, and this warp's
    const int per = ((n + size - 1) / size + kSelThreads - 1) / kSelThreads * kSelThreads, run = per / kSelWarps;
    const int w0 = min(rank * per + warp * run, n), w1 = min(w0 + run, n);
    auto key_of = [&](int i) {
        const uint32_t key = weight_key(__ldg(w + min(i, n - 1)));  // (loaded whatever it is: no branch between loads)
        return i < p.sink || i >= n - p.recent ? 0xffffffffu : key;
    };
    // The keys of the run, group by group: token i of group g lies where neither the lanes of a group
    // nor the same token of 32 groups share a bank.  0: there is none (no key is 0).
    const int groups = run / 32;
    uint32_t *mine = held + warp * run;
    auto place = [&](int g, int i) { return g * 32 + (i ^ (g & 31)); };
    constexpr int U = 8;  // tokens of a lane at a time
    // (zeros, which many tokens may have, are counted apart: additions to one bin go one by one)
    uint32_t zeros = 0;
    __syncthreads();
    if (size > 1 && n > p.budget) cluster_arrive();  // (nothing is sent to a CTA that has not started)
    if constexpr (HOLDS) {
        if (n > p.budget) {
            uint32_t *h = lane % 3 == 2 ? reinterpret_cast<uint32_t *>(sums) : hist[lane % 3];
            auto take = [&](int g, uint32_t key) {
                mine[place(g, lane)] = key;
                const bool zero = key == kZeroKey;
                zeros += zero;
                if (!zero) atomicAdd(h + (~key >> 21), 1u);
            };
            constexpr int E = 4;  // where not all 16 groups are tokens to choose among
            for (int g0 = 0; g0 < groups;) {
                const int i0 = w0 + g0 * 32;
                if (i0 >= p.sink && i0 + 2 * U * 32 <= min(w1, n - p.recent)) {
                    uint32_t key[2 * U];
#pragma unroll
                    for (int j = 0; j < 2 * U; ++j) key[j] = __float_as_uint(__ldg(w + i0 + j * 32 + lane));
#pragma unroll
                    for (int j = 0; j < 2 * U; ++j) take(g0 + j, weight_key(__uint_as_float(key[j])));
                    g0 += 2 * U;
                    continue;
                }
                uint32_t key[E];
#pragma unroll
                for (int j = 0; j < E; ++j) key[j] = key_of(i0 + j * 32 + lane);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    if (i0 + j * 32 + lane < w1) take(g0 + j, key[j]);
                    else if (g0 + j < groups) mine[place(g0 + j, lane)] = 0;
                }
                g0 += E;
            }
        }
    }
    if (tid == 0 && rank == 0 && row % p.heads == 0) {
        p.counts[b] = count;
        if (raw != n) record_status(&g_evict_status, FA_ERR_SEQ_LEN);
    }
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
    // each(f): f(token, key, whether there is one) for this warp's tokens, a lane each, in order
    auto each = [&](auto f) {
        for (int i0 = w0; i0 < w1; i0 += U * 32) {
            uint32_t key[U];
#pragma unroll
            for (int j = 0; j < U; ++j) key[j] = key_of(i0 + j * 32 + lane);
#pragma unroll
            for (int j = 0; j < U; ++j) f(i0 + j * 32 + lane, key[j], i0 + j * 32 + lane < w1);
        }
    };
    uint32_t top = 0, left = count;  // the digits found, and how many keys of that prefix stay
    // of tokens `own` + 1024 h and on: keys above that prefix, and with it
    uint32_t more[kWords] = {}, same[kWords] = {};
    const int log_own = groups >= 32 ? 5 : 32 - __clz(groups - 1), own = lane << log_own;  // (all lanes, even of few groups)
    // sort(s, f): keys without the prefix leave `same`, and f gets the others.
    auto sort = [&](int s, auto f) {
#pragma unroll
        for (int h = 0; h < kWords; ++h)
            for (uint32_t m = same[h]; m; m &= m - 1) {
                const uint32_t key = mine[place((own >> 5) + 32 * h, (own & 31) + __ffs(m) - 1)], bit = m & -m;
                if (key >> s == top) {
                    f(key);
                } else {
                    same[h] ^= bit;
                    more[h] |= key >> s > top ? bit : 0;
                }
            }
    };
    // Nobody leaves while others may still send to it, or while what they have sent is on its way: whoever has waited
    // in vain does not know what that is, so it stays for far longer than a store takes.
    auto give_up = [&] {
        if (lane == 0) record_status(&g_evict_status, FA_ERR_WATCHDOG);
        cluster_arrive();
        cluster_wait();
        for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < kLandNs;) {}
    };
    int shift = 32;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass == 2 ? 10 : 11, above = shift;
        shift -= bits;
        uint32_t *h = hist[lane & 1];
        if (!HOLDS || pass > 0) zeros = 0;
        auto add = [&](uint32_t key) {
            if (key == kZeroKey) ++zeros;
            else atomicAdd(h + (~(key >> shift) & ((1u << bits) - 1u)), 1u);
        };
        if constexpr (!HOLDS) {
            each([&](int, uint32_t key, bool is) {
                if (is && (pass == 0 || key >> above == top)) add(key);
            });
        } else if (pass == 1) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                const int g1 = min(groups, w * 32 + 32);
#pragma unroll 8
                for (int g = w * 32; g < g1; ++g) {
                    const uint32_t digit = mine[place(g, lane)] >> above;
                    const uint32_t is_more = __ballot_sync(0xffffffffu, digit > top);
                    const uint32_t is_same = __ballot_sync(0xffffffffu, digit == top);
                    if ((own >> 5) == (g & 31)) more[w] = is_more, same[w] = is_same;
                }
                const uint32_t bits_own = (2u << ((1 << log_own) - 1)) - 1u;
                more[w] = more[w] >> (own & 31) & bits_own;
                same[w] = same[w] >> (own & 31) & bits_own;
            }
        }
        if (HOLDS && pass > 0) sort(above, add);
        zeros = __reduce_add_sync(0xffffffffu, zeros);
        if (lane == 0 && zeros) atomicAdd(h + (~(kZeroKey >> shift) & ((1u << bits) - 1u)), zeros);
        // four bins a thread; a CTA adds up an equal part of them for all, and sends the sums round
        __syncthreads();
        uint4 *own_bins = reinterpret_cast<uint4 *>(hist[0]) + tid;
        uint4 sum4 = add4(own_bins[0], own_bins[kBins / 4]);
        if (HOLDS && pass == 0) sum4 = add4(sum4, sums[tid]);  // (its part of the sums comes after this thread's counts have gone)
        own_bins[0] = own_bins[kBins / 4] = make_uint4(0, 0, 0, 0);
        bool ok = true;
        if (size > 1) {
            const int part = kBins / 4 / size, to = tid / part, at = tid % part;
            if (pass == 0) cluster_wait();
            cluster_send(sent + rank * part + at, to, &sent_bar, sum4);
            ok = cluster_receive(&sent_bar, pass & 1);
            if (tid == 0 && ok) mbar_arrive_expect_tx(&sent_bar, sizeof(sent));
            sum4 = sent[at];
#pragma unroll
            for (int r = 1; r < kMaxCluster; ++r)
                if (r < size) sum4 = add4(sum4, sent[r * part + at]);
            __syncthreads();  // whoever gets sums from here may send its next counts over the ones that are read above
            if (ok) cluster_send(sums + rank * part + at, to, &sums_bar, sum4);  // (else nobody goes on)
            ok = ok && cluster_receive(&sums_bar, pass & 1);
            if (tid == 0 && ok) mbar_arrive_expect_tx(&sums_bar, sizeof(sums));
            sum4 = sums[tid];
        }
        const uint32_t c[4] = {sum4.x, sum4.y, sum4.z, sum4.w};
        const uint32_t all = c[0] + c[1] + c[2] + c[3], incl = scan_up(all, lane);
        if (lane == 31) warp_sum[warp] = incl;
        if (size == 1) {
            __syncthreads();
        } else if (__syncthreads_or(!ok)) {
            give_up();
            return;
        }
        uint32_t sum = incl - all;
#pragma unroll
        for (int k = 0; k < kSelWarps - 1; ++k) sum += k < warp ? warp_sum[k] : 0u;
        if (sum < left && left <= sum + all) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (sum < left && left <= sum + c[k]) {
                    found[0] = ~static_cast<uint32_t>(4 * tid + k) & ((1u << bits) - 1u);
                    found[1] = left - sum;
                }
                sum += c[k];
            }
        }
        __syncthreads();
        top = pass == 0 ? found[0] : top << bits | found[0];
        left = found[1];
    }
    // top: the smallest key that stays; left: how many of those equal to it
    uint32_t above = 0, equal = 0;
    uint32_t ups[kWords] = {}, ups_all = 0;  // above | equal << 16 before this lane's groups, and in the run
    if constexpr (HOLDS) {
        sort(0, [](uint32_t) {});
#pragma unroll
        for (int h = 0; h < kWords; ++h) {
            const uint32_t c = __popc(more[h]) | __popc(same[h]) << 16, incl = scan_up(c, lane);
            ups[h] = ups_all + incl - c;
            ups_all += __shfl_sync(0xffffffffu, incl, 31);
        }
        above = ups_all & 0xffffu;
        equal = ups_all >> 16;
    } else {
        each([&](int, uint32_t key, bool is) {
            above += is && key > top;
            equal += is && key == top;
        });
        above = __reduce_add_sync(0xffffffffu, above);
        equal = __reduce_add_sync(0xffffffffu, equal);
    }
    if (lane == 0) warp_has[warp] = make_uint2(above, equal);
    __syncthreads();
    uint2 has = lane < kSelWarps ? warp_has[lane] : make_uint2(0, 0);
    has.x = scan_up(has.x, lane);
    has.y = scan_up(has.y, lane);
    above = __shfl_sync(0xffffffffu, has.x, max(warp - 1, 0));
    equal = __shfl_sync(0xffffffffu, has.y, max(warp - 1, 0));
    if (warp == 0) above = equal = 0;
    if (size > 1) {  // to the CTAs of the tokens behind
        const uint2 cta = make_uint2(__shfl_sync(0xffffffffu, has.x, kSelWarps - 1), __shfl_sync(0xffffffffu, has.y, kSelWarps - 1));
        if (warp == 0 && lane > rank && lane < size) cluster_send(cta_has + rank, lane, &has_bar, cta);
        if (!__all_sync(0xffffffffu, cluster_receive(&has_bar, 0))) {
            give_up();
            return;
        }
        const uint2 v = lane < rank ? cta_has[lane] : make_uint2(0, 0);
        above += __reduce_add_sync(0xffffffffu, v.x);
        equal += __reduce_add_sync(0xffffffffu, v.y);
    }
    if (size > 1) cluster_arrive();  // nothing is sent any more
    const uint32_t to0 = above + min(equal, left);
    if constexpr (HOLDS) {
        // The tokens that stay, in order: first to where the warp's keys were, so that the lists are then
        // written, and the weights read, side by side.
        uint32_t stay = 0;
        __syncwarp();
#pragma unroll
        for (int h = 0; h < kWords; ++h) {
            const uint32_t e = equal + (ups[h] >> 16);
            uint32_t at = above + (ups[h] & 0xffffu) + min(e, left) - to0;
            int more_of_same = static_cast<int>(left) - static_cast<int>(min(e, left));
            for (uint32_t m = more[h] | same[h]; m; m &= m - 1) {
                if (same[h] & m & -m && more_of_same-- <= 0) continue;
                mine[at++] = w0 + own + 1024 * h + __ffs(m) - 1;
            }
            stay = max(stay, at);
        }
        stay = __reduce_max_sync(0xffffffffu, stay);
        __syncwarp();
        for (uint32_t k0 = lane; k0 < stay; k0 += U * 32) {
            uint32_t i[U];
            float x[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                i[j] = mine[min(k0 + j * 32, stay - 1)];
                x[j] = kept ? __ldg(w + i[j]) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (k0 + j * 32 < stay) {
                    keep[to0 + k0 + j * 32] = i[j];
                    if (kept) kept[to0 + k0 + j * 32] = x[j];
                }
        }
    } else {
        const uint32_t before = (1u << lane) - 1u;
        uint32_t stay = to0;
        each([&](int i, uint32_t key, bool is) {
            const uint32_t is_above = __ballot_sync(0xffffffffu, is && key > top);
            const uint32_t is_equal = __ballot_sync(0xffffffffu, is && key == top);
            if (!(is_above | is_equal)) return;
            const bool stays = is && (key > top || (key == top && equal + __popc(is_equal & before) < left));
            const uint32_t who = __ballot_sync(0xffffffffu, stays), at = stay + __popc(who & before);
            if (stays) {
                keep[at] = i;
                if (kept) kept[at] = __ldg(w + i);
            }
            stay += __popc(who);
            equal += __popc(is_equal);
        });
    }
    if (size > 1) cluster_wait();
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

// One sequence and kv head: its list, checked token by token.
struct KeepRow {
    const int *list, *table, *out_table;
    int len, first, count, mask, status;

    __device__ __forceinline__ KeepRow(const KeepParams &p, int b, int h) {
        const int raw_len = __ldg(p.seq_lens + b), raw_count = __ldg(p.counts + b), raw_first = p.first ? __ldg(p.first + b) : 0;
        const int max_len = p.max_pages << p.page_shift, out_len = p.out_max_pages << p.page_shift;
        len = min(max(raw_len, 0), max_len);
        first = min(max(raw_first, 0), out_len);
        count = min(min(max(raw_count, 0), p.keep_len), out_len - first);
        status = len != raw_len || count != raw_count || first != raw_first ? FA_ERR_SEQ_LEN : 0;
        list = p.keep + (static_cast<long long>(b) * p.heads + (p.heads > 1 ? h : 0)) * p.keep_len;
        table = p.page_table + static_cast<long long>(b) * p.max_pages;
        out_table = p.out_table + static_cast<long long>(b) * p.out_max_pages;
        mask = (1 << p.page_shift) - 1;
    }
    __device__ __forceinline__ void fault(int s) {
        if (!status) status = s;
    }
    // The i-th token to keep, or -1: there is none, or it is not to be moved.
    __device__ __forceinline__ int number(const KeepParams &p, int i) {
        if (i >= count) return -1;
        const int src = __ldg(list + i);
        if (src >= (p.in_place ? first + i : 0) && src < len) return src;
        fault(FA_ERR_INDEX);
        return -1;
    }
    __device__ __forceinline__ void pages(const KeepParams &p, int src, int i, int &page, int &out_page) const {
        page = __ldg(table + (src >> p.page_shift));
        out_page = __ldg(out_table + ((first + i) >> p.page_shift));
    }
    // Where it is and goes to, in elements from a head's first: to -1: nothing to do; from -1: zeros.
    __device__ __forceinline__ void places(const KeepParams &p, int src, int i, int page, int out_page, long long &from,
                                           long long &to) {
        from = to = -1;
        if (out_page < 0 || out_page >= p.num_pages) {
            fault(FA_ERR_PAGE);
            return;
        }
        to = out_page * p.page_stride + ((first + i) & mask) * p.slot_stride;
        if (page < 0 || page >= p.num_pages) {
            fault(FA_ERR_PAGE);
            return;
        }
        from = page * p.page_stride + (src & mask) * p.slot_stride;
        if (from == to) to = -1;
    }
};

// A CTA moves some columns (16 << lane_shift bytes) of a row (sequence, kv head, keys
// or values) in the order of the list, a batch of 256 >> lane_shift tokens after another, a thread 16
// bytes of one token.  kAhead batches are on their way in shared memory ahead of the one that is
// written, and the places of 256 tokens at a time, a token a thread, ahead of those: a token's
// number, its pages and itself are loads that wait for one another.
constexpr int kAhead = 7;
constexpr int kPlaces = 4;  // lots of 256 places
constexpr int kKeepSmem = (kAhead + 1 + kPlaces) * kKeepThreads * 16;

__global__ void __launch_bounds__(kKeepThreads, 4) keep_rows_kernel(const KeepParams p, const int lane_shift) {
    extern __shared__ __align__(16) uint8_t smem[];
    uint4 *data = reinterpret_cast<uint4 *>(smem) + threadIdx.x;  // [stage][thread]
    longlong2 *places = reinterpret_cast<longlong2 *>(smem + (kAhead + 1) * kKeepThreads * 16);  // [lot][token]: from, to
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    const int slices = p.chunks >> lane_shift, slice = blockIdx.x % slices, pair = blockIdx.x / slices;
    const int h = pair / 2 % p.Hkv, b = pair / 2 / p.Hkv;
    const int chunk = (slice << lane_shift) + (threadIdx.x & ((1 << lane_shift) - 1));
    const int token = threadIdx.x >> lane_shift, each = kKeepThreads >> lane_shift;  // of a batch
    uint16_t *base = (pair & 1 ? p.v_pages : p.k_pages) + h * p.head_stride + chunk * 8;
    KeepRow r(p, b, h);
    const int batches = (r.count + each - 1) / each;
    int src1 = -1, src0 = -1, page0 = 0, out_page0 = 0;
    auto number = [&](int lot) { src1 = r.number(p, lot * kKeepThreads + static_cast<int>(threadIdx.x)); };
    auto pages = [&](int lot) {
        src0 = src1;
        if (src0 >= 0) r.pages(p, src0, lot * kKeepThreads + threadIdx.x, page0, out_page0);
    };
    auto publish = [&](int lot) {
        longlong2 at = make_longlong2(-1, -1);
        if (src0 >= 0) r.places(p, src0, lot * kKeepThreads + threadIdx.x, page0, out_page0, at.x, at.y);
        places[lot % kPlaces * kKeepThreads + threadIdx.x] = at;
    };
    // batch n lies in lot n >> lane_shift
    auto place = [&](int n) { return places[(n >> lane_shift) % kPlaces * kKeepThreads + (n & ((1 << lane_shift) - 1)) * each + token]; };
    auto fetch = [&](int n) {  // (always one group of copies, empty or not)
        if (n < batches) {
            const longlong2 at = place(n);
            uint4 *to = data + n % (kAhead + 1) * kKeepThreads;
            if (at.x >= 0 && at.y >= 0)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(base + at.x) : "memory");
            else
                *to = make_uint4(0, 0, 0, 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    number(0);
    pages(0);
    number(1);
    for (int lot = 0; lot < 2; ++lot) {
        publish(lot);
        pages(lot + 1);
        number(lot + 2);
    }
    __syncthreads();
    for (int n = 0; n < kAhead; ++n) fetch(n);  // (of lots 0 and 1)
    for (int n = 0; n < batches; ++n) {
        // The first batch of lot l: lot l + 2 is published in the place of lot l - 2, and read behind the next
        // barrier (batch n + kAhead is of lot l + 1 at most).
        if ((n & ((1 << lane_shift) - 1)) == 0) {
            const int lot = (n >> lane_shift) + 2;
            publish(lot);
            pages(lot + 1);
            number(lot + 2);
        }
        fetch(n + kAhead);
        // Batch n is here, the other threads' too: what is written now holds none of the tokens still on their way
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
        __syncthreads();
        const long long to = place(n).y;
        if (to >= 0) *reinterpret_cast<uint4 *>(base + to) = data[n % (kAhead + 1) * kKeepThreads];
    }
    if (r.status && slice == 0) record_status(&g_evict_status, r.status);
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
    // CTAs per row: as few as hold it, more where rows leave SMs idle
    auto tokens = [&](int size) { return ((a.weights_len + size - 1LL) / size + kSelThreads - 1) / kSelThreads * kSelThreads; };
    int size = 1;
    while (size < kMaxCluster && (tokens(size) > kHeld || (tokens(size) > 2048 && rows * size < dev.num_sms))) size *= 2;
    const bool holds = tokens(size) <= kHeld;
    const auto kernel = holds ? select_kernel<true> : select_kernel<false>;
    static std::atomic<bool> ready[kMaxDevices];
    if (!ready[dev.device].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld * 4);
        if (e != cudaSuccess) return cuda_fail(e);
        ready[dev.device].store(true, std::memory_order_release);
    }
    const SelectParams p = {a.weights, a.seq_lens, a.keep, a.counts, a.kept, a.heads, a.weights_len, a.budget, a.sink, a.recent};
    Launch cfg(static_cast<unsigned>(rows * size), kSelThreads, holds ? tokens(size) * 4 : 0, size > 1 ? size : 0, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, kernel, p, size);
    return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

int launch_keep(const KeepLaunch &a, const DeviceInfo &dev, cudaStream_t stream) {
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
    const long long rows = 2LL * a.B * p.Hkv;
    // 16-byte pieces of a token side by side, in as few slices of the row as give every SM a CTA, or four where
    // lists are long and the copies in flight set the rate (8 sequences, 8 heads of 128: 64 tokens 2.8 us with 256
    // CTAs, 3.6 with 512; 8192 of 32768 tokens 101 and 93)
    int lane_shift = p.chunks == 16 ? 4 : 3;
    while (lane_shift > 2 && rows * (p.chunks >> lane_shift) < (a.keep_len > 1024 ? 4LL : 1LL) * dev.num_sms) --lane_shift;
    Launch cfg(static_cast<unsigned>(rows * (p.chunks >> lane_shift)), kKeepThreads, kKeepSmem, 0, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg.c, keep_rows_kernel, p, lane_shift);
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
