// fa_weigh_cut.cuh -- how the weighing of cached tokens is cut into equal ranges of work.
// Plain arithmetic: tests/test_weigh_cut_host.py and tests/test_weigh_plan_host.py compile this file for the host.
//
// weigh_tiles_kernel.  A sequence's n query tokens give each kv head n * G query rows, in
// chunks of tile_tokens whole tokens (kWeighRows rows at most).  A unit = (sequence, kv head, 256
// keys); it costs kWeighUnit steps for its start and end and one for every chunk with rows that
// see any of its keys: the chunks from the first such to the last.  The W steps of the call, in
// the order (sequence, kv head, keys), are cut into one equal range per CTA, by every CTA for
// itself from the lengths on the device.  A range has the chunks whose steps lie in it; the sums
// of a unit that ranges cut are added by weigh_join_kernel in the order of the CTAs.
#pragma once

#include <cstdint>

namespace fa {

struct WeighParams {
    const uint16_t *q, *k_pages;
    const float *lse, *in;
    float *out;
    long long page_stride, head_stride, slot_stride;
    const int *page_table, *seq_lens, *cu_q;
    int B, Hq, Hkv, G, total_q, max_q, nq_each;
    int max_pages, max_len, num_pages, page_shift, len;  // len: of a row of weights
    int causal, in_place;  // in_place: in is out
    float scale_log2, decay;
    // weigh_tiles_kernel
    int tile_tokens;
    float *part;  // [gridDim.x][2][256]: sums of the unit that a CTA continues, and of the one that it leaves open
    int4 *open;   // [gridDim.x]: the latter: last CTA, sequence, kv head, first key; or last CTA -1
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

// Without query tokens a sequence's keys and pages are not asked for, and in place there is nothing to do:
// no steps.  (32 sequences of 200 to 8192 tokens, one of them with a token, 32 heads over 8, d = 128: 5 us in place, 20
// into other weights, 41 with all keys loaded.)
__device__ __forceinline__ bool weigh_stays(const WeighParams &p, const WeighSeq &s) {
    return s.nq == 0 && p.in_place;
}

constexpr int kWeighKeys = 256;  // of a unit
constexpr int kWeighRows = 128;  // of a chunk, at most
constexpr int kWeighUnit = 2;

// The first query token that sees key k: all of them where k lies in front of the query tokens.
__device__ __forceinline__ int weigh_first_token(const WeighParams &p, const WeighSeq &s, int k) {
    return p.causal ? min(max(k - (s.len - s.nq), 0), s.nq) : 0;
}
__device__ __forceinline__ int weigh_units(const WeighParams &p, const WeighSeq &s) {
    return weigh_stays(p, s) ? 0 : (s.len + kWeighKeys - 1) / kWeighKeys;
}
// Chunks of a sequence, at least one: a unit without rows still writes its keys' weights.
__device__ __forceinline__ int weigh_chunks(const WeighParams &p, const WeighSeq &s) {
    return max(1, (s.nq + p.tile_tokens - 1) / p.tile_tokens);
}
// The first chunk of unit u with rows that see its keys.
__device__ __forceinline__ int weigh_first_chunk(const WeighParams &p, const WeighSeq &s, int chunks, int u) {
    return min(weigh_first_token(p, s, u * kWeighKeys) / p.tile_tokens, chunks - 1);
}
// Units of a sequence whose first key all of its tokens see.
__device__ __forceinline__ int weigh_whole(const WeighParams &p, const WeighSeq &s) {
    const int units = weigh_units(p, s), past = s.len - s.nq;
    return !p.causal ? units : (past < 0 ? 0 : min(units, past / kWeighKeys + 1));
}
// Steps of one kv head of a sequence.
__device__ __forceinline__ long long weigh_head_steps(const WeighParams &p, const WeighSeq &s) {
    const int units = weigh_units(p, s), chunks = weigh_chunks(p, s), whole = weigh_whole(p, s);
    long long sum = static_cast<long long>(units) * (kWeighUnit + chunks);
    for (int u = whole; u < units; ++u) sum -= weigh_first_chunk(p, s, chunks, u);
    return sum;
}

// A CTA's range [first, end) of the W steps; it starts rem steps into sequence b.
struct WeighStart {
    long long W, first, end, rem;
    int b, G;  // G: CTAs with work
};

// Thread `tid` of NT adds up the steps of sequences [b0, b1).
struct WeighShare {
    int b0, b1;
};
__device__ __forceinline__ WeighShare weigh_share(const WeighParams &p, int tid, int NT) {
    const int per = (p.B + NT - 1) / NT, b0 = min(tid * per, p.B);
    return {b0, min(b0 + per, p.B)};
}
template <typename StepsOf>
__device__ __forceinline__ long long weigh_sum(const WeighParams &p, const WeighShare &x, StepsOf steps_of, bool &bad) {
    long long sum = 0;
    for (int b = x.b0; b < x.b1; ++b) {
        sum += steps_of(weigh_seq(p, b)) * p.Hkv;
        bad |= weigh_seq_bad(p, b);
    }
    return sum;
}
// What CTA c of `ctas` gets of W steps; no more CTAs get any than there are lots of `least` steps.
__device__ __forceinline__ WeighStart weigh_range(long long W, int c, int ctas, int least) {
    WeighStart st;
    st.W = W;
    st.G = static_cast<int>(min(static_cast<long long>(ctas), max(W / least, 1LL)));
    st.first = c < st.G ? c * W / st.G : W;
    st.end = c < st.G ? (c + 1) * W / st.G : W;
    return st;
}
// Where the range starts, if it is in this thread's share: `mine` steps behind `before` others.
template <typename StepsOf>
__device__ __forceinline__ void weigh_find(const WeighParams &p, const WeighStart &range, const WeighShare &x, long long before,
                                           long long mine, StepsOf steps_of, WeighStart &st) {
    if (range.first >= range.end || range.first < before || range.first >= before + mine) return;
    long long rem = range.first - before;
    int b = x.b0;
    for (; b < x.b1 - 1; ++b) {
        const long long n = steps_of(weigh_seq(p, b)) * p.Hkv;
        if (rem < n) break;
        rem -= n;
    }
    st.b = b;
    st.rem = rem;
}

// The CTA whose range holds `step`.
__device__ __forceinline__ int weigh_cta_of(long long step, long long W, int G) {
    long long c = ((step + 1) * G - 1) / W;
    if (c >= G) c = G - 1;
    while (c > 0 && c * W / G > step) --c;
    while (c + 1 < G && (c + 1) * W / G <= step) ++c;
    return static_cast<int>(c);
}

// Chunks [c0, c1) of unit u of kv head h of sequence b.
struct WeighPiece {
    WeighSeq s;
    int b, h, u, c0, c1;
    bool opens, closes;      // has the unit's first chunk, its last
    long long to_last;       // opens and not closes: steps from the range's end to the unit's last chunk
};

// Walks a CTA's pieces in order.
struct WeighCursor {
    WeighSeq s;
    int b, h, u, units, chunks, v;  // v: the next step of unit u
    long long left;

    __device__ __forceinline__ void sequence(const WeighParams &p, int at) {
        b = at;
        s = weigh_seq(p, b);
        units = weigh_units(p, s);
        chunks = weigh_chunks(p, s);
    }
    __device__ __forceinline__ void begin(const WeighParams &p, const WeighStart &st) {
        left = st.end - st.first;
        if (left <= 0) return;
        sequence(p, st.b);
        const long long per_head = max(weigh_head_steps(p, s), 1LL);
        h = static_cast<int>(st.rem / per_head);
        long long rem = st.rem - h * per_head;
        const int whole = weigh_whole(p, s), cost = kWeighUnit + chunks;
        u = static_cast<int>(min(rem / cost, static_cast<long long>(whole)));
        rem -= static_cast<long long>(u) * cost;
        for (; u >= whole && u < units - 1; ++u) {
            const int c = cost - weigh_first_chunk(p, s, chunks, u);
            if (rem < c) break;
            rem -= c;
        }
        v = static_cast<int>(rem);
    }
    // The next piece with chunks; false when the range is used up.
    __device__ __forceinline__ bool next(const WeighParams &p, WeighPiece &x) {
        while (left > 0) {
            const int first = weigh_first_chunk(p, s, chunks, u), total = kWeighUnit + chunks - first;
            const int end = static_cast<int>(min(static_cast<long long>(total), v + left));
            x.c0 = first + max(v - kWeighUnit, 0);
            x.c1 = first + max(end - kWeighUnit, 0);
            const bool some = x.c1 > x.c0;
            if (some) {
                x.s = s;
                x.b = b;
                x.h = h;
                x.u = u;
                x.opens = x.c0 == first;
                x.closes = x.c1 == chunks;
                x.to_last = total - 1 - end;
            }
            left -= end - v;
            v = 0;
            if (left > 0 && ++u == units) {
                u = 0;
                if (++h == p.Hkv) {
                    h = 0;
                    do {  // steps are left, so a later sequence has units
                        sequence(p, b + 1);
                    } while (units == 0 && b + 1 < p.B);
                    if (units == 0) left = 0;
                }
            }
            if (some) return true;
        }
        return false;
    }
};

}  // namespace fa
