// fa_paged_rows.cuh -- the arithmetic of up to 64 query rows against 64-key tiles
// of K and V in shared memory, in warp matrix products: what paged_rows_kernel and
// paged_cluster_kernel have in common.
//
// Four consumer warps split a tile by row tiles of 16 (RT of them) and by keys
// (4 / RT groups).  Each keeps its own m, l and O for its 16 rows and its keys;
// write() joins the key groups at the end of a unit.
#pragma once

#include "fa_paged.cuh"

namespace fa {

constexpr int kConsumers = 4;
constexpr int kPagedThreads = 32 * (kConsumers + 1);  // and a producer warp
constexpr int kTile = 64;        // keys of a tile
constexpr int kJoinCols = 32;    // columns per pass of the join between key groups, for 16 rows

// Four 8x8 16-bit matrices from shared memory; lane l gives the 16-byte row l % 8 of matrix l / 8.
__device__ __forceinline__ void ldmatrix4(uint32_t saddr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(saddr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t saddr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(saddr)
                 : "memory");
}
// C (16 x 8, fp32) += A (16 x 16) B (16 x 8), 16-bit operands.
template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int RT, bool BF16>
struct PagedRows {
    static constexpr float kTau = 8.0f;          // lazy-rescale threshold, log2 units
    static constexpr int KG = kConsumers / RT;   // key groups
    static constexpr int NK = kTile / KG;        // keys of a tile per warp
    static constexpr int kSlab = kTile * 128;    // 64 keys x 64 columns
    static constexpr int kOperand = (D / 64) * kSlab;  // a K or V tile
    static constexpr int kJoinBytes = KG > 1 ? kConsumers * 16 * (kJoinCols * 4 + 8) : 0;
    // fp16 weights keep 7 bits of headroom below the largest (2^kTau), which
    // pushes the smallest ones that do not vanish down to 2^-31 of the reference
    static constexpr float kShift = BF16 ? 0.f : 7.f;

    int lane, quad, qrow, rw, kw;  // lane = 4 qrow + quad; row tile, key group
    uint32_t qf[D / 16][4];
    float o[D / 8][4];
    // rows qrow and qrow + 8 of the row tile: running maximum and sum, and kShift - m
    // once a key has been seen (0 before, when masked scores of -inf still give weight 0)
    float m0, m1, l0, l1, n0, n1;
    uint32_t joins;
    uint32_t loads;  // of begin() or tile(): a register of each, or-ed

    __device__ __forceinline__ explicit PagedRows(int warp, int lane_)
        : lane(lane_), quad(lane_ & 3), qrow(lane_ >> 2), rw(warp % RT), kw(warp / RT), joins(0) {}

    // A new unit: its query rows, `pitch` bytes apart at shared address q.
    __device__ __forceinline__ void begin(uint32_t q, int pitch) {
        const uint32_t addr = q + (rw * 16 + (lane & 7) + ((lane >> 3) & 1) * 8) * pitch + (lane >> 4) * 16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) ldmatrix4(addr + kk * 32, qf[kk]);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = n0 = n1 = 0.f;
        loads = 0;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) loads |= qf[kk][0];
    }

    // True never, and known only when the shared-memory loads of begin() or tile() have
    // arrived in every lane: what hands their place back hangs on it.  (zero: a mask that
    // is zero, which the compiler does not know.)  A barrier arrival alone comes after the
    // loads' issue, not their end, and nothing else binds the copy engine that writes the
    // place next: without this, most calls of many short units of 32 rows took a query
    // row, and a few in thousands a piece of a V tile, from the data that came behind.
    __device__ __forceinline__ bool loads_pending(uint32_t zero) const {
        return __any_sync(0xffffffffu, (loads & zero) != 0);
    }

    // One tile: K at shared address kt, V behind it (128-byte swizzled slabs of 64
    // columns); the rows see keys up to lim0 and lim1 of the tile, of which the first
    // `keys` exist.
    __device__ __forceinline__ void tile(uint32_t kt, int lim0, int lim1, int keys, float scale_log2) {
        lim0 -= kw * NK;
        lim1 -= kw * NK;
        products(kt, keys, scale_log2, min(lim0, lim1) < NK - 1, [&](int key) { return key > lim0; },
                 [&](int key) { return key > lim1; });
    }
    // The same where the rows see the keys whose bits are set.
    __device__ __forceinline__ void tile_seen(uint32_t kt, uint64_t see0, uint64_t see1, int keys, float scale_log2) {
        constexpr uint64_t kAll = NK == 64 ? ~0ull : (1ull << (NK & 63)) - 1;
        see0 >>= kw * NK;
        see1 >>= kw * NK;
        products(kt, keys, scale_log2, (see0 & see1 & kAll) != kAll, [&](int key) { return !(see0 >> key & 1); },
                 [&](int key) { return !(see1 >> key & 1); });
    }

    // hidden0 and hidden1: whether this thread's two rows do not see one of its group's keys, asked
    // where `tail` says that any is hidden.
    template <typename Hidden0, typename Hidden1>
    __device__ __forceinline__ void products(uint32_t kt, int keys, float scale_log2, bool tail, Hidden0 hidden0,
                                             Hidden1 hidden1) {
        kt += kw * NK * 128;
        const uint32_t vt = kt + kOperand;
        keys -= kw * NK;
        // K fragments: lane = key row lane % 8 of an 8-key block, 16-byte chunk lane / 8 of four
        const uint32_t k_row = (lane & 7) * 128;
        // V fragments (transposed): lane = key row of a 16-key block, chunk lane / 16 of two
        const uint32_t v_row = ((lane & 7) + ((lane >> 3) & 1) * 8) * 128;
        // ---- S = Q K^T
        float s[NK / 8][4];
#pragma unroll
        for (int nb = 0; nb < NK / 8; ++nb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nb][e] = 0.f;
#pragma unroll
            for (int k2 = 0; k2 < D / 32; ++k2) {
                uint32_t kb[4];
                const int chunk = (k2 & 1) * 4 + (lane >> 3);
                ldmatrix4(kt + (k2 >> 1) * kSlab + nb * 1024 + k_row + ((chunk ^ (lane & 7)) << 4), kb);
                mma_16816<BF16>(s[nb], qf[2 * k2], kb[0], kb[1]);
                mma_16816<BF16>(s[nb], qf[2 * k2 + 1], kb[2], kb[3]);
            }
        }
        // ---- scores in log2 units, masked; the tile's row maxima
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < NK / 8; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int key = nb * 8 + quad * 2 + e;
                s[nb][e] *= scale_log2;
                s[nb][2 + e] *= scale_log2;
                if (tail) {
                    if (hidden0(key)) s[nb][e] = -INFINITY;
                    if (hidden1(key)) s[nb][2 + e] = -INFINITY;
                }
                x0 = fmaxf(x0, s[nb][e]);
                x1 = fmaxf(x1, s[nb][2 + e]);
            }
        __syncwarp();
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
        }
        const bool up0 = x0 > m0 + kTau, up1 = x1 > m1 + kTau;
        if (__any_sync(0xffffffffu, up0 || up1)) {
            float a0 = 1.f, a1 = 1.f;
            if (up0) { a0 = ex2_approx(m0 - x0); m0 = x0; n0 = kShift - x0; }
            if (up1) { a1 = ex2_approx(m1 - x1); m1 = x1; n1 = kShift - x1; }
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                o[i][0] *= a0;
                o[i][1] *= a0;
                o[i][2] *= a1;
                o[i][3] *= a1;
            }
        }
        // ---- weights 2^(s - m), rounded to the 16-bit type of V; l adds the rounded ones,
        // so a row that one key dominates returns that key's value row
        uint32_t pf[NK / 16][4];
#pragma unroll
        for (int nb = 0; nb < NK / 8; ++nb) {
            const uint32_t lo = pack2t<BF16>(ex2_approx(s[nb][0] + n0), ex2_approx(s[nb][1] + n0));
            const uint32_t hi = pack2t<BF16>(ex2_approx(s[nb][2] + n1), ex2_approx(s[nb][3] + n1));
            float e0 = 0.f, e1 = 0.f;
            add_pair16<BF16>(l0, e0, lo);
            add_pair16<BF16>(l1, e1, hi);
            l0 += e0;
            l1 += e1;
            pf[nb >> 1][(nb & 1) * 2] = lo;
            pf[nb >> 1][(nb & 1) * 2 + 1] = hi;
        }
        loads = 0;  // (those of K are through: the weights come from them)
        // ---- O += P V.  Slots behind the last key hold anything at all, so their V
        // rows are read as zero (0 x NaN would be NaN).
#pragma unroll
        for (int kb = 0; kb < NK / 16; ++kb) {
            uint32_t mask0 = 0xffffffffu, mask1 = 0xffffffffu;
            if (keys < NK) {
                const int a = kb * 16 + quad * 2;
                mask0 = (a < keys ? 0xffffu : 0u) | (a + 1 < keys ? 0xffff0000u : 0u);
                mask1 = (a + 8 < keys ? 0xffffu : 0u) | (a + 9 < keys ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                uint32_t vb[4];
                const int chunk = (c & 3) * 2 + (lane >> 4);
                ldmatrix4_trans(vt + (c >> 2) * kSlab + kb * 2048 + v_row + ((chunk ^ (lane & 7)) << 4), vb);
                loads |= vb[0];
                mma_16816<BF16>(o[2 * c], pf[kb], vb[0] & mask0, vb[1] & mask1);
                mma_16816<BF16>(o[2 * c + 1], pf[kb], vb[2] & mask0, vb[3] & mask1);
            }
        }
    }

    // The unit's sums: l over the four lanes that share a row, m without the headroom.
    __device__ __forceinline__ void end() {
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, off);
            l1 += __shfl_xor_sync(0xffffffffu, l1, off);
        }
        m0 -= kShift;  // (-inf stays)
        m1 -= kShift;
    }

    // Hands out the unit's first `rows` rows: emit(row, row_of(row), column, columns, m, l) with
    // two or four unnormalised columns at a time.  join: kJoinBytes of shared memory;
    // j_full, j_empty: barriers for KG warps, one per row tile.  False when a wait ran out.
    template <typename RowOf, typename Emit>
    __device__ __forceinline__ bool write(int rows, uint8_t *join, uint64_t *j_full, uint64_t *j_empty,
                                          volatile int *abort_flag, RowOf row_of, Emit emit) {
        bool ok = true;
        if constexpr (KG == 1) {
            auto half = [&](int r, float m, float l, auto which) {
                constexpr int H = decltype(which)::value;
                if (r >= rows) return;
                const auto row = row_of(r);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    float a[2] = {o[i][2 * H], o[i][2 * H + 1]};
                    emit(r, row, i * 8 + quad * 2, a, m, l);
                }
            };
            half(rw * 16 + qrow, m0, l0, std::integral_constant<int, 0>{});
            half(rw * 16 + qrow + 8, m1, l1, std::integral_constant<int, 1>{});
        } else {
            // join the KG key groups of row tile rw through shared memory: as many columns per
            // pass as the unit's rows leave room for
            float *buf = reinterpret_cast<float *>(join) + rw * KG * 16 * kJoinCols;
            float2 *buf_ml = reinterpret_cast<float2 *>(join + kConsumers * 16 * kJoinCols * 4) + rw * KG * 16;
            auto passes = [&](auto used) {
                constexpr int RU = decltype(used)::value;    // rows that exist, rounded up
                constexpr int C = kJoinCols * 16 / RU < D ? kJoinCols * 16 / RU : D;  // columns per pass
                constexpr int kCells = RU * C / 4, kPer = (kCells + KG * 32 - 1) / (KG * 32);
                const int cell = kw * 32 + lane;
                auto cell_row = [&](int i) { return (cell + i * KG * 32) / (C / 4); };
                const int cell_col = cell % (C / 4) * 4;
                // 16-byte chunks of a row change places by row, against bank conflicts
                auto at = [&](int g, int r, int col) {
                    return buf + (g * RU + r) * C + (((col >> 2) ^ (r & 7)) << 2) + (col & 3);
                };
                decltype(row_of(0)) row[kPer];
                bool live[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    live[i] = cell + i * KG * 32 < kCells && rw * 16 + cell_row(i) < rows;
                    row[i] = row_of(rw * 16 + cell_row(i));
                }
#pragma unroll
                for (int pass = 0; pass < D / C; ++pass) {
                    if (joins > 0 && !lanes_wait(j_empty + rw, (joins - 1) & 1, abort_flag)) { ok = false; return; }
#pragma unroll
                    for (int i = 0; i < C / 8; ++i) {
                        const int nb = pass * (C / 8) + i, col = i * 8 + quad * 2;
                        if (RU >= 8 || qrow < RU)
                            *reinterpret_cast<float2 *>(at(kw, qrow, col)) = make_float2(o[nb][0], o[nb][1]);
                        if constexpr (RU == 16)
                            *reinterpret_cast<float2 *>(at(kw, qrow + 8, col)) = make_float2(o[nb][2], o[nb][3]);
                    }
                    if (pass == 0 && quad == 0) {
                        buf_ml[kw * 16 + qrow] = make_float2(m0, l0);
                        buf_ml[kw * 16 + qrow + 8] = make_float2(m1, l1);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(j_full + rw);
                    if (!lanes_wait(j_full + rw, joins & 1, abort_flag)) { ok = false; return; }
                    ++joins;
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        if (!live[i]) continue;
                        const int r = cell_row(i);
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
                        float M = -INFINITY, Ls = 0.f;
#pragma unroll
                        for (int g = 0; g < KG; ++g) M = fmaxf(M, buf_ml[g * 16 + r].x);
#pragma unroll
                        for (int g = 0; g < KG; ++g) {
                            const float4 v = *reinterpret_cast<const float4 *>(at(g, r, cell_col));
                            const float2 ml = buf_ml[g * 16 + r];
                            const float w = ex2_from(ml.x, M);
                            Ls = fmaf(w, ml.y, Ls);
                            acc[0] = fmaf(w, v.x, acc[0]);
                            acc[1] = fmaf(w, v.y, acc[1]);
                            acc[2] = fmaf(w, v.z, acc[2]);
                            acc[3] = fmaf(w, v.w, acc[3]);
                        }
                        emit(rw * 16 + r, row[i], pass * C + cell_col, acc, M, Ls);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(j_empty + rw);
                }
            };
            const int used = rows - rw * 16;
            if (RT == 1 && used <= 8) passes(std::integral_constant<int, 8>{});
            else passes(std::integral_constant<int, 16>{});
        }
        return ok;
    }
};

}  // namespace fa
