"""How a paged call is cut (csrc/fa_paged_cut.cuh compiled for the host, no GPU).  The two passes of a shared-prefix call
share the SMs: each adds up its own steps and the other one's, from the lengths, and both have to come to the same
split.  A call runs in clusters only where the longest sequence that its table allows stays short."""
import os
import random
import subprocess

import pytest

from attention_forward_prefill_gb300 import build

HARNESS = r"""
// arguments: none, shared-prefix calls; "form", sizes of calls that may run in clusters
#include <algorithm>
#include <cstdio>
#include <vector>
#define __device__
#define __forceinline__ inline
struct int2 { int x, y; };
struct int4 { int x, y, z, w; };
using std::max;
using std::min;
inline int __ldg(const int *p) { return *p; }
#include "fa_paged_cut.cuh"
using namespace fa;

struct Pass {
    PagedParams p{};
    PagedPlan plan;
};

// as the launch of a pass of nq_each tokens for each of B sequences
Pass pass_of(int B, int nq_each, int G, int Hkv, int d, const std::vector<int> &lens, int max_len, int first, int sms) {
    Pass x;
    x.plan = plan_paged(nq_each, G, d);
    PagedParams &p = x.p;
    p.seq_lens = lens.data();
    p.nq_each = p.max_q = nq_each;
    p.B = B;
    p.G = G;
    p.Hkv = Hkv;
    p.max_len = max_len;
    p.block_rows = x.plan.block_rows;
    p.unit_steps = x.plan.unit_steps;
    p.tile_tokens = x.plan.tiles ? x.plan.block_rows / G / 2 : 0;
    p.first = first;
    p.num_sms = sms;
    p.step_ns = paged_step_ns(x.plan, d);
    return x;
}

long long steps_of(const Pass &x, int d) {
    long long sum = 0;
    for (int b = 0; b < x.p.B; ++b) {
        const SeqView s = paged_seq(x.p, b);
        sum += (!x.plan.tiles ? paged_head_steps<RowsCut>(x.p, s)
                : d == 64     ? paged_head_steps<TilesCut<64>>(x.p, s)
                              : paged_head_steps<TilesCut<128>>(x.p, s)) * x.p.Hkv;
    }
    return sum;
}

long long peer_of(const Pass &x) {
    long long sum = 0;
    for (int b = 0; b < x.p.peer_B; ++b) sum += paged_peer_steps(x.p, b);
    return sum * x.p.Hkv;
}

int main(int argc, char **) {
    if (argc > 1) {
        long long units, max_len, prefix;
        int rows, d, sms;
        while (std::scanf("%d %d %lld %lld %lld %d", &rows, &d, &units, &max_len, &prefix, &sms) == 6)
            std::printf("%d\n", paged_cluster_size(plan_paged(1, rows, d), d, units, max_len, prefix, sms));
        return 0;
    }
    int B, G, Hkv, d, prefix, max_len, sms;
    while (std::scanf("%d %d %d %d %d %d %d", &B, &G, &Hkv, &d, &prefix, &max_len, &sms) == 7) {
        std::vector<int> front{prefix}, lens(B);
        for (int &n : lens)
            if (std::scanf("%d", &n) != 1) return 1;
        Pass a = pass_of(1, B, G, Hkv, d, front, 1 << 20, 1, sms), b = pass_of(B, 1, G, Hkv, d, lens, max_len, 0, sms);
        paged_set_peer(a.p, b.p, b.plan);
        paged_set_peer(b.p, a.p, a.plan);
        const long long wa = steps_of(a, d), wb = steps_of(b, d);
        std::printf("%lld %lld %lld %lld %d %d\n", wa, peer_of(b), wb, peer_of(a), paged_first_sms(a.p, wa, peer_of(a)),
                    paged_first_sms(b.p, wb, peer_of(b)));
    }
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    at = tmp_path_factory.mktemp("split")
    (at / "split.cpp").write_text(HARNESS)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-I", build.CSRC, str(at / "split.cpp"), "-o",
                    str(at / "split")], check=True)

    def run(cases, *how):
        if how:
            out = subprocess.run([str(at / "split"), *how], input="\n".join(" ".join(map(str, c)) for c in cases),
                                 capture_output=True, text=True, check=True).stdout
            return [int(line) for line in out.split()]
        text = "\n".join(" ".join(map(str, [B, G, Hkv, d, prefix, max_len, sms, *lens]))
                         for B, G, Hkv, d, prefix, max_len, sms, lens in cases)
        out = subprocess.run([str(at / "split")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return run


def tiles(n, keys):
    return max(1, -(-n // keys))


def steps(B, nq, G, Hkv, d, lens):
    """Steps of a pass, counted block by block as csrc/fa_paged_cut.cuh describes them."""
    rows = nq * G
    if rows <= 64 or G > 128:  # warp products: 64 keys, one step each
        block = 16 if rows <= 16 else 32 if rows <= 32 else 64
        return Hkv * sum(-(-rows // block) * (2 + tiles(n, 64)) for n in lens)
    both, one, unit = (3, 2, 5) if d == 64 else (1, 1, 2)
    tokens = 128 // G  # of a query tile, of which a block has two
    cost = [one if at + tokens >= nq else both for at in range(0, nq, 2 * tokens)]
    return Hkv * sum(unit + tiles(n, 128) * c for n in lens for c in cost)


CASES = [(100, 12 // 12, 12, 64, 16000, 4096, 148, [100] * 100), (18, 7, 2, 64, 16000, 4096, 148, [100] * 18),
         (18, 7, 2, 64, 16000, 4096, 152, [100] * 18), (5, 100, 1, 64, 3000, 4096, 152, [0, 900, 64, 65, 4097]),
         (256, 8, 8, 128, 16500, 1024, 152, [i * 4 for i in range(256)]), (1, 1, 1, 64, 0, 16, 2, [0])]


def random_case(rng):
    B, G = rng.choice([1, 2, rng.randint(1, 20), rng.randint(1, 300)]), rng.choice([1, 2, 3, 7, 8, 16, 40, 65, 71, 128, 140])
    max_len = rng.choice([16, 512, 8192])
    lens = [rng.choice([0, 1, rng.randint(-3, max_len + 5), rng.randint(0, max_len)]) for _ in range(B)]
    return (B, G, rng.choice([1, 2, 8]), rng.choice([64, 128]), rng.choice([0, 1, rng.randint(1, 60000)]), max_len,
            rng.choice([2, 148, 152]), lens)


def test_both_passes_come_to_the_same_split(split):
    rng = random.Random(5)
    cases = CASES + [random_case(rng) for _ in range(400)]
    got = split(cases)
    assert len(got) == len(cases)
    for (B, G, Hkv, d, prefix, max_len, sms, lens), (wa, wa_seen, wb, wb_seen, mine, theirs) in zip(cases, got):
        clamped = [min(max(n, 0), max_len) for n in lens]
        assert wa == wa_seen == steps(1, B, G, Hkv, d, [prefix])
        assert wb == wb_seen == steps(B, 1, G, Hkv, d, clamped)
        assert mine == theirs and 1 <= mine <= max(sms - 1, 1)


def test_clusters_are_kept_for_short_sequences_whatever_the_number_of_units(split):
    """No CTA of a cluster may be given more than a few microseconds of tiles in a row: a batch whose units times the
    cluster's size nearly fill the GPU is no exception, as its longest sequence would set the time alone."""
    cases = [(rows, d, units, max_len, prefix, sms) for rows in (1, 8, 16, 32, 64) for d in (64, 128)
             for units in (1, 8, 30, 35, 36, 38, 70, 72, 76, 144, 150, 151, 152, 153, 160, 296, 303, 304, 305, 312)
             for max_len in (16, 64, 200, 1008, 2000, 4112, 8192, 131072) for prefix in (0, 64, 784, 8192, 65536)
             for sms in (148, 152)]
    seen = set()
    for (rows, d, units, max_len, prefix, sms), size in zip(cases, split(cases, "form")):
        if size == 0:
            continue
        seen.add(size)
        in_a_row = -(-(-(-max_len // 64) + -(-prefix // 64)) // size)
        assert in_a_row <= (40 if prefix else 22) and units * size <= 2 * sms
        if rows == 64 and d == 128:
            assert in_a_row <= (10 if prefix else 5)
        if size > 2:  # clusters that all run at once
            assert units * size <= 2 * sms * 20 / 21 + 1
    assert seen == {1, 2, 4, 8}
    # 8 kv heads and a table of 8192 tokens: neighbouring batch sizes take the same form
    assert split([(4, 128, 8 * B, 8192, 0, 152) for B in (9, 18, 19, 20, 37, 38, 39)], "form") == [0] * 7
    assert split([(4, 128, 8 * B, 131072, 0, 152) for B in (1, 19, 38)], "form") == [0] * 3
    # short tables stay in clusters
    assert split([(1, 64, 12, 1008, 0, 152), (1, 64, 48, 64, 784, 152), (42, 64, 32, 4128, 0, 152)], "form") == [8, 4, 8]
    # behind a prefix too, unless its tiles in a row are many
    assert split([(7, 64, 36, 4096, prefix, 152) for prefix in (784, 16000, 65536)], "form") == [8, 8, 0]
