"""How the threads of a CTA that weighs cached tokens find its range (csrc/fa_weigh_cut.cuh compiled for the host, no GPU): batches
of more sequences than threads, sequences without steps among them, and ranges that cover all steps once."""
import os
import random
import subprocess

import pytest

from attention_forward_prefill_gb300 import build

HARNESS = r"""
#include <algorithm>
#include <cstdio>
#include <vector>
#define __device__
#define __forceinline__ inline
struct int4 { int x, y, z, w; };
using std::max;
using std::min;
inline int __ldg(const int *p) { return *p; }
#include "fa_weigh_cut.cuh"
using namespace fa;

int main() {
    int B, Hkv, in_place, tiles, threads, ctas;
    while (std::scanf("%d %d %d %d %d %d", &B, &Hkv, &in_place, &tiles, &threads, &ctas) == 6) {
        std::vector<int> lens(B), cu(B + 1);
        for (int &n : lens) if (std::scanf("%d", &n) != 1) return 1;
        for (int &n : cu) if (std::scanf("%d", &n) != 1) return 1;
        WeighParams p{};
        p.seq_lens = lens.data();
        p.cu_q = cu.data();
        p.B = B;
        p.Hkv = Hkv;
        p.causal = 1;
        p.in_place = in_place;
        p.max_len = 1 << 20;
        p.total_q = cu[B];
        p.max_q = 1 << 30;
        p.tile_tokens = 16;
        // (weigh_rows_kernel's steps are 128 keys)
        auto steps = [&](const WeighSeq &s) { return tiles ? weigh_head_steps(p, s) : weigh_stays(p, s) ? 0LL : (s.len + 127LL) / 128; };
        std::vector<long long> before(threads + 1, 0);
        bool bad = false;
        for (int t = 0; t < threads; ++t) before[t + 1] = before[t] + weigh_sum(p, weigh_share(p, t, threads), steps, bad);
        const long long W = before[threads];
        std::printf("W %lld %d\n", W, bad);
        for (int b = 0; b < B; ++b) std::printf("%lld ", steps(weigh_seq(p, b)) * Hkv);
        std::printf("\n");
        for (int c = 0; c < ctas; ++c) {
            const WeighStart range = weigh_range(W, c, ctas, tiles ? kWeighUnit + 1 : 1);
            int found = 0;
            WeighStart st{};
            for (int t = 0; t < threads; ++t) {
                st.b = -1;
                WeighStart one = st;
                weigh_find(p, range, weigh_share(p, t, threads), before[t], before[t + 1] - before[t], steps, one);
                if (one.b < 0) continue;
                ++found;
                std::printf("%lld %lld %d %d %lld\n", range.first, range.end, range.G, one.b, one.rem);
            }
            if (!found) std::printf("%lld %lld %d none 0\n", range.first, range.end, range.G);
        }
        std::printf("E\n");
    }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("weigh_plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(HARNESS)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-Wall", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)

    def run(lens, cu, Hkv, in_place, tiles, threads, ctas):
        text = f"{len(lens)} {Hkv} {int(in_place)} {int(tiles)} {threads} {ctas} {' '.join(map(str, lens))} {' '.join(map(str, cu))}\n"
        return subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split("E\n")[0].splitlines()
    return run


@pytest.mark.parametrize("tiles,threads,ctas", [(False, 256, 304), (True, 640, 152)], ids=["rows", "tiles"])
@pytest.mark.parametrize("B", [1, 2, 255, 256, 257, 513, 640, 641, 1500, 5000])
@pytest.mark.parametrize("kind", ["full", "holes", "idle in place", "one", "none"])
def test_every_range_is_found_once(plan, tiles, threads, ctas, B, kind):
    rng = random.Random(B + threads)
    lens = [rng.randint(1, 900) for _ in range(B)]
    counts = [rng.randint(1, 40) for _ in range(B)]
    if kind == "holes":
        lens = [n if rng.random() < 0.4 else 0 for n in lens]
    elif kind == "idle in place":
        counts = [n if rng.random() < 0.3 else 0 for n in counts]
    elif kind == "one":
        lens = [0] * B
        lens[rng.randrange(B)] = 70000
    elif kind == "none":
        lens = [0] * B
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    Hkv, in_place = rng.randint(1, 8), kind == "idle in place"
    head, steps, *ranges = plan(lens, cu, Hkv, in_place, tiles, threads, ctas)
    steps = [int(x) for x in steps.split()]
    W = sum(steps)
    assert head.split() == ["W", str(W), "0"] and len(ranges) == ctas
    for n, c, s in zip(lens, counts, steps):
        assert (s > 0) == (n > 0 and not (in_place and c == 0))
    used, at, b, into = max(1, min(ctas, W // (3 if tiles else 1))), 0, 0, 0
    for c, line in enumerate(ranges):
        first, end, G, found, rem = line.split()
        assert (int(first), int(G)) == (at if c < used else W, used)
        if int(first) == int(end):
            assert found == "none"
            continue
        while at >= into + steps[b]:
            into, b = into + steps[b], b + 1
        assert (int(found), int(rem)) == (b, at - into)
        at = int(end)
        assert at - int(first) in (W // used, W // used + 1)
    assert at == W
