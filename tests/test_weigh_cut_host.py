"""How the weighing of cached tokens is cut (csrc/fa_weigh_cut.cuh compiled for the host, no GPU): every chunk of every unit
belongs to one CTA, the pieces of a unit follow one another in the order of the CTAs, and what a CTA notes of the unit that it
leaves open names the CTA that closes it."""
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
    int B, Hkv, tokens, causal, max_len, ctas;
    while (std::scanf("%d %d %d %d %d %d", &B, &Hkv, &tokens, &causal, &max_len, &ctas) == 6) {
        std::vector<int> lens(B), cu(B + 1);
        for (int &n : lens) if (std::scanf("%d", &n) != 1) return 1;
        for (int &n : cu) if (std::scanf("%d", &n) != 1) return 1;
        WeighParams p{};
        p.seq_lens = lens.data();
        p.cu_q = cu.data();
        p.B = B;
        p.Hkv = Hkv;
        p.causal = causal;
        p.max_len = max_len;
        p.total_q = cu[B];
        p.max_q = 1 << 30;
        p.tile_tokens = tokens;
        std::vector<long long> steps(B);
        long long W = 0;
        for (int b = 0; b < B; ++b) W += steps[b] = weigh_head_steps(p, weigh_seq(p, b)) * Hkv;
        const int used = static_cast<int>(min(static_cast<long long>(ctas), max(W, 1LL)));
        std::printf("W %lld %d\n", W, used);
        for (int c = 0; c < used; ++c) {
            WeighStart st{};
            st.W = W;
            st.G = used;
            st.first = c * W / used;
            st.end = (c + 1) * W / used;
            st.rem = st.first;
            for (st.b = 0; st.b < B - 1 && st.rem >= steps[st.b]; ++st.b) st.rem -= steps[st.b];
            WeighCursor cur;
            cur.begin(p, st);
            WeighPiece x;
            while (cur.next(p, x))
                std::printf("P %d %d %d %d %d %d %d %d %d\n", c, x.b, x.h, x.u, x.c0, x.c1, x.opens, x.closes,
                            x.opens && !x.closes ? weigh_cta_of(st.end + x.to_last, W, used) : -1);
        }
        std::printf("E\n");
    }
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    d = tmp_path_factory.mktemp("weigh_cut")
    src, exe = d / "cut.cpp", d / "cut"
    src.write_text(HARNESS)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-Wall", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)

    def run(calls):
        text = "".join(f"{len(lens)} {Hkv} {tokens} {int(causal)} {max_len} {ctas} {' '.join(map(str, lens))} {' '.join(map(str, cu))}\n"
                       for lens, cu, Hkv, tokens, causal, max_len, ctas in calls)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [c.strip().splitlines() for c in out.split("E\n") if c.strip()]
    return run


def calls():
    rng = random.Random(4)
    some = [([1], [0, 1], 1, 1, True, 1, 152), ([0], [0, 5], 2, 4, True, 64, 152), ([0, 0], [0, 0, 0], 1, 1, False, 64, 3),
            ([256], [0, 256], 1, 96, True, 256, 152), ([4096], [0, 4096], 8, 4, True, 4096, 152), ([100], [0, 300], 2, 7, True, 128, 9),
            ([131072], [0, 131072], 1, 8, True, 131072, 152)]
    for _ in range(150):
        B = rng.randint(1, 9)
        lens = [rng.choice([0, 1, 255, 256, 257, rng.randint(0, 3000)]) for _ in range(B)]
        cu = [rng.randint(0, 3)]
        for n in lens:
            cu.append(cu[-1] + rng.choice([0, 1, n, n + 5, rng.randint(0, 900)]))
        some.append((lens, cu, rng.randint(1, 8), rng.choice([1, 2, 12, 24, 27, 48, 96, 192]), rng.random() < 0.7, 4096,
                     rng.choice([1, 2, 7, 152])))
    return some


def test_every_chunk_once(cut):
    asked = calls()
    for (lens, cu, Hkv, tokens, causal, _, ctas), lines in zip(asked, cut(asked), strict=True):
        W, used = (int(x) for x in lines[0].split()[1:])
        want, total = [], 0
        for b, n in enumerate(lens):
            nq = cu[b + 1] - cu[b]
            chunks = max(1, -(-nq // tokens))
            for h in range(Hkv):
                for u in range(-(-n // 256)):
                    # the first chunk of which any row sees the unit's first key
                    see = [i for i in range(nq) if not causal or u * 256 <= n - nq + i]
                    first = see[0] // tokens if see else chunks - 1
                    total += 2 + chunks - first
                    want += [(b, h, u, c) for c in range(first, chunks)]
        assert W == total
        pieces = [tuple(int(x) for x in line.split()[1:]) for line in lines[1:]]
        assert [(b, h, u, c) for _, b, h, u, c0, c1, *_ in pieces for c in range(c0, c1)] == want
        assert all(c1 > c0 for _, _, _, _, c0, c1, *_ in pieces)
        per = {}
        for c, b, h, u, c0, c1, opens, closes, last in pieces:
            per.setdefault((b, h, u), []).append((c, c0, c1, opens, closes, last))
        for unit in per.values():
            assert [x[3] for x in unit] == [1] + [0] * (len(unit) - 1) and [x[4] for x in unit] == [0] * (len(unit) - 1) + [1]
            assert [x[0] for x in unit] == list(range(unit[0][0], unit[0][0] + len(unit)))
            assert unit[0][5] == (unit[-1][0] if len(unit) > 1 else -1)
        # a CTA's range is as long as any other's, to a step
        for c in range(used):
            mine = [x for x in pieces if x[0] == c]
            assert sum(x[5] - x[4] for x in mine) <= W // used + 1
            assert sum(1 for x in mine if not x[6]) <= 1 and sum(1 for x in mine if x[6] and not x[7]) <= 1
