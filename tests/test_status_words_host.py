"""How the kernels record what they meet in their status words (no GPU): a wait that ran out must not be lost behind a
clamped length or a bad page that the same call, or one before it, recorded in the same word."""
import os
import re
import subprocess

from attention_forward_prefill_gb300 import build
from attention_forward_prefill_gb300.binding import FA_ERR_WATCHDOG


def sources():
    for name in sorted(os.listdir(build.CSRC)):
        if name.endswith((".cu", ".cuh")):
            with open(os.path.join(build.CSRC, name)) as f:
                yield name, f.read()


def records(text):
    """(how, status) of every report: an atomic on a status word, or record_status."""
    return re.findall(r"\b(atomicCAS|atomicExch|record_status)\([^;]*?(FA_ERR_\w+)", text)


def test_a_watchdog_report_is_never_the_second_of_two_compare_and_swaps():
    seen = 0
    for name, text in sources():
        if not name.startswith(("fa_paged", "fa_prefill")):
            continue
        for how, status in records(text):
            seen += 1
            assert status != "FA_ERR_WATCHDOG" or how != "atomicCAS", name
    assert seen >= 11


HARNESS = """
#define __device__
#define __forceinline__ inline
static int atomicCAS(int *p, int want, int v) { const int old = *p; if (old == want) *p = v; return old; }
static int atomicExch(int *p, int v) { const int old = *p; *p = v; return old; }
#include "fa_status.cuh"
#include <cstdio>
int main() {
    const int codes[3] = {FA_ERR_SEQ_LEN, FA_ERR_PAGE, FA_ERR_WATCHDOG};
    for (int a : codes)
        for (int b : codes) {
            int word = 0;
            fa::record_status(&word, a);
            fa::record_status(&word, b);
            std::printf("%d %d %d\\n", a, b, word);
        }
}
"""


def test_the_first_report_stays_unless_a_wait_ran_out(tmp_path):
    src, exe = tmp_path / "status.cpp", tmp_path / "status"
    src.write_text(HARNESS)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-I", build.CSRC, "-I", os.path.join(build.HERE, "..", "include"),
                    str(src), "-o", str(exe)], check=True)
    lines = [tuple(map(int, x.split())) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines()]
    assert len(lines) == 9
    for first, second, word in lines:
        assert word == (FA_ERR_WATCHDOG if FA_ERR_WATCHDOG in (first, second) else first)
