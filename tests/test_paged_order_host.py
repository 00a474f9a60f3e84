"""What the paged kernels' sources have to keep in order (no GPU): a mistake here may work by luck of the compiler or
of what runs beside it."""
import os
import re

from attention_forward_prefill_gb300 import build


def source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_aligned_cluster_barriers_see_whole_warps():
    """barrier.cluster.*.aligned needs all lanes of a warp at once, and the branches before it may part them."""
    text = source("fa_paged_cluster_sm103.cu")
    helper = re.search(r"void cluster_sync\(\) \{(.*?)\n\}", text, re.S)
    assert helper.group(1).lstrip().startswith("__syncwarp();")
    outside = text[:helper.start()] + text[helper.end():]
    assert "barrier.cluster" not in outside and outside.count("cluster_sync();") == 2


def test_tensor_memory_is_taken_behind_the_wait_and_before_followers_start():
    """A kernel that takes columns and then waits for one that still needs some would wait forever, and so would this
    one if what follows it took them first."""
    text = source("fa_paged_tiles_sm103.cu")
    order = [text.index(x) for x in ("paged_wait(p);", "tmem_alloc(", "paged_let_go();", "paged_plan<")]
    assert order == sorted(order)
    assert "paged_enter" not in text and "launch_dependents" not in text and text.count("paged_let_go();") == 1
    assert text.count("tmem_alloc(") == 1
