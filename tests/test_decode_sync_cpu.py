"""Races that no run shows, held off by the form of the source: what the kernels of a decoding
step may not do between two barriers, read from their text."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_layer_fp32_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*", "", text)


def body(text, head):
    """The function whose definition begins with `head`, to its closing brace."""
    at = text.index(head)
    end = at = text.index("{", at)
    depth = 0
    while True:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
        if depth == 0:
            return text[at:end]


def test_an_answer_is_read_by_all_before_the_next_is_written():
    """grid_barrier, expert_ready and tile_done follow one another within a block in any order, and
    each leaves thread 0's answer in one word of shared memory.  Every one of them has a barrier
    of the block before it writes, as a warp may not have read the last answer yet, and one before
    it reads."""
    text = source("few.cu")
    assert len(re.findall(r"plan\.on\s*=[^=]", text)) == 3
    for head in ("bool grid_barrier(", "bool expert_ready(", "void tile_done("):
        f = body(text, head)
        write = re.search(r"plan\.on\s*=[^=]", f).start()
        read = re.search(r"plan\.on(?!\s*=[^=])", f).start()
        sync = [m.start() for m in re.finditer(r"__syncthreads\(\);", f)]
        assert any(s < write for s in sync), head
        assert any(write < s < read for s in sync), head
        first = min(sync)   # for the whole block, before thread 0's part
        assert first < f.index("threadIdx.x == 0"), head


def test_no_store_into_another_block_before_it_has_begun():
    """sample_kernel's clusters: distributed shared memory may be touched once all blocks of the
    cluster run, which only a barrier of the cluster says."""
    f = body(source("sample.cu"), "sample_kernel(")
    first = f.index("put(there(")
    arrive, wait = f.index("cluster_arrive()"), f.index("cluster_wait()")
    assert arrive < wait < first
    # both by all threads: nothing but the whole cluster's exit stands before them
    assert f[:arrive].count("return;") == 1 and f.index("if (r >= a.rows) return;") < arrive
    assert "return;" not in f[arrive:wait]
    for helper in ("get32(there(", "get64(there(", "add32(there("):
        assert helper not in f[:wait]
