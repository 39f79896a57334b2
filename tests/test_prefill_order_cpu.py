"""What one CTA of a pair writes into the other's shared memory is ordered by fences that no result shows
reliably when they are missing: the source is read for them (csrc/prefill.cu)."""
import os
import re

from sparse_mla_paged_gb300 import build as B


def body(name):
    """The text of a __device__ function, without comments."""
    with open(os.path.join(B.CSRC, "prefill.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = re.search(r"(?:__device__|__global__) [\w (),]*\b%s\(" % name, text).end()
    depth, start = 0, text.index("{", at)
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]
    raise AssertionError(name)


def in_order(text, *parts):
    at = 0
    for part in parts:
        at = text.index(part, at) + len(part)


def test_marks_are_acquired_from_the_cluster():
    """The warp that issues P V: between the arrival of a tile's probabilities and the look at the marks."""
    in_order(body("run_pv"), "c.wait(BAR_PFULL0", "fence_acquire_shared_cluster();", "flags[")


def test_marks_are_released_to_the_cluster():
    """The softmax: factors and marks of all lanes, then a fence by the lane that arrives."""
    in_order(body("run_softmax"), "st_cluster(to + kOffAlpha", "st_cluster(to + kOffFlags", "__syncwarp();", "fence_cluster();",
             "c.arrive(BAR_PFULL0")


def test_events_are_acquired_by_the_epilogue():
    in_order(body("run_epilogue"), "BAR_EVENT", "fence_cluster();", "kOffFlags", "kOffAlpha")


def test_nothing_is_sent_before_the_last_was_used():
    """What a CTA sends to the other without a wait there: after an abort at most one unit's factors and one
    event are on their way, and both are waited for before either CTA leaves."""
    in_order(body("run_softmax"), "c.wait(BAR_FEMPTY", "abort_flag", "return units;", "st_async(")
    in_order(body("run_pv"), "abort_flag", "return;", "st_async(")
    in_order(body("receive_rest"), "BAR_FFULL", "wait(BAR_FFULL", "wait(BAR_EVENT")
    end = body("prefill_kernel")
    in_order(end, "run_softmax(c)", "cluster_wait();", "if (*c.abort_flag", "receive_rest(", "cluster_wait();", "tmem_dealloc_pair")
    assert "globaltimer_ns() - t0 < 20000" not in end


def test_both_ctas_wait_for_the_last_products():
    """A commit arrives at barriers of both CTAs: neither leaves before the last ones are there."""
    for name in ("run_qk", "run_pv"):
        in_order(body(name), "commit_both_el", "commit_both_el(c.bar(BAR_DRAIN)")
    in_order(body("prefill_kernel"), "run_forward(c)", "if (warp == 2 || c.rank == 0)", "c.bar(BAR_DRAIN), 0)")
