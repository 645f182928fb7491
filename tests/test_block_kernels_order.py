"""How the block operators' kernels order what one thread writes and another reads (CPU).

A missing release or wait gives right results on the GPU nearly always, so the order is held to the
sources: comments are dropped and white space is squeezed before they are looked at.
"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ring_collectives_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return re.sub(r"\s+", " ", text)


def body(text, head):
    """From `head` to the end of the block that it opens."""
    at = text.index(head)
    depth, i = 0, text.index("{", at)
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[at:j + 1]
    raise AssertionError(head)


# ---------------------------------------------------------------- weight gradient: a pair of CTAs
def test_widened_steps_reach_the_other_cta_by_a_release():
    """MMAs of the even CTA read what warps of the odd one wrote: the arrival that says so is a release at cluster
    scope, and a relaxed one hands back accumulators only."""
    kernel = body(source("wgrad.cu"), "k_wgrad(const __grid_constant__")
    assert set(re.findall(r"arrive_remote_relaxed\((\w+)", kernel)) == {"tempty_even"}
    assert "full_even = mapa_shared(full_b + 8 * stage, 0)" in kernel and "mbar_arrive_remote(full_even)" in kernel


def test_the_mmas_wait_at_cluster_scope():
    """For both operands, each of which lies in the other CTA as well."""
    kernel = body(source("wgrad.cu"), "k_wgrad(const __grid_constant__")
    assert re.search(r"wait_all<true>\(full_a \+ 8 \* stage, phase, ab, 4, full_b \+ 8 \* stage\)", kernel)
    wait = body(source("warp.cuh"), "bool wait_all(")
    asked = re.findall(r"mbar_try_wait(?:_cluster)?\((\w+), parity\)", wait)
    assert len(asked) == 2 and asked[0] == asked[1] and "CLUSTER ? mbar_try_wait_cluster(" in wait


# ---------------------------------------------------------------- norm's gradient
def test_copies_land_before_their_space_is_used_again():
    """Past the last row copies still write zeros, and a barrier does not wait for them: every thread waits for its own
    before the barrier after which the groups' sums lie where the rows were staged."""
    text = source("block_norm.cu")
    assert "cp.async.wait_all;" in body(text, "void wait_copies()")
    kernel = body(text, "k_block_norm_bwd(const Params p)")
    end = kernel.index("total.leave();")
    assert kernel[:end].rstrip().endswith("wait_copies();")
    assert end < kernel.index("__syncthreads();", end) < kernel.index("red + me.group * p.N")
    kernel = body(text, "k_block_norm(const Params p)")
    assert kernel[:kernel.index("total.leave();")].rstrip().endswith("wait_copies();")


def test_sums_of_other_blocks_are_acquired_at_cluster_scope():
    """They arrive by st.async, whose count on the mbarrier is a release at that scope."""
    sums = body(source("block_norm.cu"), "struct Sums")
    assert "st.async.shared::cluster" in sums
    assert re.findall(r"wait_all(?:<\w+>)?\(", sums) == ["wait_all<true>("]
