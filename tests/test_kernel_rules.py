"""Rules that the kernels' sources keep and that no run can show: what they
guard against holds or fails by the compiler's or the scheduler's choice."""
from __future__ import annotations

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "activation_sparse_gated_relu_b200", "csrc")


def code(name: str) -> str:
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_warp_mask_from_the_lanes_that_happen_to_be_there():
    # the lanes that reach a point together after a branch are the compiler's choice: a shuffle whose mask asks for them
    # may leave a lane's partner out
    for name in sorted(os.listdir(CSRC)):
        assert "__activemask" not in code(name), name


def test_what_another_cta_cleared_is_acquired_at_cluster_scope():
    # weight gradient: the clearing warp of each CTA of a pair releases its writes at cluster scope, so the one thread
    # that issues the pair's MMAs has to acquire them at that scope, on the blocks that were cleared
    ptx, kernel = code("ptx_pair.cuh"), code("grouped.cuh")
    wait = ptx[ptx.index("mbar_wait_cluster("):]
    assert "acquire.cluster" in wait[:wait.index("\n}")]
    assert "arrive.release.cluster" in ptx[ptx.index("mbar_release_cluster("):].split("\n}")[0]
    fix = kernel[kernel.index("warp == GT_FIX"):kernel.index("warp == GT_MMA) {")]
    issue = kernel[kernel.index("warp == GT_MMA) {"):]
    assert "mbar_release_cluster(" in fix
    assert "mbar_wait_cluster(&full[s]" in issue


def test_a_failed_wait_keeps_every_cta_of_a_cluster_from_storing():
    # where a cluster adds up its CTAs' parts, a CTA whose wait failed has none to give: all of them have to know before
    # the barrier behind which the parts are read
    sites = 0
    for name in ("qlinear.cuh", "grouped.cuh"):
        text = code(name)
        for m in re.finditer(r"cluster_sums<", text):
            before = text[:m.start()]
            sync = before.rindex("cluster_sync();")
            assert re.search(r"spread_abort\(abort_flag, \S+\);\s*$", before[:sync]), name
            assert "!*abort_flag" in before[sync:], name
            sites += 1
    assert sites == 3
    helper = code("ptx_pair.cuh")
    helper = helper[helper.index("void spread_abort("):].split("\n}")[0]
    assert "cluster_addr(" in helper and "st.shared::cluster" in helper


def test_nothing_is_under_way_when_a_cta_that_gave_up_leaves():
    # a wait can fail in any role, after the producer has issued its last copy: what is under way then (copies into
    # shared memory, MMAs that read it and write TMEM) has to be over before TMEM is freed and the CTA exits, whichever
    # role gave up
    for name, kernels in (("qlinear.cuh", 2), ("grouped.cuh", 1)):
        text = code(name)
        bodies = re.split(r"__global__", text)[1:]
        assert len(bodies) == kernels
        for body in bodies:
            assert not re.search(r"mbar_wait\w*\(&?mma_done", body), name       # returns at once where a wait failed
            assert "mbar_drain(mma_done" in body, name
            last = body[body.rindex("__syncthreads();"):]                      # every role is over
            assert re.search(r"if \(\*abort_flag\)\s*\{?\s*drain_copies\(\);", last), name
            assert last.index("drain_copies();") < last.index("tmem_dealloc"), name
    grouped = code("grouped.cuh")
    end = grouped[grouped.rindex("__syncthreads();"):]                          # the pair's CTAs signal each other
    assert re.search(r"spread_abort\(abort_flag, 2\);\s*cluster_sync\(\);.*drain_copies\(\);\s*if \(CTAS == 2\) cluster_sync\(\);",
                     end, re.S)
